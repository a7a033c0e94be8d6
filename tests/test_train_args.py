"""Argument checks of the training-head operators (no GPU needed: every call
here is refused, or has nothing to do, before any device work)."""
import pytest
import torch

FAKE = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def mp():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_adamw_gb300 as mp
    return mp


def call(mp, name, order, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(mp.lib(), name)(*[a[k] for k in order])


LNF = dict(y=FAKE, mean=FAKE, rstd=FAKE, x=2 * FAKE, weight=FAKE, bias=FAKE, rows=4, d=100, y_stride=100,
           x_stride=100, eps=1e-5, type=0, weight_type=0, stream=None)
LNB = dict(dx=FAKE, dweight=FAKE, dbias=FAKE, dy=2 * FAKE, x=3 * FAKE, weight=FAKE, mean=FAKE, rstd=FAKE, rows=4,
           d=100, dx_stride=100, dy_stride=100, x_stride=100, type=0, weight_type=2, ws=FAKE, wsn=1 << 40, stream=None)
LPF = dict(logp=FAKE, lse=FAKE, entropy=FAKE, top_logp=FAKE, top_index=FAKE, logits=FAKE, targets=FAKE, rows=4,
           vocab=100, stride=100, scale=1.0, top_k=5, type=0, index_type=1, d_status=None, stream=None)
LPB = dict(dlogits=FAKE, logits=2 * FAKE, targets=FAKE, lse=FAKE, entropy=FAKE, dlogp=FAKE, dentropy=FAKE, rows=4,
           vocab=100, dlogits_stride=100, stride=100, scale=1.0, type=0, index_type=1, d_status=None, stream=None)
DST = dict(loss=FAKE, dlogits=FAKE, logits=2 * FAKE, teacher=FAKE, index=FAKE, row_weight=FAKE, rows=4, vocab=100,
           k=5, dlogits_stride=100, stride=100, teacher_stride=5, index_stride=5, scale=1.0, type=0, index_type=1,
           d_status=None, stream=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("name,base,kw,status", [
    ("mp_layernorm_forward", LNF, dict(rows=0), "MP_OK"),
    ("mp_layernorm_forward", LNF, dict(y=None), "MP_ERR_NULL"),
    ("mp_layernorm_forward", LNF, dict(x=None), "MP_ERR_NULL"),
    ("mp_layernorm_forward", LNF, dict(x=FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_layernorm_forward", LNF, dict(type=2, x=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_layernorm_forward", LNF, dict(weight=FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_layernorm_forward", LNF, dict(mean=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_layernorm_forward", LNF, dict(type=3), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(weight_type=-1), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(rows=-1), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(d=0), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(d=(1 << 24) + 1, x_stride=1 << 25, y_stride=1 << 25), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(x_stride=99), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(y_stride=99), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(y=2 * FAKE, y_stride=101), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(eps=-1e-5), "MP_ERR_RANGE"),
    ("mp_layernorm_forward", LNF, dict(eps=NAN), "MP_ERR_RANGE"),
    ("mp_layernorm_backward", LNB, dict(dx=None, dweight=None, dbias=None), "MP_ERR_NULL"),
    ("mp_layernorm_backward", LNB, dict(dy=None), "MP_ERR_NULL"),
    ("mp_layernorm_backward", LNB, dict(mean=None), "MP_ERR_NULL"),
    ("mp_layernorm_backward", LNB, dict(ws=None), "MP_ERR_WORKSPACE"),
    ("mp_layernorm_backward", LNB, dict(wsn=8), "MP_ERR_WORKSPACE"),
    ("mp_layernorm_backward", LNB, dict(ws=FAKE + 8), "MP_ERR_ALIGN"),
    ("mp_layernorm_backward", LNB, dict(dweight=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_layernorm_backward", LNB, dict(dx=2 * FAKE, dx_stride=101), "MP_ERR_RANGE"),
    ("mp_layernorm_backward", LNB, dict(dy_stride=0), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(rows=0), "MP_OK"),
    ("mp_token_logprob_forward", LPF, dict(logits=None), "MP_ERR_NULL"),
    ("mp_token_logprob_forward", LPF, dict(targets=None), "MP_ERR_NULL"),
    ("mp_token_logprob_forward", LPF, dict(logp=None), "MP_ERR_NULL"),
    ("mp_token_logprob_forward", LPF, dict(top_index=None), "MP_ERR_NULL"),
    ("mp_token_logprob_forward", LPF, dict(logp=None, targets=None, lse=None, entropy=None, top_k=0), "MP_ERR_NULL"),
    ("mp_token_logprob_forward", LPF, dict(top_k=33), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(top_k=-1), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(vocab=4, top_k=5), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(vocab=0, top_k=0), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(vocab=1 << 31, stride=1 << 31), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(stride=99), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(scale=0.0), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(scale=INF), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(scale=NAN), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(index_type=2), "MP_ERR_RANGE"),
    ("mp_token_logprob_forward", LPF, dict(targets=FAKE + 4), "MP_ERR_ALIGN"),
    ("mp_token_logprob_forward", LPF, dict(logits=FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_token_logprob_backward", LPB, dict(rows=0), "MP_OK"),
    ("mp_token_logprob_backward", LPB, dict(dlogits=None), "MP_ERR_NULL"),
    ("mp_token_logprob_backward", LPB, dict(lse=None), "MP_ERR_NULL"),
    ("mp_token_logprob_backward", LPB, dict(dlogp=None), "MP_ERR_NULL"),
    ("mp_token_logprob_backward", LPB, dict(entropy=None), "MP_ERR_NULL"),
    ("mp_token_logprob_backward", LPB, dict(dlogp=None, targets=None, entropy=None, dentropy=None), "MP_ERR_NULL"),
    ("mp_token_logprob_backward", LPB, dict(dlogits=2 * FAKE, dlogits_stride=104), "MP_ERR_RANGE"),
    ("mp_token_logprob_backward", LPB, dict(lse=FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_distill_topk", DST, dict(rows=0), "MP_OK"),
    ("mp_distill_topk", DST, dict(loss=None), "MP_ERR_NULL"),
    ("mp_distill_topk", DST, dict(teacher=None), "MP_ERR_NULL"),
    ("mp_distill_topk", DST, dict(k=0), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(k=1025, teacher_stride=1025, index_stride=1025), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(teacher_stride=4), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(index_stride=4), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(dlogits_stride=99), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(dlogits=2 * FAKE, dlogits_stride=101), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(scale=-1.0), "MP_ERR_RANGE"),
    ("mp_distill_topk", DST, dict(index=FAKE + 4), "MP_ERR_ALIGN"),
    ("mp_distill_topk", DST, dict(teacher=FAKE + 1), "MP_ERR_ALIGN"),
])
def test_abi_checks(mp, name, base, kw, status):
    assert call(mp, name, list(base), base, **kw) == getattr(mp, status)


def test_workspace_bytes(mp):
    assert mp.mp_layernorm_workspace_bytes(-1, 8) == 0 and mp.mp_layernorm_workspace_bytes(4, 0) == 0


def test_the_binding_refuses_host_tensors(mp, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mp.mp_layernorm_forward(x.clone(), x)
    with pytest.raises(ValueError):
        mp.mp_token_logprob_forward(x, lse=torch.zeros(4))
    with pytest.raises(TypeError):
        mp.mp_layernorm_forward(x.clone(), x.double())
    with pytest.raises(TypeError):
        mp.mp_distill_topk(torch.zeros(4), None, [1.0], x, torch.zeros(4, 8, dtype=torch.int64))
