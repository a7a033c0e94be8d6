"""The training-head operators on the paths that sizes, masks and alignment
select, beyond tests/test_gpu_train_ops.py: against the same 64-bit references
and bounds (tests/train_ref.py)."""
import math

import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_adamw_gb300 as mp
    return mp


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, std=1.0, dtype=FF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def f32(*shape, fill=-7.0):
    return torch.full(shape, fill, dtype=FF, device="cuda")


# --- rows split over the blocks of a cluster --------------------------------------

@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,vocab", [(1, 4100), (1, 8200), (3, 16391), (1, 128256), (37, 50304), (75, 20001)])
def test_logprob_clusters_started_one_after_the_other(mp, rows, vocab, dtype):
    # calls in flight on two streams, each cluster's blocks taking what the other leaves free:
    # the blocks of a row start and finish at different times
    g = gen(rows + vocab)
    x = randn((rows, vocab), g, 2.5, dtype)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(60):
        o = (f32(rows), f32(rows), f32(rows), f32(rows, 8),
             torch.full((rows, 8), -9, dtype=torch.int32, device="cuda"))
        torch.cuda.current_stream().synchronize()  # the fills, before another stream writes
        mp.mp_token_logprob_forward(x, t, logp=o[0], lse=o[1], entropy=o[2], top_logp=o[3], top_index=o[4],
                                    stream=streams[i % 2])
        outs.append(o)
    torch.cuda.synchronize()
    ref, tol = R.lp_forward(x, t, 1.0, 8)
    for name, got in zip(("logp", "lse", "entropy", "top_logp"), outs[0]):
        R.assert_within(got, ref[name], tol[name], f"{rows}x{vocab} {dtype} {name}")
    assert torch.equal(outs[0][4], ref["top_index"])
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


# --- layer norm, staged rows -------------------------------------------------------

def among_nan(t, off, pad):
    """t at an offset of `off` elements, NaN between its rows."""
    rows, cols = t.shape
    buf = torch.full((off + rows * (cols + pad) + 64,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def ln_check(mp, x, dy, w, b, eps=1e-5, what="", slices=4):
    """Forward and backward of x and dy against the references, which are taken a slice of the rows at a time."""
    rows, d = x.shape
    dtype, wtype = x.dtype, w.dtype
    y, dx = (torch.full((rows, d), -7.0, dtype=dtype, device="cuda") for _ in range(2))
    mean, rstd, dw, db = f32(rows), f32(rows), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_forward(y, x, w, b, eps, mean=mean, rstd=rstd)
    mp.mp_layernorm_backward(dx, dw, db, dy, x, w, mean, rstd, workspace=ws)
    torch.cuda.synchronize()
    what = f"{what} {rows}x{d} {dtype}"
    sums = [0.0] * 4
    step = (rows + slices - 1) // slices
    for a in range(0, rows, step):
        s = slice(a, min(rows, a + step))
        (ry, rm, rr), (ty, tm, tr) = R.ln_forward(x[s], w, b, eps)
        R.assert_within(mean[s], rm, tm, what + " mean")
        R.assert_within(rstd[s], rr, tr, what + " rstd")
        R.assert_within(y[s], ry, R.rounded(ry, ty, dtype), what + " y")
        (rdx, rdw, rdb), (tdx, _, _) = R.ln_backward(dy[s], x[s], w, mean[s], rstd[s])
        R.assert_within(dx[s], rdx, R.rounded(rdx, tdx, dtype), what + " dx")
        xh, g = (x[s].double() - mean[s].double()[:, None]) * rstd[s].double()[:, None], dy[s].double()
        for i, v in enumerate((rdw, rdb, (g * xh).abs().sum(0), g.abs().sum(0))):
            sums[i] = sums[i] + v
    # the bounds of R.ln_backward, over all the rows
    Dr = 96 + rows / 48
    for got, ref, tol, name in ((dw, sums[0], (Dr + 4) * R.U * sums[2], "dweight"), (db, sums[1], Dr * R.U * sums[3], "dbias")):
        R.assert_within(got, ref, R.rounded(ref, tol, wtype), f"{what} {name}")


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,d", [(15000, 300), (9001, 1357), (5000, 2047), (3001, 4099), (2000, 8191)])
@pytest.mark.parametrize("pad", [1, 5])
def test_layernorm_stages_used_again_at_other_offsets(mp, rows, d, dtype, pad):
    # every buffer holds many rows one after the other, each at another offset from the 16-byte grid
    g = gen(rows)
    x, dy = among_nan(randn((rows, d), g, 1.5, dtype), 1, pad), among_nan(randn((rows, d), g, 1.0, dtype), 3, pad + 2)
    ln_check(mp, x, dy, 1 + randn((d,), g, 0.2), randn((d,), g, 0.3), what=f"pad {pad}")


# --- finite logits of large magnitude ------------------------------------------------

MASKS = [-1e9, -1e10, -1e12, -1e30, "lowest / 4"]


def masked_rows(rows, vocab, dtype, value, seed):
    """Logits whose rows are masked in turn by the value: not at all, over the first half, all but one token, all
    of them, the last half, and a row that lies at its negative."""
    low = torch.finfo(dtype).min
    value = low / 4 if isinstance(value, str) else value
    x = randn((rows, vocab), gen(seed), 2.0, dtype)
    x[1::6, : vocab // 2] = value
    keep = x[2::6, vocab // 3].clone()
    x[2::6] = value
    x[2::6, vocab // 3] = keep
    x[3::6] = value
    x[4::6, vocab // 2:] = value
    x[5::6] = -value
    return x


def chains_of_a_warp(monkeypatch):
    # rows far from 0 are summed by one warp or one block: n / 32 additions after one another
    monkeypatch.setattr(R, "depth", lambda n: 96 + n / 32)


def lp_large(mp, x, scale, k, entropy=True, slices=1):
    rows, vocab = x.shape
    t = torch.randint(0, vocab, (rows,), generator=gen(7), device="cuda")
    t[2::6] = vocab // 3
    logp, lse, ent = f32(rows), f32(rows), f32(rows) if entropy else None
    tl = f32(rows, k) if k else None
    ti = torch.full((rows, k), -9, dtype=torch.int32, device="cuda") if k else None
    mp.mp_token_logprob_forward(x, t, logp=logp, lse=lse, entropy=ent, top_logp=tl, top_index=ti, scale=scale)
    torch.cuda.synchronize()
    step = (rows + slices - 1) // slices
    for a in range(0, rows, step):
        s = slice(a, min(rows, a + step))
        ref, tol = R.lp_forward(x[s], t[s], scale, k)
        # log p comes from differences of logits, whatever the size of lse: R's bound of log(sum), and the difference's
        z, m, e, sums, _ = R._stats(x[s], scale)
        p = e / sums
        dist = torch.where(p > 0, p * (m - z), 0.0).sum(1)
        log_s = torch.log(sums)[:, 0]
        t_log_s = (R.depth(vocab) + 6) * R.U + 3 * R.U * dist + 2 * R.U * log_s.abs()
        tol["logp"] = t_log_s + 4 * R.U * ref["logp"].abs()
        if k:
            tol["top_logp"] = t_log_s[:, None] + 4 * R.U * ref["top_logp"].abs()
            assert torch.equal(ti[s], ref["top_index"]), "top_index"
        for name, got in (("lse", lse), ("logp", logp), ("entropy", ent), ("top_logp", tl)):
            if got is not None:
                R.assert_within(got[s], ref[name], tol[name], f"{rows}x{vocab} {x.dtype} {name}")


@pytest.mark.parametrize("scale", [0.5, 1.0, 1 / 0.6])
@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("dtype", [BF, FF])
def test_logprob_large_masks(mp, monkeypatch, dtype, value, scale):
    chains_of_a_warp(monkeypatch)
    for rows, vocab in ((6, 8192), (6, 131), (6, 50304), (300, 5000)):
        lp_large(mp, masked_rows(rows, vocab, dtype, value, rows), scale, 5)
    lp_large(mp, masked_rows(6, 8192, dtype, value, 3)[1:2], scale, 0)


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("dtype", [BF, FF])
def test_logprob_large_masks_many_long_rows(mp, monkeypatch, dtype, value):
    chains_of_a_warp(monkeypatch)
    lp_large(mp, masked_rows(2100, 16391, dtype, value, 4), 1.0, 5, slices=4)


@pytest.mark.parametrize("scale", [0.5, 1.0, 1 / 0.6])
@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("dtype", [BF, FF])
def test_distill_large_masks(mp, monkeypatch, dtype, value, scale):
    chains_of_a_warp(monkeypatch)
    for rows, vocab in ((6, 8192), (6, 131), (300, 5000), (6, 128256), (400, 40000)):
        x = masked_rows(rows, vocab, dtype, value, rows)
        g = gen(8)
        idx = torch.rand(rows, vocab, generator=g, device="cuda").topk(12, dim=1).indices
        idx[1::6] = vocab // 2 + idx[1::6] % (vocab // 2)
        idx[2::6] = vocab // 3
        idx[4::6] %= vocab // 2
        t = randn((rows, 12), g, 2.0, dtype)
        (rl, rd), (tl, td) = R.distill(x, t, idx, None, scale)
        loss, dx, alone = f32(rows), torch.full_like(x, -7.0), f32(rows)
        mp.mp_distill_topk(loss, dx, x, t, idx, scale=scale)
        mp.mp_distill_topk(alone, None, x, t, idx, scale=scale)
        torch.cuda.synchronize()
        what = f"{rows}x{vocab} {dtype} {value} {scale}"
        R.assert_within(loss, rl, tl, what + " loss")
        R.assert_within(alone, rl, tl, what + " loss alone")
        R.assert_within(dx, rd, R.rounded(rd, td, dtype), what + " dlogits")


@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** -126])
def test_extreme_scales(mp, scale):
    # the largest scale accepted; equal logits, and logits whose scaled differences are far apart or nearly 0
    x = torch.zeros(3, 900, device="cuda")
    x[1] = torch.arange(900, device="cuda") * 2.0 ** -120
    x[2] = torch.arange(900, device="cuda").float()
    t = torch.tensor([5, 899, 899], device="cuda")
    logp, lse, ent = f32(3), f32(3), f32(3)
    mp.mp_token_logprob_forward(x, t, logp=logp, lse=lse, entropy=ent, scale=scale)
    z = x.double() * scale
    p = torch.log_softmax(z, 1)
    ref = p.gather(1, t[:, None])[:, 0]
    tol = 200 * R.U * (1 + math.log(900))
    assert ((logp.double() - ref).abs() <= tol).all()
    assert ((ent.double() - torch.special.entr(p.exp()).sum(1)).abs() <= tol).all()
    loss, dx = f32(3), torch.empty_like(x)
    mp.mp_distill_topk(loss, dx, x, torch.zeros(3, 1, device="cuda"), t[:, None], scale=scale)
    assert ((loss.double() + ref).abs() <= tol).all()
    one = torch.nn.functional.one_hot(t, 900)
    assert (((dx.double() / scale) - (p.exp() - one)).abs() <= tol).all()


@pytest.mark.parametrize("d", [64, 1000, 9000])
def test_layernorm_backward_of_no_rows(mp, d):
    x, none = torch.empty(0, d, dtype=BF, device="cuda"), torch.empty(0, device="cuda")
    mp.mp_layernorm_backward(x.clone(), None, None, x, x, None, none, none)
    dw = f32(d)
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(0, d), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_backward(x.clone(), dw, None, x, x, None, none, none, workspace=ws)
    assert (dw == 0).all()


# --- layer norm of rows with a common offset -------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("d", [96, 200, 768, 1357, 1600, 4096, 4100, 5632, 8192, 9001])
def test_layernorm_common_offset(mp, d, dtype):
    # a row's values lie around one offset a thousand times their spread (fp32), or as far out as the type tells them
    # apart; constant rows, whose normalised values are 0 and whose 1/std is the largest; fp32 weight gradients
    g = gen(d)
    rows = 300
    at = {BF: 100.0, HF: 1000.0, FF: 1500.0}[dtype]
    x = (randn((rows, d), g, 1.5) + at * torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.5, -1.0, 1.0)).to(dtype)
    x[::3] = (torch.arange(100, device="cuda") * 41.0 - 2000.0)[:, None].to(dtype)
    dy = randn((rows, d), g, 1.0, dtype)
    ln_check(mp, x, dy, 1 + randn((d,), g, 0.2), randn((d,), g, 0.3), what="offset")


# --- the kernels of many rows ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("d", [264, 520, 1024, 1600, 2048, 2056, 4096, 4104, 8192, 261, 1013, 1029, 2047, 4099, 8191])
def test_layernorm_warps_of_a_row(mp, d, dtype):
    # row counts on either side of those at which fewer warps take a row: from one to eight, one to eight units a thread
    g = gen(d)
    for rows in (37, 151, 153, 303, 305, 607, 609, 1215, 1217, 2500):
        x, dy = randn((rows, d), g, 1.5, dtype), randn((rows, d), g, 1.0, dtype)
        ln_check(mp, x, dy, 1 + randn((d,), g, 0.2), randn((d,), g, 0.3), slices=1)


def hard_rows(x, every):
    """Rows that go wrong first, where one block takes every `every`-th row: three of them one after the other."""
    dtype, vocab = x.dtype, x.shape[1]
    kinds = [
        lambda r: r.fill_(-INF),
        lambda r: r.fill_(torch.finfo(dtype).min),
        lambda r: r[vocab // 2].fill_(math.nan),
        lambda r: r[vocab // 3].fill_(INF),
        lambda r: r.fill_(0.5),                                            # all equal
        lambda r: r.copy_(torch.sort(r.float()).values.to(dtype)),         # rising
        lambda r: r.copy_(torch.sort(r.float(), descending=True).values.to(dtype)),
        lambda r: r.copy_(r.float().round().clamp(-2, 2).to(dtype)),       # thousands of equal ones at the top
        lambda r: r[: vocab - 1].fill_(-INF),                              # one token
        lambda r: r[: vocab // 2].fill_(-1e4),
        lambda r: r.fill_(math.nan),
        lambda r: r[7:].copy_(r[7:] * 0),
        lambda r: r.fill_(-3e4),
    ]
    n = 0
    for block in range(len(kinds)):
        for turn in range(block, x.shape[0], every):
            kinds[n % len(kinds)](x[turn])
            n += 1
        n += 1  # the next block begins with another


@pytest.mark.parametrize("entropy", [True, False])
@pytest.mark.parametrize("k", [0, 1, 32])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_logprob_many_long_rows(mp, monkeypatch, dtype, k, entropy):
    chains_of_a_warp(monkeypatch)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # either side of the row count and of the vocabulary from which blocks read one row after the other
    for rows, vocab, pad, off in ((12 * sms - 1, 16384, 0, 0), (12 * sms, 16384, 8, 0), (12 * sms + 276, 16383, 1, 0),
                                  (12 * sms + 276, 16391, 3, 5), (12 * sms + 276, 50304, 0, 0), (3000, 20001, 0, 1)):
        x = randn((rows, vocab), gen(rows + vocab), 2.0, dtype)
        hard_rows(x, 6 * sms)
        x = among_nan(x, off, pad)
        lp_any(mp, x, k, entropy)


def lp_any(mp, x, k, entropy, slices=6):
    rows, vocab = x.shape
    t = torch.randint(0, vocab, (rows,), generator=gen(9), device="cuda", dtype=torch.int32)
    t[5::11] = -1
    outs = []
    for _ in range(3):
        o = {"lse": f32(rows), "logp": f32(rows)}
        if entropy:
            o["entropy"] = f32(rows)
        if k:
            o["top_logp"] = f32(rows, k)
            o["top_index"] = torch.full((rows, k), -9, dtype=torch.int32, device="cuda")
        mp.mp_token_logprob_forward(x, t, **o)
        outs.append(o)
    torch.cuda.synchronize()
    for o in outs[1:]:  # the same bits on every run (NaN included)
        assert all(torch.equal(v.view(torch.int32), outs[0][n].view(torch.int32)) for n, v in o.items())
    step = (rows + slices - 1) // slices
    for a in range(0, rows, step):
        s = slice(a, min(rows, a + step))
        ref, tol = R.lp_forward(x[s], t[s], 1.0, k)
        given = t[s] >= 0
        assert (outs[0]["logp"][s][~given] == 0).all()  # exactly, whatever the row holds
        for name, got in outs[0].items():
            if name == "logp":
                R.assert_within(got[s][given], ref[name][given], tol[name][given], f"{rows}x{vocab} {x.dtype} logp")
            elif name == "top_index":
                assert torch.equal(got[s], ref[name]), f"{rows}x{vocab} {x.dtype} top_index"
            else:
                R.assert_within(got[s], ref[name], tol[name], f"{rows}x{vocab} {x.dtype} {name}")


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,vocab", [(1, 4099), (1, 128256), (3, 50261), (40, 20001), (300, 5000)])
def test_logprob_gradient_over_split_rows(mp, rows, vocab, dtype):
    # a row over its own logits by several blocks; the given token in each of their parts, and at the row's ends
    g = gen(vocab)
    x = randn((rows, vocab), g, 2.0, dtype)
    dlogp, dent = randn((rows,), g), randn((rows,), g)
    for at in (0, 1, vocab // 3, vocab // 2, vocab - 9, vocab - 1):
        t = torch.full((rows,), at, device="cuda")
        t[rows // 2:] = vocab - 1 - at
        logp, lse, ent = f32(rows), f32(rows), f32(rows)
        mp.mp_token_logprob_forward(x, t, logp=logp, lse=lse, entropy=ent)
        apart, over = torch.empty_like(x), x.clone()
        kw = dict(lse=lse, dlogp=dlogp, entropy=ent, dentropy=dent)
        mp.mp_token_logprob_backward(apart, x, t, **kw)
        mp.mp_token_logprob_backward(over, over, t, **kw)
        rd, td = R.lp_backward(x, t, lse, ent, dlogp, dent, 1.0)
        R.assert_within(apart, rd, R.rounded(rd, td, dtype), f"{at}")
        assert torch.equal(over, apart)


# --- NaN and infinities anywhere in a row ---------------------------------------------------

@pytest.mark.parametrize("value", [math.nan, INF])
@pytest.mark.parametrize("masked", [0, 1, 3])
@pytest.mark.parametrize("dtype,vocab", [(HF, 37041), (BF, 46090), (BF, 50304), (FF, 19016), (BF, 128256), (FF, 33000),
                                         (BF, 5000), (FF, 777), (BF, 20001)])
def test_nan_anywhere_shows(mp, dtype, vocab, masked, value):
    # one NaN or +inf a row, at each of many places; with `masked`, thirds of the row after it hold -inf alone
    g = gen(vocab)
    for rows in (5, 608, 1900 if vocab < 60000 else 700):
        x = randn((rows, vocab), g, 2.5, dtype)
        keep = vocab - masked * (vocab // 4)
        x[:, keep:] = -INF
        at = torch.randint(0, keep, (rows,), generator=g, device="cuda")
        at[:4] = torch.tensor([0, keep - 1, keep // 2, keep - 2], device="cuda")
        x.scatter_(1, at[:, None], value)
        idx = (at[:, None] + 1 + torch.randint(0, max(1, keep - 1), (rows, 4), generator=g, device="cuda")) % keep
        t = randn((rows, 4), g, 1.0, dtype)
        loss, alone, dx, lse, ent = f32(rows), f32(rows), torch.full_like(x, -7.0), f32(rows), f32(rows)
        mp.mp_distill_topk(loss, dx, x, t, idx)
        mp.mp_distill_topk(alone, None, x, t, idx)
        mp.mp_token_logprob_forward(x, lse=lse, entropy=ent)
        for name, v in (("loss", loss), ("loss alone", alone), ("lse", lse), ("entropy", ent), ("dlogits", dx)):
            assert torch.isnan(v).all(), f"{name}: {int((~torch.isnan(v)).sum())} of {v.numel()} are not NaN, {rows} rows"


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,vocab", [(6, 500), (3, 40000), (400, 40000), (2000, 3000)])
def test_distill_of_tokens_at_the_lowest_value(mp, dtype, rows, vocab):
    # every listed token has the type's lowest logit: the loss is near the end of fp32, and finite
    g = gen(rows)
    x = randn((rows, vocab), g, 2.0, dtype)
    x[:, vocab // 2:] = torch.finfo(dtype).min
    idx = torch.randint(vocab // 2, vocab, (rows, 24), generator=g, device="cuda")
    t = randn((rows, 24), g, 2.0, dtype)
    w = torch.rand(rows, generator=g, device="cuda") * 1.8 - 0.9
    loss, alone, dx = f32(rows), f32(rows), torch.full_like(x, -7.0)
    mp.mp_distill_topk(loss, dx, x, t, idx, row_weight=w)
    mp.mp_distill_topk(alone, None, x, t, idx, row_weight=w)
    (rl, rd), (tl, td) = R.distill(x, t, idx, w, 1.0)
    R.assert_within(loss, rl, tl, "loss")
    R.assert_within(alone, rl, tl, "loss alone")
    R.assert_within(dx, rd, R.rounded(rd, td, dtype), "dlogits")
