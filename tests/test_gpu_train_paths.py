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
