"""The RMS norm once for every set of outputs, at row counts and widths that take
each of its variants, and the gated activation with one of its inputs kept.
References and bounds: tests/block_ref.py."""
import pytest
import torch

import block_ref as R
from test_gpu_block_ops import Guarded8, contiguous8, scales
from test_gpu_train_ops import BF, FF, HF, Guarded, f32, gen, mp, randn  # noqa: F401

pytestmark = pytest.mark.gpu

# residual, h, y, kind of y8, h8
SETS = {"y": (0, 0, 1, None, 0), "row8": (0, 0, 0, "row", 0), "block8": (0, 0, 0, "block", 0),
        "y h8": (0, 0, 1, None, 1), "res y": (1, 0, 1, None, 0), "res h y": (1, 1, 1, None, 0),
        "res h y h8": (1, 1, 1, None, 1), "res h row8": (1, 1, 0, "row", 0), "res h row8 h8": (1, 1, 0, "row", 1),
        "res h block8": (1, 1, 0, "block", 0), "res h block8 h8": (1, 1, 0, "block", 1)}
# one, two and four units a thread, on the 16-byte grid and off it
SHAPES = [(40, 1600), (400, 1600), (1300, 48), (1300, 512), (1300, 1280), (1300, 1600), (1300, 4096), (1300, 5120),
          (700, 8192), (40, 1365), (1300, 100), (1300, 700), (1300, 1365), (1300, 4097), (700, 5121), (7, 8200),
          (7, 9001)]


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("outputs", SETS)
def test_rmsnorm_each_set_of_outputs(mp, outputs, rows, d, dtype):  # noqa: F811
    outputs_case(mp, outputs, rows, d, dtype)


@pytest.mark.parametrize("rows,d", [(1300, 512), (1300, 1600), (1300, 4097)])
@pytest.mark.parametrize("outputs", SETS)
def test_rmsnorm_each_set_of_outputs_fp16(mp, outputs, rows, d):  # noqa: F811
    outputs_case(mp, outputs, rows, d, HF)


def outputs_case(mp, outputs, rows, d, dtype):  # noqa: F811
    residual, has_h, has_y, kind, has_h8 = SETS[outputs]
    g = gen(rows + d)
    x = randn((rows, d), g, 1.5, dtype)
    res = randn((rows, d), g, 1.0, dtype) if residual else None
    w = (1 + randn((d,), g, 0.2)).to(dtype)
    rstd = f32(rows)
    h, y = (Guarded(rows, d, dtype) if on else None for on in (has_h, has_y))
    y8, h8 = Guarded8(rows, d) if kind else None, Guarded8(rows, d) if has_h8 else None
    ys, hs = scales(rows, d, kind) if kind else None, scales(rows, d, "block") if has_h8 else None

    def view(o):
        return None if o is None else o.view

    mp.mp_rmsnorm_forward(view(y), x, w, residual=res, h=view(h), rstd=rstd, y8=view(y8), y8_scale=ys, h8=view(h8),
                          h8_scale=hs)
    torch.cuda.synchronize()
    stored = (x.float() + res.float()).to(dtype) if residual else x
    (ry, rr), (ty, tr) = R.rms_forward(stored, w, 1e-5)
    R.assert_within(rstd, rr, tr, "rstd")
    if has_h:
        assert torch.equal(h.view, stored), "h"
    if has_y:
        R.assert_within(y.view, ry, R.rounded(ry, ty, dtype), "y")
    if kind == "row":
        R.check_row8(contiguous8(y8.view), ys, ry, ty, "y8")
    elif kind:
        R.check_block8(contiguous8(y8.view), ys, ry, ty, None, "y8")
    if has_h8:
        R.check_block8(contiguous8(h8.view), hs, stored.double(), 0.0 * ry, dtype, "h8")
    for o, name in ((h, "h"), (y, "y"), (y8, "y8"), (h8, "h8")):
        if o is not None:
            o.check(name)


def test_rmsnorm_same_bits_on_every_run(mp):  # noqa: F811
    # to 8 bits with a scale a row, whose rounding shows a change of the last bit of a sum; beside other work
    g = gen(31)
    rows, d = 4096, 4096
    x, res, w = randn((rows, d), g, 1.0, BF), randn((rows, d), g, 1.0, BF), (1 + randn((d,), g, 0.1)).to(BF)
    other, side = torch.ones(1 << 29, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()

    def once():
        out = [torch.empty_like(x), f32(rows), torch.empty(rows, d, dtype=torch.uint8, device="cuda"), f32(rows)]
        mp.mp_rmsnorm_forward(None, x, w, residual=res, h=out[0], rstd=out[1], y8=out[2], y8_scale=out[3])
        return out

    want = once()
    for _ in range(30):
        with torch.cuda.stream(side):
            other.add_(1)
        for a, b in zip(once(), want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()


# dh, dx, dweight
WANTED = {"dx": (0, 1, 0), "dweight": (0, 0, 1), "dx dweight": (0, 1, 1), "dh dx": (1, 1, 0), "dh dx dweight": (1, 1, 1)}


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("rows,d", [(9, 64), (1300, 64), (1300, 100), (1300, 512), (700, 1600), (700, 1365), (700, 4096),
                                    (300, 4097), (7, 8200), (70, 9001)])
@pytest.mark.parametrize("wanted", WANTED)
def test_rmsnorm_each_set_of_gradients(mp, wanted, rows, d, kept, dtype):  # noqa: F811
    has_dh, has_dx, has_dw = WANTED[wanted]
    g = gen(rows + d)
    h, dy = randn((rows, d), g, 1.5, dtype), randn((rows, d), g, 1.0, dtype)
    dh = randn((rows, d), g, 1.0, dtype) if has_dh else None
    w = (1 + randn((d,), g, 0.2)).to(dtype)
    rstd = R.rms_forward(h, w, 1e-5)[0][1].float()
    src, s, hd = h, None, h.double()
    if kept:
        src, s = torch.empty(rows, d, dtype=torch.uint8, device="cuda"), scales(rows, d, "block")
        mp.mp_pack8(src, s, h)
        hd = R.unpack(src, s)
    dx = Guarded(rows, d, dtype) if has_dx else None
    dw = torch.full((d + 2,), 77.0, dtype=dtype, device="cuda") if has_dw else None
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda") if has_dw else None
    mp.mp_rmsnorm_backward(dx.view if has_dx else None, dw[1:1 + d] if has_dw else None, dy, src, w, rstd, dh=dh,
                           h_scale=s, workspace=ws)
    (rdx, rdw), (tdx, tdw) = R.rms_backward(dy, dh, hd, w, rstd)
    if has_dx:
        R.assert_within(dx.view, rdx, R.rounded(rdx, tdx, dtype), "dx")
        dx.check("dx")
    if has_dw:
        R.assert_within(dw[1:1 + d], rdw, R.rounded(rdw, tdw, dtype), "dweight")
        assert dw[0] == 77.0 and dw[-1] == 77.0


@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,d", [(5, 64), (300, 1600), (301, 1365)])
def test_gated_keeps_one(mp, rows, d, dtype, which):  # noqa: F811
    g = gen(d)
    a, b = randn((rows, d), g, 2.0, dtype), randn((rows, d), g, 2.0, dtype)
    y, want, q, s = torch.empty_like(a), torch.empty_like(a), Guarded8(rows, d), scales(rows, d, "block")
    mp.mp_gated_forward(want, a, b)
    mp.mp_gated_forward(y, a, b, **{which + "8": q.view, which + "8_scale": s})
    assert torch.equal(y, want)
    v = (a if which == "gate" else b).double()
    R.check_block8(contiguous8(q.view), s, v, 0.0 * v, dtype, which)
    q.check(which)
