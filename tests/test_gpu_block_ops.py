"""RMS norm, rotary positions, the gated activation and rows in 8 bits against
their 64-bit definitions, at the sizes, strides and values where they can go
wrong. Bounds: tests/block_ref.py."""
import math

import pytest
import torch

import block_ref as R
from test_gpu_train_ops import BF, FF, HF, INF, Guarded, f32, gen, mp, placed, randn  # noqa: F401

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


class Guarded8:
    """[rows, cols] bytes inside a buffer of sentinels."""

    def __init__(self, rows, cols, pad=0, off=0):
        self.buf = torch.full((off + rows * (cols + pad) + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        self.view = self.buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False

    def check(self, what):
        assert (self.buf[self.mask] == 0x5A).all(), f"{what}: written outside"


def scales(rows, d, kind):
    return f32(rows) if kind == "row" else torch.full((rows, -(-d // 32)), 77, dtype=torch.uint8, device="cuda")


def contiguous8(q):
    return q.contiguous()


# --- RMS norm ----------------------------------------------------------------------

SHAPES = [(1, 1), (3, 2), (5, 7), (4, 64), (700, 48), (33, 100), (2, 255), (17, 768), (9, 1000), (5, 1365),
          (300, 1600), (3, 1601), (7, 2048), (4, 4096), (3, 4099), (5, 5120), (3, 8192), (2, 8200), (2, 10007),
          (1, 40000), (2100, 96), (5000, 16), (1300, 8), (1, 4096), (12, 31), (12, 33)]


def rms_case(mp, rows, d, dtype, wtype, *, weight=True, residual=True, y8="row", pad=0, off=0, seed=1, eps=1e-5,
             stream=None):
    g = gen(seed)
    what = f"{rows}x{d} {dtype}"
    x = placed(randn((rows, d), g, 1.5, dtype), pad, off)
    res = placed(randn((rows, d), g, 1.0, dtype), pad, off) if residual else None
    wb = torch.zeros(d + 1, dtype=wtype, device="cuda")
    wb[1:] = 1 + randn((d,), g, 0.2)
    w = wb[1:] if weight else None
    y, h, rstd = Guarded(rows, d, dtype, pad, off), Guarded(rows, d, dtype, pad, off), f32(rows)
    q, h8 = Guarded8(rows, d, pad, off), Guarded8(rows, d, pad, off)
    qs, hs = scales(rows, d, y8), scales(rows, d, "block")
    mp.mp_rmsnorm_forward(y.view, x, w, eps, residual=res, h=h.view if residual else None, rstd=rstd, y8=q.view,
                          y8_scale=qs, h8=h8.view, h8_scale=hs, stream=stream)
    torch.cuda.synchronize()
    stored = (x.float() + res.float()).to(dtype) if residual else x
    if residual:
        assert torch.equal(h.view, stored), what + " h"
    (ry, rr), (ty, tr) = R.rms_forward(stored, w, eps)
    R.assert_within(rstd, rr, tr, what + " rstd")
    R.assert_within(y.view, ry, R.rounded(ry, ty, dtype), what + " y")
    R.check_block8(contiguous8(h8.view), hs, stored.double(), 0.0 * ry, dtype, what + " h8")
    if y8 == "row":
        R.check_row8(contiguous8(q.view), qs, ry, ty, what + " y8")
    else:
        R.check_block8(contiguous8(q.view), qs, ry, ty, None, what + " y8")
    for o, n in ((y, "y"), (h, "h"), (q, "y8"), (h8, "h8")):
        o.check(n)
    # backward, from h and from its 8 bits
    dy = placed(randn((rows, d), g, 1.0, dtype), pad, off)
    dh = placed(randn((rows, d), g, 1.0, dtype), pad, off) if residual else None
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    for kept in (False, True):
        dx, dwb = Guarded(rows, d, dtype, pad, off), torch.full((d + 2,), 77.0, dtype=wtype, device="cuda")
        src = h8.view if kept else placed(stored, pad, off)
        mp.mp_rmsnorm_backward(dx.view, dwb[1:1 + d], dy, src, w, rstd, dh=dh, h_scale=hs if kept else None,
                               workspace=ws, stream=stream)
        torch.cuda.synchronize()
        hd = R.unpack(contiguous8(h8.view), hs) if kept else stored.double()
        (rdx, rdw), (tdx, tdw) = R.rms_backward(dy, dh, hd, w, rstd)
        R.assert_within(dx.view, rdx, R.rounded(rdx, tdx, dtype), f"{what} dx kept={kept}")
        R.assert_within(dwb[1:1 + d], rdw, R.rounded(rdw, tdw, wtype), f"{what} dweight kept={kept}")
        dx.check("dx")
        assert dwb[0] == 77.0 and dwb[-1] == 77.0


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_rmsnorm_shapes(mp, rows, d, dtype):  # noqa: F811
    rms_case(mp, rows, d, dtype, dtype, y8="row" if rows % 2 else "block")


@pytest.mark.parametrize("dtype,wtype", [(BF, FF), (FF, BF), (HF, BF), (BF, HF)])
@pytest.mark.parametrize("weight,residual", [(True, False), (False, True), (False, False)])
def test_rmsnorm_weight_types(mp, dtype, wtype, weight, residual):  # noqa: F811
    rms_case(mp, 37, 776, dtype, wtype, weight=weight, residual=residual, y8="block")


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [64, 768, 1600, 4096, 8192, 9000])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_rmsnorm_strides_and_alignment(mp, dtype, d, pad, off):  # noqa: F811
    rms_case(mp, 21, d, dtype, dtype, pad=pad, off=off, y8="block" if pad == 3 else "row")


@pytest.mark.parametrize("rows", [1, 151, 152, 153, 1216, 1217, 4864, 20001])
@pytest.mark.parametrize("d", [64, 100, 800])
def test_rmsnorm_row_counts(mp, rows, d):  # noqa: F811
    rms_case(mp, rows, d, BF, FF)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [128, 136, 256, 264, 512, 520, 2048, 2056, 4096, 4104, 4160, 8184, 8192, 8224])
def test_rmsnorm_classes(mp, d, dtype):  # noqa: F811
    rms_case(mp, 701, d, dtype, dtype)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [257, 513, 769, 1025, 2049, 2561, 4097, 5121, 6145, 7681, 8191, 8193])
def test_rmsnorm_one_column_more(mp, d, dtype):  # noqa: F811
    # one column past what a number of warps holds
    rms_case(mp, 33, d, dtype, dtype)


@pytest.mark.parametrize("d", [48, 1600, 1365, 9000])
@pytest.mark.parametrize("dtype", [BF, FF])
def test_rmsnorm_in_place_and_optional_outputs(mp, d, dtype):  # noqa: F811
    g = gen(3)
    rows = 19
    x, res, dy, dh = (randn((rows, d), g, 1.0, dtype) for _ in range(4))
    w = randn((d,), g, 1.0, dtype)
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), f32(rows)
    mp.mp_rmsnorm_forward(y, x, w, residual=res, h=h, rstd=rstd)
    for yo, ho in ((0, 1), (1, 0)):  # y over x and h over the residual, and the other way round
        a = [x.clone(), res.clone()]
        mp.mp_rmsnorm_forward(a[yo], a[0], w, residual=a[1], h=a[ho])
        assert torch.equal(a[yo], y) and torch.equal(a[ho], h)
    a = x.clone()
    mp.mp_rmsnorm_forward(a, a, w, residual=res)  # the sum is not kept
    assert torch.equal(a, y)
    only = torch.empty_like(x)
    mp.mp_rmsnorm_forward(None, x, w, residual=res, h=only)  # the sum alone
    assert torch.equal(only, h)
    r2, q, s = f32(rows), torch.empty(rows, d, dtype=E4, device="cuda"), f32(rows)
    mp.mp_rmsnorm_forward(None, h, w, rstd=r2, y8=q, y8_scale=s)
    assert torch.equal(r2, rstd)
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    mp.mp_rmsnorm_backward(dx, dw, dy, h, w, rstd, dh=dh, workspace=ws)
    for k in range(3):  # over dy, dh, h
        a = [dy.clone(), dh.clone(), h.clone()]
        dw2 = torch.empty_like(w)
        mp.mp_rmsnorm_backward(a[k], dw2, a[0], a[2], w, rstd, dh=a[1], workspace=ws)
        assert torch.equal(a[k], dx) and torch.equal(dw2, dw)
    dw2, dx2 = torch.empty_like(w), torch.empty_like(dx)
    mp.mp_rmsnorm_backward(None, dw2, dy, h, w, rstd, workspace=ws)
    mp.mp_rmsnorm_backward(dx2, None, dy, h, w, rstd, dh=dh)
    assert torch.equal(dw2, dw) and torch.equal(dx2, dx)


def test_rmsnorm_no_rows(mp):  # noqa: F811
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    mp.mp_rmsnorm_forward(x.clone(), x)
    dw, none = f32(64), torch.empty(0, device="cuda")
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    mp.mp_rmsnorm_backward(x.clone(), dw, x, x, None, none, workspace=ws)
    assert (dw == 0).all()


@pytest.mark.parametrize("d", [64, 1600, 1365, 9000])
def test_rmsnorm_special_rows(mp, d):  # noqa: F811
    g = gen(4)
    x = randn((7, d), g)
    x[1] = 0.0
    x[2, d // 2], x[3, 3], x[4, d - 1] = math.nan, INF, -INF
    x[5] *= 1e-30
    y, rstd = f32(7, d), f32(7)
    q, s = torch.empty(7, d, dtype=E4, device="cuda"), f32(7)
    b, bs = torch.empty(7, d, dtype=E4, device="cuda"), scales(7, d, "block")
    mp.mp_rmsnorm_forward(y, x, eps=1e-5, rstd=rstd, y8=q, y8_scale=s, h8=b, h8_scale=bs)
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and float(s[1]) == 2.0 ** -126 and (bs[1] == 0).all()
    assert abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-4
    assert torch.isnan(y[2]).all() and torch.isnan(R.unpack(q, s)[2]).all()
    for r, c in ((3, 3), (4, d - 1)):  # rstd is 0: the infinity is NaN, the others are 0
        assert float(rstd[r]) == 0.0 and torch.isnan(y[r, c]) and torch.isnan(s[r])
        assert (torch.cat((y[r, :c], y[r, c + 1:])) == 0).all()
        assert int(bs[r, c // 32]) == 255 and torch.isnan(R.unpack(b, bs)[r, c // 32 * 32])
        assert (bs[r] == 255).sum() == 1
    assert torch.isfinite(y[[0, 5, 6]]).all() and torch.isfinite(s[[0, 5, 6]]).all()


def test_rmsnorm_differences(mp):  # noqa: F811
    # dx, dweight against central differences of the kernel's own forward pass, L = sum(c y) + sum(e h)
    g = gen(8)
    rows, d, h = 3, 24, 2.0 ** -5
    x, c, e, w = randn((rows, d), g), randn((rows, d), g), randn((rows, d), g), randn((d,), g)
    rstd = f32(rows)

    def fwd(x, w):
        y = f32(rows, d)
        mp.mp_rmsnorm_forward(y, x.contiguous(), w)
        return y.double()

    mp.mp_rmsnorm_forward(f32(rows, d), x, w, rstd=rstd)
    dx, dw = f32(rows, d), f32(d)
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_rmsnorm_backward(dx, dw, c, x, w, rstd, dh=e, workspace=ws)
    # truncation h^2 / 6 times the third derivative, rounding 200 u sum|c y| / h
    bound = 40 * h * h / 6 * float(c.abs().max() * w.abs().max() * rstd.max() ** 3) + 200 * R.U * 60 / h
    for j in range(d):
        t = torch.zeros(d, device="cuda")
        t[j] = h
        num = ((fwd(x + t, w) - fwd(x - t, w)) * c.double()).sum(1) / (2 * h) + e[:, j].double()
        assert (num - dx[:, j].double()).abs().max() <= bound
        num = ((fwd(x, w + t) - fwd(x, w - t)) * c.double()).sum() / (2 * h)
        assert abs(num - dw[j].double()) <= bound


# --- rows in 8 bits -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_pack_shapes(mp, rows, d, kind, dtype):  # noqa: F811
    pack_case(mp, rows, d, kind, dtype)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("kind", ["row", "block"])
@pytest.mark.parametrize("d", [64, 1600, 4099, 9000])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_pack_strides_and_alignment(mp, d, kind, dtype, pad, off):  # noqa: F811
    pack_case(mp, 13, d, kind, dtype, pad=pad, off=off)


def pack_case(mp, rows, d, kind, dtype, pad=0, off=0):  # noqa: F811
    g = gen(rows + d)
    x = randn((rows, d), g) * torch.exp(randn((d,), g, 2.0)) * torch.exp(randn((rows, 1), g, 3.0))
    x = placed(x.clamp(-6e4, 6e4).to(dtype), pad, off)
    q, s, back = Guarded8(rows, d, pad, off), scales(rows, d, kind), Guarded(rows, d, dtype, pad, off)
    mp.mp_pack8(q.view, s, x)
    mp.mp_unpack8(back.view, q.view, s)
    torch.cuda.synchronize()
    what = f"{rows}x{d} {dtype} {kind}"
    bytes8, v = contiguous8(q.view), x.double()
    if kind == "row":
        R.check_row8(bytes8, s, v, None, what)
    else:
        R.check_block8(bytes8, s, v, 0.0 * v, dtype, what)
        # the products with powers of two are exact: so are the bits
        w = torch.exp2(127.0 - s.double()).repeat_interleave(32, 1)[:, :d]
        assert torch.equal(bytes8, (v * w).float().to(E4).view(torch.uint8)), what + " bits"
    R.assert_within(back.view, R.unpack(bytes8, s), R.rounded(R.unpack(bytes8, s), 2 * R.U * v.abs(), dtype), what)
    q.check("q")
    back.check("x")


def test_pack_ends_of_the_range(mp):  # noqa: F811
    for dtype in (BF, HF, FF):
        top, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
        x = torch.zeros(10, 64, device="cuda", dtype=dtype)
        x[0] = top                       # reads back finite
        x[1, 3], x[1, 40] = -top, 1.0
        x[2, :] = tiny
        x[3, 5] = tiny * 2.0 ** -3       # below the normal numbers
        x[4, 7] = 448.0                  # the largest e4m3 value: scale 1
        x[5, 7] = 450.0 if dtype != BF else 452.0
        x[6, 7], x[6, 8] = math.nan, 3.0
        x[7, 33], x[7, 0] = INF, 3.0
        x[8, 9] = -0.0
        x[9, 0], x[9, 1] = 448.0, 0.0009765625  # half of the smallest step beside the largest value: to even, 0
        q, s = torch.empty(10, 64, dtype=E4, device="cuda"), scales(10, 64, "block")
        mp.mp_pack8(q, s, x)
        back = torch.empty_like(x)
        mp.mp_unpack8(back, q, s)
        assert torch.equal(s, R.block_exponents(x.double()))
        assert torch.isfinite(back[:6]).all() and (back[0].double() >= top * (1 - 2.0 ** -4)).all()
        assert float(back[1, 3].double()) <= -top * (1 - 2.0 ** -4) and float(back[1, 40]) == 1.0
        assert (back[2].double() == tiny).all()
        assert back[4, 7] == 448.0 and int(s[4, 0]) == 127 and int(s[5, 0]) == 128 and int(s[4, 1]) == 0
        assert torch.isnan(back[6, :32]).all() and (back[6, 32:] == 0).all()
        assert torch.isnan(back[7, 32:]).all() and back[7, 0] == 3.0
        assert back[9, 1] == 0.0
        r = f32(10)
        mp.mp_pack8(q, r, x)
        R.check_row8(q, r, x.double(), None, str(dtype))
        mp.mp_unpack8(back, q, r)
        assert torch.isnan(back[6]).all() and torch.isnan(back[7]).all() and (back[8] == 0).all()


def test_unpack_every_byte(mp):  # noqa: F811
    q = torch.arange(256, dtype=torch.uint8, device="cuda").view(8, 32)
    for e in (0, 1, 100, 127, 140, 255):
        s = torch.full((8, 1), e, dtype=torch.uint8, device="cuda")
        x = f32(8, 32)
        mp.mp_unpack8(x, q, s)
        R.assert_within(x, R.unpack(q, s), torch.zeros(8, 32, device="cuda", dtype=torch.float64), str(e))


# --- the gated activation -----------------------------------------------------------------

def gated_case(mp, rows, d, dtype, act, *, up=True, fused=True, pad=0, off=0, std=2.0, seed=2, stream=None):
    g = gen(seed)
    what = f"{rows}x{d} {dtype} {act}"
    if fused and up:
        both = placed(randn((rows, 2 * d), g, std, dtype), pad, off)
        a, b = both[:, :d], both[:, d:]
    else:
        a, b = placed(randn((rows, d), g, std, dtype), pad, off), placed(randn((rows, d), g, std, dtype), pad, off)
    b = b if up else None
    y = Guarded(rows, d, dtype, pad, off)
    a8, b8 = Guarded8(rows, d, pad, off), Guarded8(rows, d, pad, off)
    sa, sb = scales(rows, d, "block"), scales(rows, d, "block")
    kept = dict(gate8=a8.view, gate8_scale=sa, **(dict(up8=b8.view, up8_scale=sb) if up else {}))
    mp.mp_gated_forward(y.view, a, b, activation=act, stream=stream, **kept)
    plain = torch.empty_like(y.view)
    mp.mp_gated_forward(plain, a, b, activation=act, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(plain, y.view)
    ref, tol = R.gated(None, a.double(), None if b is None else b.double(), act)
    R.assert_within(y.view, ref["y"], R.rounded(ref["y"], tol["y"], dtype), what + " y")
    R.check_block8(contiguous8(a8.view), sa, a.double(), 0.0 * ref["y"], dtype, what + " gate8")
    if up:
        R.check_block8(contiguous8(b8.view), sb, b.double(), 0.0 * ref["y"], dtype, what + " up8")
    dy = placed(randn((rows, d), g, 1.0, dtype), pad, off)
    for k in (False, True):
        da, db, y2 = (Guarded(rows, d, dtype, pad, off) for _ in range(3))
        if k:
            src = (a8.view, b8.view if up else None, dict(gate_scale=sa, up_scale=sb if up else None))
            ad, bd = R.unpack(contiguous8(a8.view), sa), R.unpack(contiguous8(b8.view), sb) if up else None
        else:
            src, ad, bd = (a, b, {}), a.double(), b.double() if up else None
        mp.mp_gated_backward(da.view, db.view if up else None, dy, src[0], src[1], activation=act, y=y2.view,
                             stream=stream, **src[2])
        torch.cuda.synchronize()
        ref, tol = R.gated(dy, ad, bd, act)
        for name, got in (("dgate", da), ("y", y2)) + ((("dup", db),) if up else ()):
            R.assert_within(got.view, ref[name], R.rounded(ref[name], tol[name], dtype), f"{what} {name} kept={k}")
            got.check(name)
    for o in (y, a8, b8):
        o.check("outputs")


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_gated_shapes(mp, rows, d, act, dtype):  # noqa: F811
    gated_case(mp, rows, d, dtype, act)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("up,fused", [(False, False), (True, False)])
@pytest.mark.parametrize("d", [64, 1000, 2731, 14336])
def test_gated_forms(mp, d, up, fused, act, dtype):  # noqa: F811
    gated_case(mp, 6, d, dtype, act, up=up, fused=fused)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [64, 1600, 2731])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_gated_strides_and_alignment(mp, d, dtype, pad, off):  # noqa: F811
    gated_case(mp, 13, d, dtype, "silu", pad=pad, off=off)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_far_out(mp, act):  # noqa: F811
    a = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 60.0, -60.0, 100.0, -100.0, 1e10, -1e10, 1e30, -1e30,
                       3e38, -3e38, INF, -INF, math.nan]], device="cuda")
    n = a.shape[1]
    b, dy = torch.full_like(a, 0.5), torch.full_like(a, 2.0)
    y, da, db = (torch.empty_like(a) for _ in range(3))
    mp.mp_gated_forward(y, a, b, activation=act)
    mp.mp_gated_backward(da, db, dy, a, b, activation=act)
    fin = slice(0, n - 3)
    ref, tol = R.gated(dy[:, fin], a[:, fin].double(), b[:, fin].double(), act)
    # act(a) overflows nowhere: |act(a)| <= |a|; v beyond fp32 is as good as infinite, sigma 0 or 1
    for name, got in (("y", y), ("dgate", da), ("dup", db)):
        want = torch.where(a[:, fin].abs() > 200, torch.where(a[:, fin] > 0, {
            "y": 0.5 * a, "dgate": torch.ones_like(a), "dup": 2.0 * a}[name][:, fin].double(), 0.0), ref[name])
        lim = torch.where(a[:, fin].abs() > 200, 4 * R.U * want.abs(), tol[name] + R.U * want.abs() + 2.0 ** -117)
        R.assert_within(got[:, fin], want, lim, name)
    assert float(y[0, n - 3]) == INF and torch.isnan(y[0, n - 2]) and torch.isnan(y[0, n - 1])
    assert float(da[0, n - 3]) == 1.0 and torch.isnan(da[0, n - 1])


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [96, 1365])
def test_gated_in_place(mp, d, dtype):  # noqa: F811
    g = gen(6)
    a, b, dy = (randn((11, d), g, 1.0, dtype) for _ in range(3))
    y, da, db, y2 = (torch.empty_like(a) for _ in range(4))
    mp.mp_gated_forward(y, a, b)
    for k in (0, 1):
        t = [a.clone(), b.clone()]
        mp.mp_gated_forward(t[k], t[0], t[1])
        assert torch.equal(t[k], y)
    mp.mp_gated_backward(da, db, dy, a, b, y=y2)
    assert torch.equal(y2, y)
    for i, j, k in ((0, 1, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)):  # dgate, dup and y over gate, up and dy
        t = [a.clone(), b.clone(), dy.clone()]
        mp.mp_gated_backward(t[i], t[j], t[2], t[0], t[1], y=t[k])
        assert torch.equal(t[i], da) and torch.equal(t[j], db) and torch.equal(t[k], y)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_differences(mp, act):  # noqa: F811
    g = gen(9)
    a, b, c = (randn((3, 40), g, 1.5) for _ in range(3))
    da, db = torch.empty_like(a), torch.empty_like(a)
    mp.mp_gated_backward(da, db, c, a, b, activation=act)
    h = 2.0 ** -6

    def fwd(a, b):
        y = torch.empty_like(a)
        mp.mp_gated_forward(y, a, b, activation=act)
        return y.double()

    # elementwise: truncation h^2 / 6 |act'''| (below 2 for both), rounding 40 u |y| / h (|a| below 8)
    size = (c * b).abs().double()
    num = (fwd(a + h, b) - fwd(a - h, b)) * c.double() / (2 * h)
    assert ((num - da.double()).abs() <= size * (2 * h * h / 6 + 40 * R.U * 8 / h)).all()
    num = (fwd(a, b + h) - fwd(a, b - h)) * c.double() / (2 * h)
    assert ((num - db.double()).abs() <= c.abs().double() * (40 * R.U * 8 * (b.abs().double() + 1) / h)).all()


# --- rotary positions ------------------------------------------------------------------------

def heads(tokens, n, dim, g, dtype, extra=0, off=0):
    """[tokens, n, dim] in the middle of rows `extra` wider."""
    buf = torch.full((off + tokens * (n * dim + extra) + 64,), 77.0, device="cuda").to(dtype)
    v = buf[off:off + tokens * (n * dim + extra)].view(tokens, n * dim + extra)[:, :n * dim].view(tokens, n, dim)
    if g is not None:
        v.copy_(randn((tokens, n, dim), g, 1.0, dtype))
    return buf, v


def rope_case(mp, tokens, hq, hk, dim, rot, dtype, *, interleaved=False, inverse=False, extra=0, off=0, far=1000,
              positions=torch.int64, base=10000.0, scaling=None, seed=3, stream=None):
    g = gen(seed)
    turns, factor = mp.mp_rope_frequencies(rot, base, scaling)
    q, k = heads(tokens, hq, dim, g, dtype, extra, off)[1], heads(tokens, hk, dim, g, dtype, extra, off)[1] if hk else None
    (qb, qo), (kb, ko) = heads(tokens, hq, dim, None, dtype, extra, off), heads(tokens, max(hk, 1), dim, None, dtype, extra, off)
    ko = ko if hk else None
    if positions is None:
        first = far
        p = torch.arange(tokens, device="cuda") + first
        given = None
    else:
        first = 0
        p = torch.randint(-5, far, (tokens,), generator=g, device="cuda").to(positions)
        given = p
    mp.mp_rope(qo, q, ko, k, turns, given, first_position=first, interleaved=interleaved, inverse=inverse,
               factor=factor, stream=stream)
    torch.cuda.synchronize()
    for name, x, o, buf in (("q", q, qo, qb),) + ((("k", k, ko, kb),) if hk else ()):
        ref, tol = R.rope(x, turns, p.long(), factor, interleaved, inverse)
        R.assert_within(o[..., :rot], ref[..., :rot], R.rounded(ref, tol, dtype)[..., :rot], f"{name} {tokens}x{dim}/{rot}")
        assert torch.equal(o[..., rot:], x[..., rot:])
        n = o.shape[1] * dim
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[off:off + tokens * (n + extra)].view(tokens, n + extra)[:, :n] = False
        assert (buf[mask] == 77.0).all(), "written outside"
        # over the input
        y = x.clone() if extra == 0 else x
        mp.mp_rope(y, y, None, None, turns, given, first_position=first, interleaved=interleaved, inverse=inverse,
                   factor=factor, stream=stream)
        assert torch.equal(y, o)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [(1, 32, 8, 128, 128), (1, 1, 0, 2, 2), (7, 4, 4, 64, 32),
                                                  (33, 3, 1, 80, 80), (5, 12, 12, 64, 64), (300, 8, 2, 96, 24),
                                                  (19, 2, 1, 6, 4), (1000, 1, 1, 256, 256), (3, 5, 3, 33, 10),
                                                  (700, 2, 2, 128, 126), (2, 64, 64, 128, 64), (2, 1, 1, 1024, 1024)])
def test_rope_shapes(mp, tokens, hq, hk, dim, rot, interleaved, dtype):  # noqa: F811
    rope_case(mp, tokens, hq, hk, dim, rot, dtype, interleaved=interleaved, inverse=tokens % 2 == 0)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("extra,off", [(128, 0), (8, 8), (1, 0), (3, 5), (64, 1)])
def test_rope_strides_and_alignment(mp, extra, off, interleaved, dtype):  # noqa: F811
    rope_case(mp, 9, 4, 2, 64, 48, dtype, interleaved=interleaved, extra=extra, off=off)


@pytest.mark.parametrize("positions", [None, torch.int32, torch.int64])
@pytest.mark.parametrize("far", [1, 131072, (1 << 31) - 5])
def test_rope_positions(mp, positions, far):  # noqa: F811
    rope_case(mp, 40, 2, 2, 128, 128, FF, far=far, positions=positions, base=500000.0,
              scaling=mp.RopeScaling("ramp", 16.0))


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("dim", [8, 16, 40])
def test_rope_any_number_of_pairs(mp, dim, dtype):  # noqa: F811
    for rot in range(2, dim + 1, 2):
        rope_case(mp, 11, 3, 2, dim, rot, dtype, inverse=rot % 4 == 0)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_rope_many_uneven_pairs(mp, dtype):  # noqa: F811
    rope_case(mp, 5, 3, 1, 1024, 1022, dtype)
    rope_case(mp, 2500, 5, 1, 80, 50, dtype)  # several tokens a block, the last one short
    rope_case(mp, 2500, 1, 0, 24, 6, dtype)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("rot", [2, 6, 14, 16, 18, 26, 30, 32])
def test_rope_copied_columns_keep_their_bits(mp, rot, dtype):  # noqa: F811
    """Whatever they hold, and none of it gets into the rotated ones."""
    turns, _ = mp.mp_rope_frequencies(rot, 10000.0)
    g = gen(rot)
    x = randn((70, 3, 32), g, 1.0, dtype)
    bits = x.view(torch.int32 if dtype == FF else torch.int16)
    n = bits[..., rot:].shape
    special = [0x7F800001, -0x00000001, -0x80000000, 0x7F800000, 0x00000001] if dtype == FF else \
        [0x7F81, 0x7C01, -1, -0x8000, 0x7F80, 0x7C00, 1]
    pick = torch.randint(0, len(special), n, generator=g, device=x.device)
    bits[..., rot:] = torch.tensor(special, device=x.device, dtype=torch.int64).to(bits.dtype)[pick]
    clean = x.clone()
    clean[..., rot:] = 0
    o, c = torch.empty_like(x), torch.empty_like(x)
    mp.mp_rope(o, x, None, None, turns, first_position=3)
    mp.mp_rope(c, clean, None, None, turns, first_position=3)
    assert torch.equal(o.view(bits.dtype)[..., rot:], bits[..., rot:])
    assert torch.equal(o[..., :rot], c[..., :rot])
    keep = bits[..., rot:].clone()
    mp.mp_rope(x, x, None, None, turns, first_position=3)
    assert torch.equal(bits[..., rot:], keep) and torch.equal(x[..., :rot], c[..., :rot])


def test_rope_far_positions(mp):  # noqa: F811
    # positions that 32 bits do not hold, and negative ones
    turns, _ = mp.mp_rope_frequencies(64, 10000.0)
    p = torch.tensor([0, -1, 1 << 33, -(1 << 40), (1 << 62) + 12345, -(1 << 63), (1 << 63) - 1], device="cuda")
    x = randn((7, 2, 64), gen(1))
    o = torch.empty_like(x)
    mp.mp_rope(o, x, None, None, turns, p)
    ref, tol = R.rope(x, turns, p, 1.0, False, False)
    R.assert_within(o, ref, R.rounded(ref, tol, FF), "far")
    assert torch.equal(o[0], x[0])
    o2 = torch.empty_like(x[:1])
    mp.mp_rope(o2, x[2:3], None, None, turns, first_position=1 << 33)
    assert torch.equal(o2[0], o[2])


@pytest.mark.parametrize("dtype", [BF, FF])
def test_rope_head_orders(mp, dtype):  # noqa: F811
    # heads with room between them, and heads outermost in memory
    g = gen(2)
    turns, _ = mp.mp_rope_frequencies(32, 10000.0)
    for x in (randn((6, 3, 40), g, 1.0, dtype)[..., :32], randn((3, 6, 32), g, 1.0, dtype).transpose(0, 1),
              randn((3, 6, 33), g, 1.0, dtype)[..., :32].transpose(0, 1)):
        o, c = torch.empty(6, 3, 32, device="cuda", dtype=dtype), torch.empty(6, 3, 32, device="cuda", dtype=dtype)
        mp.mp_rope(o, x, None, None, turns)
        mp.mp_rope(c, x.contiguous(), None, None, turns)
        assert torch.equal(o, c)
        mp.mp_rope(x, x, None, None, turns)
        assert torch.equal(x, c)
    with pytest.raises(ValueError):  # heads that overlap
        mp.mp_rope(o, torch.zeros(1, 1, 32, device="cuda", dtype=dtype).expand(6, 3, 32), None, None, turns)


def test_rope_is_a_rotation(mp):  # noqa: F811
    # inverse undoes it, and is its transpose: <rope x, z> = <x, inverse z>
    g = gen(5)
    turns, _ = mp.mp_rope_frequencies(96, 10000.0)
    p = torch.randint(0, 1 << 20, (50,), generator=g, device="cuda")
    for inter in (False, True):
        x, z = randn((50, 3, 128), g), randn((50, 3, 128), g)
        y, back, t = (torch.empty_like(x) for _ in range(3))
        mp.mp_rope(y, x, None, None, turns, p, interleaved=inter)
        mp.mp_rope(back, y, None, None, turns, p, interleaved=inter, inverse=True)
        mp.mp_rope(t, z, None, None, turns, p, interleaved=inter, inverse=True)
        size = x.abs() + y.abs()
        i = torch.arange(48, device="cuda")
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 48)
        pair = size.clone()
        pair[..., a] = pair[..., b] = size[..., a] + size[..., b]
        assert ((back - x).abs() <= 20 * R.U * pair).all()
        lhs, rhs = (y.double() * z.double()).sum((1, 2)), (x.double() * t.double()).sum((1, 2))
        assert ((lhs - rhs).abs() <= 20 * R.U * (pair.double() * (z.abs() + t.abs()).double()).sum((1, 2))).all()


# --- each matrix on a place of its own, rows far apart -------------------------------------------

def somewhere(t, k):
    """A copy of a matrix at the k-th of several kinds of places; bytes for 8-bit rows."""
    pad, off = ((0, 0), (8, 8), (1, 0), (3, 5), (16, 16), (2, 2), (0, 1))[k % 7]
    return placed(t, pad, off)


def like8(rows, d, k):
    pad, off = ((0, 0), (8, 8), (1, 0), (3, 5), (16, 16), (2, 2), (0, 1))[k % 7]
    return Guarded8(rows, d, pad, off)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [64, 200, 1360, 1365, 4096])
@pytest.mark.parametrize("k", range(7))
def test_unlike_places(mp, k, d, dtype):  # noqa: F811
    g = gen(k)
    rows = 11
    vals = [randn((rows, d), g, 1.0, dtype) for _ in range(4)]
    x, res, dy, dh = (somewhere(v, k + i) for i, v in enumerate(vals))
    w = randn((d + 1,), g, 1.0, dtype)[k % 2:][:d]
    h, y, rstd = somewhere(vals[0], k + 4), somewhere(vals[0], k + 5), f32(rows)
    h8, y8, hs, ys = like8(rows, d, k + 6), like8(rows, d, k + 1), scales(rows, d, "block"), scales(rows, d, "row")
    mp.mp_rmsnorm_forward(y, x, w, residual=res, h=h, rstd=rstd, y8=y8.view, y8_scale=ys, h8=h8.view, h8_scale=hs)
    stored = (vals[0].float() + vals[1].float()).to(dtype)
    (ry, rr), (ty, tr) = R.rms_forward(stored, w, 1e-5)
    assert torch.equal(h, stored)
    R.assert_within(y, ry, R.rounded(ry, ty, dtype), "y")
    R.assert_within(rstd, rr, tr, "rstd")
    R.check_row8(contiguous8(y8.view), ys, ry, ty, "y8")
    R.check_block8(contiguous8(h8.view), hs, stored.double(), 0.0 * ry, dtype, "h8")
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    for src, sc, hd in ((h, None, stored.double()), (h8.view, hs, R.unpack(contiguous8(h8.view), hs))):
        dx, dw = somewhere(vals[0], k + 3), torch.empty_like(w)
        mp.mp_rmsnorm_backward(dx, dw, dy, src, w, rstd, dh=dh, h_scale=sc, workspace=ws)
        (rdx, rdw), (tdx, tdw) = R.rms_backward(vals[2], vals[3], hd, w, rstd)
        R.assert_within(dx, rdx, R.rounded(rdx, tdx, dtype), "dx")
        R.assert_within(dw, rdw, R.rounded(rdw, tdw, dtype), "dweight")
    u8, us = like8(rows, d, k + 2), scales(rows, d, "block")
    mp.mp_gated_forward(y, x, res, gate8=h8.view, gate8_scale=hs, up8=u8.view, up8_scale=us)
    ref, tol = R.gated(None, vals[0].double(), vals[1].double(), "silu")
    R.assert_within(y, ref["y"], R.rounded(ref["y"], tol["y"], dtype), "gated y")
    for a, b, kw, ad, bd in ((x, res, {}, vals[0].double(), vals[1].double()),
                             (h8.view, u8.view, dict(gate_scale=hs, up_scale=us),
                              R.unpack(contiguous8(h8.view), hs), R.unpack(contiguous8(u8.view), us))):
        da, db = somewhere(vals[0], k + 4), somewhere(vals[0], k + 6)
        mp.mp_gated_backward(da, db, dy, a, b, y=y, **kw)
        ref, tol = R.gated(vals[2], ad, bd, "silu")
        for name, got in (("dgate", da), ("dup", db), ("y", y)):
            R.assert_within(got, ref[name], R.rounded(ref[name], tol[name], dtype), name)
    for o in (h8, y8, u8):
        o.check("8 bits")


@pytest.mark.parametrize("d", [1600, 1365])
def test_rows_far_apart(mp, d):  # noqa: F811
    # offsets of elements pass 2^31, of bytes 2^32
    g = gen(20)
    rows, stride = 5, (1 << 29) + 8 * (d % 2 == 0)
    buf = torch.empty(rows * stride, dtype=BF, device="cuda")
    out = torch.empty(rows * stride, dtype=BF, device="cuda")

    def far(t):
        return t.view(rows, stride)[:, :d]

    x, y = far(buf), far(out)
    x.copy_(randn((rows, d), g, 1.0, BF))
    c, want, w = x.contiguous(), torch.empty(rows, d, dtype=BF, device="cuda"), randn((d,), g, 1.0, BF)
    rstd, r2 = f32(rows), f32(rows)
    mp.mp_rmsnorm_forward(y, x, w, rstd=rstd)
    mp.mp_rmsnorm_forward(want, c, w, rstd=r2)
    (ry, _), (ty, _) = R.rms_forward(c, w, 1e-5)
    for got in (y, want):  # of other strides, of other variants: both right
        R.assert_within(got, ry, R.rounded(ry, ty, BF), "y")
    dx, dw = y, f32(d)
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_rmsnorm_backward(dx, dw.to(BF), x, x, w, rstd, workspace=ws)
    (rdx, _), (tdx, _) = R.rms_backward(c, None, c.double(), w, rstd)
    R.assert_within(dx, rdx, R.rounded(rdx, tdx, BF), "dx")
    mp.mp_gated_forward(y, x, x)
    mp.mp_gated_forward(want, c, c)
    assert torch.equal(y, want)
    q, s = torch.empty(rows, d, dtype=E4, device="cuda"), scales(rows, d, "block")
    mp.mp_pack8(q, s, x)
    mp.mp_unpack8(y, q, s)
    q2, s2 = torch.empty(rows, d, dtype=E4, device="cuda"), scales(rows, d, "block")
    mp.mp_pack8(q2, s2, c)
    mp.mp_unpack8(want, q2, s2)
    assert torch.equal(y, want) and torch.equal(s, s2)
    turns, _ = mp.mp_rope_frequencies(64)
    n = d // 64
    mp.mp_rope(y[:, :n * 64].unflatten(1, (n, 64)), x[:, :n * 64].unflatten(1, (n, 64)), None, None, turns,
               first_position=7)
    o = torch.empty(rows, n, 64, dtype=BF, device="cuda")
    mp.mp_rope(o, c[:, :n * 64].reshape(rows, n, 64), None, None, turns, first_position=7)
    assert torch.equal(y[:, :n * 64].unflatten(1, (n, 64)), o)


@pytest.mark.parametrize("rows,d", [(4_500_011, 8), (1_200_013, 5), (70_001, 1100)])
def test_many_rows(mp, rows, d):  # noqa: F811
    """More strips of rows than one dimension of a grid counts: what calls of fewer rows give."""
    g = gen(21)
    part = 60_000  # rows of the calls to compare with
    a, b, dy = (randn((rows, d), g, 1.0, BF) for _ in range(3))

    def rows8():
        return torch.zeros(rows, d, dtype=torch.uint8, device="cuda"), scales(rows, d, "block")

    def calls(r, o):
        mp.mp_gated_forward(o["y"][r], a[r], b[r], gate8=o["a8"][0][r], gate8_scale=o["a8"][1][r], up8=o["b8"][0][r],
                            up8_scale=o["b8"][1][r])
        mp.mp_gated_backward(o["da"][r], o["db"][r], dy[r], a[r], b[r])
        mp.mp_gated_backward(o["ka"][r], o["kb"][r], dy[r], o["a8"][0][r], o["b8"][0][r], gate_scale=o["a8"][1][r],
                             up_scale=o["b8"][1][r])
        mp.mp_pack8(o["q"][0][r], o["q"][1][r], dy[r])
        mp.mp_pack8(o["p"][r], o["s"][r], dy[r])
        mp.mp_unpack8(o["x"][r], o["q"][0][r], o["q"][1][r])
        mp.mp_rmsnorm_forward(o["n"][r], a[r], None, residual=b[r], h=o["h"][r], rstd=o["r"][r])
        mp.mp_rmsnorm_backward(o["dx"][r], None, dy[r], o["h"][r], None, o["r"][r])

    def outputs():
        o = {k: torch.zeros_like(a) for k in ("y", "da", "db", "ka", "kb", "x", "n", "h", "dx")}
        return {**o, "a8": rows8(), "b8": rows8(), "q": rows8(), "p": torch.zeros_like(a, dtype=torch.uint8),
                "s": f32(rows), "r": f32(rows)}

    whole, parts = outputs(), outputs()
    calls(slice(0, rows), whole)
    for i in range(0, rows, part):
        calls(slice(i, min(i + part, rows)), parts)
    for k in ("y", "da", "db", "ka", "kb", "x", "p", "s"):
        assert torch.equal(whole[k], parts[k]), k
    for k in ("a8", "b8", "q"):
        assert torch.equal(whole[k][0], parts[k][0]) and torch.equal(whole[k][1], parts[k][1]), k
    # another number of rows may be summed by another split of a row
    (ry, rr), (ty, tr) = R.rms_forward(whole["h"][-999:], None, 1e-5)
    R.assert_within(whole["n"][-999:], ry, R.rounded(ry, ty, BF), "n")
    R.assert_within(whole["r"][-999:], rr, tr, "rstd")
    (rdx, _), (tdx, _) = R.rms_backward(dy[-999:], None, whole["h"][-999:].double(), None, whole["r"][-999:])
    R.assert_within(whole["dx"][-999:], rdx, R.rounded(rdx, tdx, BF), "dx")
    if d > 1024:  # longer than a head may be
        return
    turns, _ = mp.mp_rope_frequencies(d // 2 * 2)
    o, c, x = (t.view(rows, 1, d) for t in (torch.zeros_like(a), torch.zeros_like(a), a))
    mp.mp_rope(o, x, None, None, turns, first_position=5)
    for i in range(0, rows, part):
        r = slice(i, min(i + part, rows))
        mp.mp_rope(c[r], x[r], None, None, turns, first_position=5 + i)
    assert torch.equal(o, c)


# --- streams, graphs, two at once ---------------------------------------------------------------

def test_on_another_stream(mp):  # noqa: F811
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (s, s.cuda_stream):
        rms_case(mp, 37, 1600, BF, BF, stream=st)
        gated_case(mp, 9, 1365, BF, "silu", stream=st)
        rope_case(mp, 9, 4, 2, 64, 48, BF, stream=st)


def test_captured_and_replayed(mp):  # noqa: F811
    g = gen(12)
    rows, d = 65, 1600
    x, res, dy = (randn((rows, d), g, 1.0, BF) for _ in range(3))
    w = randn((d,), g, 1.0, BF)
    y, h, dx, dw, rstd = (torch.empty_like(t) for t in (x, x, x, w, f32(rows)))
    q, qs = torch.empty(rows, d, dtype=E4, device="cuda"), scales(rows, d, "block")
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    turns, _ = mp.mp_rope_frequencies(64)
    pos = torch.arange(rows, device="cuda")
    r = torch.empty(rows, 25, 64, dtype=BF, device="cuda")
    da, db = torch.empty(rows, d // 2, dtype=BF, device="cuda"), torch.empty(rows, d // 2, dtype=BF, device="cuda")

    def step():
        mp.mp_rmsnorm_forward(y, x, w, residual=res, h=h, rstd=rstd, h8=q, h8_scale=qs)
        mp.mp_rope(r, y.view(rows, 25, 64), None, None, turns, pos)
        mp.mp_rmsnorm_backward(dx, dw, dy, q, w, rstd, h_scale=qs, workspace=ws)
        mp.mp_gated_backward(da, db, dy[:, :d // 2], y[:, :d // 2], y[:, d // 2:])
        return [t.clone() for t in (y, h, rstd, r, dx, dw, da, db)] if not torch.cuda.is_current_stream_capturing() else None

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        x.copy_(randn((rows, d), g, 1.0, BF))
        pos.add_(1000)
        graph.replay()
        got = [t.clone() for t in (y, h, rstd, r, dx, dw, da, db)]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_two_calls_at_once(mp):  # noqa: F811
    g = gen(13)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    sets = []
    for i in range(2):
        rows, d = 3000 + i, 1365 + 3 * i
        x, dy, w = randn((rows, d), g, 1.0, BF), randn((rows, d), g, 1.0, BF), randn((d,), g)
        sets.append((x, dy, w, f32(rows), torch.empty_like(x), torch.empty_like(x), f32(d),
                     torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")))

    def go(s, stream):
        x, dy, w, rstd, y, dx, dw, ws = s
        mp.mp_rmsnorm_forward(y, x, w, rstd=rstd, stream=stream)
        mp.mp_rmsnorm_backward(dx, dw, dy, x, w, rstd, workspace=ws, stream=stream)

    torch.cuda.synchronize()
    alone = []
    for s in sets:
        go(s, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in s[3:7]])
    for _ in range(10):
        go(sets[0], a)
        go(sets[1], b)
    torch.cuda.synchronize()
    for s, want in zip(sets, alone):
        for got, ref in zip(s[3:7], want):
            assert torch.equal(got, ref)
