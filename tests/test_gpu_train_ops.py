"""The training-head operators (layer norm, token log probabilities, top-logit
distillation) against their 64-bit definitions, at the sizes, strides, masks
and values where they can go wrong. Bounds: tests/train_ref.py."""
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


class Guarded:
    """A [rows, cols] view inside a buffer of sentinels, `pad` columns wider
    than a row and starting `off` elements in."""

    def __init__(self, rows, cols, dtype, pad=0, off=0):
        self.buf = torch.full((off + rows * (cols + pad) + 64,), 77.0, dtype=dtype, device="cuda")
        self.view = self.buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False

    def check(self, what):
        assert (self.buf[self.mask] == 77.0).all(), f"{what}: written outside"


def placed(t, pad, off):
    g = Guarded(t.shape[0], t.shape[1], t.dtype, pad, off)
    g.view.copy_(t)
    return g.view


# --- layer norm ----------------------------------------------------------------

LN_SHAPES = [(1, 1), (3, 2), (5, 7), (4, 64), (700, 48), (33, 100), (2, 255), (17, 768), (9, 1000), (5, 1365),
             (300, 1600), (3, 1601), (7, 2048), (4, 4096), (3, 4099), (5, 5120), (3, 8192), (2, 8200), (2, 10007),
             (1, 40000), (2100, 96), (5000, 16), (1300, 8)]


def ln_case(mp, rows, d, dtype, wtype, *, affine=3, pad=0, off=0, shift=0.5, seed=1, eps=1e-5, stream=None):
    g = gen(seed)
    x = placed(randn((rows, d), g, 1.5, dtype) + randn((d,), g, shift, dtype), pad, off)
    dy = placed(randn((rows, d), g, 1.0, dtype), pad, off)
    wb = torch.zeros(2 * d + 1, dtype=wtype, device="cuda")  # at element-aligned places, as in a flat buffer
    wb[1:1 + d] = 1 + randn((d,), g, 0.2)
    wb[1 + d:] = randn((d,), g, 0.3)
    w = wb[1:1 + d] if affine & 1 else None
    b = wb[1 + d:] if affine & 2 else None
    y, mean, rstd = Guarded(rows, d, dtype, pad, off), f32(rows), f32(rows)
    dx, dwb = Guarded(rows, d, dtype, pad, off), torch.full((2 * d + 2,), 77.0, dtype=wtype, device="cuda")
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_forward(y.view, x, w, b, eps, mean=mean, rstd=rstd, stream=stream)
    dw, db = dwb[1:1 + d], dwb[1 + d:1 + 2 * d]
    mp.mp_layernorm_backward(dx.view, dw, db, dy, x, w, mean, rstd, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    (ry, rm, rr), (ty, tm, tr) = R.ln_forward(x, w, b, eps)
    what = f"{rows}x{d} {dtype}"
    R.assert_within(mean, rm, tm, what + " mean")
    R.assert_within(rstd, rr, tr, what + " rstd")
    R.assert_within(y.view, ry, R.rounded(ry, ty, dtype), what + " y")
    (rdx, rdw, rdb), (tdx, tdw, tdb) = R.ln_backward(dy, x, w, mean, rstd)
    R.assert_within(dx.view, rdx, R.rounded(rdx, tdx, dtype), what + " dx")
    R.assert_within(dw, rdw, R.rounded(rdw, tdw, wtype), what + " dweight")
    R.assert_within(db, rdb, R.rounded(rdb, tdb, wtype), what + " dbias")
    y.check("y")
    dx.check("dx")
    assert dwb[0] == 77.0 and dwb[-1] == 77.0


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("rows,d", LN_SHAPES)
def test_layernorm_shapes(mp, rows, d, dtype):
    ln_case(mp, rows, d, dtype, dtype)


@pytest.mark.parametrize("dtype,wtype", [(BF, FF), (FF, BF), (HF, BF), (BF, HF)])
@pytest.mark.parametrize("affine", [0, 1, 2, 3])
def test_layernorm_weight_types(mp, dtype, wtype, affine):
    ln_case(mp, 37, 776, dtype, wtype, affine=affine)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [64, 768, 1600, 4096, 8192, 9000])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_layernorm_strides_and_alignment(mp, dtype, d, pad, off):
    ln_case(mp, 21, d, dtype, dtype, pad=pad, off=off)


@pytest.mark.parametrize("rows", [151, 152, 153, 1216, 1217, 4864, 20001])
@pytest.mark.parametrize("d", [64, 800])
def test_layernorm_row_counts(mp, rows, d):
    ln_case(mp, rows, d, BF, FF)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [3840, 3841, 4096, 4097, 5632, 5633, 7680, 7681, 8191, 8192])
def test_layernorm_register_classes(mp, d, dtype):
    # either side of each change of units a thread; several rounds a block, the last one partly filled
    ln_case(mp, 701, d, dtype, dtype)


@pytest.mark.parametrize("d", [100, 768, 4096])
def test_layernorm_large_offset(mp, d):
    # a common offset a thousand times the spread: two passes lose nothing to cancellation
    ln_case(mp, 12, d, FF, FF, shift=1000.0)


def test_layernorm_constant_rows_and_eps(mp):
    x = torch.full((4, 320), 3.0, device="cuda")
    y, mean, rstd = f32(4, 320), f32(4), f32(4)
    mp.mp_layernorm_forward(y, x, eps=1e-5, mean=mean, rstd=rstd)
    assert (y == 0).all() and (mean == 3).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=3e-7, atol=0)


def test_layernorm_nonfinite_stays_in_its_row(mp):
    g = gen(4)
    x = randn((6, 256), g)
    x[2, 7], x[4, 9] = math.nan, INF
    y = f32(6, 256)
    mp.mp_layernorm_forward(y, x)
    bad = torch.isnan(y).any(1)
    assert bad.tolist() == [False, False, True, False, True, False]


@pytest.mark.parametrize("d", [48, 1600, 9000])
@pytest.mark.parametrize("dtype", [BF, FF])
def test_layernorm_in_place_and_optional_outputs(mp, d, dtype):
    g = gen(3)
    rows = 19
    x, dy, w = randn((rows, d), g, 1.0, dtype), randn((rows, d), g, 1.0, dtype), randn((d,), g, 1.0, dtype)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    mp.mp_layernorm_forward(y, x, w, mean=mean, rstd=rstd)
    x2 = x.clone()
    mp.mp_layernorm_forward(x2, x2, w)  # over its input, no statistics kept
    assert torch.equal(x2, y)
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    mp.mp_layernorm_backward(dx, dw, db, dy, x, w, mean, rstd, workspace=ws)
    only_dx = dy.clone()
    mp.mp_layernorm_backward(only_dx, None, None, only_dx, x, w, mean, rstd)  # over dy
    assert torch.equal(only_dx, dx)
    dw2, db2, dy2 = torch.empty_like(w), torch.empty_like(w), dy.clone()
    mp.mp_layernorm_backward(None, dw2, None, dy, x, w, mean, rstd, workspace=ws)
    mp.mp_layernorm_backward(dy2, None, db2, dy2, x, w, mean, rstd, workspace=ws)
    assert torch.equal(dw2, dw) and torch.equal(db2, db) and torch.equal(dy2, dx)


def test_layernorm_no_rows(mp):
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    mp.mp_layernorm_forward(x.clone(), x)
    dw, db, none = f32(64), f32(64), torch.empty(0, device="cuda")
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_backward(x.clone(), dw, db, x, x, None, none, none, workspace=ws)
    assert (dw == 0).all() and (db == 0).all()


def test_layernorm_differences(mp):
    # dx, dweight and dbias against central differences of the kernel's own forward pass, L = sum(c * y)
    g = gen(8)
    rows, d, h = 3, 24, 2.0 ** -5
    x, c, w, b = randn((rows, d), g), randn((rows, d), g), randn((d,), g), randn((d,), g)
    mean, rstd = f32(rows), f32(rows)

    def fwd(x, w, b):
        y = f32(x.shape[0], d)
        mp.mp_layernorm_forward(y, x.contiguous(), w, b, mean=f32(x.shape[0]), rstd=f32(x.shape[0]))
        return y.double()

    mp.mp_layernorm_forward(f32(rows, d), x, w, b, mean=mean, rstd=rstd)
    dx, dw, db = f32(rows, d), f32(d), f32(d)
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_backward(dx, dw, db, c, x, w, mean, rstd, workspace=ws)
    # truncation h^2/6 times the third derivative (of order |c| |w| rstd^3 sqrt(d)), rounding 200 u sum|c y| / h
    bound = 40 * h * h / 6 * float(c.abs().max() * w.abs().max() * rstd.max() ** 3) + 200 * R.U * 60 / h
    for j in range(d):
        e = torch.zeros(d, device="cuda")
        e[j] = h
        num = ((fwd(x + e, w, b) - fwd(x - e, w, b)) * c.double()).sum(1) / (2 * h)
        assert (num - dx[:, j].double()).abs().max() <= bound
        num = ((fwd(x, w + e, b) - fwd(x, w - e, b)) * c.double()).sum() / (2 * h)
        assert abs(num - dw[j].double()) <= bound
        num = ((fwd(x, w, b + e) - fwd(x, w, b - e)) * c.double()).sum() / (2 * h)
        assert abs(num - db[j].double()) <= bound


# --- token log probabilities -----------------------------------------------------

VOCABS = [1, 2, 7, 31, 64, 100, 257, 1000, 1024, 4099, 32003, 50304, 50261, 128256]


def lp_case(mp, x, targets, scale=1.0, k=0, dentropy=True, seed=5, backward=True, stream=None, status=0):
    rows, vocab = x.shape
    what = f"{rows}x{vocab} {x.dtype}"
    logp, lse, ent = f32(rows), f32(rows), f32(rows)
    tl = f32(rows, k) if k else None
    ti = torch.full((rows, k), -9, dtype=torch.int32, device="cuda") if k else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mp.mp_token_logprob_forward(x, targets, logp=logp, lse=lse, entropy=ent, top_logp=tl, top_index=ti, scale=scale,
                                d_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st) == status
    ref, tol = R.lp_forward(x, targets, scale, k)
    if k:
        assert torch.equal(ti, ref["top_index"]), what + " top_index"
        R.assert_within(tl, ref["top_logp"], tol["top_logp"], what + " top_logp")
    R.assert_within(lse, ref["lse"], tol["lse"], what + " lse")
    R.assert_within(logp, ref["logp"], tol["logp"], what + " logp")
    R.assert_within(ent, ref["entropy"], tol["entropy"], what + " entropy")
    if not backward:
        return logp, lse, ent, tl, ti
    g = gen(seed)
    dlogp = randn((rows,), g)
    dent = randn((rows,), g) if dentropy else None
    dx = Guarded(rows, vocab, x.dtype, x.stride(0) - vocab if rows > 1 else 0, x.storage_offset() % 8)
    mp.mp_token_logprob_backward(dx.view, x, targets, lse=lse, dlogp=dlogp, entropy=ent, dentropy=dent, scale=scale,
                                 stream=stream)
    torch.cuda.synchronize()
    rd, td = R.lp_backward(x, targets, lse, ent, dlogp, dent, scale)
    R.assert_within(dx.view, rd, R.rounded(rd, td, x.dtype), what + " dlogits")
    dx.check("dlogits")
    return logp, lse, ent, tl, ti


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprob_vocabularies(mp, vocab, dtype):
    g = gen(vocab)
    rows = 5
    x = randn((rows, vocab), g, 2.5, dtype)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    t[rows // 2] = -100
    lp_case(mp, x, t, k=min(20, vocab))


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 19, 20, 75, 76, 77, 151, 153, 305, 700])
@pytest.mark.parametrize("vocab", [64, 3000, 50304])
def test_logprob_row_counts(mp, rows, vocab):
    g = gen(rows)
    x = randn((rows, vocab), g, 2.0, BF)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    lp_case(mp, x, t, k=5)


@pytest.mark.parametrize("k", [0, 1, 2, 3, 8, 31, 32])
@pytest.mark.parametrize("rows,vocab", [(3, 40), (2, 777), (3, 32000), (2, 128256)])
def test_logprob_top_counts(mp, k, rows, vocab):
    g = gen(k + 1)
    x = randn((rows, vocab), g, 3.0, BF)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    lp_case(mp, x, t, k=k, backward=False)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("vocab", [70, 2048, 5001, 50304])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_logprob_strides_and_alignment(mp, dtype, vocab, pad, off):
    g = gen(9)
    x = placed(randn((6, vocab), g, 2.0, dtype), pad, off)
    t = torch.randint(0, vocab, (6,), generator=g, device="cuda")
    lp_case(mp, x, t, k=7, scale=0.7)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("vocab", [40, 1000, 20001, 128256])
def test_logprob_masks_and_extremes(mp, dtype, vocab):
    low = torch.finfo(dtype).min
    g = gen(11)
    x = randn((14, vocab), g, 2.0, dtype)
    x[0] = -INF                       # nothing allowed
    x[1, 1:] = -INF                   # one token allowed
    x[2, : vocab // 2] = -INF         # the first half masked
    x[3] = low                        # the type's lowest value everywhere: uniform
    x[4, vocab // 3:] = low           # masked by it
    x[5] = low
    x[5, vocab - 1] = 1.0
    x[6, vocab // 2] = math.nan
    x[7, vocab // 2] = INF
    x[8] = 0.0                        # all equal
    x[9, ::2] = -0.0                  # zeros of both signs are equal
    x[9, 1::2] = 0.0
    x[10] = torch.sort(x[10].float()).values.to(dtype)
    x[11] = torch.sort(x[11].float(), descending=True).values.to(dtype)
    x[12, : vocab - 1] = -INF
    x[13] = (x[13].float() * 2).round().to(dtype) / 2  # few distinct values
    t = torch.tensor([3, 0, 1, 5, 2, vocab - 1, 4, 4, 9, 1, 0, 0, 7, 2], device="cuda")
    logp, lse, ent, tl, ti = lp_case(mp, x, t, k=10)
    assert logp[0] == -INF and lse[0] == -INF and ent[0] == 0
    assert ti[0].tolist() == list(range(10)) and ti[8].tolist() == list(range(10)) and ti[3].tolist() == list(range(10))
    assert abs(float(ent[3]) - math.log(vocab)) < 1e-4 and float(ent[1]) == 0.0 and float(logp[1]) == 0.0
    assert torch.isnan(logp[6]) and torch.isnan(logp[7]) and int(ti[6, 0]) == vocab // 2


@pytest.mark.parametrize("spread", [0.0, 1e-3, 30.0, 1000.0])
def test_logprob_spreads(mp, spread):
    g = gen(12)
    x = randn((4, 9000), g, spread) + 500.0
    t = torch.randint(0, 9000, (4,), generator=g, device="cuda")
    for scale in (0.1, 1.0, 3.0):
        lp_case(mp, x, t, k=4, scale=scale)


def test_logprob_rising_rows(mp):
    # every later value is larger: the running maximum moves at every step
    for vocab in (1000, 40000):
        x = torch.arange(vocab, device="cuda", dtype=FF)[None].repeat(3, 1)
        x[1] = x[1] * 1e-3
        x[2] = x[2].flip(0) * 0.5
        lp_case(mp, x, torch.tensor([vocab - 1, 0, 5], device="cuda"), k=32)


def test_logprob_optional_outputs(mp):
    g = gen(13)
    x = randn((9, 5000), g, 2.0, BF)
    t = torch.randint(0, 5000, (9,), generator=g, device="cuda")
    logp, lse, ent, tl, ti = lp_case(mp, x, t, k=6)
    a, b, c = f32(9), f32(9), f32(9)
    mp.mp_token_logprob_forward(x, t, logp=a)
    mp.mp_token_logprob_forward(x, lse=b)
    mp.mp_token_logprob_forward(x, entropy=c)
    tl2, ti2 = torch.empty_like(tl), torch.empty_like(ti)
    mp.mp_token_logprob_forward(x, top_logp=tl2, top_index=ti2)
    for p, q in ((a, logp), (b, lse), (tl2, tl)):
        assert (p - q).abs().max() <= 1e-5
    assert (c - ent).abs().max() <= 1e-5 and torch.equal(ti, ti2)


def test_logprob_backward_forms(mp):
    g = gen(14)
    rows, vocab = 12, 3000
    x = randn((rows, vocab), g, 2.0, BF)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    t[3] = -1
    logp, lse, ent, _, _ = lp_case(mp, x, t)
    dlogp, dent = randn((rows,), g), randn((rows,), g)
    dlogp[5], dent[5] = 0.0, 0.0
    x[5, 9] = math.nan  # a row of zero gradients is not looked at
    lse[7] = -INF
    full = torch.empty_like(x)
    mp.mp_token_logprob_backward(full, x, t, lse=lse, dlogp=dlogp, entropy=ent, dentropy=dent)
    assert (full[5] == 0).all() and (full[7] == 0).all()
    over = x.clone()
    mp.mp_token_logprob_backward(over, over, t, lse=lse, dlogp=dlogp, entropy=ent, dentropy=dent)
    assert torch.equal(over, full)
    only = torch.empty_like(x)
    mp.mp_token_logprob_backward(only, x, None, lse=lse, entropy=ent, dentropy=dent)
    rd, td = R.lp_backward(x[:5], None, lse[:5], ent[:5], None, dent[:5], 1.0)
    R.assert_within(only[:5], rd, R.rounded(rd, td, BF), "entropy alone")
    mp.mp_token_logprob_backward(only, x, t, lse=lse, dlogp=dlogp)
    rd, td = R.lp_backward(x[:5], t[:5], lse[:5], None, dlogp[:5], None, 1.0)
    R.assert_within(only[:5], rd, R.rounded(rd, td, BF), "logp alone")
    assert (only[3] == 0).all()


def test_logprob_targets_out_of_range(mp):
    g = gen(15)
    x = randn((4, 1000), g, 2.0, BF)
    t = torch.tensor([5, 1000, 1 << 40, -1], device="cuda")
    logp, lse, ent, _, _ = lp_case(mp, x, t, status=mp.MP_ERR_RANGE)
    assert torch.isnan(logp[1:3]).all() and logp[3] == 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx = torch.empty_like(x)
    mp.mp_token_logprob_backward(dx, x, t, lse=lse, dlogp=f32(4, fill=1.0), d_status=st)
    assert int(st) == mp.MP_ERR_RANGE and (dx[1:] == 0).all()


def test_logprob_differences(mp):
    # central differences of the kernel's own forward pass, L = sum(a logp + b entropy)
    g = gen(16)
    rows, vocab, h, scale = 3, 29, 2.0 ** -5, 0.9
    x = randn((rows, vocab), g, 1.5)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    a, b = randn((rows,), g), randn((rows,), g)

    def fwd(x):
        logp, lse, ent = f32(rows), f32(rows), f32(rows)
        mp.mp_token_logprob_forward(x, t, logp=logp, lse=lse, entropy=ent, scale=scale)
        return a.double() * logp.double() + b.double() * ent.double(), lse, ent

    _, lse, ent = fwd(x)
    dx = torch.empty_like(x)
    mp.mp_token_logprob_backward(dx, x, t, lse=lse, dlogp=a, entropy=ent, dentropy=b, scale=scale)
    # third derivatives of logp and entropy are below 1 and 8; forward error below 300 u (1 + |entropy|)
    bound = h * h / 6 * (a.abs() + 8 * b.abs()).double() + 300 * R.U * 5 * (a.abs() + b.abs()).double() / h
    for j in range(vocab):
        e = torch.zeros(vocab, device="cuda")
        e[j] = h
        num = (fwd(x + e)[0] - fwd(x - e)[0]) / (2 * h)
        assert ((num - dx[:, j].double()).abs() <= bound).all()


# --- distillation ------------------------------------------------------------------

def teacher_for(x, K, g, cut=True):
    rows, vocab = x.shape
    idx = torch.rand(rows, vocab, generator=g, device="cuda").topk(K, dim=1).indices
    t = (x.float().nan_to_num(0.0, 0.0, 0.0).gather(1, idx) + torch.randn(rows, K, generator=g, device="cuda")).to(x.dtype)
    if cut and K > 2:
        idx[0, K // 2:] = -1
    return t, idx


def distill_case(mp, x, t, idx, w=None, scale=1.0, stream=None, status=0):
    rows, vocab = x.shape
    loss, dx = f32(rows), Guarded(rows, vocab, x.dtype, x.stride(0) - vocab if rows > 1 else 0, x.storage_offset() % 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mp.mp_distill_topk(loss, dx.view, x, t, idx, row_weight=w, scale=scale, d_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st) == status
    (rl, rd), (tl, td) = R.distill(x, t, idx, w, scale)
    what = f"{rows}x{vocab} K{t.shape[1]} {x.dtype}"
    R.assert_within(loss, rl, tl, what + " loss")
    R.assert_within(dx.view, rd, R.rounded(rd, td, x.dtype), what + " dlogits")
    dx.check("dlogits")
    alone = f32(rows)
    mp.mp_distill_topk(alone, None, x, t, idx, row_weight=w, scale=scale, stream=stream)
    over = x.clone()
    mp.mp_distill_topk(loss, over, over, t, idx, row_weight=w, scale=scale, stream=stream)
    torch.cuda.synchronize()
    R.assert_within(alone, rl, tl, what + " loss alone")
    R.assert_within(over, rd, R.rounded(rd, td, x.dtype), what + " over the logits")
    return loss, dx.view


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill_vocabularies(mp, vocab, dtype):
    g = gen(vocab)
    x = randn((5, vocab), g, 2.5, dtype)
    t, idx = teacher_for(x, min(vocab, 33), g)
    w = torch.tensor([1.0, 0.25, 0.0, -2.0, 3.0], device="cuda")
    distill_case(mp, x, t, idx, w)


@pytest.mark.parametrize("rows", [1, 2, 8, 19, 20, 75, 77, 153, 305, 620])
@pytest.mark.parametrize("vocab", [64, 3000, 50304])
def test_distill_row_counts(mp, rows, vocab):
    g = gen(rows)
    x = randn((rows, vocab), g, 2.0, BF)
    t, idx = teacher_for(x, 20, g)
    distill_case(mp, x, t, idx.int())


@pytest.mark.parametrize("K", [1, 2, 3, 31, 64, 65, 257, 1024])
@pytest.mark.parametrize("vocab", [1500, 50304])
def test_distill_list_lengths(mp, K, vocab):
    g = gen(K)
    x = randn((4, vocab), g, 2.0, BF)
    t, idx = teacher_for(x, K, g)
    distill_case(mp, x, t, idx, scale=0.5)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("vocab", [70, 2048, 5001, 50304])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 1), (1, 0), (3, 5)])
def test_distill_strides_and_alignment(mp, dtype, vocab, pad, off):
    g = gen(19)
    x = placed(randn((6, vocab), g, 2.0, dtype), pad, off)
    t, idx = teacher_for(x, 12, g)
    wide_t, wide_i = placed(t, 3, 1), torch.full((6, 17), -5, device="cuda")
    wide_i[:, 2:14] = idx
    distill_case(mp, x, wide_t, wide_i[:, 2:14], scale=1.5)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("vocab", [60, 3001, 60000, 128256])
def test_distill_masks_and_extremes(mp, dtype, vocab):
    g = gen(21)
    low = torch.finfo(dtype).min
    x = randn((13, vocab), g, 2.0, dtype)
    t, idx = teacher_for(x, 20, g, cut=False)
    idx[0] = -1                                   # nothing listed
    t[1] = -INF                                   # nothing of q > 0
    t[2, 3:] = -INF                               # three of them
    x[3] = -INF                                   # the student's row is empty
    x[4, idx[4, 0]] = -INF                        # a listed token the student masks
    x[5] = low                                    # uniform at the type's lowest value
    x[6, : vocab // 2] = -INF
    idx[6] = vocab // 2 + torch.arange(20, device="cuda") % (vocab - vocab // 2)
    idx[7] = 11                                   # one token listed twenty times
    idx[8, :6] = idx[8, 6:12]                     # some listed twice
    x[9, vocab // 2] = math.nan
    x[10, 1] = INF
    t[11, 2] = math.nan
    x[12, 5], t[12, 0] = math.nan, 1.0            # a row of weight 0 is not looked at
    w = torch.ones(13, device="cuda")
    w[12] = 0.0
    loss, dx = distill_case(mp, x, t, idx, w)
    assert loss[0] == 0 and loss[1] == 0 and loss[12] == 0 and loss[3] == INF and loss[4] == INF
    assert (dx[0] == 0).all() and (dx[1] == 0).all() and (dx[3] == 0).all() and (dx[12] == 0).all()
    assert torch.isnan(loss[9:12]).all()


@pytest.mark.parametrize("dtype,vocab,pad", [(BF, 32768, 0), (BF, 50304, 24), (HF, 50261, 3), (BF, 128256, 0),
                                             (FF, 60001, 0), (FF, 128256, 4), (BF, 180007, 1)])
def test_distill_many_long_rows(mp, dtype, vocab, pad):
    g = gen(25)
    rows = 470
    x = placed(randn((rows, vocab), g, 2.0, dtype), pad, 8)
    t, idx = teacher_for(x, 40, g)
    low = torch.finfo(dtype).min
    w = torch.rand(rows, generator=g, device="cuda") + 0.5
    w[5:9] = 0.0                       # rows of weight 0, several in one block's turn too
    w[150:460:152] = 0.0
    w[151:460:152] = 0.0
    w[7] = -1.5
    idx[10] = -1
    t[11] = -INF
    x[12] = -INF
    x[13, idx[13, 1]] = -INF
    x[14] = low
    idx[15] = 11
    idx[16, :6] = idx[16, 6:12]
    x[17, vocab // 2] = math.nan
    t[18, 2] = math.nan
    x[19, : vocab // 2] = -INF
    idx[20, 0], idx[20, 1], idx[20, 2] = 0, vocab - 1, vocab - 2  # the ends of the row
    x[21] = torch.sort(x[21].float()).values.to(dtype)
    x[6, 3] = math.nan                 # of weight 0
    distill_case(mp, x, t, idx, w, scale=0.75)
    big_t, big_i = teacher_for(x, 256, g)
    distill_case(mp, x, big_t, big_i.int(), None)


def test_distill_index_out_of_range(mp):
    g = gen(22)
    x = randn((3, 500), g, 2.0, BF)
    t, idx = teacher_for(x, 8, g, cut=False)
    idx[1, 2] = 500
    idx[2, 0] = 1 << 50
    loss, dx = distill_case(mp, x, t, idx, status=mp.MP_ERR_RANGE)
    assert torch.isnan(loss[1:]).all() and not torch.isnan(loss[0]) and not torch.isnan(dx).any()


def test_distill_of_one_token_is_cross_entropy(mp):
    g = gen(23)
    rows, vocab = 7, 4000
    x = randn((rows, vocab), g, 2.0, FF)
    tgt = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    loss, dx = distill_case(mp, x, torch.zeros(rows, 1, device="cuda"), tgt[:, None])
    logp, lse, _, _, _ = lp_case(mp, x, tgt)
    dx2 = torch.empty_like(x)
    mp.mp_token_logprob_backward(dx2, x, tgt, lse=lse, dlogp=f32(rows, fill=-1.0))
    # both are within their bounds of the same value
    assert (loss + logp).abs().max() <= 1e-5 and (dx - dx2).abs().max() <= 1e-5


def test_distill_differences(mp):
    # central differences of the kernel's own loss
    g = gen(24)
    rows, vocab, h, scale = 3, 31, 2.0 ** -5, 0.8
    x = randn((rows, vocab), g, 1.5)
    t, idx = teacher_for(x, 6, g)
    w = torch.tensor([1.0, 2.0, 0.5], device="cuda")

    def fwd(x):
        loss = f32(rows)
        mp.mp_distill_topk(loss, None, x, t, idx, row_weight=w, scale=scale)
        return loss.double()

    dx = torch.empty_like(x)
    mp.mp_distill_topk(f32(rows), dx, x, t, idx, row_weight=w, scale=scale)
    bound = (h * h / 6 + 300 * R.U * 8 / h) * w.double()
    for j in range(vocab):
        e = torch.zeros(vocab, device="cuda")
        e[j] = h
        num = (fwd(x + e) - fwd(x - e)) / (2 * h)
        assert ((num - dx[:, j].double()).abs() <= bound).all()


# --- all of them --------------------------------------------------------------------

def test_offsets_past_32_bits(mp):
    """Rows that start more than 2^32 elements apart."""
    stride = (1 << 32) + 24
    g = gen(30)
    for vocab in (3000, 50304):
        big = torch.empty(stride + vocab, dtype=BF, device="cuda")
        x = big.as_strided((2, vocab), (stride, 1))
        x.copy_(randn((2, vocab), g, 2.0, BF))
        t, idx = teacher_for(x, 9, g)
        c = x.contiguous()
        tgt = torch.tensor([5, vocab - 1], device="cuda")
        outs = []
        for m in (x, c):
            logp, lse, ent, tl, ti = f32(2), f32(2), f32(2), f32(2, 8), torch.empty(2, 8, dtype=torch.int32, device="cuda")
            mp.mp_token_logprob_forward(m, tgt, logp=logp, lse=lse, entropy=ent, top_logp=tl, top_index=ti)
            y = torch.empty_like(c)
            mp.mp_layernorm_forward(y, m, mean=f32(2), rstd=f32(2))
            loss, dx, dl = f32(2), torch.empty_like(c), torch.empty_like(c)
            mp.mp_distill_topk(loss, dx, m, t, idx)
            mp.mp_token_logprob_backward(dl, m, tgt, lse=lse, dlogp=f32(2, fill=1.0))
            outs.append((logp, lse, ent, tl, ti, y, loss, dx, dl))
        for p, q in zip(*outs):
            assert torch.equal(p, q)
        over = x.clone()
        mp.mp_distill_topk(f32(2), x, x, t, idx)  # the gradient over the far rows
        assert torch.equal(x, outs[1][7])
        del big, x, over


def test_other_stream(mp):
    s = torch.cuda.Stream()
    g = gen(31)
    x = randn((300, 5000), g, 2.0, BF)
    t, idx = teacher_for(x, 9, g)
    tgt = torch.randint(0, 5000, (300,), generator=g, device="cuda")
    torch.cuda.synchronize()
    lp_case(mp, x, tgt, k=3, stream=s)
    distill_case(mp, x, t, idx, stream=s)
    x = randn((400, 40000), g, 2.0, BF)
    t, idx = teacher_for(x, 9, g)
    torch.cuda.synchronize()
    distill_case(mp, x, t, idx, stream=s)
    ln_case(mp, 300, 768, BF, BF, stream=s)


def test_same_bits_on_every_run(mp):
    g = gen(32)
    for rows, vocab in ((1, 128256), (40, 50304), (700, 5001)):
        x = randn((rows, vocab), g, 2.0, BF)
        t, idx = teacher_for(x, 16, g)
        idx[:, 0] = idx[:, 5]
        tgt = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        w, dy = randn((vocab,), g, 1.0, BF), randn((rows, vocab), g, 1.0, BF)
        first = None
        for _ in range(3):
            logp, lse, ent, tl = f32(rows), f32(rows), f32(rows), f32(rows, 8)
            ti = torch.empty(rows, 8, dtype=torch.int32, device="cuda")
            mp.mp_token_logprob_forward(x, tgt, logp=logp, lse=lse, entropy=ent, top_logp=tl, top_index=ti)
            loss, dx = f32(rows), torch.empty_like(x)
            mp.mp_distill_topk(loss, dx, x, t, idx)
            mean, rstd, y, dl = f32(rows), f32(rows), torch.empty_like(x), torch.empty_like(x)
            mp.mp_layernorm_forward(y, x, w, mean=mean, rstd=rstd)
            dw, db = f32(vocab).to(BF), f32(vocab).to(BF)
            ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, vocab), dtype=torch.uint8, device="cuda")
            mp.mp_layernorm_backward(dl, dw, db, dy, x, w, mean, rstd, workspace=ws)
            got = (logp, lse, ent, tl, ti, loss, dx, y, mean, rstd, dl, dw, db)
            first = got if first is None else first
            assert all(torch.equal(p, q) for p, q in zip(got, first))


def test_in_a_graph(mp):
    """Captured once, replayed on new inputs in the same buffers."""
    g = gen(33)
    rows, vocab, d = 30, 4000, 768
    x, h = randn((rows, vocab), g, 2.0, BF), randn((rows, d), g, 1.0, BF)
    t, idx = teacher_for(x, 9, g)
    y, mean, rstd = torch.empty_like(h), f32(rows), f32(rows)
    loss, dx, logp, lse = f32(rows), torch.empty_like(x), f32(rows), f32(rows)
    tgt = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tl, ti = f32(rows, 4), torch.empty(rows, 4, dtype=torch.int32, device="cuda")
    dw = f32(d)
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    dh = torch.empty_like(h)

    def step():
        mp.mp_layernorm_forward(y, h, mean=mean, rstd=rstd)
        mp.mp_layernorm_backward(dh, dw, None, y, h, None, mean, rstd, workspace=ws)
        mp.mp_distill_topk(loss, dx, x, t, idx)
        mp.mp_token_logprob_forward(x, tgt, logp=logp, lse=lse, top_logp=tl, top_index=ti)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(randn((rows, vocab), g, 2.0, BF))
    h.copy_(randn((rows, d), g, 1.0, BF))
    graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in (y, dh, dw, loss, dx, logp, lse, tl, ti)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, (y, dh, dw, loss, dx, logp, lse, tl, ti)))


# --- inputs and outputs of unlike alignment ---------------------------------------

def among_nan(t, off, pad=8):
    """t at an offset of `off` elements, between NaNs: an element used from
    beyond a row shows."""
    rows, cols = t.shape
    buf = torch.full((off + rows * (cols + pad) + 64,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("vocab", [1, 8, 15, 16, 22, 23, 24, 31, 70, 1029, 8200])
@pytest.mark.parametrize("pad", [8, 3])
def test_softmax_gradients_of_unlike_alignment(mp, vocab, dtype, pad):
    # with pad 3 the alignment changes from row to row as well
    g = gen(vocab)
    rows = 9
    x = randn((rows, vocab), g, 2.0, dtype)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    lt, idx = teacher_for(x, min(vocab, 6), g)
    dlogp, dent = randn((rows,), g), randn((rows,), g)
    for off in range(8):
        for out in (0, 1, 2, 5):
            what = f"{vocab} {dtype} at {off} -> {out}"
            xs = among_nan(x, off, pad)
            logp, lse, ent = f32(rows), f32(rows), f32(rows)
            mp.mp_token_logprob_forward(xs, t, logp=logp, lse=lse, entropy=ent)
            dx = Guarded(rows, vocab, dtype, 8, out)
            mp.mp_token_logprob_backward(dx.view, xs, t, lse=lse, dlogp=dlogp, entropy=ent, dentropy=dent)
            rd, td = R.lp_backward(x, t, lse, ent, dlogp, dent, 1.0)
            R.assert_within(dx.view, rd, R.rounded(rd, td, dtype), "log probabilities " + what)
            dx.check("dlogits")
            loss, dx = f32(rows), Guarded(rows, vocab, dtype, 8, out)
            mp.mp_distill_topk(loss, dx.view, xs, lt, idx)
            (rl, rd), (tl, td) = R.distill(x, lt, idx, None, 1.0)
            R.assert_within(loss, rl, tl, "loss " + what)
            R.assert_within(dx.view, rd, R.rounded(rd, td, dtype), "distillation " + what)
            dx.check("dlogits")


@pytest.mark.parametrize("rows", [77, 400])
def test_distill_unlike_alignment_many_rows(mp, rows):
    g = gen(rows)
    x = randn((rows, 20001), g, 2.0, BF)
    lt, idx = teacher_for(x, 33, g)
    loss, dx = f32(rows), Guarded(rows, 20001, BF, 7, 0)
    mp.mp_distill_topk(loss, dx.view, among_nan(x, 3, 2), lt, idx)
    (rl, rd), (tl, td) = R.distill(x, lt, idx, None, 1.0)
    R.assert_within(loss, rl, tl, "loss")
    R.assert_within(dx.view, rd, R.rounded(rd, td, BF), "dlogits")
    dx.check("dlogits")


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("d", [60, 257, 1365, 4100])
@pytest.mark.parametrize("pad", [8, 5])
def test_layernorm_unlike_alignment(mp, d, dtype, pad):
    g = gen(d)
    rows = 37
    x, dy, w, b = (randn(s, g, 1.0, dtype) for s in ((rows, d), (rows, d), (d,), (d,)))
    for off, off_dy, out in ((0, 1, 0), (1, 0, 0), (3, 6, 1), (0, 0, 5)):
        y, dx = Guarded(rows, d, dtype, pad, out), Guarded(rows, d, dtype, 8, (out + 3) % 8)
        mean, rstd, dw, db = f32(rows), f32(rows), torch.empty_like(w), torch.empty_like(b)
        ws = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
        xs, dys = among_nan(x, off, pad), among_nan(dy, off_dy, 8)
        mp.mp_layernorm_forward(y.view, xs, w, b, mean=mean, rstd=rstd)
        mp.mp_layernorm_backward(dx.view, dw, db, dys, xs, w, mean, rstd, workspace=ws)
        (ry, rm, rr), (ty, tm, tr) = R.ln_forward(x, w, b, 1e-5)
        (rdx, rdw, rdb), (tdx, tdw, tdb) = R.ln_backward(dy, x, w, mean, rstd)
        for got, ref, tol, what in ((y.view, ry, ty, "y"), (dx.view, rdx, tdx, "dx"), (dw, rdw, tdw, "dweight"),
                                    (db, rdb, tdb, "dbias")):
            R.assert_within(got, ref, R.rounded(ref, tol, dtype), f"{what} {d} {dtype} {off} {off_dy} {out}")
        y.check("y")
        dx.check("dx")


def test_binding_refusals(mp):
    x = torch.zeros(4, 8, dtype=BF, device="cuda")
    v, i = f32(4), torch.zeros(4, dtype=torch.int64, device="cuda")
    ws = torch.empty(mp.mp_layernorm_workspace_bytes(4, 8), dtype=torch.uint8, device="cuda")
    for error, fn in (
            (TypeError, lambda: mp.mp_layernorm_forward(x.float(), x)),
            (ValueError, lambda: mp.mp_layernorm_forward(x[:3], x)),
            (ValueError, lambda: mp.mp_layernorm_forward(x.clone(), x.t().contiguous().t())),
            (ValueError, lambda: mp.mp_layernorm_forward(x[:1].expand(4, 8), x)),
            (ValueError, lambda: mp.mp_layernorm_forward(x[0], x[0])),
            (ValueError, lambda: mp.mp_layernorm_forward(x.clone(), x, f32(7))),
            (TypeError, lambda: mp.mp_layernorm_forward(x.clone(), x, f32(8), f32(8).half())),
            (TypeError, lambda: mp.mp_layernorm_forward(x.clone(), x, mean=v.double())),
            (ValueError, lambda: mp.mp_layernorm_forward(x.clone(), x, mean=f32(8)[::2])),
            (mp.MpError, lambda: mp.mp_layernorm_backward(x.clone(), f32(8), None, x, x, None, v, v)),
            (mp.MpError, lambda: mp.mp_layernorm_backward(x.clone(), f32(8), None, x, x, None, v, v, workspace=ws[:4])),
            (TypeError, lambda: mp.mp_token_logprob_forward(x, v, logp=v)),
            (mp.MpError, lambda: mp.mp_token_logprob_forward(x, i)),
            (ValueError, lambda: mp.mp_token_logprob_forward(x, i, logp=v, top_logp=f32(4, 2))),
            (ValueError, lambda: mp.mp_token_logprob_forward(x, i[:3], logp=v)),
            (mp.MpError, lambda: mp.mp_token_logprob_forward(x, i, logp=v, scale=0.0)),
            (mp.MpError, lambda: mp.mp_token_logprob_backward(x.clone(), x, i, lse=v)),
            (TypeError, lambda: mp.mp_distill_topk(v, None, x, x.float(), i[:, None])),
            (ValueError, lambda: mp.mp_distill_topk(v, None, x, x, i[:, None])),
            (ValueError, lambda: mp.mp_distill_topk(v, None, x, x[:3], torch.zeros(3, 8, dtype=torch.int64, device="cuda"))),
            (ValueError, lambda: mp.mp_distill_topk(v.cpu(), None, x, x, torch.zeros(4, 8, dtype=torch.int64, device="cuda")))):
        with pytest.raises(error):
            fn()
