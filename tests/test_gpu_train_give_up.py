"""What the staged kernels leave when a wait for a copy runs out. No wait does
on a working GPU, so the kernels are compiled a second time with a limit of
0: a wait whose copy has not landed when it begins gives up. Every access stays in
bounds then (no index is read from what has not arrived), every wait still
ends, and copies in flight land before a block ends. A row that was given up
has to show it: what is not NaN has to be right."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

BF, FF = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from mixed_precision_adamw_gb300 import build as B
    out = tmp_path_factory.mktemp("short_waits")
    sources = [os.path.join(os.path.dirname(os.path.abspath(__file__)), "short_waits.cu"),
               os.path.join(B.CSRC, "mp_layernorm.cu"), os.path.join(B.CSRC, "mp_distill.cu")]

    def compile(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        subprocess.run([B.nvcc(), *B.NVCC_FLAGS, "-DMP_WAIT_LIMIT_NS=0", "-c", src, "-o", obj], check=True,
                       capture_output=True)
        return obj

    with ThreadPoolExecutor() as ex:
        objs = list(ex.map(compile, sources))
    lib = str(out / "short_waits.so")
    subprocess.run([B.nvcc(), "-shared", *B.GENCODE, "-o", lib, *objs], check=True, capture_output=True)
    return ctypes.CDLL(lib)


def ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def i64(*v):
    return [ctypes.c_int64(x) for x in v]


def right_or_nan(got, ref, tol, what):
    """Elements that are not NaN are within the bound; returns whether some are NaN."""
    nan = torch.isnan(got)
    ok = nan | ((got.double() - ref).abs() <= tol)
    assert ok.all(), f"{what}: {int((~ok).sum())} wrong elements are not NaN"
    return bool(nan.any())


def test_layernorm_gives_up(short):
    # which waits give up depends on the copies' time: some of all these do
    gave = [layernorm_case(short, rows, d, pad, dtype) for dtype in (BF, FF)
            for rows, d, pad in ((20000, 1600, 0), (9001, 1357, 1), (3000, 8192, 0))]
    for which, name in enumerate(("y", "mean", "dx", "dweight", "dbias")):
        assert any(v[which] for v in gave), f"{name}: no wait gave up"


def layernorm_case(short, rows, d, pad, dtype):
    """Checks one size and type; which of y, mean, dx, dweight and dbias hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x, dy = (torch.randn(rows, d + pad, generator=g, device="cuda").to(dtype)[:, :d] for _ in range(2))
    w, b = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    y, dx = (torch.full((rows, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    mean, rstd, m2, r2 = (torch.full((rows,), 7.0, device="cuda") for _ in range(4))
    dw, db = (torch.full((d,), 7.0, device="cuda") for _ in range(2))
    short.mp_layernorm_workspace_bytes.restype = ctypes.c_size_t
    n = short.mp_layernorm_workspace_bytes(*i64(rows, d))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    code = ctypes.c_int32(0 if dtype == BF else 2)
    xd = x.double()
    m2.copy_(xd.mean(1))
    r2.copy_(1 / torch.sqrt(xd.var(1, unbiased=False) + 1e-5))
    (ry, rm, rr), (ty, tm, tr) = R.ln_forward(x, w, b, 1e-5)
    # the forward pass's copies are mostly there when they are waited for: it runs beside others that keep HBM busy
    big, side = torch.ones(1 << 31, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    gave_y = gave_mean = False
    for _ in range(20):
        for t in (y, mean, rstd):
            t.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big.add_(1)
        assert short.mp_layernorm_forward(ptr(y), ptr(mean), ptr(rstd), ptr(x), ptr(w), ptr(b),
                                          *i64(rows, d, d, d + pad), ctypes.c_float(1e-5), code, ctypes.c_int32(2),
                                          None) == 0
        torch.cuda.synchronize()
        gave_y = right_or_nan(y, ry, R.rounded(ry, ty, dtype), "y") or gave_y
        gave_mean = right_or_nan(mean, rm, tm, "mean") or gave_mean
        right_or_nan(rstd, rr, tr, "rstd")
        if gave_y and gave_mean:
            break
    assert short.mp_layernorm_backward(ptr(dx), ptr(dw), ptr(db), ptr(dy), ptr(x), ptr(w), ptr(m2), ptr(r2),
                                       *i64(rows, d, d, d + pad, d + pad), code, ctypes.c_int32(2), ptr(ws),
                                       ctypes.c_size_t(n), None) == 0
    torch.cuda.synchronize()
    (rdx, rdw, rdb), (tdx, tdw, tdb) = R.ln_backward(dy, x, w, m2, r2)
    return (gave_y, gave_mean, right_or_nan(dx, rdx, R.rounded(rdx, tdx, dtype), "dx"),
            right_or_nan(dw, rdw, R.rounded(rdw, tdw, FF), "dweight"),
            right_or_nan(db, rdb, R.rounded(rdb, tdb, FF), "dbias"))


@pytest.mark.parametrize("dtype,vocab,in_place", [(BF, 50304, False), (BF, 128256, True), (FF, 60000, True)])
def test_distill_gives_up(short, dtype, vocab, in_place):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows, k = 470, 40
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 2).to(dtype)
    idx = torch.rand(rows, vocab, generator=g, device="cuda").topk(k, dim=1).indices
    t = torch.randn(rows, k, generator=g, device="cuda").to(dtype)
    w = torch.rand(rows, generator=g, device="cuda") + 0.5
    w[::7] = 0.0
    (rl, rd), (tl, td) = R.distill(x, t, idx, w, 1.0)
    logits = x.clone()
    dx = logits if in_place else torch.full_like(x, 7.0)
    loss, status = torch.full((rows,), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.full((1 << 29,), 1, dtype=torch.uint8, device="cuda")  # x is not in L2: loads take their time
    torch.cuda.synchronize()
    args = (ptr(x if not in_place else logits), ptr(t), ptr(idx), ptr(w), *i64(rows, vocab), ctypes.c_int32(k),
            *i64(vocab, vocab, k, k), ctypes.c_float(1.0), ctypes.c_int32(0 if dtype == BF else 2), ctypes.c_int32(1))
    assert short.mp_distill_topk(ptr(loss), ptr(dx), *args, ptr(status), None) == 0
    torch.cuda.synchronize()
    gave = torch.isnan(loss)
    assert gave.any() and int(status) == 6, "no wait gave up"
    assert torch.isnan(dx[gave, 0]).all(), "a row that gave up has a gradient that looks whole"
    right_or_nan(loss, rl, tl, "loss")
    ok = (dx.double() - rd).abs() <= R.rounded(rd, td, dtype)
    ok[:, 0] |= torch.isnan(dx[:, 0])  # a row may be marked although it was whole
    assert ok[~gave].all(), "a row that did not give up is wrong"
