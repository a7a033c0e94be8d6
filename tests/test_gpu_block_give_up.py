"""What the staged RMS norm kernels leave when a wait for a copy runs out. No
wait does on a working GPU, so the kernels are compiled a second time with a
limit of 0: a wait whose copy has not landed when it begins gives up. Every access
stays in bounds then (no index is read from what has not arrived), every wait
still ends, and copies in flight land before a block ends. A row that was
given up has to show it: what is not NaN has to be right."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import block_ref as R
from test_gpu_train_give_up import i64, ptr, right_or_nan

pytestmark = pytest.mark.gpu

BF, FF = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def short(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from mixed_precision_adamw_gb300 import build as B
    out = tmp_path_factory.mktemp("short_waits")
    sources = [os.path.join(os.path.dirname(os.path.abspath(__file__)), "short_waits.cu"),
               os.path.join(B.CSRC, "mp_rmsnorm.cu")]

    def compile(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        subprocess.run([B.nvcc(), *B.NVCC_FLAGS, "-DMP_WAIT_LIMIT_NS=0", "-c", src, "-o", obj], check=True,
                       capture_output=True)
        return obj

    with ThreadPoolExecutor() as ex:
        objs = list(ex.map(compile, sources))
    lib = str(out / "short_waits.so")
    subprocess.run([B.nvcc(), "-shared", *B.GENCODE, "-o", lib, *objs], check=True, capture_output=True)
    L = ctypes.CDLL(lib)
    L.mp_rmsnorm_workspace_bytes.restype = ctypes.c_size_t
    return L


def i32(*v):
    return [ctypes.c_int32(x) for x in v]


def test_rmsnorm_gives_up(short):
    # which waits give up depends on the copies' time: some of all these do
    gave = [case(short, rows, d, pad, dtype) for dtype in (BF, FF)
            for rows, d, pad in ((20000, 1600, 0), (9001, 1357, 1), (3000, 8192, 0), (20000, 512, 0))]
    for which, name in enumerate(("y", "rstd", "h8", "y8", "dx", "dweight")):
        assert any(v[which] for v in gave), f"{name}: no wait gave up"


def case(short, rows, d, pad, dtype):
    """Checks one size and type; which of the outputs hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x, res, dy = (torch.randn(rows, d + pad, generator=g, device="cuda").to(dtype)[:, :d] for _ in range(3))
    w = torch.randn(d, generator=g, device="cuda")
    y, h, dx = (torch.full((rows, d), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    y8, h8 = (torch.zeros(rows, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    s8, hs = torch.zeros(rows, device="cuda"), torch.zeros(rows, -(-d // 32), dtype=torch.uint8, device="cuda")
    rstd, dw = torch.full((rows,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    code = ctypes.c_int32(0 if dtype == BF else 2)
    stored = (x.float() + res.float()).to(dtype)
    (ry, rr), (ty, tr) = R.rms_forward(stored, w, 1e-5)
    # the copies are mostly there when they are waited for: beside others that keep HBM busy some are not
    big, side = torch.ones(1 << 31, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    gave = [False] * 4
    for _ in range(20):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big.add_(1)
        assert short.mp_rmsnorm_forward(ptr(y), ptr(h), ptr(rstd), ptr(y8), ptr(s8), ptr(h8), ptr(hs), ptr(x),
                                        ptr(res), ptr(w), *i64(rows, d, d, d, d, d, d + pad, d + pad),
                                        ctypes.c_float(1e-5), code, *i32(2, 1), None) == 0
        torch.cuda.synchronize()
        assert (torch.isnan(h) | (h == stored)).all(), "a sum that is not NaN is wrong"
        back, kept = R.unpack(y8, s8), R.unpack(h8, hs)
        now = [right_or_nan(y, ry, R.rounded(ry, ty, dtype), "y"), right_or_nan(rstd, rr, tr, "rstd"),
               right_or_nan(kept, stored.double(), R.E4 * stored.double().abs() + 2.0 ** -10, "h8"),
               # half a step of a value, or of the smallest steps beside the row's largest value
               right_or_nan(back, ry, 1.01 * (R.E4 * ry.abs() + ry.abs().amax(1, keepdim=True) / 448 * 2.0 ** -10),
                            "y8")]
        gave = [a or b for a, b in zip(gave, now)]
        if all(gave):
            break
    r2 = rr.float()
    n = short.mp_rmsnorm_workspace_bytes(*i64(rows, d))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    (rdx, rdw), (tdx, tdw) = R.rms_backward(dy, res, stored.double(), w, r2)
    back = [False, False]
    for _ in range(20):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big.add_(1)
        assert short.mp_rmsnorm_backward(ptr(dx), ptr(dw), ptr(dy), ptr(res), ptr(stored), None, ptr(w), ptr(r2),
                                         *i64(rows, d, d, d + pad, d + pad, d), code, *i32(2), ptr(ws),
                                         ctypes.c_size_t(n), None) == 0
        torch.cuda.synchronize()
        now = [right_or_nan(dx, rdx, R.rounded(rdx, tdx, dtype), "dx"),
               right_or_nan(dw, rdw, R.rounded(rdw, tdw, FF), "dweight")]
        back = [a or b for a, b in zip(back, now)]
        if all(back):
            break
    return gave + back
