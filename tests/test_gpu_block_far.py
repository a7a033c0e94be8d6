"""Rows so far apart that offsets pass 32 bits, in every kernel of the RMS norm.
References and bounds: tests/block_ref.py."""
import pytest
import torch

import block_ref as R
from test_gpu_block_ops import contiguous8, scales
from test_gpu_train_ops import BF, f32, gen, mp, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("d", [128, 100, 1600, 1365, 8200, 9001])
def test_rmsnorm_rows_far_apart(mp, d, kept):  # noqa: F811
    # Elements' offsets pass 2^31 within the call's rows, bytes' 2^32: forward, and backward with the weight
    # gradient, of rows that one block sums and of rows that several do.
    g = gen(22)
    rows = 12
    stride = (1 << 28) + (8 if d % 8 == 0 else 1)
    a = torch.empty(rows * stride, dtype=BF, device="cuda")
    b = torch.empty(rows * stride, dtype=BF, device="cuda")
    x, y = (t.view(rows, stride)[:, :d] for t in (a, b))
    # 8-bit rows twice as far apart, behind the others in the same buffer
    bytes8 = b.view(torch.uint8).view(rows, 2 * stride)
    q, s = bytes8[:, 4 * d + 16 - 4 * d % 16:][:, :d], scales(rows, d, "block")
    c, w = randn((rows, d), g, 1.0, BF), (1 + randn((d,), g, 0.2)).to(BF)
    x.copy_(c)
    rstd = f32(rows)
    mp.mp_rmsnorm_forward(y, x, w, rstd=rstd, h8=q, h8_scale=s)
    (ry, rr), (ty, tr) = R.rms_forward(c, w, 1e-5)
    R.assert_within(rstd, rr, tr, "rstd")
    R.assert_within(y, ry, R.rounded(ry, ty, BF), "y")
    R.check_block8(contiguous8(q), s, c.double(), 0.0 * ry, BF, "h8")
    dy = y.contiguous()
    hd = R.unpack(contiguous8(q), s) if kept else c.double()
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    dw = torch.full((d,), 77.0, dtype=BF, device="cuda")
    mp.mp_rmsnorm_backward(y, dw, y, q if kept else x, w, rstd, h_scale=s if kept else None, workspace=ws)
    (rdx, rdw), (tdx, tdw) = R.rms_backward(dy, None, hd, w, rstd)
    R.assert_within(y, rdx, R.rounded(rdx, tdx, BF), "dx")
    R.assert_within(dw, rdw, R.rounded(rdw, tdw, BF), "dweight")
