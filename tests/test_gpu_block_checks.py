"""Calls of a block's operators that the binding passes on and the checks in
Python carry through."""
import pytest
import torch

from test_gpu_block_ops import E4
from test_gpu_train_ops import BF, FF, gen, mp, randn  # noqa: F401

pytestmark = pytest.mark.gpu


class Passes:
    """A binding that passes every call on to the checks in Python."""

    def __getattr__(self, name):
        return lambda *args: None


class Named(torch.Tensor):
    """A tensor of another class, which the binding passes on."""


@pytest.mark.parametrize("how", ["passes", "subclass", "vector scales"])
@pytest.mark.parametrize("d", [64, 1365])
def test_calls_through_the_checks(mp, how, d, monkeypatch):  # noqa: F811
    # they give what the binding's own calls give
    g = gen(40)
    rows, blocks = 13, -(-d // 32)
    x, res, dy, dh = (randn((rows, 2 * d), g, 1.0, BF)[:, :d] for _ in range(4))
    w, pos = randn((d,), g, 1.0, BF), torch.arange(rows, device="cuda", dtype=torch.int32) * 7
    ws = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    turns, _ = mp.mp_rope_frequencies(16)
    heads = x[:, :64].unflatten(1, (2, 32))

    def calls(wrap, scale_shape):
        def new(*shape, dtype=BF):
            return wrap(torch.zeros(*shape, dtype=dtype, device="cuda"))

        def new8():
            return new(rows, d, dtype=E4), new(*scale_shape, dtype=torch.uint8)
        xs, rs, dys, dhs, ww, hh = (wrap(t) for t in (x, res, dy, dh, w, heads))
        y, h, rstd, dx, dw, back = new(rows, d), new(rows, d), new(rows, dtype=FF), new(rows, d), new(d), new(rows, d)
        (y8, y8s), (h8, h8s), (a8, a8s), (b8, b8s), (p8, p8s) = (new8() for _ in range(5))
        r8, r8s = new(rows, d, dtype=torch.uint8), new(rows, dtype=FF)
        mp.mp_rmsnorm_forward(y, xs, ww, residual=rs, h=h, rstd=rstd, y8=y8, y8_scale=y8s, h8=h8, h8_scale=h8s)
        mp.mp_rmsnorm_backward(dx, dw, dys, h8, ww, rstd, dh=dhs, h_scale=h8s, workspace=wrap(ws))
        mp.mp_pack8(p8, p8s, xs)
        mp.mp_pack8(r8, r8s, xs)
        mp.mp_unpack8(back, p8, p8s)
        qo, ko = new(rows, 2, 32), new(rows, 2, 32)
        mp.mp_rope(qo, hh, ko, hh, wrap(turns), wrap(pos), interleaved=True)
        act, da, db, again = new(rows, d), new(rows, d), new(rows, d), new(rows, d)
        mp.mp_gated_forward(act, xs, rs, activation="gelu", gate8=a8, gate8_scale=a8s, up8=b8, up8_scale=b8s)
        mp.mp_gated_backward(da, db, dys, a8, b8, activation="gelu", gate_scale=a8s, up_scale=b8s, y=again)
        out = [y, h, rstd, dx, dw, back, qo, ko, act, da, db, again, y8, h8, a8, b8, p8, r8, r8s, y8s, h8s, a8s, b8s, p8s]
        return [t.as_subclass(torch.Tensor).view(-1) for t in out]

    want = calls(lambda t: t, (rows, blocks))
    if how == "passes":
        monkeypatch.setattr(mp.block, "_binding", Passes())
    wrap = (lambda t: t.as_subclass(Named)) if how == "subclass" else (lambda t: t)
    got = calls(wrap, (rows * blocks,) if how == "vector scales" else (rows, blocks))
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
