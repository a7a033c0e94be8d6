"""Argument checks of the operators of a block between its matrix products, and
the rotary frequencies (no GPU needed: every call here is refused, has nothing
to do, or runs on the host)."""
import ctypes
import math

import pytest
import torch

from test_train_args import FAKE, call, mp  # noqa: F401

NAN, INF = float("nan"), float("inf")
Q = 4 * FAKE
RF = dict(y=FAKE, h=2 * FAKE, rstd=FAKE, y8=3 * FAKE, y8_scale=FAKE, h8=4 * FAKE, h8_scale=FAKE, x=5 * FAKE,
          residual=6 * FAKE, weight=FAKE, rows=4, d=100, y_stride=100, h_stride=100, y8_stride=100, h8_stride=100,
          x_stride=100, residual_stride=100, eps=1e-5, type=0, weight_type=0, y8_kind=1, stream=None)
RB = dict(dx=FAKE, dweight=FAKE, dy=2 * FAKE, dh=3 * FAKE, h=4 * FAKE, h_scale=None, weight=FAKE, rstd=FAKE, rows=4,
          d=100, dx_stride=100, dy_stride=100, dh_stride=100, h_stride=100, type=0, weight_type=2, ws=FAKE,
          wsn=1 << 40, stream=None)
RO = dict(q_out=FAKE, q=2 * FAKE, k_out=3 * FAKE, k=4 * FAKE, turns=FAKE, positions=FAKE, first=0, tokens=4,
          q_heads=4, k_heads=2, head_dim=64, rotary_dim=32, qot=256, qoh=64, qt=256, qh=64, kot=128, koh=64, kt=128,
          kh=64, factor=1.0, interleaved=0, inverse=0, type=0, index_type=1, stream=None)
GF = dict(y=FAKE, gate8=2 * FAKE, gate8_scale=FAKE, up8=3 * FAKE, up8_scale=FAKE, gate=4 * FAKE, up=5 * FAKE, rows=4,
          d=100, y_stride=100, gate8_stride=100, up8_stride=100, gate_stride=200, up_stride=200, activation=0, type=0,
          stream=None)
GB = dict(dgate=FAKE, dup=2 * FAKE, y=3 * FAKE, dy=4 * FAKE, gate=5 * FAKE, gate_scale=None, up=6 * FAKE,
          up_scale=None, rows=4, d=100, dgate_stride=100, dup_stride=100, y_stride=100, dy_stride=100,
          gate_stride=100, up_stride=100, activation=1, type=0, stream=None)
PK = dict(q=FAKE, scale=FAKE, x=2 * FAKE, rows=4, d=100, q_stride=100, x_stride=100, type=0, kind=2, stream=None)
UP = dict(x=FAKE, q=2 * FAKE, scale=FAKE, rows=4, d=100, x_stride=100, q_stride=100, type=0, kind=1, stream=None)

CASES = [
    ("mp_rmsnorm_forward", RF, dict(rows=0), "MP_OK"),
    ("mp_rmsnorm_forward", RF, dict(x=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_forward", RF, dict(y=None, h=None, rstd=None, y8=None, h8=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_forward", RF, dict(y8_scale=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_forward", RF, dict(h8_scale=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_forward", RF, dict(residual=None), "MP_ERR_NULL"),  # h without one
    ("mp_rmsnorm_forward", RF, dict(rows=-1), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(d=0), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(d=(1 << 24) + 1), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(type=3), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(weight_type=-1), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y8_kind=0), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y8_kind=3), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(x_stride=99), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(h8_stride=99), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y8_stride=99), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(residual_stride=1), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(eps=-1.0), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(eps=NAN), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y=5 * FAKE, y_stride=104), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(h=6 * FAKE, h_stride=104), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(h=FAKE), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y8=4 * FAKE), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(y8=5 * FAKE), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(h8=FAKE), "MP_ERR_RANGE"),
    ("mp_rmsnorm_forward", RF, dict(x=5 * FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_forward", RF, dict(type=2, h=2 * FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_forward", RF, dict(y8_scale=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_forward", RF, dict(rstd=FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_backward", RB, dict(rows=0, dweight=None, dy=None, h=None, rstd=None), "MP_OK"),
    ("mp_rmsnorm_backward", RB, dict(dx=None, dweight=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_backward", RB, dict(dy=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_backward", RB, dict(h=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_backward", RB, dict(rstd=None), "MP_ERR_NULL"),
    ("mp_rmsnorm_backward", RB, dict(ws=None), "MP_ERR_WORKSPACE"),
    ("mp_rmsnorm_backward", RB, dict(wsn=8), "MP_ERR_WORKSPACE"),
    ("mp_rmsnorm_backward", RB, dict(ws=FAKE + 8), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_backward", RB, dict(dweight=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_backward", RB, dict(h=4 * FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_rmsnorm_backward", RB, dict(dx=2 * FAKE, dx_stride=101), "MP_ERR_RANGE"),
    ("mp_rmsnorm_backward", RB, dict(dx=3 * FAKE, dx_stride=101), "MP_ERR_RANGE"),
    ("mp_rmsnorm_backward", RB, dict(dx=4 * FAKE, h_scale=FAKE), "MP_ERR_RANGE"),  # 8-bit h is not dx
    ("mp_rmsnorm_backward", RB, dict(dh_stride=99), "MP_ERR_RANGE"),
    ("mp_rmsnorm_backward", RB, dict(h_stride=0), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(tokens=0), "MP_OK"),
    ("mp_rope", RO, dict(tokens=-1), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(tokens=1 << 31), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(q_heads=0, k_heads=0), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(q_heads=1025, qt=1 << 20, qot=1 << 20), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(head_dim=1025), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(rotary_dim=31), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(rotary_dim=0), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(rotary_dim=66), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(qh=63), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(qt=255), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(kot=127), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(kh=1 << 62), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(kt=1 << 62), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(qt=64, qh=255), "MP_ERR_RANGE"),  # heads outermost, one element short
    ("mp_rope", RO, dict(qt=64, qh=256, q=None), "MP_ERR_NULL"),  # and not
    ("mp_rope", RO, dict(factor=INF), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(index_type=2), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(type=-1), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(q_out=2 * FAKE, qot=512), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(k_out=FAKE), "MP_ERR_RANGE"),
    ("mp_rope", RO, dict(turns=None), "MP_ERR_NULL"),
    ("mp_rope", RO, dict(q=None), "MP_ERR_NULL"),
    ("mp_rope", RO, dict(k_out=None), "MP_ERR_NULL"),
    ("mp_rope", RO, dict(turns=FAKE + 4), "MP_ERR_ALIGN"),
    ("mp_rope", RO, dict(positions=FAKE + 4), "MP_ERR_ALIGN"),
    ("mp_rope", RO, dict(k=4 * FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_gated_forward", GF, dict(rows=0), "MP_OK"),
    ("mp_gated_forward", GF, dict(y=None), "MP_ERR_NULL"),
    ("mp_gated_forward", GF, dict(gate=None), "MP_ERR_NULL"),
    ("mp_gated_forward", GF, dict(gate8_scale=None), "MP_ERR_NULL"),
    ("mp_gated_forward", GF, dict(up=None), "MP_ERR_NULL"),  # up8 without up
    ("mp_gated_forward", GF, dict(activation=2), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(up_stride=99), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(gate8_stride=99), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(y=4 * FAKE), "MP_ERR_RANGE"),  # over gate, another stride
    ("mp_gated_forward", GF, dict(up8=2 * FAKE), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(gate8=FAKE), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(rows=1 << 31), "MP_ERR_RANGE"),
    ("mp_gated_forward", GF, dict(up=5 * FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_gated_backward", GB, dict(rows=0), "MP_OK"),
    ("mp_gated_backward", GB, dict(dgate=None), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(dup=None), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(up=None), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(gate_scale=FAKE), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(up_scale=FAKE), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(up=None, dup=None, up_scale=FAKE), "MP_ERR_NULL"),
    ("mp_gated_backward", GB, dict(dgate=2 * FAKE), "MP_ERR_RANGE"),
    ("mp_gated_backward", GB, dict(y=FAKE), "MP_ERR_RANGE"),
    ("mp_gated_backward", GB, dict(dgate=4 * FAKE, dgate_stride=101), "MP_ERR_RANGE"),
    ("mp_gated_backward", GB, dict(dgate=5 * FAKE, gate_scale=FAKE, up_scale=FAKE), "MP_ERR_RANGE"),
    ("mp_gated_backward", GB, dict(activation=-1), "MP_ERR_RANGE"),
    ("mp_gated_backward", GB, dict(dy=4 * FAKE + 1), "MP_ERR_ALIGN"),
    ("mp_pack8", PK, dict(rows=0), "MP_OK"),
    ("mp_pack8", PK, dict(kind=0), "MP_ERR_RANGE"),
    ("mp_pack8", PK, dict(q_stride=99), "MP_ERR_RANGE"),
    ("mp_pack8", PK, dict(q=2 * FAKE), "MP_ERR_RANGE"),
    ("mp_pack8", PK, dict(scale=None), "MP_ERR_NULL"),
    ("mp_pack8", PK, dict(kind=1, scale=FAKE + 2), "MP_ERR_ALIGN"),
    ("mp_pack8", PK, dict(x=FAKE * 2 + 1), "MP_ERR_ALIGN"),
    ("mp_unpack8", UP, dict(rows=0), "MP_OK"),
    ("mp_unpack8", UP, dict(x=None), "MP_ERR_NULL"),
    ("mp_unpack8", UP, dict(kind=4), "MP_ERR_RANGE"),
    ("mp_unpack8", UP, dict(type=9), "MP_ERR_RANGE"),
    ("mp_unpack8", UP, dict(scale=FAKE + 1), "MP_ERR_ALIGN"),
]


@pytest.mark.parametrize("name,base,kw,status", CASES)
def test_abi_checks(mp, name, base, kw, status):  # noqa: F811
    assert call(mp, name, list(base), base, **kw) == getattr(mp, status)


def test_workspace_bytes(mp):  # noqa: F811
    assert mp.mp_rmsnorm_workspace_bytes(-1, 8) == 0 and mp.mp_rmsnorm_workspace_bytes(4, 0) == 0
    assert mp.mp_rmsnorm_workspace_bytes(4, (1 << 24) + 1) == 0
    assert mp.mp_rmsnorm_workspace_bytes(0, 64) >= 256


def test_the_binding_refuses(mp, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mp.mp_rmsnorm_forward(x.clone(), x)
    with pytest.raises(TypeError):
        mp.mp_rmsnorm_forward(x.clone(), x.double())
    with pytest.raises(ValueError):
        mp.mp_gated_forward(x.clone(), x)
    with pytest.raises(ValueError):
        mp.mp_pack8(q, s, x)
    with pytest.raises(ValueError):
        mp.mp_rope(x[None], x[None], None, None, torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError):
        mp.RopeScaling("spiral", 2.0)


def test_struct_layout(mp):  # noqa: F811
    assert ctypes.sizeof(mp.MpRopeScaling) == 40


# --- frequencies -----------------------------------------------------------------

# A frequency is held to the nearest 2^-64 turns: off by at most half of that, and this is a whole one.
STEP = 2 * math.pi * 2.0 ** -64


def frequencies(mp, r, base=10000.0, scaling=None):
    t, f = mp.mp_rope_frequencies(r, base, scaling, device="cpu")
    assert t.dtype == torch.int64 and t.numel() == r // 2
    return [(int(v) % (1 << 64)) * 2 * math.pi / 2 ** 64 for v in t], f


@pytest.mark.parametrize("r,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (96, 1e6), (1024, 1.5)])
def test_frequencies(mp, r, base):  # noqa: F811
    got, factor = frequencies(mp, r, base)
    assert factor == 1.0
    for i, f in enumerate(got):
        ref = base ** (-2 * i / r)
        assert abs(f - ref) <= 1e-14 * ref + STEP


def test_scaled_frequencies(mp):  # noqa: F811
    r, base, k, L = 128, 500000.0, 8.0, 8192
    plain = [base ** (-2 * i / r) for i in range(r // 2)]

    def close(a, b):
        assert all(abs(x - y) <= 1e-13 * y + STEP for x, y in zip(a, b))

    close(frequencies(mp, r, base, mp.RopeScaling("linear", k))[0], [f / k for f in plain])
    got = frequencies(mp, r, base, mp.RopeScaling("base", k))[0]
    assert abs(got[0] - 1.0) <= 1e-13 and abs(got[-1] - plain[-1] / k) <= 1e-13 * got[-1] + STEP  # the ends
    assert frequencies(mp, 2, base, mp.RopeScaling("base", k))[0][0] == pytest.approx(1.0, abs=1e-13)
    got, factor = frequencies(mp, r, base, mp.RopeScaling("bands", k, context=L, low=1.0, high=4.0))
    for f, g in zip(plain, got):
        wave = 2 * math.pi / f
        if wave < L / 4.0:
            want = f
        elif wave > L / 1.0:
            want = f / k
        else:
            s = (L / wave - 1.0) / 3.0
            want = (1 - s) * f / k + s * f
        assert abs(g - want) <= 1e-13 * want + STEP
    assert factor == 1.0
    got, factor = frequencies(mp, r, base, mp.RopeScaling("ramp", k, context=L))
    lo = math.floor(r * math.log(L / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(r * math.log(L / (2 * math.pi)) / (2 * math.log(base)))
    for i, (f, g) in enumerate(zip(plain, got)):
        s = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        want = f / k * s + f * (1 - s)
        assert abs(g - want) <= 1e-13 * want + STEP
    assert factor == pytest.approx(0.1 * math.log(k) + 1)
    for kind in ("linear", "base", "bands", "ramp"):  # no longer a context: nothing changes
        got, factor = frequencies(mp, r, base, mp.RopeScaling(kind, 1.0))
        close(got, plain)
        assert factor == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=1026), dict(base=1.0),
                                dict(base=NAN), dict(base=INF), dict(kind="linear", factor=0.5),
                                dict(kind="linear", factor=NAN), dict(kind="bands", factor=2.0, context=0.0),
                                dict(kind="bands", factor=2.0, low=4.0, high=4.0), dict(kind="ramp", factor=2.0, low=0.0),
                                dict(kind="base", factor=1e308, rotary_dim=4)])
def test_frequency_refusals(mp, kw):  # noqa: F811
    kw = dict(kw)
    r, base = kw.pop("rotary_dim", 64), kw.pop("base", 10000.0)
    scaling = mp.RopeScaling(kw.pop("kind"), kw.pop("factor"), **kw) if kw else None
    with pytest.raises(mp.MpError) as e:
        mp.mp_rope_frequencies(r, base, scaling, device="cpu")
    assert e.value.status == mp.MP_ERR_RANGE


def test_the_binding_leaves_the_rest_alone(mp):  # noqa: F811
    # whatever is not plainly right is passed on, with no error left behind
    from mixed_precision_adamw_gb300 import _binding as b
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for args in ((), (1,) * 12, (None,) * 12, (x,) * 12):
        assert b.rmsnorm_forward(*args) is None
    for f, n in ((b.rmsnorm_backward, 10), (b.rope, 11), (b.gated_forward, 9), (b.gated_backward, 10), (b.pack8, 4),
                 (b.unpack8, 4)):
        for v in (None, 1, 1.0, "x", x, 1 << 80, object()):
            assert f(*(v,) * n) is None
        assert f() is None
