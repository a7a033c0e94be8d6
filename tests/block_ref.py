"""64-bit references of the operators of a block between its matrix products,
and the error bounds their kernels are held to, derived from the formula and
the roundings of a 32-bit evaluation as in train_ref.py (U = 2^-24 a rounding
to nearest; a sum of D additions is off by at most D U sum|terms|). Further:

  rsqrt      2 ulp (4 U).   sin, cos of a part of pi: 1 ulp (2 U) absolutely.
  sigma      exp2: 2 ulp (4 U), its argument -v log2(e) is off by 2 U |v| log2(e),
             which is 2 U |v| of the exponential; adding 1 U, 1/x 1 ulp (2 U).
             What is below 2^-126 may be 0.
  e4m3       half a step is 2^-4 of the value, or 2^-10 of the scale for the
             smallest (a step of 2^-9).
"""
import math

import torch

from train_ref import TINY, U, UO, as_f32, assert_within, depth, rounded  # noqa: F401

E4 = 2.0 ** -4
TOP = {torch.bfloat16: 247, torch.float16: 135, torch.float32: 247}  # block exponent of the type's largest values


def unpack(q, scale):
    """What 8-bit rows stand for, in 64 bits."""
    v = q.view(torch.float8_e4m3fn).float().double()
    if scale.dtype == torch.float32:
        return v * scale.double()[:, None]
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale == 255, math.nan, s)
    return v * s.repeat_interleave(32, 1)[:, :q.shape[1]]


def block_exponents(v):
    """uint8 exponents of the blocks of exact fp32 or narrower values (64-bit tensor): the least e with
    amax <= 448 2^e, in integers."""
    rows, d = v.shape
    n = -(-d // 32)
    w = torch.zeros(rows, n * 32, dtype=torch.float64, device=v.device)
    w[:, :d] = v
    amax = w.view(rows, n, 32).abs().amax(2)
    m, k = torch.frexp(amax)
    e = torch.where(amax == 0, -127, k - 9 + (m > 0.875).int()).clamp(min=-127)
    return torch.where(torch.isfinite(amax), e + 127, 255).to(torch.uint8)


def check_block8(q, scale, v, t_v, dtype, what):
    """q, scale against values v (64 bits) known within t_v; dtype: of exact values, None for others."""
    s = torch.exp2(scale.double() - 127).repeat_interleave(32, 1)[:, :v.shape[1]]
    nan = (scale == 255).repeat_interleave(32, 1)[:, :v.shape[1]]
    if dtype is not None:
        assert torch.equal(scale, block_exponents(v)), what + " exponents"
    got = unpack(q, scale)
    assert torch.isnan(got[nan]).all(), what + " NaN blocks"
    ok = ~nan
    lim = E4 * (v.abs() + t_v) + s * 2.0 ** -10 + t_v
    err = (got - v).abs()
    bad = ~(err <= lim) & ok
    assert not bad.any(), f"{what}: {int(bad.sum())} values beyond, worst {float((err / lim)[ok].max())}"
    if dtype is None:
        amax = torch.zeros(v.shape[0], scale.shape[1] * 32, dtype=torch.float64, device=v.device)
        tol = amax.clone()
        amax[:, :v.shape[1]], tol[:, :v.shape[1]] = v.abs(), t_v
        amax, tol = amax.view(v.shape[0], -1, 32).amax(2), tol.view(v.shape[0], -1, 32).amax(2)
        top = 448 * torch.exp2(scale.double() - 127)
        fine = (scale == 255) | ((amax - tol <= top) & ((amax + tol > top / 2) | (scale == 0)))
        assert fine.all(), what + " exponents"


def check_row8(q, scale, v, t_v, what):
    amax = v.abs().amax(1)
    finite = torch.isfinite(amax)
    assert torch.equal(torch.isnan(scale), ~finite), what + " NaN rows"
    ref = (amax / 448).clamp(min=2.0 ** -126)
    t_amax = t_v.amax(1) if t_v is not None else torch.zeros_like(amax)
    assert ((scale.double() - ref).abs() <= t_amax / 448 + 4 * U * ref)[finite].all(), what + " scales"
    got = unpack(q, scale)
    assert torch.isnan(got[~finite]).all(), what
    t = t_v if t_v is not None else 0.0
    lim = E4 * (v.abs() + t) + scale.double()[:, None] * 2.0 ** -10 + t + 8 * U * (v.abs() + amax[:, None])
    bad = ~((got - v).abs() <= lim) & finite[:, None]
    assert not bad.any(), f"{what}: {int(bad.sum())} values beyond the bound"


# --- RMS norm ----------------------------------------------------------------

def rms_forward(h, weight, eps):
    """(y, rstd) of the stored h and their bounds (y's before its rounding)."""
    hd = h.double()
    d = h.shape[1]
    w = torch.ones(d, dtype=torch.float64, device=h.device) if weight is None else weight.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + as_f32(eps))
    y = hd * rstd * w
    t_rel = (0.5 * (depth(d) + 4) + 6) * U
    return (y, rstd[:, 0]), (y.abs() * (t_rel + 3 * U), rstd[:, 0] * t_rel)


def rms_backward(dy, dh, h, weight, rstd):
    """(dx, dweight) for the given fp32 rstd and 64-bit h, and their bounds."""
    g0 = dy.double()
    rows, d = dy.shape
    D, Dr = depth(d), 96 + rows / 48
    w = torch.ones(d, dtype=torch.float64, device=dy.device) if weight is None else weight.double()
    r = rstd.double()[:, None]
    xh, g = h * r, g0 * w
    e = torch.zeros_like(g0) if dh is None else dh.double()
    c = (g * xh).mean(1, keepdim=True)
    ca = (g * xh).abs().mean(1, keepdim=True)
    dx = e + r * (g - xh * c)
    t_dx = U * (r * xh.abs() * ca * (D + 10) + 6 * r * (g.abs() + xh.abs() * c.abs()) + 4 * e.abs())
    dw = (g0 * xh).sum(0)
    return (dx, dw), (t_dx, (Dr + 4) * U * (g0 * xh).abs().sum(0))


# --- the gated activation --------------------------------------------------------

K = 2 * math.sqrt(2 / math.pi)


def _act(a, act):
    """v, dv/da * a, and the relative roundings of v."""
    if act == "silu":
        return a, a, 0.0
    return K * (a + 0.044715 * a ** 3), K * (a + 3 * 0.044715 * a ** 3), 6.0


def gated(dy, a, b, act):
    """dict of y, dgate, dup for 64-bit gate a and up b (None: 1), and their bounds before rounding."""
    v, av, n = _act(a, act)
    s = torch.sigmoid(v)
    far = torch.sigmoid(-v)
    e_s = U * (s * (far * ((2 + n) * v.abs() + 4) + 3)) + 2.0 ** -125
    t = s * far
    e_t = e_s * far + s * (e_s + U) + U * t
    f = a * s
    e_f = a.abs() * e_s + U * f.abs()
    slope = s + torch.where(t * av.abs() > 0, av * t, torch.zeros_like(t))
    e_slope = e_s + torch.where(t > 0, e_t * av.abs() + 7 * U * (t * av).abs(), torch.zeros_like(t)) + U * slope.abs()
    one = torch.ones_like(a) if b is None else b
    y = f * one
    out, tol = {"y": y}, {"y": e_f * one.abs() + U * y.abs()}
    if dy is not None:
        g = dy.double()
        out["dgate"], out["dup"] = g * one * slope, g * f
        tol["dgate"] = (g * one).abs() * e_slope + 3 * U * out["dgate"].abs()
        tol["dup"] = g.abs() * e_f + U * out["dup"].abs()
    return out, tol


# --- rotary positions --------------------------------------------------------------

def rope(x, turns, positions, factor, interleaved, inverse):
    """The rotation of x [tokens, heads, dim] by the 64-bit turns table, and its bound."""
    import numpy as np
    with np.errstate(over="ignore"):
        p = positions.cpu().numpy().astype(np.int64).view(np.uint64)
        frac = (p[:, None] * turns.cpu().numpy().view(np.uint64)[None, :]).view(np.int64)
    angle = torch.from_numpy(frac.astype(np.float64)).to(x.device) * (2 * math.pi * 2.0 ** -64)
    if inverse:
        angle = -angle
    r = 2 * turns.numel()
    f = as_f32(factor)
    c, s = (torch.cos(angle) * f)[:, None], (torch.sin(angle) * f)[:, None]
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i = torch.arange(r // 2, device=x.device)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    t = 8 * U * abs(f) * (a.abs() + b.abs())
    tol[..., i] = tol[..., j] = t
    return y, tol
