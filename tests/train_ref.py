"""64-bit references of the training-head operators and the error bounds their
kernels are held to. Every bound is derived, element by element, from the
formula and the roundings that a 32-bit evaluation makes:

  u   = 2^-24: one fp32 rounding to nearest is off by at most u relatively.
  uo  the same for the output's type, 2^-p for a significand of p bits (p = 8
      bf16, 11 fp16, 24 fp32), with half a step of its smallest values.
  Sums: a sum whose terms pass through at most D additions is off by at most
      D u sum|terms|. A row's sum: at least 256 chains (n / 256 additions), 5
      steps in a warp, the join of warps and blocks: D = n / 256 + 96. A sum
      over rows: at least 48 chains, and the join of at most 96.
  The scale is an fp32 argument: the references take its fp32 value.
  Exponentials: 2 ulp (4 u), and the rounded argument y adds 2 u |y|.
"""
import math

import torch

U = 2.0 ** -24
UO = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}


def depth(n):
    return 96 + n / 256


def rounded(v, tol, dtype):
    """tol of a value v before its rounding to dtype -> after it."""
    return tol + UO[dtype] * (v.abs() + tol) + TINY[dtype]


def assert_within(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, what
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN positions differ"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = ~(nan | inf)
    err = (got - ref).abs()[ok]
    lim = tol.expand_as(ref)[ok]
    bad = ~(err <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, "
                           f"worst {float((err / lim).max()):.3g} of it")


def as_f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


# --- layer norm --------------------------------------------------------------

def ln_forward(x, weight, bias, eps):
    """(y, mean, rstd) and their bounds (y's before its rounding)."""
    xd = x.double()
    d = x.shape[1]
    D = depth(d)
    w = torch.ones(d, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(d, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    mean = xd.mean(1, keepdim=True)
    xc = xd - mean
    var = (xc * xc).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    y = xc * rstd * w + b
    t_mean = (D + 2) * U * xd.abs().mean(1, keepdim=True)
    # sum (x - mean')^2 with mean' = mean + e: + d e^2; each distance rounded once (2 u on its square)
    t_var = var * (D + 5) * U + t_mean ** 2
    t_rstd = rstd * (0.5 * t_var / (var + eps) + 4 * U)
    t_xh = t_mean * rstd + xc.abs() * t_rstd + 3 * U * (xc * rstd).abs()
    t_y = t_xh * w.abs() + U * y.abs()
    return (y, mean[:, 0], rstd[:, 0]), (t_y, t_mean[:, 0], t_rstd[:, 0])


def ln_backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) for the given fp32 mean and rstd, and their bounds."""
    xd, g0 = x.double(), dy.double()
    rows, d = x.shape
    D, Dr = depth(d), 96 + rows / 48
    w = torch.ones(d, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    mu, r = mean.double()[:, None], rstd.double()[:, None]
    xh = (xd - mu) * r
    g = g0 * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    t_c1 = (D + 3) * U * g.abs().mean(1, keepdim=True)
    t_c2 = (D + 6) * U * (g * xh).abs().mean(1, keepdim=True)
    t_dx = r * (t_c1 + xh.abs() * t_c2 + 6 * U * (g.abs() + c1.abs() + (xh * c2).abs()))
    dw, db = (g0 * xh).sum(0), g0.sum(0)
    t_dw = (Dr + 4) * U * (g0 * xh).abs().sum(0)
    t_db = Dr * U * g0.abs().sum(0)
    return (dx, dw, db), (t_dx, t_dw, t_db)


# --- token log probabilities ---------------------------------------------------

def _stats(x, scale):
    z = x.double() * as_f32(scale)
    m = z.amax(1, keepdim=True)
    e = torch.where(z == -math.inf, 0.0, torch.exp(z - m))
    s = e.sum(1, keepdim=True)
    lse = torch.where(m == -math.inf, m, m + torch.log(s))
    return z, m, e, s, lse


def lp_forward(x, targets, scale, k):
    """dict of logp, lse, entropy, top_index, top_logp with bounds."""
    rows, vocab = x.shape
    z, m, e, s, lse = _stats(x, scale)
    empty = (m == -math.inf)[:, 0]
    D = depth(vocab)
    p = e / s
    dist = torch.where(e > 0, p * (m - z), torch.where(torch.isnan(e), e, 0.0)).sum(1, keepdim=True)  # >= 0
    ent = torch.where(empty, 0.0, (torch.log(s) + dist)[:, 0])
    t_log_s = (D + 6) * U + 3 * U * dist + 2 * U * torch.log(s).abs()
    t_lse = (t_log_s + 3 * U * (m.abs() + lse.abs()))[:, 0]
    t_ent = (t_log_s + (2 * D + 20) * U * dist + 3 * U * (p * (m - z) ** 2).nan_to_num(0.0).sum(1, keepdim=True)
             + 2 * U * ent[:, None].abs())[:, 0]
    out, tol = {"lse": lse[:, 0], "entropy": ent}, {"lse": t_lse, "entropy": t_ent}

    def at(idx):
        zz = z.gather(1, idx)
        lp = torch.where(empty[:, None], -math.inf, (zz - m) - torch.log(s))
        return lp, t_lse[:, None] + 3 * U * (zz.abs() + lse.abs())

    if targets is not None:
        t = targets.long()
        lp, t_lp = at(t.clamp(0, vocab - 1)[:, None])
        lp = torch.where(t < 0, 0.0, torch.where(t >= vocab, math.nan, lp[:, 0]))
        out["logp"], tol["logp"] = lp, t_lp[:, 0]
    if k:
        order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :k]
        out["top_index"] = order.int()
        out["top_logp"], tol["top_logp"] = at(order)
    return out, tol


def lp_backward(x, targets, lse, entropy, dlogp, dentropy, scale):
    """(dlogits, bound before its rounding) for the given fp32 lse and entropy."""
    rows, vocab = x.shape
    scale = as_f32(scale)
    y = x.double() * scale - lse.double()[:, None]
    p = torch.exp(y)
    t = torch.full((rows,), -1, device=x.device) if targets is None else targets.long()
    has = (t >= 0) & (t < vocab)
    g = torch.where(has, dlogp.double(), 0.0)[:, None] if dlogp is not None else torch.zeros(rows, 1, device=x.device)
    h = dentropy.double()[:, None] if dentropy is not None else torch.zeros_like(g)
    en = entropy.double()[:, None] if entropy is not None else torch.zeros_like(g)
    one = torch.zeros_like(y).scatter_(1, t.clamp(0, vocab - 1)[:, None], has.double()[:, None])
    yy = torch.where(p == 0, 0.0, y)
    f = g * (one - p) - h * p * (yy + en)
    size = p * (g.abs() + h.abs() * (yy.abs() + en.abs()))
    tol = ((3 * yy.abs() + 12) * size + 3 * one * g.abs()) * U + 2.0 ** -125 * (g.abs() + h.abs() * 200)
    zero = ((g == 0) & (h == 0)) | (lse[:, None] == -math.inf)
    return torch.where(zero, 0.0, f * scale), torch.where(zero, 0.0, tol * scale)


# --- distillation ----------------------------------------------------------------

def distill(x, teacher, index, row_weight, scale):
    """(loss, dlogits) and bounds (dlogits' before its rounding)."""
    rows, vocab = x.shape
    scale = as_f32(scale)
    z, m, e, s, lse = _stats(x, scale)
    idx = index.long()
    use = (idx >= 0) & (idx < vocab)
    bad = (idx >= vocab).any(1)
    at = idx.clamp(0, vocab - 1)
    t = torch.where(use, teacher.double() * scale, -math.inf)
    tm = t.amax(1, keepdim=True)
    none = (tm == -math.inf)[:, 0]
    empty = (m == -math.inf)[:, 0]
    et = torch.where(t == -math.inf, 0.0, torch.exp(t - tm))
    ts = et.sum(1, keepdim=True)
    q = torch.where(none[:, None], 0.0, et / ts)
    lq = torch.where(q > 0, torch.log(q), torch.where(torch.isnan(q), q, 0.0))
    lz = torch.where(empty[:, None], -math.inf, (z.gather(1, at) - m) - torch.log(s))
    kl = torch.where(q == 0, 0.0, q * (lq - lz)).sum(1)
    w = torch.ones(rows, dtype=torch.float64, device=x.device) if row_weight is None else row_weight.double()
    loss = torch.where(bad, math.nan, torch.where(none, 0.0, w * kl))
    loss = torch.where(w == 0, 0.0, loss)
    D, Dk = depth(vocab), 96
    p = torch.where(empty[:, None], 0.0, e / s)
    far = torch.where(p > 0, p * (m - z), 0.0).nan_to_num(0.0).sum(1)  # argument roundings in s
    fart = torch.where(q > 0, q * (tm - t), 0.0).nan_to_num(0.0).sum(1)
    mag = torch.where(q == 0, 0.0, q * (lq.abs() + (tm - t).abs() + lz.abs() + (m - z.gather(1, at)).abs()))
    t_loss = w.abs() * U * ((D + Dk + 20) + 4 * (far + fart) + (2 * Dk + 12) * mag.nan_to_num(0.0, 0.0, 0.0).sum(1))
    t_loss = torch.where(w == 0, 0.0, t_loss)  # exact, whatever the row holds
    dense = torch.zeros_like(p).scatter_add_(1, at, torch.where(use, q, 0.0))
    zero = none | empty | (w == 0)
    ws = (w * scale)[:, None]
    dx = torch.where(zero[:, None], 0.0, (p - dense) * ws)
    dist = torch.where(p > 0, m - z, 0.0)
    t_p = p * ((D + 14) + 3 * dist + 4 * far[:, None])
    t_q = torch.zeros_like(p).scatter_add_(
        1, at, torch.where(use & (q > 0), q * ((2 * Dk + 14) + 3 * (tm - t) + 4 * fart[:, None]), 0.0))
    t_dx = ws.abs() * (U * (t_p + t_q + 4 * (p + dense)) + 2.0 ** -125)
    t_dx = torch.where(zero[:, None], 0.0, t_dx)
    return (loss, dx), (t_loss, t_dx)
