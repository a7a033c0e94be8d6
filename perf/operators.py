"""Workloads of the training-head operators: layer norm (forward and backward
with the weight gradients), log probabilities of given tokens (with entropy
and top alternatives; and their gradient), and distillation from a teacher's
top logits (loss and gradient).

Each case is one pass through one operator. `run` computes it in plain torch
operations in 32 bits, rounded once at the end (own = False), or through the
library's entry points (own = True).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-5


def listed():
    return [
        # one token's activations through a 768-wide layer norm: a launch's latency
        {"name": "ln fwd 1x768 bf16", "op": "ln", "dir": "fwd", "rows": 1, "d": 768, "type": "bf16", "wtype": "bf16",
         "bias": True, "pad": 0},
        # a micro-batch of 32 x 1024 tokens, the 1600-wide GPT-2 set
        {"name": "ln fwd 32768x1600 bf16", "op": "ln", "dir": "fwd", "rows": 32768, "d": 1600, "type": "bf16",
         "wtype": "bf16", "bias": True, "pad": 0},
        # its backward pass, the gradients of weight and bias into the bf16 gradient buffer
        {"name": "ln bwd 32768x1600 bf16", "op": "ln", "dir": "bwd", "rows": 32768, "d": 1600, "type": "bf16",
         "wtype": "bf16", "bias": True, "pad": 0},
        # 8192 tokens of the 4096-wide set, fp32 weights and weight gradients, no bias
        {"name": "ln bwd 8192x4096 bf16", "op": "ln", "dir": "bwd", "rows": 8192, "d": 4096, "type": "bf16",
         "wtype": "f32", "bias": False, "pad": 0},
        # odd width and length, fp32 activations, rows of a wider buffer
        {"name": "ln bwd 3001x1365 f32", "op": "ln", "dir": "bwd", "rows": 3001, "d": 1365, "type": "f32",
         "wtype": "f32", "bias": True, "pad": 3},
        # one token just decoded, its alternatives: a launch's latency and one long row
        {"name": "lp fwd 1x128256 bf16 k8", "op": "lp", "dir": "fwd", "rows": 1, "vocab": 128256, "type": "bf16",
         "k": 8, "scale": 1.0, "masked": 0, "pad": 0, "entropy": True},
        # scoring a micro-batch of 8 x 1024 tokens
        {"name": "lp fwd 8192x50304 bf16 k20", "op": "lp", "dir": "fwd", "rows": 8192, "vocab": 50304, "type": "bf16",
         "k": 20, "scale": 1.0, "masked": 47, "pad": 0, "entropy": True},
        # a policy-gradient step on the same micro-batch, with an entropy bonus
        {"name": "lp bwd 8192x50304 bf16", "op": "lp", "dir": "bwd", "rows": 8192, "vocab": 50304, "type": "bf16",
         "k": 0, "scale": 1.0, "masked": 47, "pad": 0, "entropy": True},
        # odd vocabulary and length, fp32 logits at a temperature of 0.8
        {"name": "lp fwd 2047x32003 f32 k5", "op": "lp", "dir": "fwd", "rows": 2047, "vocab": 32003, "type": "f32",
         "k": 5, "scale": 1.25, "masked": 100, "pad": 0, "entropy": True},
        # a few rows: the end of a ragged batch
        {"name": "distill 4x50304 bf16 K20", "op": "distill", "rows": 4, "vocab": 50304, "type": "bf16", "K": 20,
         "scale": 0.5, "masked": 47, "pad": 0},
        # a micro-batch of 8192 tokens at the largest vocabulary
        {"name": "distill 8192x128256 bf16 K64", "op": "distill", "rows": 8192, "vocab": 128256, "type": "bf16",
         "K": 64, "scale": 1.0, "masked": 0, "pad": 0},
        # odd vocabulary, length and list, fp16 with loss scaling in the row weights
        {"name": "distill 1021x50261 f16 K33", "op": "distill", "rows": 1021, "vocab": 50261, "type": "f16", "K": 33,
         "scale": 0.5, "masked": 5, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln", "lp", "lp", "distill"])
    ty = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "ln":
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:  # widths are mostly multiples of 8, some odd
            d = max(64, d // 8 * 8)
        rows = min(_log_int(rng, 1, 65536), (1 << 27) // d)
        return {"op": "ln", "dir": rng.choice(["fwd", "bwd"]), "rows": rows, "d": d, "type": ty,
                "wtype": rng.choice([ty, "f32"]), "bias": rng.random() < 0.7, "pad": rng.choice([0, 0, 0, 8, 5])}
    vocab = _log_int(rng, 64, 128256)
    if rng.random() < 0.5:
        vocab = max(64, vocab // 64 * 64)
    rows = min(_log_int(rng, 1, 8192), (1 << 29) // vocab)
    case = {"op": op, "rows": rows, "vocab": vocab, "type": ty, "scale": rng.choice([1.0, 1.0, 0.5, 1.25]),
            "masked": rng.choice([0, 7, vocab // 10]), "pad": rng.choice([0, 0, 0, 64, 3])}
    if op == "lp":
        case.update(dir=rng.choice(["fwd", "bwd"]), k=rng.choice([0, 1, 5, 20, 32]), entropy=rng.random() < 0.7)
        if case["dir"] == "bwd":
            case["k"] = 0
    else:
        case["K"] = min(_log_int(rng, 1, 128), vocab // 2)
    return case


def work(case):
    rows, e = case["rows"], _SIZE[case["type"]]
    if case["op"] == "ln":
        d, we = case["d"], _SIZE[case["wtype"]]
        affine = 2 if case["bias"] else 1
        if case["dir"] == "fwd":
            return {"bytes": 2 * e * rows * d + affine * we * d + 8 * rows, "flops": 8 * rows * d}
        return {"bytes": 3 * e * rows * d + we * d * (1 + affine) + 8 * rows, "flops": 16 * rows * d}
    n = rows * case["vocab"]
    if case["op"] == "lp":
        if case["dir"] == "fwd":
            ent = 1 if case["entropy"] else 0
            return {"bytes": e * n + rows * (8 + 8 + 4 * ent + 8 * case["k"]), "flops": (5 + 2 * ent) * n}
        ent = 2 if case["entropy"] else 0
        return {"bytes": 2 * e * n + rows * (8 + 8 + 4 * ent), "flops": (4 + ent) * n}
    return {"bytes": 2 * e * n + rows * (case["K"] * (e + 8) + 8), "flops": 8 * n}


def _randn(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _logits(case, gen):
    """Logits of a trained head: spread 2.5, a masked tail of the vocabulary, rows of a wider buffer if padded."""
    rows, vocab = case["rows"], case["vocab"]
    buf = torch.empty(rows, vocab + case["pad"], dtype=_DT[case["type"]], device="cuda")
    step = max(1, (1 << 28) // (vocab + case["pad"]))
    for a in range(0, rows, step):
        b = min(rows, a + step)
        buf[a:b] = torch.randn(b - a, buf.shape[1], generator=gen, device="cuda").mul_(2.5)
    x = buf[:, :vocab]
    if case["masked"]:
        x[:, vocab - case["masked"]:] = -math.inf
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, dt = case["rows"], _DT[case["type"]]
    st = {"case": dict(case)}
    if case["op"] == "ln":
        d, wdt = case["d"], _DT[case["wtype"]]
        shape = (rows, d + case["pad"])
        # activations with a per-channel offset, as a residual stream has
        x = (torch.randn(shape, generator=gen, device="cuda") * 1.5
             + torch.randn(shape[1], generator=gen, device="cuda") * 0.5).to(dt)[:, :d]
        st["x"] = x
        st["weight"] = (1.0 + torch.randn(d, generator=gen, device="cuda") * 0.1).to(wdt)
        st["bias"] = _randn((d,), gen, 0.1, wdt) if case["bias"] else None
        st["mean"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        st["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        if case["dir"] == "fwd":
            st["y"] = torch.empty(rows, d, dtype=dt, device="cuda")
        else:
            # what the forward pass kept
            xf = x.double()
            st["mean"].copy_(xf.mean(1))
            st["rstd"].copy_((xf.var(1, unbiased=False) + _EPS).rsqrt())
            st["dy"] = _randn((rows, d), gen, 1.0, dt)
            st["dx"] = torch.empty(rows, d, dtype=dt, device="cuda")
            st["dweight"] = torch.empty(d, dtype=wdt, device="cuda")
            st["dbias"] = torch.empty(d, dtype=wdt, device="cuda") if case["bias"] else None
        return st
    vocab = case["vocab"]
    x = st["logits"] = _logits(case, gen)
    allowed = vocab - case["masked"]
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] == "lp":
        tgt = torch.randint(0, allowed, (rows,), generator=gen, device="cuda")
        if rows > 1:  # some positions have no given token
            tgt = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.05, torch.full_like(tgt, -1), tgt)
        # the given token is mostly a likely one
        at = tgt.clamp(min=0)[:, None]
        x.scatter_(1, at, (x.gather(1, at).float() + 6.0).to(dt))
        st["targets"] = tgt
        if case["dir"] == "fwd":
            st["logp"], st["lse"] = torch.empty(rows, **f32), torch.empty(rows, **f32)
            st["ent"] = torch.empty(rows, **f32) if case["entropy"] else None
            k = case["k"]
            st["top_logp"] = torch.empty(rows, k, **f32) if k else None
            st["top_index"] = torch.empty(rows, k, dtype=torch.int32, device="cuda") if k else None
        else:
            # what the forward pass kept
            st["lse"], st["ent"] = torch.empty(rows, **f32), torch.empty(rows, **f32)
            step = max(1, (1 << 27) // vocab)
            for a in range(0, rows, step):
                z = x[a:a + step].double() * case["scale"]
                lse = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[:, None])
                st["lse"][a:a + step] = lse
                st["ent"][a:a + step] = lse - torch.where(p > 0, p * z, 0.0).sum(1)
            st["dlogp"] = torch.randn(rows, generator=gen, device="cuda") * (1.0 / rows)
            st["dent"] = torch.full((rows,), -0.01 / rows, **f32) if case["entropy"] else None
            st["dlogits"] = torch.empty(rows, vocab, dtype=dt, device="cuda")
        return st
    # a teacher that mostly agrees: the student's value at the listed tokens, with noise and a lead for some
    K = case["K"]
    step = max(1, (1 << 24) // vocab)
    idx = torch.empty(rows, K, dtype=torch.int64, device="cuda")
    for a in range(0, rows, step):
        b = min(rows, a + step)
        noise = torch.rand(b - a, allowed, generator=gen, device="cuda")
        idx[a:b] = noise.topk(K, dim=1).indices if K > 1 else noise.argmax(1, keepdim=True)
    got = x.gather(1, idx).float()
    st["teacher"] = (got + torch.randn(rows, K, generator=gen, device="cuda") * 1.5 + 4.0).to(dt)
    if rows > 1:  # some lists are shorter
        cut = torch.randint(0, 4 * K, (rows, 1), generator=gen, device="cuda")
        idx = torch.where(torch.arange(K, device="cuda")[None] <= cut, idx, torch.full_like(idx, -1))
    x.scatter_(1, idx.clamp(min=0), (x.gather(1, idx.clamp(min=0)).float() + 4.0).to(dt))
    st["index"] = idx
    unit = 64.0 if case["type"] == "f16" else 1.0 / rows  # fp16 gradients are kept in range by loss scaling
    w = torch.full((rows,), unit, **f32)
    if rows > 1:  # prompt positions take no part
        w = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.1, torch.zeros_like(w), w)
    st["row_weight"] = w
    st["loss"] = torch.empty(rows, **f32)
    st["dlogits"] = torch.empty(rows, vocab, dtype=dt, device="cuda")
    return st


# --- the plain forms ---------------------------------------------------------

def _plain_ln(st):
    c = st["case"]
    dt = st["x"].dtype
    x = st["x"].float()
    w = st["weight"].float()
    if c["dir"] == "fwd":
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + _EPS)
        y = xc * rstd[:, None] * w
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    dy = st["dy"].float()
    rstd = st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    out = {"dx": dx.to(dt), "dweight": (dy * xh).sum(0).to(st["weight"].dtype)}
    if st["bias"] is not None:
        out["dbias"] = dy.sum(0).to(st["bias"].dtype)
    return out


def _ordered(x):
    """int64 keys in the order (value falling, index rising), all different."""
    b = (x + 0.0).view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -1 - (b & 0x7FFFFFFF), b)
    n = x.shape[1]
    return b * (1 << 20) + (n - 1 - torch.arange(n, device=x.device))


def _plain_lp(st):
    c = st["case"]
    x = st["logits"].float()
    z = x * c["scale"]
    tgt = st["targets"]
    has = tgt >= 0
    at = tgt.clamp(min=0)[:, None]
    if c["dir"] == "fwd":
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        s = e.sum(1, keepdim=True)
        lse = (m + torch.log(s))[:, 0]
        out = {"lse": lse, "logp": torch.where(has, z.gather(1, at)[:, 0] - lse, 0.0)}
        if c["entropy"]:
            t = torch.where(e > 0, e * (z - m), 0.0).sum(1, keepdim=True)
            out["entropy"] = (torch.log(s) - t / s)[:, 0]
        if c["k"]:
            idx = x.shape[1] - 1 - (torch.topk(_ordered(x), c["k"], dim=1).values & ((1 << 20) - 1))
            out["top_index"] = idx.to(torch.int32)
            out["top_logp"] = z.gather(1, idx) - lse[:, None]
        return out
    lp = z - st["lse"][:, None]
    p = torch.exp(lp)
    d = torch.where(has, st["dlogp"], 0.0)[:, None]
    f = -d * p
    if c["entropy"]:
        f = f - st["dent"][:, None] * torch.where(p > 0, p * (lp + st["ent"][:, None]), 0.0)
    f = f.scatter_add(1, at, d)
    return {"dlogits": (f * c["scale"]).to(st["logits"].dtype)}


def _plain_distill(st):
    c = st["case"]
    z = st["logits"].float() * c["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    lse = m + torch.log(s)
    use = st["index"] >= 0
    at = st["index"].clamp(min=0)
    t = torch.where(use, st["teacher"].float() * c["scale"], -math.inf)
    t = t - t.amax(1, keepdim=True)
    logq = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    q = torch.exp(logq)
    w = st["row_weight"]
    kl = torch.where(q > 0, q * (logq - (z.gather(1, at) - lse)), 0.0).sum(1)
    f = (e / s).scatter_add(1, at, -q) * (w * c["scale"])[:, None]
    return {"loss": kl * w, "dlogits": f.to(st["logits"].dtype)}


# --- the library's calls -----------------------------------------------------

def _own_ln(st):
    import mixed_precision_adamw_gb300 as mp
    if st["case"]["dir"] == "fwd":
        mp.mp_layernorm_forward(st["y"], st["x"], st["weight"], st["bias"], _EPS, mean=st["mean"], rstd=st["rstd"])
        return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if "workspace" not in st:  # kept for the next pass, as a training loop does
        rows, d = st["x"].shape
        st["workspace"] = torch.empty(mp.mp_layernorm_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    mp.mp_layernorm_backward(st["dx"], st["dweight"], st["dbias"], st["dy"], st["x"], st["weight"], st["mean"],
                             st["rstd"], workspace=st["workspace"])
    out = {"dx": st["dx"], "dweight": st["dweight"]}
    if st["dbias"] is not None:
        out["dbias"] = st["dbias"]
    return out


def _own_lp(st):
    import mixed_precision_adamw_gb300 as mp
    c = st["case"]
    if c["dir"] == "fwd":
        mp.mp_token_logprob_forward(st["logits"], st["targets"], logp=st["logp"], lse=st["lse"], entropy=st["ent"],
                                    top_logp=st["top_logp"], top_index=st["top_index"], scale=c["scale"])
        out = {"lse": st["lse"], "logp": st["logp"]}
        if c["entropy"]:
            out["entropy"] = st["ent"]
        if c["k"]:
            out["top_index"], out["top_logp"] = st["top_index"], st["top_logp"]
        return out
    mp.mp_token_logprob_backward(st["dlogits"], st["logits"], st["targets"], lse=st["lse"], dlogp=st["dlogp"],
                                 entropy=st["ent"], dentropy=st["dent"], scale=c["scale"])
    return {"dlogits": st["dlogits"]}


def _own_distill(st):
    import mixed_precision_adamw_gb300 as mp
    mp.mp_distill_topk(st["loss"], st["dlogits"], st["logits"], st["teacher"], st["index"],
                       row_weight=st["row_weight"], scale=st["case"]["scale"])
    return {"loss": st["loss"], "dlogits": st["dlogits"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ln": _own_ln, "lp": _own_lp, "distill": _own_distill}[op](state)
    return {"ln": _plain_ln, "lp": _plain_lp, "distill": _plain_distill}[op](state)


# --- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ln":
        x, w = st["x"].double(), st["weight"].double()
        n = x.shape[1]
        mu = x.sum(1) / n
        var = ((x - mu[:, None]) ** 2).sum(1) / n
        r = (var + _EPS) ** -0.5
        xh = torch.einsum("rc,r->rc", x - mu[:, None], r)
        if case["dir"] == "fwd":
            y = xh * w + (st["bias"].double() if st["bias"] is not None else 0.0)
            return {"y": y, "mean": mu, "rstd": r}
        dy = st["dy"].double()
        # the transposed Jacobian of w * xh, row by row
        a = torch.einsum("rc,c->r", dy, w) / n
        b = torch.einsum("rc,c,rc->r", dy, w, xh) / n
        dx = (dy * w - a[:, None] - b[:, None] * xh) * r[:, None]
        out = {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xh)}
        if st["bias"] is not None:
            out["dbias"] = torch.einsum("rc->c", dy)
        return out
    rows, vocab = st["logits"].shape
    step = max(1, (1 << 27) // vocab)
    parts = []
    for a in range(0, rows, step):
        z = st["logits"][a:a + step].double() * case["scale"]
        n = z.shape[0]
        r = torch.arange(n, device=z.device)
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        p = torch.softmax(z, 1)
        if case["op"] == "lp":
            tgt = st["targets"][a:a + step]
            given = (tgt >= 0).double()
            at = tgt.clamp(min=0)
            if case["dir"] == "fwd":
                out = {"lse": lse, "logp": torch.where(tgt >= 0, lp[r, at], 0.0)}
                if case["entropy"]:
                    out["entropy"] = torch.special.entr(p).sum(1)
                if case["k"]:
                    out["top_logp"] = lp.sort(1, descending=True).values[:, :case["k"]]
            else:
                g = torch.zeros_like(p)
                g[r, at] = given * st["dlogp"][a:a + step].double()
                g -= p * g.sum(1, keepdim=True)
                if case["entropy"]:
                    h = torch.special.entr(p)
                    g += st["dent"][a:a + step].double()[:, None] * (h - p * h.sum(1, keepdim=True))
                out = {"dlogits": g * case["scale"]}
        else:
            idx = st["index"][a:a + step]
            t = (st["teacher"][a:a + step].double() * case["scale"]).masked_fill(idx < 0, -math.inf)
            q = torch.softmax(t, 1)
            w = st["row_weight"][a:a + step].double()
            at = idx.clamp(min=0)
            ce = -(q * torch.where(idx >= 0, lp.gather(1, at), 0.0)).sum(1)
            dense = torch.zeros_like(p).scatter_add_(1, at, q)
            out = {"loss": w * (ce - torch.special.entr(q).sum(1)),
                   "dlogits": (p - dense) * w[:, None] * case["scale"]}
        parts.append(out)
    got = {k: torch.cat([q[k] for q in parts]) for k in parts[0]}
    if case["op"] == "lp" and case["dir"] == "fwd" and case["k"]:
        got["top_index"] = None
    return got
