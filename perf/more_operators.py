"""Workloads of the operators of a transformer block between its matrix
products: RMS norm with the residual's addition (forward, with the output in
type or in 8 bits; backward with the weight gradient), rotary positions
(forward and inverse), the gated activation (forward and backward), and
activations kept in 8 bits for the backward pass (written and read by the two
above, or by themselves).

Each case is one pass through one operator. `run` computes it in plain torch
operations in 32 bits, rounded once at the end (own = False), or through the
library's entry points (own = True).

8 bits are e4m3 values with scales: one fp32 number a row, or one power of two
for every 32 columns, held as its exponent + 127.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-5
_E4M3 = torch.float8_e4m3fn
_MOST = {"bf16": 1 << 26, "f16": 1 << 26, "f32": 1 << 25}  # elements of a drawn case
_PLAIN = {"factor": 1.0, "context": 8192}


def listed():
    return [
        # one decoded token's residual stream: a launch's latency
        {"name": "rms fwd 1x4096 bf16", "op": "rms", "dir": "fwd", "rows": 1, "d": 4096, "type": "bf16",
         "wtype": "bf16", "residual": True, "out": "y", "kept": False, "pad": 0},
        # a micro-batch of 2 x 8192 tokens in front of an 8-bit product: a scale for each token
        {"name": "rms fwd 16384x4096 bf16 to 8 bits", "op": "rms", "dir": "fwd", "rows": 16384, "d": 4096,
         "type": "bf16", "wtype": "bf16", "residual": True, "out": "row8", "kept": False, "pad": 0},
        # the backward pass of 8192 tokens, the residual stream kept in 8 bits
        {"name": "rms bwd 8192x4096 bf16 from 8 bits", "op": "rms", "dir": "bwd", "rows": 8192, "d": 4096,
         "type": "bf16", "wtype": "bf16", "residual": True, "out": "y", "kept": True, "pad": 0},
        # odd width and length, fp32, no residual
        {"name": "rms bwd 3001x1365 f32", "op": "rms", "dir": "bwd", "rows": 3001, "d": 1365, "type": "f32",
         "wtype": "f32", "residual": False, "out": "y", "kept": False, "pad": 0},
        # one decoded token's queries and keys far into a long context
        {"name": "rope 1x(32+8)x128 bf16 bands", "op": "rope", "dir": "fwd", "tokens": 1, "q_heads": 32, "k_heads": 8,
         "head": 128, "rotary": 128, "layout": "half", "type": "bf16", "base": 500000.0, "scaling": "bands",
         "far": 131072},
        # a prompt of 16384 tokens
        {"name": "rope 16384x(32+8)x128 bf16 bands", "op": "rope", "dir": "fwd", "tokens": 16384, "q_heads": 32,
         "k_heads": 8, "head": 128, "rotary": 128, "layout": "half", "type": "bf16", "base": 500000.0,
         "scaling": "bands", "far": 131072},
        # gradients of a batch of odd length, half of each head rotated, neighbouring pairs
        {"name": "rope bwd 4097x(12+12)x64 f32 interleaved", "op": "rope", "dir": "bwd", "tokens": 4097, "q_heads": 12,
         "k_heads": 12, "head": 64, "rotary": 32, "layout": "interleaved", "type": "f32", "base": 10000.0,
         "scaling": "none", "far": 1024},
        # 8192 tokens of the 14336-wide activation, gate and up kept in 8 bits on the way
        {"name": "gated fwd 8192x14336 bf16 kept", "op": "gated", "dir": "fwd", "rows": 8192, "d": 14336,
         "type": "bf16", "act": "silu", "kept": True, "again": False, "fused": True},
        # the backward pass from what was kept, with the output again for the product behind it
        {"name": "gated bwd 8192x14336 bf16 from 8 bits", "op": "gated", "dir": "bwd", "rows": 8192, "d": 14336,
         "type": "bf16", "act": "silu", "kept": True, "again": True, "fused": True},
        # odd width and length, fp16, from gate and up themselves
        {"name": "gated bwd 1021x2731 f16 gelu", "op": "gated", "dir": "bwd", "rows": 1021, "d": 2731, "type": "f16",
         "act": "gelu", "kept": False, "again": False, "fused": True},
        # a layer's activations put away in 8 bits
        {"name": "pack 16384x4096 bf16", "op": "pack", "dir": "pack", "rows": 16384, "d": 4096, "type": "bf16",
         "scales": "block", "pad": 0},
        # and read back, odd width and length, a scale for each row
        {"name": "unpack 2047x1365 f32 rows", "op": "pack", "dir": "unpack", "rows": 2047, "d": 1365, "type": "f32",
         "scales": "row", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    d = _log_int(rng, lo, hi)
    if rng.random() < 0.6:  # widths are mostly multiples of 32, some odd
        d = max(lo, d // 32 * 32)
    return d


def draw(rng):
    op = rng.choice(["rms", "rms", "rope", "rope", "gated", "gated", "pack"])
    ty = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = _MOST[ty]
    if op == "rope":
        head = rng.choice([32, 64, 80, 96, 128, 128, 256])
        k_heads = rng.choice([1, 2, 4, 8, 12])
        q_heads = k_heads * rng.choice([1, 1, 2, 4, 8])
        tokens = min(_log_int(rng, 1, 32768), most // (head * (q_heads + k_heads)))
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "tokens": tokens, "q_heads": q_heads,
                "k_heads": k_heads, "head": head, "rotary": head if rng.random() < 0.6 else 2 * rng.randint(1, head // 2),
                "layout": rng.choice(["half", "interleaved"]), "type": ty,
                "base": rng.choice([10000.0, 500000.0, 1000000.0]),
                "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]),
                "far": rng.choice([1024, 8192, 131072, 1 << 20])}
    if op == "gated":
        d = _width(rng, 64, 28672)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "rows": min(_log_int(rng, 1, 32768), most // d), "d": d,
                "type": ty, "act": rng.choice(["silu", "silu", "gelu"]), "kept": rng.random() < 0.5,
                "again": rng.random() < 0.4, "fused": rng.random() < 0.7}
    d = _width(rng, 64, 8192)
    case = {"op": op, "rows": min(_log_int(rng, 1, 65536), most // d), "d": d, "type": ty,
            "pad": rng.choice([0, 0, 0, 8, 5])}
    if op == "pack":
        return {**case, "dir": rng.choice(["pack", "unpack"]), "scales": rng.choice(["row", "block"])}
    return {**case, "dir": rng.choice(["fwd", "bwd"]), "wtype": rng.choice([ty, "f32"]),
            "residual": rng.random() < 0.7, "out": rng.choice(["y", "y", "row8", "block8"]),
            "kept": rng.random() < 0.4}


def _bytes8(rows, d, scales):
    return rows * d + (4 * rows if scales == "row" else rows * -(-d // 32))


def work(case):
    e = _SIZE[case["type"]]
    if case["op"] == "rope":
        n = case["tokens"] * case["head"] * (case["q_heads"] + case["k_heads"])
        turned = case["tokens"] * case["rotary"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": 2 * e * n + 8 * case["tokens"] + 4 * case["rotary"], "flops": 3 * turned}
    rows, d = case["rows"], case["d"]
    n = rows * d
    kept = _bytes8(rows, d, "block")
    if case["op"] == "rms":
        we = _SIZE[case["wtype"]]
        if case["dir"] == "fwd":
            out = {"y": e * n, "row8": _bytes8(rows, d, "row"), "block8": kept}[case["out"]]
            b = e * n * (3 if case["residual"] else 1) + out + 4 * rows + we * d + (kept if case["kept"] else 0)
            return {"bytes": b, "flops": 6 * n}
        b = e * n * (3 if case["residual"] else 2) + (kept if case["kept"] else e * n) + 4 * rows + 2 * we * d
        return {"bytes": b, "flops": 12 * n}
    if case["op"] == "gated":
        if case["dir"] == "fwd":
            return {"bytes": 3 * e * n + (2 * kept if case["kept"] else 0), "flops": 12 * n}
        source = 2 * kept if case["kept"] else 2 * e * n
        return {"bytes": 3 * e * n + source + (e * n if case["again"] else 0), "flops": 20 * n}
    return {"bytes": e * n + _bytes8(rows, d, case["scales"]), "flops": 2 * n}


# --- 8 bits --------------------------------------------------------------------

def _pack(v, scales):
    """fp32 [rows, d] -> e4m3 values and scales, elementary operations."""
    rows, d = v.shape
    if scales == "row":
        s = torch.clamp(v.abs().amax(1) / 448.0, min=2.0 ** -126)
        return (v / s[:, None]).clamp(-448.0, 448.0).to(_E4M3), s
    blocks = -(-d // 32)
    w = torch.zeros(rows, blocks * 32, device=v.device)
    w[:, :d] = v
    w = w.view(rows, blocks, 32)
    m, k = torch.frexp(w.abs().amax(2))  # amax = m 2^k, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m == 0, -127, k - 9 + (m > 0.875).to(torch.int32)).clamp(min=-127)
    q = torch.ldexp(w, -e[:, :, None]).view(rows, blocks * 32)[:, :d].to(_E4M3)
    return q.contiguous(), (e + 127).to(torch.uint8)


def _unpack(q, s):
    v = q.float()
    if s.dtype == torch.float32:
        return v * s[:, None]
    rows, d = v.shape
    f = torch.ldexp(torch.ones((), device=v.device), s.to(torch.int32) - 127)
    return v * f.repeat_interleave(32, dim=1)[:, :d]


def _new8(rows, d, scales):
    s = (torch.empty(rows, device="cuda") if scales == "row"
         else torch.empty(rows, -(-d // 32), dtype=torch.uint8, device="cuda"))
    return torch.empty(rows, d, dtype=_E4M3, device="cuda"), s


# --- inputs --------------------------------------------------------------------

def _randn(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _stream(rows, width, gen, dtype):
    """A residual stream: some channels a good deal larger than the others."""
    channel = torch.exp(torch.randn(width, generator=gen, device="cuda") * 0.8)
    return (torch.randn(rows, width, generator=gen, device="cuda") * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["type"]]
    st = {"case": dict(case)}
    if case["op"] == "rope":
        return _prepare_rope(st, case, gen, dt)
    rows, d = case["rows"], case["d"]
    if case["op"] == "rms":
        wdt = _DT[case["wtype"]]
        st["weight"] = (1.0 + torch.randn(d, generator=gen, device="cuda") * 0.1).to(wdt)
        x = _stream(rows, d + case["pad"], gen, dt)[:, :d]
        if case["dir"] == "fwd":
            st["x"] = x
            st["residual"] = _stream(rows, d + case["pad"], gen, dt)[:, :d] if case["residual"] else None
            st["h"] = torch.empty(rows, d, dtype=dt, device="cuda") if case["residual"] else None
            st["rstd"] = torch.empty(rows, device="cuda")
            st["y"] = torch.empty(rows, d, dtype=dt, device="cuda") if case["out"] == "y" else None
            st["y8"] = _new8(rows, d, case["out"][:-1]) if case["out"] != "y" else None
            st["h8"] = _new8(rows, d, "block") if case["kept"] else None
            return st
        # what the forward pass kept
        st["rstd"] = ((x.double() ** 2).mean(1) + _EPS).rsqrt().float()
        if case["kept"]:
            st["h"], st["h_scale"] = _pack(x.float(), "block")
        else:
            st["h"], st["h_scale"] = x, None
        st["dy"] = _randn((rows, d), gen, 1.0, dt)
        st["dh"] = _randn((rows, d), gen, 1.0, dt) if case["residual"] else None
        st["dx"] = torch.empty(rows, d, dtype=dt, device="cuda")
        st["dweight"] = torch.empty(d, dtype=wdt, device="cuda")
        return st
    if case["op"] == "gated":
        if case["fused"]:  # one product's output holds both
            both = _randn((rows, 2 * d), gen, 1.5, dt)
            gate, up = both[:, :d], both[:, d:]
        else:
            gate, up = _randn((rows, d), gen, 1.5, dt), _randn((rows, d), gen, 1.5, dt)
        st["gate"], st["up"], st["gate_scale"], st["up_scale"] = gate, up, None, None
        if case["dir"] == "fwd":
            st["y"] = torch.empty(rows, d, dtype=dt, device="cuda")
            st["gate8"] = _new8(rows, d, "block") if case["kept"] else None
            st["up8"] = _new8(rows, d, "block") if case["kept"] else None
            return st
        if case["kept"]:
            st["gate"], st["gate_scale"] = _pack(gate.float(), "block")
            st["up"], st["up_scale"] = _pack(up.float(), "block")
        st["dy"] = _randn((rows, d), gen, 1.0, dt)
        if case["fused"]:
            both = torch.empty(rows, 2 * d, dtype=dt, device="cuda")
            st["dgate"], st["dup"] = both[:, :d], both[:, d:]
        else:
            st["dgate"], st["dup"] = (torch.empty(rows, d, dtype=dt, device="cuda") for _ in range(2))
        st["y"] = torch.empty(rows, d, dtype=dt, device="cuda") if case["again"] else None
        return st
    x = _stream(rows, d + case["pad"], gen, dt)[:, :d]
    if case["dir"] == "pack":
        st["x"] = x
        st["q"], st["scale"] = _new8(rows, d, case["scales"])
    else:
        st["q"], st["scale"] = _pack(x.float(), case["scales"])
        st["x"] = torch.empty(rows, d, dtype=dt, device="cuda")
    return st


def _frequencies(case):
    """Radians a position of each pair, fp64, and the factor of the result."""
    r, base, context = case["rotary"], case["base"], _PLAIN["context"]
    stretch = max(1.0, case["far"] / context) if case["scaling"] != "none" else 1.0
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "base" and r > 2:  # a larger base, so that the slowest pair is stretched by the factor
        base = base * stretch ** (r / (r - 2))
    f = base ** (-i / r)
    if case["scaling"] == "linear":
        return f / stretch, 1.0
    if case["scaling"] == "bands":  # long waves stretched, short ones kept, a blend between
        s = ((context * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * ((1 - s) / stretch + s), 1.0
    if case["scaling"] == "ramp":  # the same over the pair's index, between those of 32 turns and 1 turn in the context
        def index(turns):
            return r * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(index(32.0))), min(r - 1.0, math.ceil(index(1.0)))
        s = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (s / stretch + 1 - s), 0.1 * math.log(stretch) + 1.0
    return f, 1.0


def _prepare_rope(st, case, gen, dt):
    t, hq, hk, D = case["tokens"], case["q_heads"], case["k_heads"], case["head"]
    # queries, keys and values come out of one product
    qkv = _randn((t, (hq + 2 * hk) * D), gen, 1.0, dt)
    st["q"] = qkv[:, :hq * D].view(t, hq, D)
    st["k"] = qkv[:, hq * D:(hq + hk) * D].view(t, hk, D)
    st["q_out"] = torch.empty(t, hq, D, dtype=dt, device="cuda")
    st["k_out"] = torch.empty(t, hk, D, dtype=dt, device="cuda")
    # the sequences of a batch one after the other, each from a place of its own
    run = max(1, t // 3)
    at = torch.arange(t, device="cuda") % run
    start = torch.randint(0, max(1, case["far"] - run), (-(-t // run),), generator=gen, device="cuda")
    st["positions"] = at + start[torch.arange(t, device="cuda") // run]
    st["frequencies"], st["factor"] = _frequencies(case)
    return st


# --- the plain forms -----------------------------------------------------------

def _plain_rms(st):
    c = st["case"]
    w = st["weight"].float()
    if c["dir"] == "fwd":
        x = st["x"].float()
        if st["residual"] is not None:
            x = (x + st["residual"].float()).to(st["x"].dtype).float()  # the norm is of the stored sum
        rstd = 1.0 / torch.sqrt((x * x).mean(1) + _EPS)
        y = x * rstd[:, None] * w
        out = {"rstd": rstd}
        if st["residual"] is not None:
            out["h"] = x.to(st["x"].dtype)
        if c["out"] == "y":
            out["y"] = y.to(st["x"].dtype)
        elif c["out"] == "row8":
            out["y8"], out["y8_scale"] = _pack(y, "row")
        else:
            out["y8"] = _unpack(*_pack(y, "block")).to(torch.bfloat16)
        if c["kept"]:
            out["h8"], out["h8_scale"] = _pack(x, "block")
        return out
    h = st["h"].float() if st["h_scale"] is None else _unpack(st["h"], st["h_scale"])
    rstd = st["rstd"][:, None]
    dy = st["dy"].float()
    xh = h * rstd
    g = dy * w
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(st["dy"].dtype), "dweight": (dy * xh).sum(0).to(st["weight"].dtype)}


def _plain_rope(st):
    c = st["case"]
    r = c["rotary"]
    angle = st["positions"].double()[:, None] * st["frequencies"]
    cos = (torch.cos(angle) * st["factor"]).float()[:, None, :]
    sin = (torch.sin(angle) * st["factor"]).float()[:, None, :]
    if c["dir"] == "bwd":
        sin = -sin
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        a, b = (x[..., :r // 2], x[..., r // 2:r]) if c["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
        u, v = a * cos - b * sin, a * sin + b * cos
        turned = torch.cat((u, v), -1) if c["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
        out[name] = torch.cat((turned, x[..., r:]), -1).to(st[name].dtype)
    return out


def _plain_gated(st):
    c = st["case"]
    a = st["gate"].float() if st["gate_scale"] is None else _unpack(st["gate"], st["gate_scale"])
    b = st["up"].float() if st["up_scale"] is None else _unpack(st["up"], st["up_scale"])
    dt = _DT[c["type"]]
    k = 2.0 * math.sqrt(2.0 / math.pi)
    v = a if c["act"] == "silu" else k * (a + 0.044715 * a * a * a)
    s = 1.0 / (1.0 + torch.exp(-v))
    if c["dir"] == "fwd":
        out = {"y": (a * s * b).to(dt)}
        if c["kept"]:
            out["gate8"], out["gate8_scale"] = _pack(a, "block")
            out["up8"], out["up8_scale"] = _pack(b, "block")
        return out
    dv = 1.0 if c["act"] == "silu" else k * (1.0 + 3.0 * 0.044715 * a * a)
    dy = st["dy"].float()
    out = {"dgate": (dy * b * (s + a * s * (1.0 - s) * dv)).to(dt), "dup": (dy * a * s).to(dt)}
    if c["again"]:
        out["y"] = (a * s * b).to(dt)
    return out


def _plain_pack(st):
    if st["case"]["dir"] == "pack":
        q, s = _pack(st["x"].float(), st["case"]["scales"])
        return {"q": q, "scale": s}
    return {"x": _unpack(st["q"], st["scale"]).to(st["x"].dtype)}


# --- the library's calls -------------------------------------------------------

def _own_rms(st):
    import mixed_precision_adamw_gb300 as mp
    c = st["case"]
    if c["dir"] == "fwd":
        y8, h8 = st["y8"] or (None, None), st["h8"] or (None, None)
        mp.mp_rmsnorm_forward(st["y"], st["x"], st["weight"], _EPS, residual=st["residual"], h=st["h"],
                              rstd=st["rstd"], y8=y8[0], y8_scale=y8[1], h8=h8[0], h8_scale=h8[1])
        out = {"rstd": st["rstd"]}
        if st["residual"] is not None:
            out["h"] = st["h"]
        if c["out"] == "y":
            out["y"] = st["y"]
        elif c["out"] == "row8":
            out["y8"], out["y8_scale"] = y8
        else:  # read back as the values that it stands for
            out["y8"] = torch.empty(y8[0].shape, dtype=torch.bfloat16, device="cuda")
            mp.mp_unpack8(out["y8"], *y8)
        if c["kept"]:
            out["h8"], out["h8_scale"] = h8
        return out
    if "workspace" not in st:  # kept for the next pass, as a training loop does
        n = mp.mp_rmsnorm_workspace_bytes(*st["dy"].shape)
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    mp.mp_rmsnorm_backward(st["dx"], st["dweight"], st["dy"], st["h"], st["weight"], st["rstd"], dh=st["dh"],
                           h_scale=st["h_scale"], workspace=st["workspace"])
    return {"dx": st["dx"], "dweight": st["dweight"]}


def _own_rope(st):
    import mixed_precision_adamw_gb300 as mp
    c = st["case"]
    if "turns" not in st:  # a model's table, made once
        stretch = max(1.0, c["far"] / _PLAIN["context"])
        scaling = None if c["scaling"] == "none" else mp.RopeScaling(c["scaling"], stretch, context=_PLAIN["context"])
        st["turns"], st["result"] = mp.mp_rope_frequencies(c["rotary"], c["base"], scaling, device="cuda")
    mp.mp_rope(st["q_out"], st["q"], st["k_out"], st["k"], st["turns"], st["positions"],
               interleaved=c["layout"] == "interleaved", inverse=c["dir"] == "bwd", factor=st["result"])
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_gated(st):
    import mixed_precision_adamw_gb300 as mp
    c = st["case"]
    if c["dir"] == "fwd":
        g8, u8 = st["gate8"] or (None, None), st["up8"] or (None, None)
        mp.mp_gated_forward(st["y"], st["gate"], st["up"], activation=c["act"], gate8=g8[0], gate8_scale=g8[1],
                            up8=u8[0], up8_scale=u8[1])
        out = {"y": st["y"]}
        if c["kept"]:
            out["gate8"], out["gate8_scale"] = g8
            out["up8"], out["up8_scale"] = u8
        return out
    mp.mp_gated_backward(st["dgate"], st["dup"], st["dy"], st["gate"], st["up"], activation=c["act"],
                         gate_scale=st["gate_scale"], up_scale=st["up_scale"], y=st["y"])
    out = {"dgate": st["dgate"], "dup": st["dup"]}
    if c["again"]:
        out["y"] = st["y"]
    return out


def _own_pack(st):
    import mixed_precision_adamw_gb300 as mp
    if st["case"]["dir"] == "pack":
        mp.mp_pack8(st["q"], st["scale"], st["x"])
        return {"q": st["q"], "scale": st["scale"]}
    mp.mp_unpack8(st["x"], st["q"], st["scale"])
    return {"x": st["x"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rms": _own_rms, "rope": _own_rope, "gated": _own_gated, "pack": _own_pack}[op](state)
    return {"rms": _plain_rms, "rope": _plain_rope, "gated": _plain_gated, "pack": _plain_pack}[op](state)


# --- the definitions in 64 bits --------------------------------------------------

def _read8(q, s):
    """What 8-bit values stand for, in 64 bits."""
    rows, d = q.shape
    if s.dtype == torch.float32:
        return q.double() * s.double()[:, None]
    column = torch.arange(d, device=q.device) // 32
    return q.double() * torch.exp2(s.double() - 127.0)[:, column]


def _scaled8(v, scales):
    """v over its scale before the rounding to 8 bits, and the scale (64 bits)."""
    rows, d = v.shape
    if scales == "row":
        s = (v.abs().max(1).values / 448.0).clamp(min=2.0 ** -126)
        return v / s[:, None], s
    column = torch.arange(d, device=v.device) // 32
    top = torch.zeros(rows, -(-d // 32), dtype=torch.float64, device=v.device)
    top.scatter_reduce_(1, column.expand(rows, d), v.abs(), "amax")
    m, k = torch.frexp(top / 448.0)  # the least power of two not below it, exactly
    e = torch.where(top > 0, k - (m == 0.5).to(k.dtype), -127).clamp(min=-127)
    return v / torch.exp2(e.double())[:, column], None


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rms":
        w = st["weight"].double()
        if case["dir"] == "fwd":
            h = st["x"].double()
            out = {}
            if st["residual"] is not None:
                out["h"] = h + st["residual"].double()
                # the norm is of the sum as it is stored; 32-bit inputs' sum is rounded once
                h = out["h"].to(st["x"].dtype).double()
            r = (torch.einsum("rc,rc->r", h, h) / h.shape[1] + _EPS) ** -0.5
            y = torch.einsum("rc,r,c->rc", h, r, w)
            out["rstd"] = r
            if case["out"] == "y":
                out["y"] = y
            elif case["out"] == "row8":
                out["y8"], out["y8_scale"] = _scaled8(y, "row")
            else:
                out["y8"] = y
            if case["kept"]:
                out["h8"], out["h8_scale"] = _scaled8(h, "block")
            return out
        h = st["h"].double() if st["h_scale"] is None else _read8(st["h"], st["h_scale"])
        r, dy = st["rstd"].double(), st["dy"].double()
        # the transposed Jacobian of h r(h) w, row by row
        along = torch.einsum("rc,c,rc->r", dy, w, h) * r ** 3 / h.shape[1]
        dx = torch.einsum("rc,c,r->rc", dy, w, r) - along[:, None] * h
        if st["dh"] is not None:
            dx = dx + st["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, h, r)}
    if case["op"] == "rope":
        r = case["rotary"]
        sign = -1.0 if case["dir"] == "bwd" else 1.0
        angle = sign * torch.outer(st["positions"].double(), st["frequencies"])
        turn = torch.polar(torch.full_like(angle, st["factor"]), angle)[:, None, :]
        out = {}
        for name in ("q", "k"):
            x = st[name].double().clone()
            half = case["layout"] == "half"
            z = (torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) if half
                 else torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2))) * turn
            x[..., :r] = torch.cat((z.real, z.imag), -1) if half else torch.view_as_real(z).flatten(-2)
            out[name] = x
        return out
    if case["op"] == "gated":
        a = st["gate"].double() if st["gate_scale"] is None else _read8(st["gate"], st["gate_scale"])
        b = st["up"].double() if st["up_scale"] is None else _read8(st["up"], st["up_scale"])
        if case["act"] == "silu":
            s = torch.sigmoid(a)
            f, df = a * s, s + a * s * torch.sigmoid(-a)
        else:
            c = math.sqrt(2.0 / math.pi)
            t = torch.tanh(c * (a + 0.044715 * a ** 3))
            f = 0.5 * a * (1.0 + t)
            df = 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t ** 2) * c * (1.0 + 0.134145 * a ** 2)
        if case["dir"] == "fwd":
            out = {"y": f * b}
            if case["kept"]:
                out["gate8"], out["gate8_scale"] = _scaled8(a, "block")
                out["up8"], out["up8_scale"] = _scaled8(b, "block")
            return out
        dy = st["dy"].double()
        out = {"dgate": dy * b * df, "dup": dy * f}
        if case["again"]:
            out["y"] = f * b
        return out
    if case["dir"] == "pack":
        q, s = _scaled8(st["x"].double(), case["scales"])
        return {"q": q, "scale": s}
    return {"x": _read8(st["q"], st["scale"])}
