"""Python entry points of include/mp_block.h: what a transformer block computes
between its matrix products, forward and backward, and activations kept in 8
bits.

As in the rest of the package every buffer is the caller's, every call only
enqueues work on the stream (the current one unless given) and a non-OK status
raises MpError. Matrices are as in train.py. Rows in 8 bits are 2-D tensors of
float8_e4m3fn (or uint8) with contiguous rows; their scales tell the kind: a
contiguous float32 [rows], or uint8 [rows, ceil(d / 32)] of exponents + 127.
"""
from __future__ import annotations

import ctypes
import importlib.util
from typing import Optional, Tuple

import torch

from . import _check, _lib, _raw_stream, _stream
from .train import MP_FP32, MP_INT64, _F32, _INDEX_TYPES, _TYPES, _U8, _index_type, _matrix, _on, _rows, _vector, _weight_type

MP_SCALE_ROW, MP_SCALE_BLOCK = 1, 2
MP_ACT_SILU, MP_ACT_GELU = 0, 1
ACTIVATIONS = {"silu": MP_ACT_SILU, "gelu": MP_ACT_GELU}
ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

_E4M3 = torch.float8_e4m3fn
_BYTES = frozenset((_E4M3, torch.uint8))


class MpRopeScaling(ctypes.Structure):
    """mp_rope_scaling_t."""
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", ctypes.c_double),
                ("context", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double)]


def _declare():
    vp, i64, i32, f32, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    for name, res, args in (
            ("mp_rmsnorm_forward", ctypes.c_int, [vp] * 10 + [i64] * 8 + [f32, i32, i32, i32, vp]),
            ("mp_rmsnorm_workspace_bytes", size, [i64, i64]),
            ("mp_rmsnorm_backward", ctypes.c_int, [vp] * 8 + [i64] * 6 + [i32, i32, vp, size, vp]),
            ("mp_rope", ctypes.c_int,
             [vp] * 6 + [i64, i64] + [i32] * 4 + [i64] * 8 + [f32] + [i32] * 4 + [vp]),
            ("mp_rope_frequencies", ctypes.c_int,
             [vp, ctypes.POINTER(f32), i32, ctypes.c_double, ctypes.POINTER(MpRopeScaling)]),
            ("mp_gated_forward", ctypes.c_int, [vp] * 7 + [i64] * 7 + [i32, i32, vp]),
            ("mp_gated_backward", ctypes.c_int, [vp] * 8 + [i64] * 8 + [i32, i32, vp]),
            ("mp_pack8", ctypes.c_int, [vp] * 3 + [i64] * 4 + [i32, i32, vp]),
            ("mp_unpack8", ctypes.c_int, [vp] * 3 + [i64] * 4 + [i32, i32, vp])):
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = res, args


_declare()

_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_current_stream = _raw_stream or _current_stream  # without a Stream object, where PyTorch can


class _NoBinding:
    """In place of _binding where it was not built (or by another Python): makes no call."""

    def __getattr__(self, name):
        return lambda *args: None


# _binding makes the ordinary calls (each function below begins with it) and
# returns None for all others: those go through the checks here, which name
# what is wrong.
if importlib.util.find_spec("._binding", __package__) is None:
    _binding = _NoBinding()
else:
    from . import _binding
_binding.bind(torch.Tensor, torch.nn.Parameter,
              (torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32,
               torch.int64), _device, _current_stream,
              tuple(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in
                    ("mp_rmsnorm_forward", "mp_rmsnorm_backward", "mp_rope", "mp_gated_forward",
                     "mp_gated_backward", "mp_pack8", "mp_unpack8")))


def _matrix8(t, scale, name: str, dev: int, rows: int, d: int):
    """(pointer, row stride, scale pointer, kind) of rows in 8 bits; Nones for None."""
    if t is None:
        if scale is not None:
            raise ValueError(f"{name}_scale: given without {name}")
        return None, 0, None, 0
    if scale is None:
        raise ValueError(f"{name}: given without its scales")
    if not isinstance(t, torch.Tensor) or not isinstance(scale, torch.Tensor):
        raise TypeError(f"{name}: expected torch.Tensors")
    if t.dtype not in _BYTES:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_BYTES)}")
    _on(t, name, dev)
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != d:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, d)}")
    p, stride = _rows(t, name, None)
    if scale.dtype == torch.float32:
        return p, stride, _vector(scale, name + "_scale", dev, rows, _F32), MP_SCALE_ROW
    return p, stride, _vector(scale, name + "_scale", dev, rows * ((d + 31) // 32), _U8), MP_SCALE_BLOCK


def _block_scaled(kind: int, name: str) -> None:
    if kind == MP_SCALE_ROW:
        raise TypeError(f"{name}_scale: one power of two for 32 columns (uint8) expected")


def mp_rmsnorm_forward(y: Optional[torch.Tensor], x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, *, residual: Optional[torch.Tensor] = None,
                       h: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                       y8: Optional[torch.Tensor] = None, y8_scale: Optional[torch.Tensor] = None,
                       h8: Optional[torch.Tensor] = None, h8_scale: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Enqueue y = RMS norm of h = x + residual over its last dimension, times
    weight. h (the sum, the next residual), rstd (float32 [rows], for the
    backward pass), y8 (y in 8 bits, scales of either kind) and h8 (h in 8 bits for the
    backward pass, scales of 32 columns) are written if given; y may be None.
    y and h may be x or residual themselves."""
    st = _binding.rmsnorm_forward(y, x, weight, eps, residual, h, rstd, y8, y8_scale, h8, h8_scale, stream)
    if st is None:
        st = _rmsnorm_forward(y, x, weight, eps, residual, h, rstd, y8, y8_scale, h8, h8_scale, stream)
    if st:
        _check(st, "mp_rmsnorm_forward")


def _rmsnorm_forward(y, x, weight, eps, residual, h, rstd, y8, y8_scale, h8, h8_scale, stream) -> int:
    dev = torch.cuda.current_device()
    xp, xs, code = _matrix(x, "x", dev)
    rows, d = x.shape
    yp, ys, _ = (None, 0, 0) if y is None else _matrix(y, "y", dev, x)
    rp, rs, _ = (None, 0, 0) if residual is None else _matrix(residual, "residual", dev, x)
    hp, hs, _ = (None, 0, 0) if h is None else _matrix(h, "h", dev, x)
    y8p, y8n, y8s, kind = _matrix8(y8, y8_scale, "y8", dev, rows, d)
    h8p, h8n, h8s, hkind = _matrix8(h8, h8_scale, "h8", dev, rows, d)
    _block_scaled(hkind, "h8")
    return _lib.mp_rmsnorm_forward(
        yp, hp, _vector(rstd, "rstd", dev, rows, _F32), y8p, y8s, h8p, h8s, xp, rp,
        _vector(weight, "weight", dev, d, _TYPES), rows, d, ys, hs, y8n, h8n, xs, rs, eps, code,
        MP_FP32 if weight is None else _TYPES[weight.dtype], kind, _stream(stream))


def mp_rmsnorm_workspace_bytes(rows: int, d: int) -> int:
    """Bytes of scratch that mp_rmsnorm_backward needs for the weight gradient."""
    return int(_lib.mp_rmsnorm_workspace_bytes(rows, d))


def mp_rmsnorm_backward(dx: Optional[torch.Tensor], dweight: Optional[torch.Tensor], dy: torch.Tensor,
                        h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor, *,
                        dh: Optional[torch.Tensor] = None, h_scale: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the RMS norm's backward pass: dx [rows, d], the gradient of x and
    of the residual (with dh, the gradient that reaches h otherwise, added), and the
    weight's gradient summed over the rows (written, not added to). h: the
    forward pass's h (or x), or h8 with h_scale. dx may be dy, dh or h itself. workspace: uint8 of
    mp_rmsnorm_workspace_bytes(rows, d) bytes, when dweight is given."""
    st = _binding.rmsnorm_backward(dx, dweight, dy, h, weight, rstd, dh, h_scale, workspace, stream)
    if st is None:
        st = _rmsnorm_backward(dx, dweight, dy, h, weight, rstd, dh, h_scale, workspace, stream)
    if st:
        _check(st, "mp_rmsnorm_backward")


def _rmsnorm_backward(dx, dweight, dy, h, weight, rstd, dh, h_scale, workspace, stream) -> int:
    dev = torch.cuda.current_device()
    dyp, dys, code = _matrix(dy, "dy", dev)
    rows, d = dy.shape
    if h_scale is None:
        hp, hs, _ = _matrix(h, "h", dev, dy)
        hsp = None
    else:
        hp, hs, hsp, kind = _matrix8(h, h_scale, "h", dev, rows, d)
        _block_scaled(kind, "h")
    dxp, dxs, _ = (None, 0, 0) if dx is None else _matrix(dx, "dx", dev, dy)
    dhp, dhs, _ = (None, 0, 0) if dh is None else _matrix(dh, "dh", dev, dy)
    wsp, wsn = None, 0
    if workspace is not None:
        wsn = workspace.numel()
        wsp = _vector(workspace, "workspace", dev, wsn, _U8)
    return _lib.mp_rmsnorm_backward(
        dxp, _vector(dweight, "dweight", dev, d, _TYPES), dyp, dhp, hp, hsp, _vector(weight, "weight", dev, d, _TYPES),
        _vector(rstd, "rstd", dev, rows, _F32), rows, d, dxs, dys, dhs, hs, code, _weight_type(weight, dweight), wsp,
        wsn, _stream(stream))


class RopeScaling:
    """How rotary frequencies are changed for contexts `factor` times as long as
    the `context` positions trained with: "linear", "base", "bands" or "ramp"
    (see mp_rope_kind_t in include/mp_block.h). low and high: turns of a pair
    in the context between which the last two blend (1 and 4; 1 and 32)."""

    def __init__(self, kind: str, factor: float, *, context: float = 8192, low: float = 1.0,
                 high: Optional[float] = None):
        if kind not in ROPE_KINDS:
            raise ValueError(f"kind: one of {sorted(ROPE_KINDS)}")
        self._s = MpRopeScaling(ROPE_KINDS[kind], 0, float(factor), float(context), float(low),
                                float(high if high is not None else 32.0 if kind == "ramp" else 4.0))


def mp_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[RopeScaling] = None,
                        device=None) -> Tuple[torch.Tensor, float]:
    """(turns, factor) for mp_rope: int64 [rotary_dim / 2], each frequency as a
    64-bit fraction of a turn, copied to `device` (the current CUDA device unless given)."""
    rotary_dim = max(0, min(rotary_dim, 1 << 20))  # within 32 bits; longer than a head may be: refused below
    turns = torch.empty(rotary_dim // 2, dtype=torch.int64)
    factor = ctypes.c_float()
    _check(_lib.mp_rope_frequencies(turns.data_ptr(), ctypes.byref(factor), rotary_dim, base,
                                    None if scaling is None else ctypes.byref(scaling._s)), "mp_rope_frequencies")
    return turns.to("cuda" if device is None else device), factor.value


def _heads(t, name: str, dev: int, like=None):
    """(pointer, token stride, head stride, code) of [tokens, heads, head_dim]
    with contiguous heads' values, tokens or heads outermost, of the shape and
    type of `like` if given."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev:
        code = _TYPES.get(t.dtype)
        if code is not None and t.dim() == 3 and (like is None or (t.shape == like.shape and t.dtype == like.dtype)):
            tokens, heads, dim = t.shape
            ts, hs, last = t.stride()
            if last == 1 and hs >= dim and ts >= (heads - 1) * hs + dim:
                return t.data_ptr(), ts, hs, code
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_TYPES)}")
    _on(t, name, dev)
    if t.dim() != 3:
        raise ValueError(f"{name}: {t.dim()}-D, expected [tokens, heads, head_dim]")
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {like.dtype}")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    tokens, heads, dim = t.shape
    ts, hs, last = t.stride()
    if last != 1 and dim > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if heads > 1 and hs < dim or tokens > 1 and ts < dim:
        raise ValueError(f"{name}: strides {ts}, {hs} < {dim}")
    if heads > 1 and tokens > 1 and ts < (heads - 1) * hs + dim and hs < (tokens - 1) * ts + dim:
        raise ValueError(f"{name}: strides {ts}, {hs}: heads overlap")
    return t.data_ptr(), ts if tokens > 1 else max(ts, dim), hs if heads > 1 else max(hs, dim), code


def mp_rope(q_out: torch.Tensor, q: torch.Tensor, k_out: Optional[torch.Tensor], k: Optional[torch.Tensor],
            turns: torch.Tensor, positions: Optional[torch.Tensor] = None, *, first_position: int = 0,
            interleaved: bool = False, inverse: bool = False, factor: float = 1.0, stream=None) -> None:
    """Enqueue the rotation of queries [tokens, heads, head_dim] and keys (heads of
    their own number; None: none) by their positions (int32 or int64 [tokens];
    None: first_position, first_position + 1, ...). turns and factor are
    mp_rope_frequencies' (rotary_dim = 2 len(turns); a head's further columns are
    copied). inverse: the rotation back, which is the gradient. Outputs may be the inputs themselves."""
    st = _binding.rope(q_out, q, k_out, k, turns, positions, first_position, interleaved, inverse, factor, stream)
    if st is None:
        st = _rope(q_out, q, k_out, k, turns, positions, first_position, interleaved, inverse, factor, stream)
    if st:
        _check(st, "mp_rope")


def _rope(q_out, q, k_out, k, turns, positions, first_position, interleaved, inverse, factor, stream) -> int:
    dev = torch.cuda.current_device()
    qp, qts, qhs, code = _heads(q, "q", dev)
    qop, qots, qohs, _ = _heads(q_out, "q_out", dev, q)
    tokens, q_heads, dim = q.shape
    kp = kop = None
    kts = khs = kots = kohs = k_heads = 0
    if k is not None:
        if k_out is None:
            raise ValueError("k_out: missing")
        kp, kts, khs, kcode = _heads(k, "k", dev)
        kop, kots, kohs, _ = _heads(k_out, "k_out", dev, k)
        if kcode != code:
            raise TypeError(f"k: dtype {k.dtype}, expected {q.dtype}")
        if k.shape[0] != tokens or k.shape[2] != dim:
            raise ValueError(f"k: shape {tuple(k.shape)}, expected {tokens} tokens, head_dim {dim}")
        k_heads = k.shape[1]
    elif k_out is not None:
        raise ValueError("k: missing")
    pairs = turns.numel()
    icode = MP_INT64 if positions is None else _index_type(positions, "positions")
    return _lib.mp_rope(
        qop, qp, kop, kp, _vector(turns, "turns", dev, pairs, (torch.int64,)),
        _vector(positions, "positions", dev, tokens, _INDEX_TYPES), first_position, tokens, q_heads, k_heads, dim,
        2 * pairs, qots, qohs, qts, qhs, kots, kohs, kts, khs, factor, interleaved, inverse, code, icode,
        _stream(stream))


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation: one of {sorted(ACTIVATIONS)}")
    return code


def mp_gated_forward(y: torch.Tensor, gate: torch.Tensor, up: Optional[torch.Tensor] = None, *,
                     activation: str = "silu", gate8: Optional[torch.Tensor] = None,
                     gate8_scale: Optional[torch.Tensor] = None, up8: Optional[torch.Tensor] = None,
                     up8_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue y = act(gate) * up (act(gate) without up), and gate and up in 8
    bits (scales of 32 columns) for the backward pass if wanted. y may be gate
    or up itself. activation: "silu", or "gelu", which is its form with tanh
    (PyTorch's approximate="tanh")."""
    act = _activation(activation)
    st = _binding.gated_forward(y, gate, up, act, gate8, gate8_scale, up8, up8_scale, stream)
    if st is None:
        st = _gated_forward(y, gate, up, act, gate8, gate8_scale, up8, up8_scale, stream)
    if st:
        _check(st, "mp_gated_forward")


def _gated_forward(y, gate, up, act, gate8, gate8_scale, up8, up8_scale, stream) -> int:
    dev = torch.cuda.current_device()
    gp, gs, code = _matrix(gate, "gate", dev)
    yp, ys, _ = _matrix(y, "y", dev, gate)
    up_, us, _ = (None, 0, 0) if up is None else _matrix(up, "up", dev, gate)
    rows, d = gate.shape
    g8p, g8n, g8s, gkind = _matrix8(gate8, gate8_scale, "gate8", dev, rows, d)
    u8p, u8n, u8s, ukind = _matrix8(up8, up8_scale, "up8", dev, rows, d)
    _block_scaled(gkind, "gate8")
    _block_scaled(ukind, "up8")
    return _lib.mp_gated_forward(yp, g8p, g8s, u8p, u8s, gp, up_, rows, d, ys, g8n, u8n, gs, us, act, code,
                                 _stream(stream))


def mp_gated_backward(dgate: torch.Tensor, dup: Optional[torch.Tensor], dy: torch.Tensor, gate: torch.Tensor,
                      up: Optional[torch.Tensor] = None, *, activation: str = "silu",
                      gate_scale: Optional[torch.Tensor] = None, up_scale: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the gradients of gate and up, from gate and up themselves or (with
    gate_scale and up_scale) from what the forward pass kept in 8 bits; and, if
    wanted, y = act(gate) * up again. dgate and dup may be dy, gate or up
    themselves."""
    act = _activation(activation)
    st = _binding.gated_backward(dgate, dup, dy, gate, up, act, gate_scale, up_scale, y, stream)
    if st is None:
        st = _gated_backward(dgate, dup, dy, gate, up, act, gate_scale, up_scale, y, stream)
    if st:
        _check(st, "mp_gated_backward")


def _gated_backward(dgate, dup, dy, gate, up, act, gate_scale, up_scale, y, stream) -> int:
    dev = torch.cuda.current_device()
    dyp, dys, code = _matrix(dy, "dy", dev)
    dgp, dgs, _ = _matrix(dgate, "dgate", dev, dy)
    rows, d = dy.shape
    if (up is None) != (dup is None):
        raise ValueError("up and dup: both or neither")
    if gate_scale is None:
        if up_scale is not None:
            raise ValueError("gate_scale: missing")
        gp, gs, _ = _matrix(gate, "gate", dev, dy)
        up_, us, _ = (None, 0, 0) if up is None else _matrix(up, "up", dev, dy)
        gsp = usp = None
    else:
        gp, gs, gsp, gkind = _matrix8(gate, gate_scale, "gate", dev, rows, d)
        up_, us, usp, ukind = _matrix8(up, up_scale, "up", dev, rows, d)
        _block_scaled(gkind, "gate")
        _block_scaled(ukind, "up")
    dup_, dus, _ = (None, 0, 0) if dup is None else _matrix(dup, "dup", dev, dy)
    yp, ys, _ = (None, 0, 0) if y is None else _matrix(y, "y", dev, dy)
    return _lib.mp_gated_backward(dgp, dup_, yp, dyp, gp, gsp, up_, usp, rows, d, dgs, dus, ys, dys, gs, us, act, code,
                                  _stream(stream))


def mp_pack8(q: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, *, stream=None) -> None:
    """Enqueue q, scale = x in 8 bits (scales of either kind)."""
    st = _binding.pack8(q, scale, x, stream)
    if st is None:
        xp, xs, code, qp, qs, sp, kind = _rows8(x, q, scale)
        st = _lib.mp_pack8(qp, sp, xp, x.shape[0], x.shape[1], qs, xs, code, kind, _stream(stream))
    if st:
        _check(st, "mp_pack8")


def mp_unpack8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, *, stream=None) -> None:
    """Enqueue x = the values that q and scale stand for."""
    st = _binding.unpack8(x, q, scale, stream)
    if st is None:
        xp, xs, code, qp, qs, sp, kind = _rows8(x, q, scale)
        st = _lib.mp_unpack8(xp, qp, sp, x.shape[0], x.shape[1], xs, qs, code, kind, _stream(stream))
    if st:
        _check(st, "mp_unpack8")


def _rows8(x, q, scale):
    dev = torch.cuda.current_device()
    xp, xs, code = _matrix(x, "x", dev)
    if q is None:
        raise TypeError("q: expected a torch.Tensor")
    return (xp, xs, code) + _matrix8(q, scale, "q", dev, *x.shape)


__all__ = [
    "MP_SCALE_ROW", "MP_SCALE_BLOCK", "MP_ACT_SILU", "MP_ACT_GELU", "ACTIVATIONS", "ROPE_KINDS", "MpRopeScaling",
    "RopeScaling", "mp_rmsnorm_forward", "mp_rmsnorm_workspace_bytes", "mp_rmsnorm_backward", "mp_rope_frequencies",
    "mp_rope", "mp_gated_forward", "mp_gated_backward", "mp_pack8", "mp_unpack8",
]
