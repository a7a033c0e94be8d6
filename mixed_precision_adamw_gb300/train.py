"""Python entry points of include/mp_train.h: the operators at the head of a
bf16 training step, whose gradients Optimizer.step takes.

As in the rest of the package every buffer is the caller's, every call only
enqueues work on the stream (the current one unless given) and a non-OK status
raises MpError. Matrices are 2-D CUDA tensors whose last dimension is
contiguous (rows may be strided, e.g. a column range of a wider buffer), of
bfloat16, float16 or float32; weights have a type of their own. Per-row
vectors are contiguous.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _check, _lib, _stream

MP_BF16, MP_FP16, MP_FP32 = 0, 1, 2
MP_INT32, MP_INT64 = 0, 1

_TYPES = {torch.bfloat16: MP_BF16, torch.float16: MP_FP16, torch.float32: MP_FP32}
_INDEX_TYPES = {torch.int32: MP_INT32, torch.int64: MP_INT64}


def _declare():
    vp, i64, i32, f32, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    for name, res, args in (
            ("mp_layernorm_forward", ctypes.c_int, [vp] * 6 + [i64] * 4 + [f32, i32, i32, vp]),
            ("mp_layernorm_workspace_bytes", size, [i64, i64]),
            ("mp_layernorm_backward", ctypes.c_int, [vp] * 8 + [i64] * 5 + [i32, i32, vp, size, vp]),
            ("mp_token_logprob_forward", ctypes.c_int,
             [vp] * 7 + [i64] * 3 + [f32, i32, i32, i32, vp, vp]),
            ("mp_token_logprob_backward", ctypes.c_int, [vp] * 7 + [i64] * 4 + [f32, i32, i32, vp, vp]),
            ("mp_distill_topk", ctypes.c_int,
             [vp] * 6 + [i64, i64, i32] + [i64] * 4 + [f32, i32, i32, vp, vp])):
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = res, args


_declare()


def _on(t, name: str, dev: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


# The checks below run on every call, in front of kernels of a few
# microseconds: the common case is one condition, and what is wrong with the
# others is found out afterwards.

def _matrix(t, name: str, dev: int, like=None):
    """(pointer, row stride, code of the element type) of a 2-D tensor with
    contiguous rows, of the shape and type of the tensor `like` if given."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev:
        code = _TYPES.get(t.dtype)
        shape = t.shape
        if code is not None and len(shape) == 2 and (like is None or (shape == like.shape and t.dtype == like.dtype)):
            stride, last = t.stride()
            if last == 1 and stride >= shape[1]:
                return t.data_ptr(), stride, code
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_TYPES)}")
    _on(t, name, dev)
    return _rows(t, name, like) + (code,)


def _index_matrix(t, name: str, dev: int, like):
    """The same of an int32 or int64 matrix of the shape of `like`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    code = _INDEX_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_INDEX_TYPES)}")
    _on(t, name, dev)
    if t.shape != like.shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    return _rows(t, name, None) + (code,)


def _rows(t, name: str, like):
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()}-D, expected [rows, length]")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {like.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    stride, last = t.stride()
    rows, cols = t.shape
    if last != 1 and cols > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if stride < cols:
        if rows > 1:  # rows that overlap (an expanded tensor)
            raise ValueError(f"{name}: row stride {stride} < {cols}")
        stride = cols
    return t.data_ptr(), stride


def _vector(t, name: str, dev: int, n: int, dtypes):
    """Pointer of a contiguous tensor of n elements; None stays None."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in dtypes and t.numel() == n
            and t.is_contiguous()):
        return t.data_ptr()
    _on(t, name, dev)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    if t.numel() != n:
        raise ValueError(f"{name}: {t.numel()} elements, expected {n}")
    raise ValueError(f"{name}: must be contiguous")


_F32 = frozenset((torch.float32,))
_I32 = frozenset((torch.int32,))
_U8 = frozenset((torch.uint8,))


def _weight_type(*weights) -> int:
    """The common type of the given weight tensors (float32 if none is given)."""
    dtype = None
    for t in weights:
        if t is not None:
            if dtype is None:
                dtype = t.dtype
            elif t.dtype != dtype:
                raise TypeError("weight, bias and their gradients must have one dtype")
    return MP_FP32 if dtype is None else _TYPES[dtype]


def mp_layernorm_forward(y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                         bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                         mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Enqueue y = layer norm of x over its last dimension, with weight and
    bias if given; mean and rstd (float32 [rows]) are kept for the backward
    pass. y may be x itself."""
    dev = torch.cuda.current_device()
    xp, xs, code = _matrix(x, "x", dev)
    yp, ys, _ = _matrix(y, "y", dev, x)
    rows, d = x.shape
    st = _lib.mp_layernorm_forward(
        yp, _vector(mean, "mean", dev, rows, _F32), _vector(rstd, "rstd", dev, rows, _F32), xp,
        _vector(weight, "weight", dev, d, _TYPES), _vector(bias, "bias", dev, d, _TYPES), rows, d, ys, xs, eps, code,
        _weight_type(weight, bias), _stream(stream))
    if st:
        _check(st, "mp_layernorm_forward")


def mp_layernorm_workspace_bytes(rows: int, d: int) -> int:
    """Bytes of scratch that mp_layernorm_backward needs for the weight gradients."""
    return int(_lib.mp_layernorm_workspace_bytes(rows, d))


def mp_layernorm_backward(dx: Optional[torch.Tensor], dweight: Optional[torch.Tensor],
                          dbias: Optional[torch.Tensor], dy: torch.Tensor, x: torch.Tensor,
                          weight: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, *,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the layer norm's backward pass: dx [rows, d], and the gradients
    of weight and bias summed over the rows (written, not added to; any of the
    three may be None). dx may be dy itself. workspace: uint8 of
    mp_layernorm_workspace_bytes(rows, d) bytes, when dweight or dbias is given."""
    dev = torch.cuda.current_device()
    xp, xs, code = _matrix(x, "x", dev)
    rows, d = x.shape
    dyp, dys, _ = _matrix(dy, "dy", dev, x)
    dxp, dxs, _ = (None, 0, 0) if dx is None else _matrix(dx, "dx", dev, x)
    wsp, wsn = None, 0
    if workspace is not None:
        wsn = workspace.numel()
        wsp = _vector(workspace, "workspace", dev, wsn, _U8)
    st = _lib.mp_layernorm_backward(
        dxp, _vector(dweight, "dweight", dev, d, _TYPES), _vector(dbias, "dbias", dev, d, _TYPES), dyp, xp,
        _vector(weight, "weight", dev, d, _TYPES), _vector(mean, "mean", dev, rows, _F32),
        _vector(rstd, "rstd", dev, rows, _F32), rows, d, dxs, dys, xs, code, _weight_type(weight, dweight, dbias), wsp,
        wsn, _stream(stream))
    if st:
        _check(st, "mp_layernorm_backward")


def _index_type(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    code = _INDEX_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_INDEX_TYPES)}")
    return code


def mp_token_logprob_forward(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *,
                             logp: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                             entropy: Optional[torch.Tensor] = None, top_logp: Optional[torch.Tensor] = None,
                             top_index: Optional[torch.Tensor] = None, scale: float = 1.0,
                             d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the log probabilities of the given tokens under softmax(scale *
    logits), each row's log-sum-exp and entropy, and its top alternatives
    (top_logp float32 and top_index int32, both [rows, k], k <= 32; largest
    first, equal ones by rising index). Negative targets: no given token."""
    dev = torch.cuda.current_device()
    lp, ls, code = _matrix(logits, "logits", dev)
    rows, vocab = logits.shape
    icode = MP_INT64 if targets is None else _index_type(targets, "targets")
    k, tlp, tip = 0, None, None
    if top_logp is not None or top_index is not None:
        if top_logp is None or top_index is None:
            raise ValueError("top_logp and top_index: both or neither")
        if top_logp.dim() != 2 or top_logp.shape[0] != rows or top_index.shape != top_logp.shape:
            raise ValueError(f"top_logp, top_index: shape [{rows}, k] expected")
        k = top_logp.shape[1]
        tlp = _vector(top_logp, "top_logp", dev, rows * k, _F32)
        tip = _vector(top_index, "top_index", dev, rows * k, _I32)
    st = _lib.mp_token_logprob_forward(
        _vector(logp, "logp", dev, rows, _F32), _vector(lse, "lse", dev, rows, _F32),
        _vector(entropy, "entropy", dev, rows, _F32), tlp, tip, lp, _vector(targets, "targets", dev, rows, _INDEX_TYPES),
        rows, vocab, ls, scale, k, code, icode, _vector(d_status, "d_status", dev, 1, _I32), _stream(stream))
    if st:
        _check(st, "mp_token_logprob_forward")


def mp_token_logprob_backward(dlogits: torch.Tensor, logits: torch.Tensor, targets: Optional[torch.Tensor], *,
                              lse: torch.Tensor, dlogp: Optional[torch.Tensor] = None,
                              entropy: Optional[torch.Tensor] = None, dentropy: Optional[torch.Tensor] = None,
                              scale: float = 1.0, d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue the gradient of the logits for the gradients dlogp of the log
    probabilities and dentropy of the entropies (with the forward pass's lse
    and entropy). dlogits may be logits itself."""
    dev = torch.cuda.current_device()
    lp, ls, code = _matrix(logits, "logits", dev)
    rows, vocab = logits.shape
    dp, ds, _ = _matrix(dlogits, "dlogits", dev, logits)
    icode = MP_INT64 if targets is None else _index_type(targets, "targets")
    if dentropy is None:
        entropy = None  # only its own gradient needs it
    st = _lib.mp_token_logprob_backward(
        dp, lp, _vector(targets, "targets", dev, rows, _INDEX_TYPES), _vector(lse, "lse", dev, rows, _F32),
        _vector(entropy, "entropy", dev, rows, _F32), _vector(dlogp, "dlogp", dev, rows, _F32),
        _vector(dentropy, "dentropy", dev, rows, _F32), rows, vocab, ds, ls, scale, code, icode,
        _vector(d_status, "d_status", dev, 1, _I32), _stream(stream))
    if st:
        _check(st, "mp_token_logprob_backward")


def mp_distill_topk(loss: torch.Tensor, dlogits: Optional[torch.Tensor], logits: torch.Tensor,
                    teacher: torch.Tensor, index: torch.Tensor, *, row_weight: Optional[torch.Tensor] = None,
                    scale: float = 1.0, d_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue loss[r] = row_weight[r] * KL(softmax of the teacher's listed
    logits || softmax of the student's logits), both at scale = 1 /
    temperature, and its gradient dlogits (None: the loss alone). teacher and
    index: [rows, k], k <= 1024, negative indices unused. dlogits may be logits
    itself."""
    dev = torch.cuda.current_device()
    lp, ls, code = _matrix(logits, "logits", dev)
    rows, vocab = logits.shape
    dp, ds, _ = (None, 0, 0) if dlogits is None else _matrix(dlogits, "dlogits", dev, logits)
    tp, ts, tcode = _matrix(teacher, "teacher", dev)
    if tcode != code:
        raise TypeError(f"teacher: dtype {teacher.dtype}, expected {logits.dtype}")
    ip, istride, icode = _index_matrix(index, "index", dev, teacher)
    if teacher.shape[0] != rows:
        raise ValueError(f"teacher: {teacher.shape[0]} rows, expected {rows}")
    st = _lib.mp_distill_topk(
        _vector(loss, "loss", dev, rows, _F32), dp, lp, tp, ip, _vector(row_weight, "row_weight", dev, rows, _F32),
        rows, vocab, teacher.shape[1], ds, ls, ts, istride, scale, code, icode,
        _vector(d_status, "d_status", dev, 1, _I32), _stream(stream))
    if st:
        _check(st, "mp_distill_topk")


__all__ = [
    "MP_BF16", "MP_FP16", "MP_FP32", "MP_INT32", "MP_INT64", "mp_layernorm_forward",
    "mp_layernorm_workspace_bytes", "mp_layernorm_backward", "mp_token_logprob_forward",
    "mp_token_logprob_backward", "mp_distill_topk",
]
