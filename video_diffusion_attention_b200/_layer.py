"""The operators around the attention (argument marshalling only, see include/tara_attn.h):
rotary tables over several axes, the norm and rotation of Q and K, the linear layer and the
Q/K/V projection.

Tensors are CUDA tensors of one dtype (bf16, fp16 or fp32) on one device with the last dimension
contiguous; other strides are passed on, so a part of a fused projection, a transposed view or
rows of a packed tensor needs no copy.  Outputs the caller does not give are allocated on the
stream the call runs on.  Forward only, like the attention: nothing is recorded for a gradient, and
results do not require one.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional, Sequence

import numpy as np

from ._binding import (ROPE_MAX_AXES, TaraEpilogue, TaraError, TaraGrid, TaraNormRope, TaraRope,
                       TaraView, _dtype_code, load_library)

ACTS = {None: 0, "none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}
PAIRINGS = {"interleaved": 0, "halves": 1}


@dataclasses.dataclass
class TokenGrid:
    """`frames` x `rows` x `cols` tokens in packing order; token (f, r, c) has on axis a the
    position origin[a] + f*frame_step[a] + r*row_step[a] + c*col_step[a].

    The defaults give a video on (time, height, width); text of n tokens on the time axis is
    TokenGrid(frames=n)."""
    frames: int
    rows: int = 1
    cols: int = 1
    origin: Sequence[float] = (0.0, 0.0, 0.0)
    frame_step: Sequence[float] = (1.0, 0.0, 0.0)
    row_step: Sequence[float] = (0.0, 1.0, 0.0)
    col_step: Sequence[float] = (0.0, 0.0, 1.0)


def pack_token_positions(grids: Sequence[TokenGrid], n_axes: int = 3) -> np.ndarray:
    """Positions [N][n_axes] (float32, host) of the grids in packing order."""
    arr = (TaraGrid * max(1, len(grids)))()
    for c, g in zip(arr, grids):
        c.frames, c.rows, c.cols = int(g.frames), int(g.rows), int(g.cols)
        for name in ("origin", "frame_step", "row_step", "col_step"):
            src, dst = getattr(g, name), getattr(c, name)
            for a in range(min(n_axes, ROPE_MAX_AXES, len(src))):
                dst[a] = float(src[a])
    N = sum(max(0, int(g.frames)) * max(0, int(g.rows)) * max(0, int(g.cols)) for g in grids)
    pos = np.empty((N, max(0, n_axes)), np.float32)
    rc = load_library().tara_pack_token_positions(arr, len(grids), n_axes, pos.ctypes.data, N)
    if rc != 0:
        raise TaraError(rc, "tara_pack_token_positions")
    return pos


# ---------------------------------------------------------------------------------------
# marshalling
# ---------------------------------------------------------------------------------------
_DTYPES = {}   # torch dtype -> tara_dtype, filled on first use (torch is imported late)


def _dtype(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        code = _DTYPES[t.dtype] = _dtype_code(t)
    return code


def _view(t) -> TaraView:
    """View of [B][H][N][D], [B][N][C] or [N][C] (any strides, last dimension contiguous)."""
    shape, stride = t.shape, t.stride()
    nd = len(stride)
    if nd < 2 or nd > 4:
        raise ValueError("expected [B][H][N][D], [B][N][C] or [N][C]")
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    if max(shape) > 0x7fffffff:
        raise ValueError("a dimension is longer than 2^31 - 1")
    if nd == 3:
        return TaraView(t.data_ptr(), _dtype(t), shape[0], 1, shape[1], shape[2], stride[0], 0,
                        stride[1])
    if nd == 4:
        return TaraView(t.data_ptr(), _dtype(t), *shape, *stride[:3])
    return TaraView(t.data_ptr(), _dtype(t), 1, 1, shape[0], shape[1], 0, 0, stride[0])


def _new(like, B, H, N, D):
    """A new contiguous [B][H][N][D] tensor like `like`, and its view."""
    t = like.new_empty((B, H, N, D))
    return t, TaraView(t.data_ptr(), _dtype(like), B, H, N, D, H * N * D, N * D, D)


def _vector(t, name: str, like, *shapes) -> Optional[int]:
    """Pointer of an optional contiguous parameter of one of the given shapes."""
    if t is None:
        return None
    if t.shape not in shapes or not t.is_contiguous():
        raise ValueError("%s must be contiguous of shape %s" % (name, " or ".join(map(str, shapes))))
    if t.dtype != like.dtype:
        raise TypeError("%s must have the tensors' dtype" % name)
    if t.get_device() != like.get_device():
        raise ValueError("all tensors must be on one device")
    return t.data_ptr()


def _same_device(like, *tensors) -> None:
    device = like.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("all tensors must be on one device")


def _elsewhere(t, stream):
    """None when a call on t runs where the caller is (its current device and stream);
    otherwise a context that makes t's device, and the stream that was given, current."""
    import torch
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    if stream is None and torch.cuda.current_device() == t.get_device():
        return None
    if stream is not None and stream.device != t.device:
        raise ValueError("the stream and the tensors must be on one device")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(t.device))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


_raw_stream = None   # device index -> handle of its current stream


def _current_stream(t) -> int:
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(t.get_device())


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise TaraError(rc, what)


# ---------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------
def rope_table(pos, dims: Sequence[int], theta=10000.0, out=None, stream=None):
    """(cos, sin) of every rotated pair: [..., N, sum(dims)/2, 2] float32 from positions
    [..., N, axes] (float32, contiguous).  dims: columns of each axis; theta: one base or one
    per axis."""
    import torch
    away = _elsewhere(pos, stream)
    if away is not None:
        with away:
            return rope_table(pos, dims, theta, out)
    if pos.dtype != torch.float32 or not pos.is_contiguous() or pos.dim() < 2:
        raise ValueError("pos must be a contiguous float32 [..., N, axes] tensor")
    n_axes = len(dims)
    thetas = list(theta) if isinstance(theta, (list, tuple)) else [theta] * n_axes
    if pos.shape[-1] != n_axes or len(thetas) != n_axes or n_axes > ROPE_MAX_AXES:
        raise ValueError("pos, dims and theta must agree on the axes (at most %d)" % ROPE_MAX_AXES)
    r = TaraRope(n_axes, tuple(dims), tuple(thetas))
    shape = tuple(pos.shape[:-1]) + (sum(dims) // 2, 2)
    if out is None:
        out = pos.new_empty(shape)
    elif tuple(out.shape) != shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous float32 of shape %s" % (shape,))
    else:
        _same_device(pos, out)
    _check(load_library().tara_rope_table(pos.data_ptr(), pos.numel() // max(1, n_axes),
                                          ctypes.byref(r), out.data_ptr(), _current_stream(pos)),
           "tara_rope_table")
    return out


def _norm_rope_struct(like, H, N, D, B, q_weight, k_weight, eps, norm, table, pairing):
    code = PAIRINGS.get(pairing)
    if code is None:
        raise ValueError("pairing must be one of %s" % sorted(PAIRINGS))
    qw = kw = None
    stride = 0
    if norm:
        if q_weight is not None and k_weight is not None and q_weight.dim() != k_weight.dim():
            raise ValueError("q_weight and k_weight must both be [D] or both [H][D]")
        qw = _vector(q_weight, "q_weight", like, (D,), (H, D))
        kw = _vector(k_weight, "k_weight", like, (D,), (H, D))
        one = q_weight if q_weight is not None else k_weight
        stride = D if one is not None and one.dim() == 2 else 0
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights are only used with the norm")
    if table is None:
        return TaraNormRope(1 if norm else 0, eps, qw, kw, stride, None, 0, 0, code)
    import torch
    shape = table.shape
    if table.dtype != torch.float32 or not table.is_contiguous() or len(shape) not in (3, 4):
        raise ValueError("table must be a contiguous float32 [N][R/2][2] or [B][N][R/2][2]")
    if shape[-3] != N or shape[-1] != 2 or (len(shape) == 4 and shape[0] != B):
        raise ValueError("table does not match the tokens")
    _same_device(like, table)
    return TaraNormRope(1 if norm else 0, eps, qw, kw, stride, table.data_ptr(),
                        table.stride(0) if len(shape) == 4 and B > 1 else 0, 2 * shape[-2], code)


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 table=None, pairing: str = "interleaved", q_out=None, k_out=None, stream=None):
    """q, k after the per-head root-mean-square norm (weights [D] or [H][D], None: 1) and the
    rotation by `table` (None: none), in one pass over both.

    q, k: [B][H][N][D] views with any strides; the outputs are new contiguous tensors unless
    q_out / k_out are given (an output may be its own input).  k = None processes q alone and
    returns one tensor."""
    away = _elsewhere(q, stream)
    if away is not None:
        with away:
            return qk_norm_rope(q, k, q_weight, k_weight, eps, norm, table, pairing, q_out, k_out)
    _same_device(q, k, q_out, k_out)
    if q.dim() != 4:
        raise ValueError("q must be [B][H][N][D]")
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out and k_weight need k")
    B, H, N, D = q.shape
    p = _norm_rope_struct(q, H, N, D, B, q_weight, k_weight, eps, norm, table, pairing)
    qv = _view(q)
    q_out, qo = _new(q, B, H, N, D) if q_out is None else (q_out, _view(q_out))
    kv = ko = None
    if k is not None:
        k_out, ko = _new(q, B, H, N, D) if k_out is None else (k_out, _view(k_out))
        kv, ko = ctypes.byref(_view(k)), ctypes.byref(ko)
    _check(load_library().tara_qk_norm_rope(ctypes.byref(qv), kv, ctypes.byref(p),
                                            ctypes.byref(qo), ko, _current_stream(q)),
           "tara_qk_norm_rope")
    return q_out if k is None else (q_out, k_out)


def linear(x, w, bias=None, act: Optional[str] = None, gate=None, residual=None,
           heads: Optional[int] = None, out=None, stream=None):
    """residual + gate * act(x w^T + bias).

    x: [N][C_in], [B][N][C_in], or [B][H][N][D] with C_in = H*D (the attention's output as it
    is); w: [C_out][C_in]; bias [C_out]; gate [C_out] or [B][C_out]; act: None, "gelu",
    "gelu_tanh" or "silu"; residual: columns of out in any of the layouts.  The result is
    [N][C_out] or [B][N][C_out], or [B][heads][N][C_out/heads] when heads is given."""
    away = _elsewhere(x, stream)
    if away is not None:
        with away:
            return linear(x, w, bias, act, gate, residual, heads, out)
    _same_device(x, w, residual, out)
    if act not in ACTS:
        raise ValueError("act must be one of %s" % sorted(a for a in ACTS if a))
    xv = _view(x)
    if w.dim() != 2 or w.shape[1] != xv.H * xv.D or w.dtype != x.dtype or not w.is_contiguous():
        raise ValueError("w must be contiguous [C_out][C_in] of x's dtype")
    B, N, C = xv.B, xv.N, w.shape[0]
    if heads is not None and (heads < 1 or C % heads != 0):
        raise ValueError("heads must divide the output columns")
    e = TaraEpilogue(_vector(bias, "bias", x, (C,)), ACTS[act],
                     _vector(gate, "gate", x, (C,), (B, C)),
                     C if gate is not None and gate.dim() == 2 and B > 1 else 0)
    if residual is not None:
        e.residual = ctypes.pointer(_view(residual))
    if out is None:
        if heads is not None:
            shape = (B, heads, N, C // heads)
        else:
            shape = (N, C) if x.dim() == 2 else (B, N, C)
        out = x.new_empty(shape)
    elif heads is not None and (out.dim() != 4 or out.shape[1] != heads):
        raise ValueError("out must be [B][heads][N][D]")
    yv = _view(out)
    if yv.H * yv.D != C:
        raise ValueError("out must have %d columns" % C)
    _check(load_library().tara_linear(ctypes.byref(xv), w.data_ptr(), ctypes.byref(e),
                                      ctypes.byref(yv), _current_stream(x)), "tara_linear")
    return out


def qkv_project(x, w, heads: int, bias=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                norm: bool = True, table=None, pairing: str = "interleaved", out=None,
                stream=None):
    """q, k, v [B][heads][N][D] = x w^T + bias split into three, q and k through the norm and
    rotation of qk_norm_rope (norm=False and table=None: neither).

    x: [N][C_in], [B][N][C_in] or [B][H][N][D]; w: [3*heads*D][C_in]; out: three tensors or
    views [B][heads][N][D] to write, for instance rows of the packed sequence's q, k, v."""
    away = _elsewhere(x, stream)
    if away is not None:
        with away:
            return qkv_project(x, w, heads, bias, q_weight, k_weight, eps, norm, table, pairing, out)
    _same_device(x, w)
    xv = _view(x)
    if w.dim() != 2 or w.shape[1] != xv.H * xv.D or w.dtype != x.dtype or not w.is_contiguous():
        raise ValueError("w must be contiguous [3*heads*D][C_in] of x's dtype")
    rows = w.shape[0]
    if heads < 1 or rows % (3 * heads) != 0:
        raise ValueError("w must have 3*heads*D rows")
    B, N, D = xv.B, xv.N, rows // (3 * heads)
    p = None
    if norm or table is not None:
        p = ctypes.byref(_norm_rope_struct(x, heads, N, D, B, q_weight, k_weight, eps, norm,
                                           table, pairing))
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights are only used with the norm")
    bias_ptr = _vector(bias, "bias", x, (rows,))
    if out is None:
        (q, qv), (k, kv), (v, vv) = (_new(x, B, heads, N, D) for _ in range(3))
    else:
        q, k, v = out
        _same_device(x, q, k, v)
        qv, kv, vv = _view(q), _view(k), _view(v)
        # the library takes w's rows, and those of bias and weights, from the outputs' sizes
        for o in (qv, kv, vv):
            if (o.B, o.H, o.N, o.D) != (B, heads, N, D):
                raise ValueError("out must be three [%d][%d][%d][%d] tensors" % (B, heads, N, D))
    _check(load_library().tara_qkv_project(
        ctypes.byref(xv), w.data_ptr(), bias_ptr, p, ctypes.byref(qv), ctypes.byref(kv),
        ctypes.byref(vv), _current_stream(x)), "tara_qkv_project")
    return q, k, v
