"""The operators that a layer needs beside its router, moves and products: the norm
that makes its input, low-rank adapters beside its projections, dropout, and the
gradient of its combine.

    y, x = rms_norm(attention_out, weight, residual=x)             # x: the residual stream
    (y, payload), x = rms_norm(attention_out, weight, residual=x, cast_fp8=SCALE_F32, return_bf16=True)
    recv, _, handle = dispatch(payload, topk_idx, num_experts, num_ranks)
    out = linear(y, w, residual=adapter_linear(y, a, b, adapter_idx, scale))
    x = dropout(combined, 0.1, seed, offset=layer, residual=x)

As in experts.py each has its gradient as a call of its own and nothing is
recorded. A layer's way back goes through combine_backward to the experts' rows
and the routing weights; a dispatch's gradient is combine with weights of 1.

This module only marshals arguments to libcgd (include/cgd_layer.h), on the
caller's current stream of the inputs' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import DispatchHandle, PackedHandle, _check, _dev_tensor, _fp8_empty, load
from .experts import _BF16, _F32, _ptr, _shaped

__all__ = ["rms_norm", "rms_norm_backward", "adapter_linear", "adapter_linear_backward", "dropout", "dropout_backward",
           "combine_backward"]


def configure(lib):
    """Declare the C signatures of cgd_layer.h on a loaded library."""
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    u64, f64 = ctypes.c_uint64, ctypes.c_double
    lib.cgd_rms_norm.restype = i32
    lib.cgd_rms_norm.argtypes = [vp, vp, vp, i32, f32, i64, i32, vp, vp, vp, i32, vp, vp]
    lib.cgd_rms_norm_backward_workspace_bytes.restype = sz
    lib.cgd_rms_norm_backward_workspace_bytes.argtypes = [i64, i32]
    lib.cgd_rms_norm_backward.restype = i32
    lib.cgd_rms_norm_backward.argtypes = [vp, vp, vp, i32, f32, i64, i32, vp, vp, vp, vp, sz, vp]
    lib.cgd_adapter_linear_workspace_bytes.restype = sz
    lib.cgd_adapter_linear_workspace_bytes.argtypes = [i64, i32, i32, i64, i64]
    lib.cgd_adapter_linear.restype = i32
    lib.cgd_adapter_linear.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.cgd_adapter_linear_backward_workspace_bytes.restype = sz
    lib.cgd_adapter_linear_backward_workspace_bytes.argtypes = [i64, i32, i32, i64, i64]
    lib.cgd_adapter_linear_backward.restype = i32
    lib.cgd_adapter_linear_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, vp, vp, vp, vp, sz,
                                                vp]
    lib.cgd_dropout.restype = i32
    lib.cgd_dropout.argtypes = [vp, vp, i64, f64, u64, u64, vp, vp, vp]
    lib.cgd_combine_backward.restype = i32
    lib.cgd_combine_backward.argtypes = [vp, vp, i64, i32, vp, vp, i64, i32, vp, vp, vp]
    return lib


# The smallest of these calls take longer on the host than on the GPU, so a tensor that
# is as it should be is told by the fewest questions (a device by its number), and
# the device is only changed where it has to be.
_BFLOAT16, _FLOAT32 = torch.bfloat16, torch.float32
_Tensor = torch.Tensor


def _like(t, name: str, dtype, shape, dev: int):
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()):
        _shaped(t, name, dtype, tuple(shape), torch.device("cuda", dev))  # says what is wrong


def _bf16(t, name: str, ndim: int) -> int:
    """The device of a contiguous bf16 tensor (ndim 0: of any dimensions, but one at least)."""
    if not (isinstance(t, _Tensor) and t.is_cuda and t.dtype is _BFLOAT16 and t.is_contiguous() and t.dim() == (ndim or t.dim() or 1)):
        _dev_tensor(t, name, _BFLOAT16, ndim or max(1, t.dim() if isinstance(t, _Tensor) else 1))
    return t.get_device()


def _out(out, name: str, shape, dev: int, inputs, over=()):
    """The caller's bf16 output: it shares no memory with the inputs (contiguous), which
    other blocks still read while it is written, but may be one of `over` itself."""
    _like(out, name, _BFLOAT16, shape, dev)
    begin = out.data_ptr()
    end = begin + out.nbytes
    for t in inputs:
        if t is not None and t.data_ptr() < end and begin < t.data_ptr() + t.nbytes:
            raise ValueError(f"{name} shares memory with an input")
    for t in over:
        if t is not None and t.data_ptr() != begin and t.data_ptr() < end and begin < t.data_ptr() + t.nbytes:
            raise ValueError(f"{name} shares memory with an input")
    return out


def _call(name: str, dev: int, *args):
    """A call of the library on the device's current stream."""
    before = torch._C._cuda_getDevice()
    if before != dev:
        torch.cuda.set_device(dev)
    try:
        status = getattr(load(), name)(*args, torch._C._cuda_getCurrentRawStream(dev))
    finally:
        if before != dev:
            torch.cuda.set_device(before)
    if status:
        _check(name, status)


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def _norm_weight(weight, H: int, dev: int) -> int:
    dtype = weight.dtype if isinstance(weight, _Tensor) else None
    if dtype is not _BFLOAT16 and dtype is not _FLOAT32:
        raise TypeError("weight must be a bfloat16 or float32 tensor")
    _like(weight, "weight", dtype, (H,), dev)
    return _F32 if dtype is _FLOAT32 else _BF16


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             cast_fp8: int | None = None, return_bf16: bool = False, sum_out: torch.Tensor | None = None):
    """s / sqrt(mean(s * s) + eps) * weight over the last dimension, s = x + residual -> y,
    or with a residual (y, sum).

    x and residual bf16 [..., H], weight bf16 or float32 [H]. y is bf16; with
    cast_fp8 = a scale format the FP8 tuple (codes [..., H], scales [..., H/128])
    that dispatch and linear take, encoded from float32; with return_bf16 as well,
    (bf16 tensor, FP8 tuple), e.g. for a gate beside the dispatch. sum is s in bf16,
    the residual stream; y is made from s before that rounding. sum_out, if given,
    receives it and may be residual or x itself."""
    dev = _bf16(x, "x", 0)
    shape = x.shape
    H = shape[-1]
    n = x.numel() // H if H else 0
    wtype = _norm_weight(weight, H, dev)
    y = q = sc = total = None
    if residual is not None:
        _like(residual, "residual", _BFLOAT16, shape, dev)
    if sum_out is not None:
        if residual is None:
            raise ValueError("sum_out goes with residual")
        total = _out(sum_out, "sum_out", shape, dev, (weight,), over=(x, residual))
    elif residual is not None:
        total = torch.empty_like(x)
    if cast_fp8 is None:
        if return_bf16:
            raise ValueError("return_bf16 goes with cast_fp8")
        y = torch.empty_like(x)
    else:
        if H % 128:
            raise ValueError(f"an FP8 output needs a last dimension that is a multiple of 128 (got {H})")
        if return_bf16:
            y = torch.empty_like(x)
        q, sc = _fp8_empty(n, H, cast_fp8, x.device)
        if len(shape) != 2:
            q, sc = q.view(shape), sc.view(*shape[:-1], H // 128)
    _call("cgd_rms_norm", dev, x.data_ptr(), _ptr(residual), weight.data_ptr(), wtype, eps, n, H, _ptr(y), _ptr(q), _ptr(sc),
          cast_fp8 or 0, _ptr(total))
    out = y if q is None else (y, (q, sc)) if return_bf16 else (q, sc)
    return out if residual is None else (out, total)


def rms_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      grad_sum: torch.Tensor | None = None):
    """Gradients of rms_norm at x, the values that were normed (with a residual: the
    sum that rms_norm returned, whose gradient is that of both terms): -> (grad_x
    bf16 like x, grad_weight like weight). grad_sum, what reaches the residual
    stream on its other way, is added to grad_x. All bf16 but a float32 weight's."""
    dev = _bf16(x, "x", 0)
    shape = x.shape
    H = shape[-1]
    n = x.numel() // H if H else 0
    wtype = _norm_weight(weight, H, dev)
    _like(grad_y, "grad_y", _BFLOAT16, shape, dev)
    if grad_sum is not None:
        _like(grad_sum, "grad_sum", _BFLOAT16, shape, dev)
    gx, gw = torch.empty_like(x), torch.empty_like(weight)
    nbytes = load().cgd_rms_norm_backward_workspace_bytes(n, H)
    wk = x.new_empty(nbytes // 2) if nbytes else None
    _call("cgd_rms_norm_backward", dev, grad_y.data_ptr(), x.data_ptr(), weight.data_ptr(), wtype, eps, n, H, _ptr(grad_sum),
          gx.data_ptr(), gw.data_ptr(), _ptr(wk), nbytes)
    return gx, gw


# ---------------------------------------------------------------------------
# Adapters
# ---------------------------------------------------------------------------

def _adapters(x, a, b, adapter_idx, scale):
    """-> (T, J, R, I, O, the device's number)."""
    dev = _bf16(x, "x", 2)
    T, I = x.shape
    if _bf16(a, "a", 3) != dev or _bf16(b, "b", 3) != dev:
        raise ValueError("a and b must be on x's device")
    J, R, in_a = a.shape
    in_b, O, out_r = b.shape
    if in_a != I or in_b != J or out_r != R:
        raise ValueError(f"a must be [num_adapters, rank, {I}] and b [num_adapters, out_features, rank] "
                         f"(got {tuple(a.shape)} and {tuple(b.shape)})")
    _like(adapter_idx, "adapter_idx", torch.int64, (T,), dev)
    if scale is not None:
        _like(scale, "scale", _FLOAT32, (J,), dev)
    return T, J, R, I, O, dev


def adapter_linear(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter_idx: torch.Tensor,
                   scale: torch.Tensor | None = None, residual: torch.Tensor | None = None, return_hidden: bool = False,
                   out: torch.Tensor | None = None):
    """Low-rank adapters of many requests: residual[t] + scale[j] * b[j] @ (a[j] @ x[t])
    with j = adapter_idx[t] -> bf16 [T, O].

    x bf16 [T, I]; a bf16 [J, R, I] and b bf16 [J, O, R], up to 512 adapters of one
    rank R (a multiple of 8 up to 256; smaller ones padded with zeros); adapter_idx
    int64 [T], any order; a token with an index outside [0, J) has no adapter: its
    row is the residual's, or 0. scale float32 [J]. Beside a shared projection the
    result is linear's residual: linear(x, w, residual=adapter_linear(x, a, b, idx)).
    It is rounded to bf16 on the way there and the sum once more: half the memory of
    a float32 result, for an error of up to 2^-8 of the adapters' part.
    With return_hidden -> (out, hidden float32 [T, R]: a[j] @ x[t]), which
    adapter_linear_backward takes. out, if given, shares no memory with an input,
    but may be residual itself."""
    T, J, R, I, O, dev = _adapters(x, a, b, adapter_idx, scale)
    if residual is not None:
        _like(residual, "residual", _BFLOAT16, (T, O), dev)
    if out is None:
        out = x.new_empty((T, O)) if residual is None else torch.empty_like(residual)
    else:
        _out(out, "out", (T, O), dev, (x, a, b, adapter_idx, scale), over=(residual,))
    hidden = torch.empty((T, R), dtype=_FLOAT32, device=x.device) if return_hidden else None
    nbytes = load().cgd_adapter_linear_workspace_bytes(T, J, R, I, O)
    wk = x.new_empty(nbytes // 2) if nbytes else None  # (bf16 elements; nothing of it outlives the call)
    _call("cgd_adapter_linear", dev, x.data_ptr(), a.data_ptr(), b.data_ptr(), _ptr(scale), adapter_idx.data_ptr(), T, J, R, I, O,
          _ptr(residual), out.data_ptr(), _ptr(hidden), _ptr(wk), nbytes)
    return (out, hidden) if return_hidden else out


def adapter_linear_backward(grad_out: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                            adapter_idx: torch.Tensor, hidden: torch.Tensor, scale: torch.Tensor | None = None):
    """Gradients of adapter_linear (bf16): -> (grad_x like x, grad_a like a, grad_b
    like b). hidden as adapter_linear returned it. An adapter without tokens gets
    zeros, a token without an adapter a zero row. The residual's gradient is
    grad_out; the shared projection's grad_x comes from linear_backward and adds to
    this one. O has to be a multiple of 8."""
    T, J, R, I, O, dev = _adapters(x, a, b, adapter_idx, scale)
    _like(grad_out, "grad_out", _BFLOAT16, (T, O), dev)
    _like(hidden, "hidden", _FLOAT32, (T, R), dev)
    gx, ga, gb = torch.empty_like(x), torch.empty_like(a), torch.empty_like(b)
    nbytes = load().cgd_adapter_linear_backward_workspace_bytes(T, J, R, I, O)
    wk = x.new_empty(nbytes // 2)
    _call("cgd_adapter_linear_backward", dev, grad_out.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), _ptr(scale),
          adapter_idx.data_ptr(), hidden.data_ptr(), T, J, R, I, O, gx.data_ptr(), ga.data_ptr(), gb.data_ptr(), _ptr(wk), nbytes)
    return gx, ga, gb


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

def dropout(x: torch.Tensor, p: float, seed, offset: int = 0, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """x with elements dropped with probability p and the others divided by 1 - p,
    plus residual; bf16, any shape. The mask comes from a counter-based generator
    (Philox4x32-10) and is nowhere stored: the same seed and offset give it again.

    p counts in steps of 1/65536, and what is kept is divided by the probability in
    use. seed: an integer, or an int64 tensor [2] on the device whose elements,
    (seed, offset), are read when the kernel runs, so that a captured graph can be
    replayed with new numbers; `offset` is added to it. Calls of one seed need
    offsets of their own (a layer's number, a step's). A dropped element is 0 even
    where x is infinite or NaN. out may be x or residual itself."""
    if not (isinstance(x, _Tensor) and x.is_cuda and x.dtype is _BFLOAT16 and x.is_contiguous()):
        _dev_tensor(x, "x", _BFLOAT16, x.dim() if isinstance(x, _Tensor) else 1)
    dev = x.get_device()
    state = None
    if isinstance(seed, torch.Tensor):
        state, seed = _shaped(seed, "seed", torch.int64, (2,), x.device), 0
    if not (isinstance(seed, int) and 0 <= seed < 1 << 64 and isinstance(offset, int) and 0 <= offset < 1 << 64):
        raise ValueError(f"seed and offset must be integers in [0, 2^64) (got {seed!r}, {offset!r})")
    if residual is not None:
        _like(residual, "residual", _BFLOAT16, x.shape, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _out(out, "out", x.shape, dev, (state,), over=(x, residual))
    _call("cgd_dropout", dev, x.data_ptr(), _ptr(residual), x.numel(), p, seed, offset, _ptr(state), out.data_ptr())
    return out


def dropout_backward(grad_out: torch.Tensor, p: float, seed, offset: int = 0, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of dropout at x, for the same p, seed and offset (the residual's is grad_out)."""
    return dropout(grad_out, p, seed, offset=offset, out=out)


# ---------------------------------------------------------------------------
# Combine's gradient
# ---------------------------------------------------------------------------

def combine_backward(grad_out: torch.Tensor, expert_out: torch.Tensor, handle, topk_weights: torch.Tensor,
                     out: torch.Tensor | None = None):
    """Gradients of combine(expert_out, handle, topk_weights), or of low_latency_combine
    with its PackedHandle: -> (grad_expert_out bf16 like expert_out,
    grad_topk_weights float32 [T, K]).

    grad_out bf16 [T, H]. Row dst_row[t, k] gets topk_weights[t, k] * grad_out[t],
    the weight the sum of grad_out[t] * expert_out[dst_row[t, k]] (0 for a slot
    without a row). Rows that hold no token are left as they were (in a new tensor:
    undefined). out, if given, receives grad_expert_out and shares no memory with
    an input."""
    packed = isinstance(handle, PackedHandle)
    if not packed and not isinstance(handle, DispatchHandle):
        raise TypeError("handle must be a DispatchHandle or a PackedHandle")
    dev = _bf16(expert_out, "expert_out", 3 if packed else 2)
    shape = expert_out.shape
    H = shape[-1]
    cap = shape[0] * shape[1] if packed else shape[0]
    if packed and shape[:2] != (handle.num_experts, handle.expert_capacity):
        raise ValueError("expert_out must be [num_experts, expert_capacity, hidden]")
    dst = handle.dst_row
    T, K = dst.shape
    _like(dst, "handle.dst_row", torch.int32, (T, K), dev)
    _like(grad_out, "grad_out", _BFLOAT16, (T, H), dev)
    _like(topk_weights, "topk_weights", _FLOAT32, (T, K), dev)
    if out is None:
        out = torch.empty_like(expert_out)
    else:
        _out(out, "out", shape, dev, (grad_out, expert_out, dst, topk_weights))
    gw = torch.empty_like(topk_weights)
    _call("cgd_combine_backward", dev, grad_out.data_ptr(), expert_out.data_ptr(), cap, H, dst.data_ptr(), topk_weights.data_ptr(),
          T, K, out.data_ptr(), gw.data_ptr())
    return out, gw
