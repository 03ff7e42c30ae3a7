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
from .experts import _BF16, _Current, _F32, _ptr, _result, _shaped, _stream, _workspace

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


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def _rows(x, name: str):
    """-> (rows, hidden) of a bf16 tensor whose last dimension is normed."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    _dev_tensor(x, name, torch.bfloat16, max(1, x.dim()))
    H = x.shape[-1]
    return (x.numel() // H if H else 0), H


def _norm_weight(weight, H: int, dev) -> int:
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("weight must be a bfloat16 or float32 tensor")
    _shaped(weight, "weight", weight.dtype, (H,), dev)
    return _F32 if weight.dtype == torch.float32 else _BF16


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
    lib = load()
    n, H = _rows(x, "x")
    dev = x.device
    wtype = _norm_weight(weight, H, dev)
    if residual is not None:
        _shaped(residual, "residual", torch.bfloat16, tuple(x.shape), dev)
    if return_bf16 and cast_fp8 is None:
        raise ValueError("return_bf16 goes with cast_fp8")
    if cast_fp8 is not None and H % 128:
        raise ValueError(f"an FP8 output needs a last dimension that is a multiple of 128 (got {H})")
    if sum_out is not None:
        if residual is None:
            raise ValueError("sum_out goes with residual")
        _result(sum_out, torch.bfloat16, tuple(x.shape), dev, weight, *([x] if sum_out.data_ptr() != x.data_ptr() else []),
                over=residual)
    with _Current(dev):
        y = torch.empty_like(x) if cast_fp8 is None or return_bf16 else None
        total = sum_out if sum_out is not None else None if residual is None else torch.empty_like(x)
        q = sc = None
        if cast_fp8 is not None:
            q, sc = _fp8_empty(n, H, cast_fp8, dev)
            q, sc = q.view(x.shape), sc.view(*x.shape[:-1], H // 128)
        _check("cgd_rms_norm",
               lib.cgd_rms_norm(_ptr(x), _ptr(residual), _ptr(weight), wtype, eps, n, H, _ptr(y), _ptr(q), _ptr(sc),
                                0 if cast_fp8 is None else cast_fp8, _ptr(total), _stream(dev)))
    out = y if q is None else (y, (q, sc)) if return_bf16 else (q, sc)
    return out if residual is None else (out, total)


def rms_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      grad_sum: torch.Tensor | None = None):
    """Gradients of rms_norm at x, the values that were normed (with a residual: the
    sum that rms_norm returned, whose gradient is that of both terms): -> (grad_x
    bf16 like x, grad_weight like weight). grad_sum, what reaches the residual
    stream on its other way, is added to grad_x. All bf16 but a float32 weight's."""
    lib = load()
    n, H = _rows(x, "x")
    dev = x.device
    wtype = _norm_weight(weight, H, dev)
    _shaped(grad_y, "grad_y", torch.bfloat16, tuple(x.shape), dev)
    if grad_sum is not None:
        _shaped(grad_sum, "grad_sum", torch.bfloat16, tuple(x.shape), dev)
    with _Current(dev):
        gx, gw = torch.empty_like(x), torch.empty_like(weight)
        nbytes = lib.cgd_rms_norm_backward_workspace_bytes(n, H)
        wk = _workspace(nbytes, dev)
        _check("cgd_rms_norm_backward",
               lib.cgd_rms_norm_backward(_ptr(grad_y), _ptr(x), _ptr(weight), wtype, eps, n, H, _ptr(grad_sum), _ptr(gx),
                                         _ptr(gw), _ptr(wk), nbytes, _stream(dev)))
    return gx, gw


# ---------------------------------------------------------------------------
# Adapters
# ---------------------------------------------------------------------------

def _adapters(x, a, b, adapter_idx, scale):
    """-> (T, J, R, I, O, device)."""
    _dev_tensor(x, "x", torch.bfloat16, 2)
    dev = x.device
    T, I = x.shape
    _dev_tensor(a, "a", torch.bfloat16, 3)
    _dev_tensor(b, "b", torch.bfloat16, 3)
    J, R = a.shape[:2]
    O = b.shape[1]
    _shaped(a, "a", torch.bfloat16, (J, R, I), dev)
    _shaped(b, "b", torch.bfloat16, (J, O, R), dev)
    _shaped(adapter_idx, "adapter_idx", torch.int64, (T,), dev)
    if scale is not None:
        _shaped(scale, "scale", torch.float32, (J,), dev)
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
    With return_hidden -> (out, hidden float32 [T, R]: a[j] @ x[t]), which
    adapter_linear_backward takes. out, if given, shares no memory with an input,
    but may be residual itself."""
    lib = load()
    T, J, R, I, O, dev = _adapters(x, a, b, adapter_idx, scale)
    if residual is not None:
        _shaped(residual, "residual", torch.bfloat16, (T, O), dev)
    with _Current(dev):
        if out is None:
            out = torch.empty((T, O), dtype=torch.bfloat16, device=dev)
        else:
            _result(out, torch.bfloat16, (T, O), dev, x, a, b, adapter_idx, scale, over=residual)
        hidden = torch.empty((T, R), dtype=torch.float32, device=dev) if return_hidden else None
        nbytes = lib.cgd_adapter_linear_workspace_bytes(T, J, R, I, O)
        wk = _workspace(nbytes, dev)
        _check("cgd_adapter_linear",
               lib.cgd_adapter_linear(_ptr(x), _ptr(a), _ptr(b), _ptr(scale), _ptr(adapter_idx), T, J, R, I, O,
                                      _ptr(residual), _ptr(out), _ptr(hidden), _ptr(wk), nbytes, _stream(dev)))
    return (out, hidden) if return_hidden else out


def adapter_linear_backward(grad_out: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                            adapter_idx: torch.Tensor, hidden: torch.Tensor, scale: torch.Tensor | None = None):
    """Gradients of adapter_linear (bf16): -> (grad_x like x, grad_a like a, grad_b
    like b). hidden as adapter_linear returned it. An adapter without tokens gets
    zeros, a token without an adapter a zero row. The residual's gradient is
    grad_out; the shared projection's grad_x comes from linear_backward and adds to
    this one. O has to be a multiple of 8."""
    lib = load()
    T, J, R, I, O, dev = _adapters(x, a, b, adapter_idx, scale)
    _shaped(grad_out, "grad_out", torch.bfloat16, (T, O), dev)
    _shaped(hidden, "hidden", torch.float32, (T, R), dev)
    with _Current(dev):
        gx, ga, gb = torch.empty_like(x), torch.empty_like(a), torch.empty_like(b)
        nbytes = lib.cgd_adapter_linear_backward_workspace_bytes(T, J, R, I, O)
        wk = _workspace(nbytes, dev)
        _check("cgd_adapter_linear_backward",
               lib.cgd_adapter_linear_backward(_ptr(grad_out), _ptr(x), _ptr(a), _ptr(b), _ptr(scale), _ptr(adapter_idx),
                                               _ptr(hidden), T, J, R, I, O, _ptr(gx), _ptr(ga), _ptr(gb), _ptr(wk),
                                               nbytes, _stream(dev)))
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
    lib = load()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    _dev_tensor(x, "x", torch.bfloat16, x.dim())
    dev = x.device
    shape = tuple(x.shape)
    if residual is not None:
        _shaped(residual, "residual", torch.bfloat16, shape, dev)
    state = None
    if isinstance(seed, torch.Tensor):
        state, seed = _shaped(seed, "seed", torch.int64, (2,), dev), 0
    for name, v in (("seed", seed), ("offset", offset)):
        if not isinstance(v, int) or not 0 <= v < 1 << 64:
            raise ValueError(f"{name} must be an integer in [0, 2^64) (got {v!r})")
    with _Current(dev):
        if out is None:
            out = torch.empty_like(x)
        else:
            _result(out, torch.bfloat16, shape, dev, state, *([x] if out.data_ptr() != x.data_ptr() else []), over=residual)
        _check("cgd_dropout",
               lib.cgd_dropout(_ptr(x), _ptr(residual), x.numel(), p, seed, offset, _ptr(state), _ptr(out), _stream(dev)))
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
    lib = load()
    packed = isinstance(handle, PackedHandle)
    if not packed and not isinstance(handle, DispatchHandle):
        raise TypeError("handle must be a DispatchHandle or a PackedHandle")
    _dev_tensor(expert_out, "expert_out", torch.bfloat16, 3 if packed else 2)
    dev = expert_out.device
    H = expert_out.shape[-1]
    cap = expert_out.shape[0] * expert_out.shape[1] if packed else expert_out.shape[0]
    if packed and expert_out.shape[:2] != (handle.num_experts, handle.expert_capacity):
        raise ValueError("expert_out must be [num_experts, expert_capacity, hidden]")
    T, K = handle.dst_row.shape
    _shaped(handle.dst_row, "handle.dst_row", torch.int32, (T, K), dev)
    _shaped(grad_out, "grad_out", torch.bfloat16, (T, H), dev)
    _shaped(topk_weights, "topk_weights", torch.float32, (T, K), dev)
    with _Current(dev):
        if out is None:
            out = torch.empty_like(expert_out)
        else:
            _result(out, torch.bfloat16, tuple(expert_out.shape), dev, grad_out, expert_out, handle.dst_row, topk_weights)
        gw = torch.empty((T, K), dtype=torch.float32, device=dev)
        _check("cgd_combine_backward",
               lib.cgd_combine_backward(_ptr(grad_out), _ptr(expert_out), cap, H, _ptr(handle.dst_row), _ptr(topk_weights),
                                        T, K, _ptr(out), _ptr(gw), _stream(dev)))
    return out, gw
