"""The computing operators around dispatch and combine: the router, the experts'
grouped products and the dense product with its epilogue.

    topk_idx, topk_weights = route(logits, num_topk, scoring="sigmoid", bias=bias)
    h = grouped_linear(recv_x, w_gate_up, handle, activation="swiglu")    # over dispatch's segments
    y = grouped_linear(h, w_down, handle)
    combined = combine(y, handle, topk_weights)
    out = linear(shared_h, w_shared_down, residual=combined)

Each has its gradient as a call of its own (route_backward,
grouped_linear_backward, linear_backward): like dispatch and combine they take
and give tensors, and record nothing. The products' gradients take bf16, a
gate's float32 ones rounded:

    grad_logits = route_backward(grad_topk_weights, logits, topk_idx, scoring="sigmoid")
    grad_x, grad_gate, _ = linear_backward(grad_logits.bfloat16(), x, gate)

Like the rest of the package this module only marshals arguments to libcgd
(include/cgd_experts.h): the kernels run on the caller's current stream of the
inputs' device. Workspaces come from torch's allocator call by call, so calls
on several streams, and graphs captured one after the other, share none.
"""
from __future__ import annotations

import ctypes

import torch

from . import DispatchHandle, SCALE_F32, SCALE_UE8M0, _check, _dev_tensor, load

__all__ = ["route", "route_backward", "linear", "linear_backward", "grouped_linear", "grouped_linear_backward"]

_BF16, _F32, _FP8 = 0, 1, 2
_SCORING = {"softmax": 0, "sigmoid": 1}
_ACTIVATION = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


def configure(lib):
    """Declare the C signatures of cgd_experts.h on a loaded library."""
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.cgd_route.restype = i32
    lib.cgd_route.argtypes = [vp, i32, i64, i32, i32, i32, vp, i32, i32, i32, i32, f32, vp, vp, vp]
    lib.cgd_route_backward.restype = i32
    lib.cgd_route_backward.argtypes = [vp, vp, i32, vp, i64, i32, i32, i32, i32, f32, vp, vp]
    lib.cgd_linear_workspace_bytes.restype = sz
    lib.cgd_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.cgd_linear.restype = i32
    lib.cgd_linear.argtypes = [vp, i32, vp, i64, i64, i32, vp, vp, i64, i64, i64, vp, i32, vp, vp, i32, vp, vp, sz, vp]
    lib.cgd_grouped_linear_workspace_bytes.restype = sz
    lib.cgd_grouped_linear_workspace_bytes.argtypes = [i64, i32, i64, i64, i64, i32, i32]
    lib.cgd_grouped_linear.restype = i32
    lib.cgd_grouped_linear.argtypes = [vp, i32, vp, i64, i64, i32, vp, vp, i64, i32, vp, i64, vp, i64, i64, vp, i32, vp,
                                       vp, vp, sz, vp]
    lib.cgd_linear_backward_workspace_bytes.restype = sz
    lib.cgd_linear_backward_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.cgd_linear_backward.restype = i32
    lib.cgd_linear_backward.argtypes = [vp, vp, vp, i64, i64, i64, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.cgd_grouped_linear_backward_workspace_bytes.restype = sz
    lib.cgd_grouped_linear_backward_workspace_bytes.argtypes = [i64, i32, i64, i64, i32, i32]
    lib.cgd_grouped_linear_backward.restype = i32
    lib.cgd_grouped_linear_backward.argtypes = [vp, vp, vp, i64, i32, vp, i64, vp, i64, i64, vp, i32, vp, vp, vp, vp,
                                                sz, vp]
    return lib


class _Current:
    """Makes a device current for a call, where it is not already (a quarter of
    the cost of torch.cuda.device there)."""

    __slots__ = ("index", "before")

    def __init__(self, dev):
        self.index = dev.index

    def __enter__(self):
        self.before = torch.cuda.current_device()
        if self.before != self.index:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.before != self.index:
            torch.cuda.set_device(self.before)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    """The current stream's handle (torch.cuda.current_stream makes an object of it first)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _choice(table: dict, value, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {list(table)} (got {value!r})")
    return table[value]


def _shaped(t, name: str, dtype, shape: tuple, dev) -> torch.Tensor:
    """A contiguous tensor of this type and shape on the device (libcgd checks its alignment)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on the inputs' device {dev} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _result(out, dtype, shape: tuple, dev, *inputs, over=None) -> torch.Tensor:
    """The caller's output tensor: it shares no memory with the inputs, which
    other blocks still read while it is written, but may be `over` itself."""
    _shaped(out, "out", dtype, shape, dev)
    begin, end = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in (*inputs, over):
        if t is None or t.numel() == 0 or (t is over and t.data_ptr() == begin and t.dtype == dtype):
            continue
        span = 1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
        if t.data_ptr() < end and begin < t.data_ptr() + span * t.element_size():
            raise ValueError("out shares memory with an input")
    return out


def _workspace(nbytes: int, dev):
    """Scratch memory for one call, from torch's allocator (a capture's own
    pool while a graph is captured): nothing of it outlives the call."""
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------

def _logits(logits):
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16 (got {logits.dtype})")
    _dev_tensor(logits, "logits", logits.dtype, 2)
    return _F32 if logits.dtype == torch.float32 else _BF16


def route(logits: torch.Tensor, num_topk: int, scoring: str = "softmax", bias: torch.Tensor | None = None,
          num_groups: int = 1, num_topk_groups: int | None = None, group_score_topk: int = 2,
          renormalize: bool = True, scale: float = 1.0):
    """The experts of each token: -> (topk_idx int64 [T, K], topk_weights float32 [T, K]),
    as get_dispatch_layout, dispatch and combine take them.

    logits [T, E] float32 or bfloat16; the score s is their softmax or sigmoid.
    The choice is by s + bias (float32 [E]; for the choice only), descending,
    ties to the lower index, compared in 64 bits. With num_topk_groups <
    num_groups only experts of the best groups of E / num_groups neighbours can
    be chosen, a group being worth the sum of its group_score_topk (1 or 2)
    largest choice values. The weight is s, divided by the sum over the chosen
    with renormalize, times scale. An expert with a logit of -inf (or NaN) is
    never chosen; slots left over hold -1 and 0."""
    lib = load()
    ltype = _logits(logits)
    T, E = logits.shape
    dev = logits.device
    mode = _choice(_SCORING, scoring, "scoring")
    if bias is not None:
        _shaped(bias, "bias", torch.float32, (E,), dev)
    if num_topk_groups is None:
        num_topk_groups = num_groups
    if not 1 <= num_topk <= E:
        raise ValueError(f"num_topk must be in [1, {E}] (got {num_topk})")
    with _Current(dev):
        idx = torch.empty((T, num_topk), dtype=torch.int64, device=dev)
        wts = torch.empty((T, num_topk), dtype=torch.float32, device=dev)
        _check("cgd_route",
               lib.cgd_route(_ptr(logits), ltype, T, E, num_topk, mode, _ptr(bias), num_groups, num_topk_groups,
                             group_score_topk, int(renormalize), scale, _ptr(idx), _ptr(wts), _stream(dev)))
    return idx, wts


def route_backward(grad_topk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                   scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """The gradient of route's topk_weights with respect to the logits (the
    choice itself has none) -> grad_logits [T, E] of the logits' type."""
    lib = load()
    ltype = _logits(logits)
    T, E = logits.shape
    dev = logits.device
    mode = _choice(_SCORING, scoring, "scoring")
    _dev_tensor(topk_idx, "topk_idx", torch.int64, 2)
    K = topk_idx.shape[1]
    _shaped(topk_idx, "topk_idx", torch.int64, (T, K), dev)
    _shaped(grad_topk_weights, "grad_topk_weights", torch.float32, (T, K), dev)
    with _Current(dev):
        out = torch.empty_like(logits)
        _check("cgd_route_backward",
               lib.cgd_route_backward(_ptr(grad_topk_weights), _ptr(logits), ltype, _ptr(topk_idx), T, E, K, mode,
                                      int(renormalize), scale, _ptr(out), _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

class _X:
    """x as the library takes it: bf16, or the FP8 tuple (codes, scales)."""

    def __init__(self, x, ndim: int):
        if isinstance(x, tuple):
            if len(x) != 2:
                raise TypeError("x must be a tensor or a (codes, scales) tuple")
            q, sc = x
            if not isinstance(q, torch.Tensor) or q.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError("x codes must be float8_e4m3fn (or uint8)")
            if not isinstance(sc, torch.Tensor) or sc.dtype not in (torch.float32, torch.uint8):
                raise TypeError("x scales must be a float32 (or uint8 UE8M0) tensor")
            _dev_tensor(q, "x codes", q.dtype, ndim)
            H = q.shape[-1]
            if H % 128 or sc.shape != (*q.shape[:-1], H // 128) or sc.device != q.device:
                raise ValueError("x scales must be [..., in_features / 128] on the codes' device")
            self.fmt = SCALE_UE8M0 if sc.dtype == torch.uint8 else SCALE_F32
            self.st, self.sb = self._strides(sc)
            self.kind, self.t, self.scales = _FP8, q, sc
        else:
            _dev_tensor(x, "x", torch.bfloat16, ndim)
            self.kind, self.t, self.scales = _BF16, x, None
            self.fmt, self.st, self.sb = SCALE_F32, 0, 0

    @staticmethod
    def _strides(sc) -> tuple:
        """Row and block stride; a dimension of size 1 has none of its own (whatever torch says)."""
        rows = [(n, st) for n, st in zip(sc.shape[:-1], sc.stride()) if n > 1]
        if not rows or not sc.numel():
            return 0, sc.stride(-1)
        if len(rows) == 2 and rows[0][1] != rows[1][0] * rows[1][1]:
            raise ValueError("x scales must have one row stride over all experts' buffers")
        return rows[-1][1], sc.stride(-1)


def _weight(weight, kind: int, lead: tuple, dev, K: int):
    """-> (weight, its scales or None, rows of one weight)."""
    nd = len(lead) + 2
    if kind == _FP8:
        if not (isinstance(weight, tuple) and len(weight) == 2):
            raise TypeError("FP8 x needs weight as a (codes, scales) tuple")
        w, ws = weight
        if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError("weight codes must be float8_e4m3fn (or uint8)")
        _dev_tensor(w, "weight codes", w.dtype, nd)
        rows = w.shape[-2]
        _shaped(w, "weight codes", w.dtype, (*lead, rows, K), dev)
        _shaped(ws, "weight scales", torch.float32, (*lead, (rows + 127) // 128, K // 128), dev)
        return w, ws, rows
    if isinstance(weight, tuple):
        raise TypeError("bf16 x needs a bf16 weight")
    _dev_tensor(weight, "weight", torch.bfloat16, nd)
    rows = weight.shape[-2]
    _shaped(weight, "weight", torch.bfloat16, (*lead, rows, K), dev)
    return weight, None, rows


def _features(rows: int, act: int) -> int:
    if act != 4:
        return rows
    if rows % 2:
        raise ValueError("a SwiGLU weight holds as many gate rows as up rows")
    return rows // 2


def linear(x, weight, bias: torch.Tensor | None = None, activation: str | None = None,
           residual: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
           return_preact: bool = False, out: torch.Tensor | None = None):
    """act(x @ weight.T + bias) + residual, [T, O].

    x bf16 [T, I] and weight bf16 [O, I]; or FP8 tuples (codes, scales) with
    one scale for 128 values of a row of x ([T, I/128], as per_token_cast_to_fp8
    gives them) and for 128 x 128 of weight ([ceil(O/128), I/128] float32).
    activation: None, "relu", "silu", "gelu" (erf) or "swiglu", whose weight
    holds O gate rows and then O up rows. bias bf16 [weight rows], residual
    bf16 [T, O]. out_dtype bfloat16, or float32 for bf16 x (a gate's logits).
    With return_preact -> (out, preact bf16 [T, weight rows]), which
    linear_backward takes. out, if given, shares no memory with an input, but
    may be residual itself."""
    lib = load()
    X = _X(x, 2)
    T, K = X.t.shape
    dev = X.t.device
    act = _choice(_ACTIVATION, activation, "activation")
    w, ws, rows = _weight(weight, X.kind, (), dev, K)
    O = _features(rows, act)
    if bias is not None:
        _shaped(bias, "bias", torch.bfloat16, (rows,), dev)
    if residual is not None:
        _shaped(residual, "residual", torch.bfloat16, (T, O), dev)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    with _Current(dev):
        if out is None:
            out = torch.empty((T, O), dtype=out_dtype, device=dev)
        else:
            _result(out, out_dtype, (T, O), dev, X.t, X.scales, w, ws, bias, over=residual)
        pre = torch.empty((T, rows), dtype=torch.bfloat16, device=dev) if return_preact else None
        nbytes = lib.cgd_linear_workspace_bytes(T, K, O, act, X.kind)
        wk = _workspace(nbytes, dev)
        _check("cgd_linear",
               lib.cgd_linear(_ptr(X.t), X.kind, _ptr(X.scales), X.st, X.sb, X.fmt, _ptr(w), _ptr(ws), T, K, O,
                              _ptr(bias), act, _ptr(residual), _ptr(out), _F32 if out_dtype == torch.float32 else _BF16,
                              _ptr(pre), _ptr(wk), nbytes, _stream(dev)))
    return (out, pre) if return_preact else out


def _groups(x3: bool, groups, counts, G: int, dev):
    """-> (offsets or None, counts or None) of the rows that hold data."""
    if x3:
        if isinstance(groups, DispatchHandle):
            raise TypeError("a 3-D x has packed buffers: give their row counts (packed_recv_count)")
        if counts is not None:
            raise ValueError("counts goes with offsets; packed buffers take their counts as groups")
        _shaped(groups, "groups (row counts)", torch.int32, (G,), dev)
        return None, groups
    off = groups.expert_offset if isinstance(groups, DispatchHandle) else groups
    _shaped(off, "groups (row offsets)", torch.int32, (G + 1,), dev)
    if counts is not None:
        _shaped(counts, "counts", torch.int32, (G,), dev)
    return off, counts


def grouped_linear(x, weight, groups, bias: torch.Tensor | None = None, activation: str | None = None,
                   counts: torch.Tensor | None = None, return_preact: bool = False, out: torch.Tensor | None = None):
    """act(x @ weight[e].T + bias[e]) for the rows of each expert e.

    x [rows, I] with weight [G, O, I]: groups is a DispatchHandle or its
    expert_offset (int32 [G + 1], segment e = rows [off[e], off[e+1])); counts
    (int32 [G], e.g. num_tokens_per_expert) limits each segment to its first
    rows, where the rest is alignment padding. x [G, cap, I], the packed
    buffers of low_latency_dispatch: groups is their packed_recv_count (int32
    [G]). Types, FP8 tuples, activation and return_preact as in linear, with
    bias [G, weight rows] and FP8 weight scales [G, ceil(O/128), I/128].
    -> bf16 [rows, O] or [G, cap, O]; rows that hold no data are left as they
    were (in a new tensor: undefined)."""
    lib = load()
    nd = (x[0] if isinstance(x, tuple) and x else x).dim() if isinstance(x, (tuple, torch.Tensor)) else 2
    X = _X(x, 3 if nd == 3 else 2)
    lead = tuple(X.t.shape[:-1])
    K = X.t.shape[-1]
    dev = X.t.device
    act = _choice(_ACTIVATION, activation, "activation")
    wt = weight[0] if isinstance(weight, tuple) and weight else weight
    if not isinstance(wt, torch.Tensor) or wt.dim() != 3:
        raise ValueError("weight must be [num_groups, rows, in_features]")
    G = X.t.shape[0] if nd == 3 else wt.shape[0]
    w, ws, rows = _weight(weight, X.kind, (G,), dev, K)
    O = _features(rows, act)
    off, cnt = _groups(nd == 3, groups, counts, G, dev)
    if bias is not None:
        _shaped(bias, "bias", torch.bfloat16, (G, rows), dev)
    cap = lead[1] if nd == 3 else 0
    N = lead[0] * lead[1] if nd == 3 else lead[0]
    with _Current(dev):
        if out is None:
            out = torch.empty((*lead, O), dtype=torch.bfloat16, device=dev)
        else:
            _result(out, torch.bfloat16, (*lead, O), dev, X.t, X.scales, w, ws, bias, off, cnt)
        pre = torch.empty((*lead, rows), dtype=torch.bfloat16, device=dev) if return_preact else None
        nbytes = lib.cgd_grouped_linear_workspace_bytes(N, G, cap, K, O, act, X.kind)
        wk = _workspace(nbytes, dev)
        _check("cgd_grouped_linear",
               lib.cgd_grouped_linear(_ptr(X.t), X.kind, _ptr(X.scales), X.st, X.sb, X.fmt, _ptr(w), _ptr(ws), N, G,
                                      _ptr(off), cap, _ptr(cnt), K, O, _ptr(bias), act, _ptr(out), _ptr(pre), _ptr(wk),
                                      nbytes, _stream(dev)))
    return (out, pre) if return_preact else out


def linear_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                    preact: torch.Tensor | None = None, activation: str | None = None, bias_grad: bool = False):
    """Gradients of linear (bf16): -> (grad_x [T, I], grad_weight like weight,
    grad_bias [weight rows] or None). grad_out bf16 [T, O] (a float32 output's,
    too: a bf16 operand of both products); preact as linear returned it, needed
    with an activation. The residual's gradient is grad_out."""
    lib = load()
    _dev_tensor(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    act = _choice(_ACTIVATION, activation, "activation")
    w, _, rows = _weight(weight, _BF16, (), dev, K)
    O = _features(rows, act)
    _shaped(grad_out, "grad_out", torch.bfloat16, (T, O), dev)
    if (preact is None) != (act == 0):
        raise ValueError("preact goes with an activation")
    if preact is not None:
        _shaped(preact, "preact", torch.bfloat16, (T, rows), dev)
    with _Current(dev):
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        gb = torch.empty(rows, dtype=torch.bfloat16, device=dev) if bias_grad else None
        nbytes = lib.cgd_linear_backward_workspace_bytes(T, K, O, act, int(bias_grad))
        wk = _workspace(nbytes, dev)
        _check("cgd_linear_backward",
               lib.cgd_linear_backward(_ptr(grad_out), _ptr(x), _ptr(w), T, K, O, _ptr(preact), act, _ptr(gx), _ptr(gw),
                                       _ptr(gb), _ptr(wk), nbytes, _stream(dev)))
    return gx, gw, gb


def grouped_linear_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, groups,
                            preact: torch.Tensor | None = None, activation: str | None = None, bias_grad: bool = False,
                            counts: torch.Tensor | None = None):
    """Gradients of grouped_linear (bf16): -> (grad_x like x, grad_weight like
    weight, grad_bias [G, weight rows] or None). Experts without rows get zero
    gradients; rows of grad_x that hold no data are undefined. With a
    DispatchHandle whose segments are padded (expert_alignment > 1), counts must
    say which rows hold data: padding rows would enter the weights' gradient."""
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise TypeError("x must be a 2-D or 3-D bf16 tensor")
    _dev_tensor(x, "x", torch.bfloat16, x.dim())
    packed = x.dim() == 3
    lead = tuple(x.shape[:-1])
    K = x.shape[-1]
    dev = x.device
    act = _choice(_ACTIVATION, activation, "activation")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 3:
        raise ValueError("weight must be [num_groups, rows, in_features]")
    G = x.shape[0] if packed else weight.shape[0]
    w, _, rows = _weight(weight, _BF16, (G,), dev, K)
    O = _features(rows, act)
    if isinstance(groups, DispatchHandle) and groups.expert_alignment > 1 and counts is None:
        raise ValueError("a handle with expert_alignment > 1 needs counts (num_tokens_per_expert): "
                         "padding rows hold no data")
    off, cnt = _groups(packed, groups, counts, G, dev)
    _shaped(grad_out, "grad_out", torch.bfloat16, (*lead, O), dev)
    if (preact is None) != (act == 0):
        raise ValueError("preact goes with an activation")
    if preact is not None:
        _shaped(preact, "preact", torch.bfloat16, (*lead, rows), dev)
    cap = lead[1] if packed else 0
    N = lead[0] * lead[1] if packed else lead[0]
    with _Current(dev):
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        gb = torch.empty((G, rows), dtype=torch.bfloat16, device=dev) if bias_grad else None
        nbytes = lib.cgd_grouped_linear_backward_workspace_bytes(N, G, K, O, act, int(bias_grad))
        wk = _workspace(nbytes, dev)
        _check("cgd_grouped_linear_backward",
               lib.cgd_grouped_linear_backward(_ptr(grad_out), _ptr(x), _ptr(w), N, G, _ptr(off), cap, _ptr(cnt), K, O,
                                               _ptr(preact), act, _ptr(gx), _ptr(gw), _ptr(gb), _ptr(wk), nbytes,
                                               _stream(dev)))
    return gx, gw, gb
