"""Gradients on their largest tiles over reductions of one to many stages, and
over packed buffers. References in 64 bits on the GPU; tolerances as derived in
test_gpu_products.py."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from test_gpu_products import BF16, F64, _bf, _d64, _gen, _offsets

pytestmark = pytest.mark.gpu


def _near(got, want, tol, what):
    bad = ~((got.to(F64) - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -120)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: "
                             f"{float(got[i])} for {float(want[i])} +- {float(tol[i])}")


def _check(grad, x, w, pre, act, O, gx, gw, gb, what):
    d, td = _d64(grad, pre, act, O)
    x, w = x.to(F64), w.to(F64)
    r = 2.0 ** -8 if act else 0.0  # d is rounded to bf16
    _near(gx, d @ w, (r + d.shape[1] * 2.0 ** -24) * (d.abs() @ w.abs()) + 1.01 * (td @ w.abs()), what + " grad_x")
    S = d.abs().mT.contiguous() @ x.abs()
    _near(gw, d.mT.contiguous() @ x, (r + d.shape[0] * 2.0 ** -24) * S + 1.01 * (td.mT.contiguous() @ x.abs()),
          what + " grad_weight")
    if gb is not None:
        _near(gb, d.sum(0), d.abs().sum(0) * d.shape[0] * 2.0 ** -24 + td.sum(0), what + " grad_bias")


def _inputs(seed, lead, G, K, O, act):
    g = _gen(seed)
    W = 2 * O if act == "swiglu" else O
    x, w = _bf(g, *lead, K), _bf(g, *G, W, K, scale=1 / math.sqrt(K))
    return [None if t is None else t.to(DEV) for t in (_bf(g, *lead, O), x, w, _bf(g, *lead, W) if act else None)]


# 9 x 24 tiles of 256 x 256 in both directions; reductions of 36 stages and a bit
@pytest.mark.parametrize("T,K,O,act,bias", [(2100, 6144, 2304, None, True), (2305, 6136, 2311, "gelu", False),
                                            (2176, 6152, 1152, "swiglu", True)])
def test_tall_tiles_over_many_stages(T, K, O, act, bias):
    say(f"tall gradients T={T} K={K} O={O} act={act}")
    grad, x, w, pre = _inputs(T, (T,), (), K, O, act)
    gx, gw, gb = cgd.linear_backward(grad, x, w, preact=pre, activation=act, bias_grad=bias)
    _check(grad, x, w, pre, act, O, gx, gw, gb, "dense")


@pytest.mark.parametrize("n", [1, 8, 63, 64, 65, 72, 128, 136, 200, 257, 320, 328, 392, 450])
def test_tall_tiles_over_few_stages(n):
    """Every turn of the operands' slots: n features for the input gradient, n rows for the weight gradient."""
    say(f"tall gradients, a reduction of {n}")
    grad, x, w, _ = _inputs(n, (2100,), (), 6144, n, None)
    gx, gw, _ = cgd.linear_backward(grad, x, w)
    _check(grad, x, w, None, None, n, gx, gw, None, "n features")
    grad, x, w, _ = _inputs(n, (n,), (), 6144, 2304, None)
    gx, gw, gb = cgd.linear_backward(grad, x, w, bias_grad=True)
    _check(grad, x, w, None, None, 2304, gx, gw, gb, "n rows")


@pytest.mark.parametrize("act,O", [(None, 1664), ("swiglu", 832), ("gelu", 1661)])
def test_tall_tiles_of_uneven_groups(act, O):
    G, N, K = 6, 3000, 3200
    say(f"tall gradients of groups act={act}")
    grad, x, w, pre = _inputs(O, (N,), (G,), K, O, act)
    off = _offsets(_gen(2), G, N, empty=(2,))
    gx, gw, gb = cgd.grouped_linear_backward(grad, x, w, off.to(DEV), preact=pre, activation=act, bias_grad=True)
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        _check(grad[a:z], x[a:z], w[e], None if pre is None else pre[a:z], act, O, gx[a:z], gw[e], gb[e], f"group {e}")


# XCDs take a weight gradient's tiles in turn: few groups, many groups; and in runs
@pytest.mark.parametrize("G,N,K,W", [(33, 600, 2048, 2048), (10, 900, 2048, 2049), (2, 300, 4096, 4104), (16, 500, 2048, 2048)])
def test_weight_gradients_shared_out(G, N, K, W):
    say(f"weight gradients G={G} N={N} K={K} W={W}")
    grad, x, w, _ = _inputs(G, (N,), (G,), K, W, None)
    off = _offsets(_gen(G), G, N, empty=(1,) if G > 2 else ())
    gx, gw, gb = cgd.grouped_linear_backward(grad, x, w, off.to(DEV), bias_grad=True)
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        _check(grad[a:z], x[a:z], w[e], None, None, W, gx[a:z], gw[e], gb[e], f"group {e}")


# few rows; odd widths; tall tiles; rows in pieces, some without any
@pytest.mark.parametrize("G,cap,K,O", [(1, 1, 64, 16), (4, 30, 128, 100), (7, 150, 136, 257), (6, 601, 3200, 1664),
                                       (2, 2100, 64, 40), (33, 70, 256, 64)])
@pytest.mark.parametrize("act,bias", [(None, True), ("swiglu", True), ("gelu", False)])
def test_packed_buffers(G, cap, K, O, act, bias):
    say(f"packed gradients G={G} cap={cap} K={K} O={O} act={act}")
    grad, x, w, pre = _inputs(G + cap, (G, cap), (G,), K, O, act)
    cnt = torch.randint(0, cap + 1, (G,), generator=_gen(cap), dtype=torch.int32)
    cnt[0] = cap
    if G > 1:
        cnt[1] = 0
    for e in range(G):  # what lies past a count may be anything
        for t in (grad, x, pre):
            if t is not None:
                t[e, int(cnt[e]):] = float("nan")
    gx, gw, gb = cgd.grouped_linear_backward(grad, x, w, cnt.to(DEV), preact=pre, activation=act, bias_grad=bias)
    assert gx.shape == x.shape and (gb is not None) == bias
    for e in range(G):
        n = int(cnt[e])
        _check(grad[e, :n], x[e, :n], w[e], None if pre is None else pre[e, :n], act, O, gx[e, :n], gw[e],
               None if gb is None else gb[e], f"buffer {e}")
