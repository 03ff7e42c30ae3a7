"""The router and its gradient against a plain computation in 64 bits.

The choice has to be equal, entry by entry. A weight is a quotient of fp32
exponentials (each good to 2^-22 for arguments this small) or of 64-bit ones,
rounded to fp32 once: 2^-20 of the value covers it. A gradient is a sum of at
most 17 such products, each good to 2^-20 of its factors: 2^-19 of the sum of
the terms' sizes, then half a step of its type."""
import math

import numpy as np
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
INF = math.inf


def _clean(logits):
    l = logits.to(torch.float64).numpy().copy()
    l[np.isnan(l)] = -INF
    return np.minimum(l, np.finfo(np.float32).max)


def _scores(l, scoring):
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    top = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isinf(l), 0.0, np.exp(l - top))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def plain_route(logits, K, scoring, bias=None, groups=1, keep=None, group_top=2, renorm=True, scale=1.0):
    l = _clean(logits)
    T, E = l.shape
    s = _scores(l, scoring)
    by_logit = bias is None and (groups == 1 or group_top == 1)
    c = l.copy() if by_logit else s + (0.0 if bias is None else bias.to(torch.float64).numpy())
    c[np.isnan(c) | np.isinf(l)] = -INF
    idx = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    n = E // groups
    for t in range(T):
        v = c[t].copy()
        if groups > 1 and keep is not None and keep < groups:
            val = []
            for q in range(groups):
                o = np.sort(v[q * n:(q + 1) * n])[::-1]
                x = o[0]
                if group_top == 2 and n > 1 and o[1] > -INF:
                    x = o[0] + o[1]
                val.append(x)
            best = sorted(range(groups), key=lambda q: (-val[q], q))[:keep]
            for q in range(groups):
                if q not in best:
                    v[q * n:(q + 1) * n] = -INF
        order = np.argsort(-v, kind="stable")[:K]
        order = [e for e in order if v[e] > -INF]
        idx[t, :len(order)] = order
        p = s[t, order]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else p * 0
        w[t, :len(order)] = p * scale
    return idx, w


def _check(logits, K, **kw):
    bias = kw.pop("bias", None)
    gi, gw = cgd.route(logits.to(DEV), K, bias=None if bias is None else bias.to(DEV), num_groups=kw.get("groups", 1),
                       num_topk_groups=kw.get("keep"), group_score_topk=kw.get("group_top", 2),
                       renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0), scoring=kw["scoring"])
    torch.cuda.synchronize()
    i, w = plain_route(logits, K, bias=bias, **kw)
    np.testing.assert_array_equal(gi.cpu().numpy(), i)
    assert gw.dtype == torch.float32
    err = np.abs(gw.cpu().numpy().astype(np.float64) - w)
    assert (err <= 2.0 ** -20 * np.abs(w) + 1e-37).all(), err.max()


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (130, 60, 6), (33, 64, 8), (17, 65, 4),
                                   (128, 128, 8), (100, 160, 6), (257, 256, 8), (64, 257, 16), (300, 512, 16),
                                   (31, 384, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased,renorm", [(False, True), (False, False), (True, True), (True, False)])
def test_route(T, E, K, scoring, dtype, biased, renorm):
    say(f"route T={T} E={E} K={K} {scoring} {dtype} biased={biased} renorm={renorm}")
    g = torch.Generator().manual_seed(T + E)
    l = (torch.randn(T, E, generator=g) * 2).to(dtype)
    l[torch.rand(T, E, generator=g) < 0.05] = -INF
    if T > 2:
        l[T // 2] = -INF
    bias = torch.randn(E, generator=g) * 0.2 if biased else None
    _check(l, K, scoring=scoring, bias=bias, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,keep,K,group_top", [(256, 8, 4, 8, 2), (256, 8, 4, 8, 1), (64, 4, 1, 6, 2),
                                                       (60, 6, 3, 5, 2), (512, 64, 9, 16, 2), (12, 12, 5, 5, 2),
                                                       (130, 2, 1, 8, 1), (48, 8, 8, 8, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_groups(E, groups, keep, K, group_top, scoring, biased, dtype):
    say(f"route groups E={E} {groups}/{keep} K={K} top{group_top} {scoring} biased={biased} {dtype}")
    g = torch.Generator().manual_seed(E + groups)
    T = 90
    l = (torch.randn(T, E, generator=g) * 2).to(dtype)
    l[torch.rand(T, E, generator=g) < 0.2] = -INF
    l[3] = -INF
    l[4, : E // 2] = -INF
    bias = torch.randn(E, generator=g) * 0.2 if biased else None
    _check(l, K, scoring=scoring, bias=bias, groups=groups, keep=keep, group_top=group_top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,K", [(16, 4), (64, 16), (256, 8), (512, 16)])
def test_route_ties_go_to_the_lowest_index(scoring, biased, E, K):
    say(f"route ties E={E} K={K} {scoring} biased={biased}")
    g = torch.Generator().manual_seed(E)
    l = torch.zeros(40, E)
    l[1:20] = torch.randint(0, 2, (19, E), generator=g).float()       # two values
    l[20:30] = torch.randint(0, E // 4, (10, E), generator=g) / 8.0   # a few of each
    l[30, E // 2:] = -0.0                                             # -0 equals +0
    l[31, 1:] = -INF                                                  # one expert
    _check(l, K, scoring=scoring, bias=torch.zeros(E) if biased else None)


def test_route_odd_values():
    """NaN counts as -inf, +inf as the largest finite value, the lowest finite value is a value."""
    E = 100
    g = torch.Generator().manual_seed(1)
    l = torch.randn(12, E, generator=g)
    l[0, 5] = float("nan")
    l[1, :] = float("nan")
    l[2, 7] = INF
    l[3, [3, 9]] = INF
    l[4, :] = torch.finfo(torch.float32).min
    l[5, 10:] = torch.finfo(torch.float32).min
    l[6, :] = -200.0
    l[7, 0] = 1e30
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            _check(l, 8, scoring=scoring, renorm=renorm)
    bias = torch.zeros(E)
    bias[:50] = -INF
    bias[60] = float("nan")
    _check(l[5:], 8, scoring="sigmoid", bias=bias)
    _check(l, 8, scoring="softmax", bias=bias)
    gi, gw = cgd.route(torch.empty(0, E, device=DEV), 8)
    assert gi.shape == (0, 8) and gw.shape == (0, 8)


def _grad64(logits, idx, g, scoring, renorm, scale):
    """-> (gradient, sum of the terms' sizes)."""
    l = _clean(logits)
    p = _scores(l, scoring)
    T, E = l.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        dp, mp = np.zeros(E), np.zeros(E)
        sel = [(k, int(e)) for k, e in enumerate(idx[t]) if 0 <= e < E]
        S = sum(p[t, e] for _, e in sel)
        for k, e in sel:
            if renorm:
                if S > 0:
                    d = sum(g[t, j] * p[t, q] for j, q in sel) / S
                    md = sum(abs(g[t, j]) * p[t, q] for j, q in sel) / S
                    dp[e] += (g[t, k] - d) / S
                    mp[e] += (abs(g[t, k]) + md) / S
            else:
                dp[e] += g[t, k]
                mp[e] += abs(g[t, k])
        dp, mp = dp * scale, mp * abs(scale)
        if scoring == "sigmoid":
            out[t], mag[t] = dp * p[t] * (1 - p[t]), mp * p[t]
        else:
            out[t] = p[t] * (dp - (p[t] * dp).sum())
            mag[t] = p[t] * (mp + (p[t] * mp).sum())
    return out, mag


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (9, 60, 6), (33, 64, 8), (130, 130, 4), (65, 256, 8),
                                   (40, 512, 16)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward(T, E, K, scoring, renorm, dtype):
    say(f"route_backward T={T} E={E} K={K} {scoring} renorm={renorm} {dtype}")
    g = torch.Generator().manual_seed(T + E + K)
    l = (torch.randn(T, E, generator=g) * 2).to(dtype)
    l[torch.rand(T, E, generator=g) < 0.05] = -INF
    idx = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :K].contiguous()
    idx[torch.rand(T, K, generator=g) < 0.1] = -1
    if T > 5:
        l[3] = -INF
        idx[4] = -1
        idx[5] = idx[5, 0]       # the same expert in every slot
        idx[1, 0] = E + 5        # out of range: no slot
    gr = torch.randn(T, K, generator=g)
    got = cgd.route_backward(gr.to(DEV), l.to(DEV), idx.to(DEV), scoring=scoring, renormalize=renorm, scale=1.7)
    torch.cuda.synchronize()
    assert got.dtype == dtype and got.shape == (T, E)
    want, mag = _grad64(l, idx.numpy(), gr.double().numpy(), scoring, renorm, 1.7)
    tol = 2.0 ** -19 * mag + 1e-36
    tol = tol + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * (np.abs(want) + tol)
    err = np.abs(got.to(torch.float64).cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(scoring, renorm):
    """The weights of a fixed choice, moved by small steps of the logits (in 64 bits)."""
    T, E, K, h = 3, 24, 4, 1e-5
    g = torch.Generator().manual_seed(2)
    l = torch.randn(T, E, generator=g)
    idx, _ = cgd.route(l.to(DEV), K, scoring=scoring)
    gr = torch.randn(T, K, generator=g)
    got = cgd.route_backward(gr.to(DEV), l.to(DEV), idx, scoring=scoring, renormalize=renorm).cpu().double().numpy()
    i = idx.cpu().numpy()

    def value(x):
        p = np.take_along_axis(_scores(x, scoring), i, 1)
        if renorm:
            p = p / p.sum(1, keepdims=True)
        return (p * gr.double().numpy()).sum(1)

    x = l.double().numpy()
    for e in range(E):
        d = np.zeros_like(x)
        d[:, e] = h
        num = (value(x + d) - value(x - d)) / (2 * h)
        # differences: h^2 / 6 of a third derivative below 10, and 64-bit rounding over h
        assert (np.abs(num - got[:, e]) <= 1e-8 + 2.0 ** -18 * np.abs(gr.numpy()).sum(1)).all()
