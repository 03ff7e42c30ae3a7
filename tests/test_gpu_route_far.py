"""Routing weights and their gradient where the chosen experts lie far below the
token's best, which a bias keeps out of the choice.

The definition in 64 bits has scores down to exp(-745); the chosen ones' shares
are as exact there as anywhere. Tolerances as in test_gpu_route.py: 2^-20 of a
weight, 2^-19 of the sum of a gradient's terms and half a step of its type."""
import math

import numpy as np
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from test_gpu_route import _check, _grad64

pytestmark = pytest.mark.gpu

GAPS = [0.0, 60.0, 90.0, 100.0, 120.0, 700.0, 800.0]  # 800: zero in 64 bits, too
# Scores themselves (not shares) this small are good to 2^-24 of the distance to the best
# logit, 2^-18 here; from 90 on they are below what the tolerances take for zero.
FAINT = (60.0,)


def _far(gap, E, T, dtype, masked):
    """The token's best expert (another one for each token, in service nowhere: the bias), the others `gap` below."""
    g = torch.Generator().manual_seed(int(gap) + E)
    l = (torch.randn(T, E, generator=g) - gap).to(dtype)
    best = torch.arange(T) % masked
    l[torch.arange(T), best] = 3.0
    bias = torch.randn(E, generator=g) * 0.2
    bias[:masked] = -math.inf
    return l, bias


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("E,K", [(8, 2), (64, 8), (256, 8), (512, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups", [1, 4])
def test_weights_of_experts_far_below_the_best(gap, E, K, dtype, groups):
    say(f"route gap={gap} E={E} K={K} {dtype} groups={groups}")
    l, bias = _far(gap, E, 21, dtype, E // 8)
    kw = dict(groups=4, keep=2, group_top=1) if groups > 1 else {}
    _check(l, K, scoring="softmax", bias=bias, renorm=True, **kw)
    if gap not in FAINT:
        _check(l, K, scoring="softmax", bias=bias, renorm=False, **kw)
    if gap < 745:
        _, w = cgd.route(l.to(DEV), K, bias=bias.to(DEV))
        # roundings of the total (6 steps over the lanes), of each weight, of the sum here
        assert ((w.sum(1) - 1).abs() <= (6 + 1 + K) * 2.0 ** -24).all()


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_experts_far_below_the_best(gap, dtype, renorm):
    say(f"route_backward gap={gap} {dtype} renorm={renorm}")
    if gap in FAINT and not renorm:
        pytest.skip("scores good to 2^-18, see FAINT")
    T, E, K = 21, 64, 8
    l, bias = _far(gap, E, T, dtype, E // 8)
    idx, _ = cgd.route(l.to(DEV), K, bias=bias.to(DEV))
    gr = torch.randn(T, K, generator=torch.Generator().manual_seed(1))
    got = cgd.route_backward(gr.to(DEV), l.to(DEV), idx, renormalize=renorm).to(torch.float64).cpu().numpy()
    want, mag = _grad64(l, idx.cpu().numpy(), gr.double().numpy(), "softmax", renorm, 1.0)
    tol = 2.0 ** -19 * mag + 1e-36
    tol = tol + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * (np.abs(want) + tol)
    assert (np.abs(got - want) <= tol).all()
    if gap > 745:
        assert not got.any()  # no weight, no gradient
