"""The activations alone: products with one term (a one-hot weight), so that no
sum's tolerance covers what the activation itself loses.

Derived before the first run. With u = |v| / sqrt 2, the argument of erfc is off by
2^-23 of itself (the constant's rounding and the product's), which moves erfc(u) by at
most (2 u^2 + 1) 2^-23 = (v^2 + 1) 2^-23 of its value; erfc and the products cost less
than 2^-20 together. A sigmoid's exponent, v log2(e), is rounded twice, each 2^-24 of
|v|: |v| 2^-23 of its value, and 2^-21 for the exponential, the sum, the division and
the products. The normal density's exponent is rounded three times, each 2^-24 of v^2 / 2: within (v^2 + 1)
2^-23 of its value as well. The slope is the sum of two such terms. Then half a step
of the result's type."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _values():
    return torch.linspace(-8, 8, 1025).to(BF16)


def _cdf(v):
    return 0.5 * torch.special.erfc(-v / math.sqrt(2))


def _value(v, act):
    """-> (value, error before its rounding)."""
    v = v.to(F64)
    if act == "gelu":
        y = v * _cdf(v)
        return y, y.abs() * (2.0 ** -20 + (v * v + 1) * 2.0 ** -23)
    if act == "silu":
        y = v / (1 + torch.exp(-v))
        return y, y.abs() * (v.abs() * 2.0 ** -23 + 2.0 ** -21)
    return v.clamp_min(0), torch.zeros_like(v)


def _slope(v, act):
    v = v.to(F64)
    if act == "gelu":
        a, b = _cdf(v), v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        return a + b, (a + b.abs()) * (2.0 ** -20 + (v * v + 1) * 2.0 ** -23)
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        a, b = s, v * s * (1 - s)
        return a + b, (a + b.abs()) * (v.abs() * 2.0 ** -23 + 2.0 ** -21)
    return (v > 0).to(F64), torch.zeros_like(v)


def _near(got, want, tol, what):
    bad = ~((got.to(F64).cpu() - want).abs() <= tol + HALF[got.dtype] * (want.abs() + tol))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for {float(want[i])}")


# small tiles (whole and odd widths), a reduction in pieces, 256 x 256 tiles
@pytest.mark.parametrize("K,O", [(8, 24), (8, 25), (1024, 24), (8, 10240)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_value(K, O, dtype, act):
    say(f"activation {act} K={K} O={O} {dtype}")
    v = _values()
    x, w = torch.zeros(len(v), K, dtype=BF16), torch.zeros(O, K, dtype=BF16)
    x[:, K // 2], w[:, K // 2] = v, 1.0
    out, pre = cgd.linear(x.to(DEV), w.to(DEV), activation=act, out_dtype=dtype, return_preact=True)
    assert torch.equal(pre.cpu(), v[:, None].expand(-1, O))
    y, tol = _value(v, act)
    _near(out, y[:, None].expand(-1, O), tol[:, None].expand(-1, O), act)


@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_slope(act):
    say(f"activation slope {act}")
    v = _values()
    want, tol = _slope(v, act)
    one = torch.ones(len(v), 8, dtype=BF16, device=DEV)
    # d itself, through a unit weight
    gx, _, _ = cgd.linear_backward(one, one, torch.eye(8, dtype=BF16, device=DEV),
                                   preact=v[:, None].expand(-1, 8).contiguous().to(DEV), activation=act)
    _near(gx, want[:, None].expand(-1, 8), tol[:, None].expand(-1, 8), "d")
    # the bias gradient of one row: from fp32
    _, _, gb = cgd.linear_backward(one.view(-1)[:len(v)].view(1, -1), one[:1], torch.zeros(len(v), 8, dtype=BF16, device=DEV),
                                   preact=v.view(1, -1).to(DEV), activation=act, bias_grad=True)
    _near(gb, want, tol, "bias gradient")
