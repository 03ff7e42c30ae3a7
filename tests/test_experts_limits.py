"""Sizes that no launch holds are refused before any HIP call (no GPU needed;
addresses are never dereferenced)."""
import ctypes

import pytest

import combine_get_dispatch_06_amd as cgd

FAKE = ctypes.c_void_p(0x10000)


def _backward(T, act, bias_grad, I=8, O=8, groups=0, capacity=0):
    lib = cgd.load()
    tail = (I, O, FAKE if act else None, act, FAKE, FAKE, FAKE if bias_grad else None, FAKE, 1 << 62, None)
    if groups:
        return lib.cgd_grouped_linear_backward(FAKE, FAKE, FAKE, T, groups, None if capacity else FAKE, capacity, FAKE, *tail)
    return lib.cgd_linear_backward(FAKE, FAKE, FAKE, T, *tail)


@pytest.mark.parametrize("act,bias_grad", [(3, False), (4, True), (0, True)])
@pytest.mark.parametrize("kw", [dict(T=(1 << 29) + 32), dict(T=(1 << 29) + 32, groups=1), dict(T=(1 << 29) - 32, groups=512),
                                dict(T=1 << 29, groups=512, capacity=1 << 20), dict(T=(1 << 30) - 512)])
def test_activation_gradients_of_too_many_rows(kw, act, bias_grad):
    """Pieces of 32 rows, 256 work-items each: fewer than 2^32 in a launch."""
    assert _backward(act=act, bias_grad=bias_grad, **kw) == -1
    assert b"launch" in cgd.load().cgd_last_error()
