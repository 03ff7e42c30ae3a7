"""Grouped products where one tile for each group just fills a round of blocks
(512): groups on both sides of 64, 128 and 192 rows, against 64 bits (tolerances
as derived in test_gpu_products.py)."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from test_gpu_products import BF16, _bf, _dev, _gen, _near, _ref

pytestmark = pytest.mark.gpu


def _lengths(G, mean):
    """Whole lengths that add up to G * mean, the edges of the tiles among them."""
    n = torch.randint(1, 2 * mean, (G,), generator=_gen(mean))
    n[:8] = torch.tensor([0, 1, 127, 128, 129, 191, 192, 193])
    n[8] = 385
    while int(n.sum()) > G * mean:
        k = 9 + int(n[9:].argmax())
        n[k] -= min(int(n[k]), int(n.sum()) - G * mean)
    n[-1] += G * mean - int(n.sum())
    return n


# 56 rows a group and fewer room keep the smaller tile
@pytest.mark.parametrize("G,mean,K,O", [(64, 60, 136, 1000), (64, 57, 1032, 1001), (64, 128, 72, 1003), (60, 100, 264, 1024),
                                        (64, 56, 136, 1000), (48, 90, 136, 1000)])
@pytest.mark.parametrize("act,bias", [(None, False), ("gelu", True), ("swiglu", True)])
def test_groups_around_the_tiles(G, mean, K, O, act, bias):
    say(f"groups around the tiles G={G} mean={mean} K={K} O={O} act={act}")
    if act == "swiglu":
        O //= 2
    W = 2 * O if act == "swiglu" else O
    n = _lengths(G, mean)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    N = int(off[-1])
    assert N == G * mean and int(n.min()) >= 0
    g = _gen(G + mean + K)
    x, w = _bf(g, N + 5, K), _bf(g, G, W, K, scale=1 / math.sqrt(K))
    b = _bf(g, G, W) if bias else None
    room = torch.full((N + 5, O), 7.0, dtype=BF16, device=DEV)
    cgd.grouped_linear(_dev(x), _dev(w), off.to(torch.int32).to(DEV), bias=_dev(b), activation=act, out=room)
    torch.cuda.synchronize()
    out = room.cpu()
    assert (out[N:] == 7.0).all()  # rows behind the last group
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        y, _, t, _ = _ref(x[a:z], w[e], None if b is None else b[e], act, O)
        _near(out[a:z], y, t, BF16, f"group {e} of {z - a} rows")
