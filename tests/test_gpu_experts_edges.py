"""Calls at the edges of what the computing operators document: scales whose
strides say nothing, more tokens than one launch holds, a gate's gradient."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from test_gpu_products import BF16, F32, _bf, _check_grads, _dev, _fp8_w, _fp8_x, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [cgd.SCALE_F32, cgd.SCALE_UE8M0])
def test_scales_of_one_row(fmt):
    """The stride of a dimension of size 1 is never stepped over, so it may be anything."""
    K, O = 384, 40
    (q, sc), _ = _fp8_x(_gen(1), 1, K, fmt=fmt)
    x, w = _dev((q, sc)), _dev(_fp8_w(_gen(2), (), O, K)[0])
    want = cgd.linear(x, w)
    for st in (1, 1 << 30):
        odd = torch.as_strided(x[1], (1, K // 128), (st, 1))
        assert torch.equal(cgd.linear((x[0], odd), w), want), st


@pytest.mark.parametrize("fmt", [cgd.SCALE_F32, cgd.SCALE_UE8M0])
@pytest.mark.parametrize("G,cap", [(5, 1), (1, 5), (1, 1)])
def test_scales_of_packed_buffers_of_one_row(G, cap, fmt):
    K, O = 384, 40
    say(f"packed scales G={G} cap={cap} fmt={fmt}")
    (q, sc), _ = _fp8_x(_gen(3), G, cap, K, fmt=fmt)
    x, w = _dev((q, sc)), _dev(_fp8_w(_gen(4), (G,), O, K)[0])
    cnt = torch.full((G,), cap, dtype=torch.int32, device=DEV)
    want = cgd.grouped_linear(x, w, cnt)
    nb = K // 128
    # column-major within each buffer: with one buffer or one row there is still one row stride
    turned = x[1].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(cgd.grouped_linear((x[0], turned), w, cnt), want)
    odd = torch.as_strided(x[1], (G, cap, nb), (nb if G > 1 else 1 << 30, nb if cap > 1 else 7, 1))
    assert torch.equal(cgd.grouped_linear((x[0], odd), w, cnt), want)


def test_scales_of_packed_buffers_column_major():
    """Several rows in several buffers need one row stride."""
    (q, sc), _ = _fp8_x(_gen(5), 3, 4, 256)
    x, w = _dev((q, sc)), _dev(_fp8_w(_gen(6), (3,), 16, 256)[0])
    cnt = torch.full((3,), 4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        cgd.grouped_linear((x[0], x[1].transpose(1, 2).contiguous().transpose(1, 2)), w, cnt)
    flat = x[1].view(12, 2).t().contiguous().t().unflatten(0, (3, 4))  # column-major over all rows
    assert torch.equal(cgd.grouped_linear((x[0], flat), w, cnt), cgd.grouped_linear(x, w, cnt))


@pytest.mark.parametrize("biased", [False, True])
def test_more_tokens_than_one_launch_holds(biased):
    """64 work-items for each token, fewer than 2^32 in a launch."""
    T, E, K = (1 << 26) + 5, 2, 1
    say(f"route T={T} biased={biased}")
    l = torch.zeros(T, E, dtype=BF16, device=DEV)
    l[:, 0] = (torch.arange(T, device=DEV) % 3 - 1).to(BF16)  # -1, 0 (a tie), 1 against 0
    l[T - 2] = -float("inf")
    bias = torch.zeros(E, device=DEV) if biased else None
    idx, w = cgd.route(l, K, bias=bias, renormalize=False, scale=2.0)
    torch.cuda.synchronize()
    first = l[:, 0]
    want = (first < 0).long()
    want[T - 2] = -1
    assert torch.equal(idx[:, 0], want)
    best = 2.0 * torch.sigmoid(first.abs().double())
    best[T - 2] = 0.0
    assert ((w[:, 0].double() - best).abs() <= 2.0 ** -20 * best).all()
    del want, w
    if not biased:
        g = cgd.route_backward(torch.ones(T, K, device=DEV), l, idx, renormalize=False)
        torch.cuda.synchronize()
        p = torch.sigmoid(first.double())
        d = p * (1 - p)  # towards the chosen expert
        d = torch.where(idx[:, 0] == 0, d, -d)
        d[T - 2] = 0.0
        for c, want in ((0, d), (1, -d)):
            assert ((g[:, c].double() - want).abs() <= (2.0 ** -19 + 2.0 ** -8) * want.abs()).all(), c


@pytest.mark.parametrize("T,E,K,H", [(1, 8, 2, 64), (300, 256, 8, 512)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_of_a_gate(T, E, K, H, scoring):
    """fp32 logits, their gradient rounded to bf16 once: the operand of both products."""
    say(f"gate gradient T={T} E={E} K={K} H={H} {scoring}")
    g = _gen(T + E)
    x, gate = _bf(g, T, H), _bf(g, E, H, scale=2 / math.sqrt(H))
    logits = cgd.linear(_dev(x), _dev(gate), out_dtype=F32)
    idx, w = cgd.route(logits, K, scoring=scoring)
    gl = cgd.route_backward(torch.randn(T, K, generator=g).to(DEV), logits, idx, scoring=scoring)
    assert gl.dtype == F32
    gx, gg, _ = cgd.linear_backward(gl.bfloat16(), _dev(x), _dev(gate))
    _check_grads(gl.cpu(), x, gate, None, None, E, gx, gg, None, True, "gate")
