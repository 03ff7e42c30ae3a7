"""The computing operators as they are used together: a layer's step forward
and backward around dispatch and combine, with padded segments, packed buffers
and FP8 payloads, on other streams, two at once and from captured graphs; the
largest tiles, offsets past 32 bits, and what the calls refuse.

Every bf16 rounding is off by at most 2^-8 of its value, fp32 sums by far less
here (at most 2^-13 of the terms' sizes). A value that went through n of them
is compared within (n + 1) * 2^-8 of the sum of its terms' sizes, the terms'
own sizes taken through the layer as absolute values: the one in excess covers
the products of two errors and the fp32 sums."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from test_gpu_products import (BF16, F32, F64, _act64, _bf, _check_grads, _dev, _fp8_w, _fp8_x, _gen, _near, _offsets,
                               _ref)

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8


def FP8(K):
    """Error of an FP8 product over K values, in units of the sum of its terms' sizes (see the products' tests)."""
    return 7 * 2.0 ** -13 + (K + 3) * 2.0 ** -24


def _within(got, want, mag, n, what):
    # the reference's own rounding: 64-bit sums of up to 2^8 terms, none above the largest of mag
    got, tol = got.to(F64).cpu(), (n + 1) * STEP * mag + 2.0 ** -44 * mag.max()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / tol).max()}"


def _layer(seed, T, E, K, H, I):
    """Inputs of a layer on the CPU (bf16; the weights of a SwiGLU expert and of a shared one)."""
    g = _gen(seed)
    return dict(x=_bf(g, T, H), gate=_bf(g, E, H, scale=2 / math.sqrt(H)), w13=_bf(g, E, 2 * I, H, scale=1 / math.sqrt(H)),
                w2=_bf(g, E, H, I, scale=1 / math.sqrt(I)), s13=_bf(g, 2 * I, H, scale=1 / math.sqrt(H)),
                s2=_bf(g, H, I, scale=1 / math.sqrt(I)))


def _mlp64(x, w13, w2, I):
    """-> (value, sum of its terms' sizes)."""
    h = _act64(x.to(F64) @ w13.to(F64).mT, "swiglu", I)
    return h @ w2.to(F64).mT, h.abs() @ w2.to(F64).abs().mT


def _layer64(p, idx, wts, I):
    y, m = _mlp64(p["x"], p["s13"], p["s2"], I)
    for k in range(idx.shape[1]):
        for e in range(p["w13"].shape[0]):
            t = (idx[:, k] == e).nonzero()[:, 0]
            if len(t):
                a, b = _mlp64(p["x"][t], p["w13"][e], p["w2"][e], I)
                y[t] += wts[t, k, None].to(F64) * a
                m[t] += wts[t, k, None].to(F64) * b
    return y, m


SIZES = [(1, 8, 2, 64, 32), (37, 16, 4, 256, 136), (300, 64, 8, 512, 256)]


@pytest.mark.parametrize("T,E,K,H,I", SIZES)
@pytest.mark.parametrize("align", [1, 16])
def test_layer(T, E, K, H, I, align):
    say(f"layer T={T} E={E} K={K} H={H} I={I} align={align}")
    p = _layer(T + E, T, E, K, H, I)
    d = {k: v.to(DEV) for k, v in p.items()}
    logits = cgd.linear(d["x"], d["gate"], out_dtype=F32)
    idx, wts = cgd.route(logits, K, scoring="sigmoid")
    (_, _, per_expert, _, _), recv, _, handle = cgd.layout_and_dispatch(d["x"], idx, E, 8, expert_alignment=align)
    recv[handle.recv_src_idx < 0] = float("nan")  # padding, and what lies behind the last segment
    h = cgd.grouped_linear(recv, d["w13"], handle, activation="swiglu", counts=per_expert)
    y = cgd.grouped_linear(h, d["w2"], handle, counts=per_expert)
    both = cgd.combine(y, handle, wts)
    s = cgd.linear(d["x"], d["s13"], activation="swiglu")
    out = cgd.linear(s, d["s2"], residual=both)
    torch.cuda.synchronize()
    want, mag = _layer64(p, idx.cpu(), wts.cpu(), I)
    _within(out, want, mag, 4, "layer")  # h, y, the combined rows, the sum
    over = cgd.linear(s, d["s2"], residual=both, out=both)  # in place
    assert over is both and torch.equal(over, out)
    # segments with their padding, taken as a whole: the rows that hold data are the same
    h2 = cgd.grouped_linear(recv, d["w13"], handle, activation="swiglu")
    data = handle.recv_src_idx >= 0
    assert torch.equal(h2[data], h[data])


@pytest.mark.parametrize("T,E,K,H,I", SIZES)
@pytest.mark.parametrize("fp8", [False, True])
def test_packed_layer(T, E, K, H, I, fp8):
    say(f"packed layer T={T} E={E} K={K} H={H} I={I} fp8={fp8}")
    if fp8:
        H, I = (H + 127) // 128 * 128, (I + 127) // 128 * 128
    p = _layer(T + E, T, E, K, H, I)
    d = {k: v.to(DEV) for k, v in p.items()}
    idx, wts = cgd.route(cgd.linear(d["x"], d["gate"], out_dtype=F32), K, scoring="softmax")
    recv, count, handle = cgd.low_latency_dispatch(d["x"], idx, E, 8, use_fp8=fp8)
    if fp8:
        (w13, f13), (w2, f2) = _fp8_w(_gen(1), (E,), 2 * I, H), _fp8_w(_gen(2), (E,), H, I)
        h = cgd.grouped_linear(recv, _dev(w13), count, activation="swiglu")
        cast = cgd.per_token_cast_to_fp8(h.view(E * T, I))
        y = cgd.grouped_linear((cast[0].view(E, T, I), cast[1].view(E, T, -1)), _dev(w2), count)
        torch.cuda.synchronize()
        # the products of what they were given, group by group
        f = recv[0].to(F32).to(F64).cpu() * recv[1].to(F64).cpu().repeat_interleave(128, -1)
        c = (cast[0].to(F32).to(F64) * cast[1].to(F64).repeat_interleave(128, -1)).cpu().view(E, T, I)
        for e in range(E):
            n = int(count[e])
            v, _, t, _ = _ref(f[e, :n], f13[e], None, "swiglu", I, steps=FP8(H))
            _near(h[e, :n], v, t, BF16, f"first product, group {e}")
            v, _, t, _ = _ref(c[e, :n], f2[e], None, None, H, steps=FP8(I))
            _near(y[e, :n], v, t, BF16, f"second product, group {e}")
    else:
        recv[torch.arange(T, device=DEV)[None, :] >= count[:, None]] = float("nan")
        y = cgd.grouped_linear(cgd.grouped_linear(recv, d["w13"], count, activation="swiglu"), d["w2"], count)
    out = cgd.low_latency_combine(y, wts, handle)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    if not fp8:
        p["s13"], p["s2"] = torch.zeros_like(p["s13"]), torch.zeros_like(p["s2"])
        want, mag = _layer64(p, idx.cpu(), wts.cpu(), I)
        _within(out, want, mag, 3, "packed layer")


@pytest.mark.parametrize("T,E,K,H,I", SIZES)
@pytest.mark.parametrize("align", [1, 8])
def test_layer_backward(T, E, K, H, I, align):
    """The layer's gradients, put together from the operators' own, against 64-bit autograd."""
    say(f"layer backward T={T} E={E} K={K} H={H} I={I} align={align}")
    p = _layer(T * 3 + E, T, E, K, H, I)
    d = {k: v.to(DEV) for k, v in p.items()}
    G = _bf(_gen(5), T, H)
    logits = cgd.linear(d["x"], d["gate"], out_dtype=F32)
    idx, wts = cgd.route(logits, K, scoring="softmax", scale=1.5)
    (_, _, cnt, _, _), recv, _, handle = cgd.layout_and_dispatch(d["x"], idx, E, 8, expert_alignment=align)
    recv[handle.recv_src_idx < 0] = float("nan")
    h, pre = cgd.grouped_linear(recv, d["w13"], handle, activation="swiglu", counts=cnt, return_preact=True)
    y = cgd.grouped_linear(h, d["w2"], handle, counts=cnt)
    # d/d weight of a slot: its row's product with G; d/d row: the weight times G
    rows = handle.dst_row.long()
    gw = (y[rows].float() * G.to(DEV).float()[:, None, :]).sum(-1)
    gy = torch.full_like(y, float("nan"))
    gy[rows.view(-1)] = (wts[..., None] * G.to(DEV).float()[:, None, :]).to(BF16).view(T * K, H)
    gh, gw2, _ = cgd.grouped_linear_backward(gy, h, d["w2"], handle, counts=cnt)
    gr, gw13, _ = cgd.grouped_linear_backward(gh, recv, d["w13"], handle, preact=pre, activation="swiglu", counts=cnt)
    gx = cgd.combine(gr, handle, torch.ones_like(wts))
    gl = cgd.route_backward(gw, logits, idx, scoring="softmax", scale=1.5)
    torch.cuda.synchronize()

    x, w13, w2 = (p[k].to(F64).requires_grad_() for k in ("x", "w13", "w2"))
    l = logits.cpu().to(F64).requires_grad_()
    i = idx.cpu()
    s = torch.softmax(l, 1).gather(1, i)
    w = 1.5 * s / s.sum(1, keepdim=True)
    g64, total = G.to(F64), 0.0
    a13, a2, ax = w13.detach().abs(), w2.detach().abs(), x.detach().abs()
    m2, m13, mx = torch.zeros(E, H, I, dtype=F64), torch.zeros(E, 2 * I, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    mw = torch.zeros(T, K, dtype=F64)
    for k in range(K):
        for e in range(E):
            t = (i[:, k] == e).nonzero()[:, 0]
            if not len(t):
                continue
            z = x[t] @ w13[e].T
            hh = _act64(z, "swiglu", I)
            total = total + (w[t, k, None] * (hh @ w2[e].T) * g64[t]).sum()
            # sizes: of the gradients of y and h, of d (silu' < 1.1, silu'' <= 0.5)
            z, hh = z.detach(), hh.detach()
            ga, u = z[:, :I].abs(), z[:, I:].abs()
            my = w[t, k, None].detach() * g64[t].abs()
            mh = my @ a2[e]
            md = torch.cat([mh * u * (1.1 + 0.5 * ga), mh * (ga + 1.1 * ga)], 1)
            m2[e] += my.T @ hh.abs()
            m13[e] += md.T @ ax[t]
            mx[t] += md @ a13[e]
            mw[t, k] = ((hh.abs() @ a2[e].T) * g64[t].abs()).sum(1)
    total.backward()
    _within(gw2, w2.grad, m2, 3, "second weight")        # h, gy, itself
    _within(gw13, w13.grad, m13, 5, "first weight")      # gy, gh, preact, d, itself
    _within(gx, x.grad, mx, 6, "x")                      # and the rows' sum
    sh, mwt = w.detach() / 1.5, mw * 1.5
    ml = torch.zeros(T, E, dtype=F64).scatter_(1, i, sh * (mwt + (sh * mwt).sum(1, keepdim=True)))
    _within(gl, l.grad, ml, 2, "logits")                 # h, y


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "swiglu"])
def test_gradients_against_differences(act):
    """Along random directions the gradients give the change of a 64-bit loss."""
    T, K, O, step = 40, 72, 48, 2.0 ** -16
    g = _gen(3)
    W = 2 * O if act == "swiglu" else O
    x, w, b = _bf(g, T, K), _bf(g, W, K, scale=1 / math.sqrt(K)), _bf(g, W)
    G = _bf(g, T, O)
    _, pre = cgd.linear(_dev(x), _dev(w), bias=_dev(b), activation=act, return_preact=True)
    # from the preact as it is kept: the loss is taken around it
    gx, gw, gb = cgd.linear_backward(_dev(G), _dev(x), _dev(w), preact=pre if act else None, activation=act, bias_grad=True)
    p64 = pre.cpu().to(F64)
    x, w, G = x.to(F64), w.to(F64), G.to(F64)
    for grad, name in ((gx, "x"), (gw, "weight"), (gb, "bias")):
        v = torch.randn(grad.shape, generator=g, dtype=F64)
        move = {"x": lambda: v @ w.T, "weight": lambda: x @ v.T, "bias": lambda: v.expand(T, W)}[name]()

        def loss(s):
            return (_act64(p64 + s * move, act, O) * G).sum()

        num = (loss(step) - loss(-step)) / (2 * step)
        # d rounded once, the gradient once; differences: the second derivative's jump of relu counts
        # where |preact| <= step * |move|, else step^2 times a bounded third derivative
        slope = torch.ones(T, W, dtype=F64)
        if act == "swiglu":
            slope = torch.cat([p64[:, O:].abs(), p64[:, :O].abs()], 1)
        size = (G.abs().repeat(1, W // O) * 1.2 * slope * move.abs()).sum()
        parts = {"x": lambda: (v.abs() @ w.abs().T), "weight": lambda: (x.abs() @ v.abs().T),
                 "bias": lambda: v.abs().expand(T, W)}[name]()
        mag = (G.abs().repeat(1, W // O) * 1.2 * slope * parts).sum()
        kink = (G.abs() * move.abs())[p64.abs() <= step * move.abs()].sum() if act == "relu" else 0.0
        got = (grad.cpu().to(F64) * v).sum()
        assert abs(got - num) <= 3 * STEP * mag + kink + 1e-6 * size, (name, float(got), float(num), float(mag))


# ---------------------------------------------------------------------------
# The largest tiles
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("K", [128, 384, 512, 1664])
@pytest.mark.parametrize("act,bias,fmt", [(None, False, cgd.SCALE_F32), ("gelu", True, cgd.SCALE_UE8M0),
                                          ("swiglu", True, cgd.SCALE_F32)])
def test_fp8_tall_tiles_over_many_steps(K, act, bias, fmt):
    say(f"fp8 tall tiles K={K} act={act} fmt={fmt}")
    G, N, O = 5, 2100, 2944 if act == "swiglu" else 5900
    g = _gen(K)
    W = 2 * O if act == "swiglu" else O
    (xq, xd), (wq, wd) = _fp8_x(g, N, K, fmt=fmt), _fp8_w(g, (G,), W, K)
    b = _bf(g, G, W) if bias else None
    off = _offsets(g, G, N, empty=(2,))
    out, pre = cgd.grouped_linear(_dev(xq), _dev(wq), _dev(off), bias=_dev(b), activation=act, return_preact=True)
    dense = cgd.linear(_dev(xq), (_dev(wq)[0][0], _dev(wq)[1][0]), bias=None if b is None else _dev(b)[0], activation=act)
    torch.cuda.synchronize()
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        y, pr, t, tp = _ref(xd[a:z].to(DEV), wd[e].to(DEV), None if b is None else b[e].to(DEV), act, O, steps=FP8(K))
        _near(out[a:z], y.cpu(), t.cpu(), BF16, f"group {e}")
        _near(pre[a:z], pr.cpu(), tp.cpu(), BF16, f"preact, group {e}")
    y, _, t, _ = _ref(xd.to(DEV), wd[0].to(DEV), None if b is None else b[0].to(DEV), act, O, steps=FP8(K))
    _near(dense, y.cpu(), t.cpu(), BF16, "dense")


@pytest.mark.parametrize("T,K,O", [(2100, 384, 6144), (2049, 256, 6152), (2303, 128, 6140)])
def test_tall_tiles_with_a_residual(T, K, O):
    """Whole tiles, tiles that stick out below and to the right, rows that are no whole number of stores."""
    say(f"tall tiles with a residual T={T} K={K} O={O}")
    g = _gen(T)
    res = _bf(g, T, O)
    (xq, xd), (wq, wd) = _fp8_x(g, T, K), _fp8_w(g, (), O, K)
    room = torch.full((T + 8, O), 7.0, dtype=BF16, device=DEV)
    cgd.linear(_dev(xq), _dev(wq), residual=_dev(res), out=room[:T])
    y, _, t, _ = _ref(xd.to(DEV), wd.to(DEV), None, None, O, res.to(DEV), steps=FP8(K))
    _near(room[:T], y.cpu(), t.cpu(), BF16, "fp8")
    x, w = _bf(g, T, K), _bf(g, O, K, scale=1 / math.sqrt(K))
    out = cgd.linear(_dev(x), _dev(w), residual=_dev(res))
    y, _, t, _ = _ref(x.to(DEV), w.to(DEV), None, None, O, res.to(DEV))
    _near(out, y.cpu(), t.cpu(), BF16, "bf16")
    assert (room[T:] == 7.0).all()


@pytest.mark.parametrize("G,N,K,O", [(1, 1, 128, 16), (1, 40, 640, 300), (1, 500, 1152, 129), (3, 70, 256, 260),
                                     (16, 900, 2048, 256), (5, 2100, 128, 5900), (5, 2100, 1664, 5900),
                                     (4, 3100, 512, 3333)])
@pytest.mark.parametrize("fmt", [cgd.SCALE_F32, cgd.SCALE_UE8M0])
def test_fp8_exact(G, N, K, O, fmt):
    """Products that differ by 2^4 at most, scales by 2^4: all sums are multiples of 2^-4 below 2^20, hence exact."""
    say(f"fp8 exact G={G} N={N} K={K} O={O} fmt={fmt}")
    g = _gen(N + K)

    def codes(*shape):
        return torch.exp2(torch.randint(-1, 2, shape, generator=g).float()) * (1 - 2.0 * torch.randint(0, 2, shape, generator=g))

    x, w = codes(N, K), codes(G, O, K)
    xs = torch.randint(-1, 2, (N, K // 128), generator=g)
    ws = torch.exp2(torch.randint(-1, 2, (G, (O + 127) // 128, K // 128), generator=g).float())
    sc = (xs + 127).to(torch.uint8) if fmt == cgd.SCALE_UE8M0 else torch.exp2(xs.float())
    off = _offsets(g, G, N)
    q = torch.float8_e4m3fn
    out = cgd.grouped_linear(_dev((x.to(q), sc)), _dev((w.to(q), ws)), _dev(off))
    xd = (x * torch.exp2(xs.float()).repeat_interleave(128, 1)).to(DEV, F64)
    wd = (w * ws.repeat_interleave(128, 1)[:, :O].repeat_interleave(128, 2)).to(DEV, F64)
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        assert torch.equal(out[a:z], (xd[a:z] @ wd[e].T).to(BF16)), e
    assert torch.equal(cgd.linear(_dev((x.to(q), sc)), _dev((w[0].to(q), ws[0]))), (xd @ wd[0].T).to(BF16))


@pytest.mark.parametrize("G,N,K,W", [(17, 900, 2048, 2048), (33, 1500, 1536, 1288), (130, 3000, 520, 1280), (1, 20000, 520, 72),
                                     (3, 5000, 264, 40), (7, 9000, 136, 257), (2, 1100, 64, 8)])
def test_weight_gradients_of_many_groups_and_of_many_rows(G, N, K, W):
    """Tiles shared out over the XCDs; a group's rows in pieces (uneven groups: some pieces without rows)."""
    say(f"weight gradients G={G} N={N} K={K} W={W}")
    g = _gen(G)
    off = _offsets(g, G, N, empty=(1, G - 2) if G > 3 else ())
    x, w, grad = _bf(g, N, K), _bf(g, G, W, K, scale=1 / math.sqrt(K)), _bf(g, N, W)
    gx, gw, gb = cgd.grouped_linear_backward(_dev(grad), _dev(x), _dev(w), _dev(off), bias_grad=True)
    torch.cuda.synchronize()
    gx, gw, gb = gx.cpu(), gw.cpu(), gb.cpu()
    for e in range(G):
        a, z = int(off[e]), int(off[e + 1])
        _check_grads(grad[a:z], x[a:z], w[e], None, None, W, gx[a:z], gw[e], gb[e], False, f"group {e}")


def test_offsets_past_32_bits():
    """More than 2^32 elements of x, of the output and of the gradient."""
    N, K, O = 600_000, 8192, 16
    g = _gen(4)
    off = torch.tensor([0, 5, N - 9, N], dtype=torch.int32)
    cnt = torch.tensor([5, 3, 9], dtype=torch.int32)
    say(f"offsets past 32 bits N={N} K={K}")
    x = torch.empty(N, K, dtype=BF16, device=DEV)
    data = torch.cat([torch.arange(0, 8), torch.arange(N - 9, N)])
    xd = _bf(g, len(data), K)
    x[data.to(DEV)] = xd.to(DEV)
    w, grad = _bf(g, 3, O, K, scale=1 / math.sqrt(K)), torch.zeros(N, O, dtype=BF16, device=DEV)
    gd = _bf(g, len(data), O)
    grad[data.to(DEV)] = gd.to(DEV)
    out = cgd.grouped_linear(x, _dev(w), _dev(off), counts=_dev(cnt))
    gx, gw, _ = cgd.grouped_linear_backward(grad, x, _dev(w), _dev(off), counts=_dev(cnt))
    torch.cuda.synchronize()
    for e, (a, z) in enumerate(((0, 5), (5, 8), (8, 17))):
        at = data[a:z].to(DEV)
        y, _, t, _ = _ref(xd[a:z], w[e], None, None, O)
        _near(out[at], y, t, BF16, f"out {e}")
        _check_grads(gd[a:z], xd[a:z], w[e], None, None, O, gx[at].cpu(), gw[e].cpu(), None, False, f"group {e}")
    del gx, x
    # the other way round: a wide output
    say(f"wide output N={N} O={K}")
    x = torch.zeros(N, O, dtype=BF16, device=DEV)
    x[data.to(DEV)] = gd.to(DEV)
    w = _bf(g, 3, K, O)
    out = cgd.grouped_linear(x, _dev(w), _dev(off), counts=_dev(cnt))
    torch.cuda.synchronize()
    for e, (a, z) in enumerate(((0, 5), (5, 8), (8, 17))):
        y, _, t, _ = _ref(gd[a:z], w[e], None, None, K)
        _near(out[data[a:z].to(DEV)], y, t, BF16, f"wide out {e}")


# ---------------------------------------------------------------------------
# Streams, graphs
# ---------------------------------------------------------------------------

def _step_inputs(seed, T=130, E=16, K=4, H=512, I=264):
    p = _layer(seed, T, E, K, H, I)
    p["G"] = _bf(_gen(seed + 1), T, H)
    return {k: v.to(DEV) for k, v in p.items()}


def _step(d, E=16, K=4):
    """A layer forward and the products' gradients: one call at least of every kind, split reductions among them."""
    logits = cgd.linear(d["x"], d["gate"], out_dtype=F32)
    idx, wts = cgd.route(logits, K, scoring="sigmoid", num_groups=4, num_topk_groups=2)
    (_, _, cnt, _, _), recv, _, handle = cgd.layout_and_dispatch(d["x"], idx, E, 8)
    h, pre = cgd.grouped_linear(recv, d["w13"], handle, activation="swiglu", return_preact=True)
    y = cgd.grouped_linear(h, d["w2"], handle)
    s, spre = cgd.linear(d["x"], d["s13"], activation="swiglu", return_preact=True)
    out = cgd.linear(s, d["s2"], residual=cgd.combine(y, handle, wts))
    gl = cgd.route_backward(wts, logits, idx, scoring="sigmoid")
    gs, gs2, _ = cgd.linear_backward(d["G"], s, d["s2"])
    gx, gs13, gb = cgd.linear_backward(gs, d["x"], d["s13"], preact=spre, activation="swiglu", bias_grad=True)
    gh, gw2, _ = cgd.grouped_linear_backward(y, h, d["w2"], handle)
    _, gw13, geb = cgd.grouped_linear_backward(gh, recv, d["w13"], handle, preact=pre, activation="swiglu", bias_grad=True)
    return [logits, idx, wts, out, gl, gs, gs2, gx, gs13, gb, gw2, gw13, geb]


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_another_stream_and_two_at_once():
    a, b = _step_inputs(1), _step_inputs(2)
    want_a, want_b = _step(a), _step(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got = {}
        for name, s, d in (("a", s1, a), ("b", s2, b)):
            with torch.cuda.stream(s):
                got[name] = _step(d)
        torch.cuda.synchronize()
        assert _same(got["a"], want_a) and _same(got["b"], want_b)


def test_graphs_replayed_with_new_inputs():
    """Two captured steps, replayed in turn and at once, with eager work in between."""
    steps = []
    for seed in (1, 2):
        d = _step_inputs(seed)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            _step(d)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            res = _step(d)
        steps.append((d, graph, res))
    for rnd in range(4):
        want = []
        for n, (d, graph, res) in enumerate(steps):
            fresh = _step_inputs(10 * rnd + n + 3)
            for k in d:
                d[k].copy_(fresh[k])
            want.append(_step(fresh))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(res, want[n]), (rnd, n)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (d, graph, res), s in zip(steps, streams):  # both at once
            for r in res:
                r.zero_()
        torch.cuda.synchronize()
        for (d, graph, res), s in zip(steps, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for n, (d, graph, res) in enumerate(steps):
            assert _same(res, want[n]), ("at once", rnd, n)


# ---------------------------------------------------------------------------
# Nothing to do, and what is refused
# ---------------------------------------------------------------------------

def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=BF16, device=DEV)
    w, w3 = torch.ones(24, 64, dtype=BF16, device=DEV), torch.ones(3, 24, 64, dtype=BF16, device=DEV)
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert cgd.linear(e(0, 64), w).shape == (0, 24)
    assert cgd.linear(e(0, 64), w, activation="swiglu").shape == (0, 12)
    assert cgd.grouped_linear(e(0, 64), w3, zero).shape == (0, 24)
    assert cgd.grouped_linear(e(3, 0, 64), w3, zero[:3].contiguous()).shape == (3, 0, 24)
    gx, gw, gb = cgd.linear_backward(e(0, 24), e(0, 64), w, bias_grad=True)
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()
    gx, gw, gb = cgd.grouped_linear_backward(e(0, 24), e(0, 64), w3, zero, bias_grad=True)
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()
    gx, gw, gb = cgd.grouped_linear_backward(e(3, 0, 12), e(3, 0, 64), w3, zero[:3].contiguous(), preact=e(3, 0, 24),
                                             activation="swiglu", bias_grad=True)
    assert gx.shape == (3, 0, 64) and not gw.any() and not gb.any()
    assert cgd.route_backward(torch.empty(0, 2, device=DEV), torch.empty(0, 8, device=DEV),
                              torch.empty(0, 2, dtype=torch.int64, device=DEV)).shape == (0, 8)
    # rows, but none that hold data: the output stays, the gradients are zero
    x, y = torch.full((70, 64), float("nan"), dtype=BF16, device=DEV), torch.full((70, 24), 3.0, dtype=BF16, device=DEV)
    cgd.grouped_linear(x, w3, zero, out=y)
    _, gw, gb = cgd.grouped_linear_backward(x[:, :24].contiguous(), x, w3, zero, bias_grad=True)
    torch.cuda.synchronize()
    assert (y == 3.0).all() and not gw.any() and not gb.any()


def test_segments_outside_the_rows_are_cut():
    """Offsets that do not fit the rows reach nothing outside them."""
    x, w = _bf(_gen(1), 100, 64), _bf(_gen(2), 3, 40, 64)
    off = torch.tensor([-50, 30, 20, 1000], dtype=torch.int32)
    room = torch.full((300, 40), 5.0, dtype=BF16, device=DEV)
    cgd.grouped_linear(_dev(x), _dev(w), _dev(off), out=room[100:200])
    gx, gw, gb = cgd.grouped_linear_backward(room[100:200], _dev(x), _dev(w), _dev(off), bias_grad=True,
                                             counts=torch.tensor([-3, 7, 9999], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (room[:100] == 5.0).all() and (room[200:] == 5.0).all()
    assert not gw[:2].any() and gw[2].any()
    # segments that overlap: far more pieces than the rows have
    off = torch.tensor([0, 100] * 64 + [0], dtype=torch.int32)
    w = _bf(_gen(3), 128, 40, 64)
    out = cgd.grouped_linear(_dev(x), _dev(w), _dev(off))
    gx, gw, gb = cgd.grouped_linear_backward(room[100:200], _dev(x), _dev(w), _dev(off), bias_grad=True)
    torch.cuda.synchronize()
    assert out.shape == (100, 40) and torch.isfinite(gb.float()).all() and not gb[1].any()


def test_refusals():
    x, w = torch.zeros(8, 64, dtype=BF16, device=DEV), torch.zeros(32, 64, dtype=BF16, device=DEV)
    w3, off = torch.zeros(2, 32, 64, dtype=BF16, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    flat = torch.zeros(8 * 64 + 8, dtype=BF16, device=DEV)
    l = torch.zeros(8, 16, device=DEV)
    bad = (ValueError, TypeError, cgd.CgdError)
    for call in (
        lambda: cgd.linear(x.cpu(), w), lambda: cgd.linear(x, w.cpu()), lambda: cgd.linear(x.float(), w),
        lambda: cgd.linear(x, w[:, :32]), lambda: cgd.linear(x.t(), w), lambda: cgd.linear(x[:, ::2], w[:, :32].contiguous()),
        lambda: cgd.linear(flat[1:513].view(8, 64), w), lambda: cgd.linear(x, w, activation="tanh"),
        lambda: cgd.linear(x, w[:31].contiguous(), activation="swiglu"), lambda: cgd.linear(x[:, :60].contiguous(), w[:, :60].contiguous()),
        lambda: cgd.linear(x, w, bias=torch.zeros(31, dtype=BF16, device=DEV)),
        lambda: cgd.linear(x, w, bias=torch.zeros(32, device=DEV)),
        lambda: cgd.linear(x, w, residual=torch.zeros(1, 32, dtype=BF16, device=DEV).expand(8, 32)),
        lambda: cgd.linear(x, w, out_dtype=torch.float16), lambda: cgd.linear(x, w, out=x[:, :32]),
        lambda: cgd.linear(x, torch.zeros(64, 64, dtype=BF16, device=DEV), out=x),
        lambda: cgd.linear(x, w, out=w[:8, :32].reshape(8, 32).t().contiguous().t()),
        lambda: cgd.linear(x, w, residual=flat[:256].view(8, 32), out=flat[64:320].view(8, 32)),
        lambda: cgd.grouped_linear(x, w3, off[:2]), lambda: cgd.grouped_linear(x, w3, off.long()),
        lambda: cgd.grouped_linear(x, w3, off.cpu()), lambda: cgd.grouped_linear(x, w, off),
        lambda: cgd.grouped_linear(x, w3, off, counts=off), lambda: cgd.grouped_linear(x.view(2, 4, 64), w3, off),
        lambda: cgd.grouped_linear(x.view(2, 4, 64), w3, off[:2], counts=off[:2]),
        lambda: cgd.grouped_linear(x, torch.zeros(2, 64, 64, dtype=BF16, device=DEV), off, out=x),
        lambda: cgd.linear_backward(x[:, :32], x, w), lambda: cgd.linear_backward(x[:1, :32].expand(8, 32), x, w),
        lambda: cgd.linear_backward(x[:, :32].contiguous(), x, w, activation="gelu"),
        lambda: cgd.linear_backward(x[:, :32].contiguous(), x, w, preact=x[:, :32].contiguous()),
        lambda: cgd.grouped_linear_backward(x[:, :32].contiguous(), x, w3, off[:2]),
        lambda: cgd.route(l, 0), lambda: cgd.route(l, 17), lambda: cgd.route(l, 1 << 40), lambda: cgd.route(l, -1),
        lambda: cgd.route(l.half(), 2), lambda: cgd.route(l.t(), 2), lambda: cgd.route(l, 2, scoring="tanh"),
        lambda: cgd.route(l, 2, bias=torch.zeros(15, device=DEV)), lambda: cgd.route(l, 2, num_groups=3),
        lambda: cgd.route(l, 2, num_groups=4, num_topk_groups=5),
        lambda: cgd.route_backward(l[:, :2], l, torch.zeros(8, 2, dtype=torch.int64, device=DEV)),
        lambda: cgd.route_backward(l[:, :2].contiguous(), l, torch.zeros(8, 2, dtype=torch.int32, device=DEV)),
        lambda: cgd.route_backward(l[:4, :2].contiguous(), l, torch.zeros(8, 2, dtype=torch.int64, device=DEV)),
    ):
        with pytest.raises(bad):
            call()
    # a padded handle's gradient needs the counts
    idx, _ = cgd.route(l, 2)
    _, _, _, handle = (None, *cgd.dispatch(x, idx, 16, 8, expert_alignment=4))
    recv = torch.zeros(handle.recv_capacity, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        cgd.grouped_linear_backward(recv[:, :32].contiguous(), recv, torch.zeros(16, 32, 64, dtype=BF16, device=DEV), handle)
