"""The norm, the adapters, dropout and combine's gradient as a layer uses them: a
step forward and backward, the FP8 payload on its way through dispatch and the
experts, other streams, two steps at once, captured graphs with new inputs, rows
and launches past 32 bits, and what the calls refuse."""
import math

import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from philox import kept
from test_gpu_experts_step import FP8, STEP, _layer, _within
from test_gpu_layer import BF16, F32, F64, I64, U, _adapters64, _bf, _case, _dev, _gen, _near, _norm64
from test_gpu_products import _fp8_w, _offsets, _ref

pytestmark = pytest.mark.gpu


def _drop64(x, p, seed, offset, res=None):
    limit = round(p * 65536)
    keep = torch.from_numpy(kept(x.numel(), seed, offset, limit)).view(x.shape)
    y = torch.where(keep, x * (65536 / max(1, 65536 - limit)), torch.zeros((), dtype=F64))
    return y if res is None else y + res


@pytest.mark.parametrize("T,I,J,R,none", [(1, 64, 1, 8, 0.0), (50, 264, 3, 16, 0.2), (700, 128, 4, 64, 0.1), (1500, 256, 6, 24, 0.1)])
def test_training_step(T, I, J, R, none):
    """Norm, a projection with adapters behind dropout, dropout to the residual stream,
    and all of it back, against 64-bit autograd.

    A bf16 rounding is off by 2^-8 of its value (STEP); a value is compared within
    (n + 1) steps of the sum of its terms' sizes, taken through the step as absolute
    values, n the roundings on its way, the one in excess for products of two errors
    and fp32 sums:  y, G's dropped form go, z (after y): 1, 1, 2;  grad_b: go, z, itself;
    grad_a the same;  grad_W: go, y, itself;  at y: go, the product, its dropped form,
    the sum of both ways: 4;  grad_x: that, the stream s once in each of s s r^3 (5
    of relative size one step each), itself: 10;  grad_w: at y, s, r, itself: 7."""
    say(f"training step T={T} I={I} J={J} R={R}")
    c = _case(T, J, R, I, I, none, 0, T + I)
    g = _gen(T * 3 + I)
    r, w, W, G = _bf(g, T, I), torch.rand(I, generator=g) + 0.5, _bf(g, I, I, scale=1 / math.sqrt(I)), _bf(g, T, I)
    d = {k: _dev(v) for k, v in c.items()}
    p = 0.25
    y, s = cgd.rms_norm(d["x"], _dev(w), residual=_dev(r))
    z = cgd.dropout(y, p, 99, offset=1)
    delta, hidden = cgd.adapter_linear(z, d["a"], d["b"], d["idx"], scale=d["scale"], return_hidden=True)
    o = cgd.linear(y, _dev(W), residual=delta)
    out = cgd.dropout(o, p, 99, offset=2, residual=s)
    go = cgd.dropout_backward(_dev(G), p, 99, offset=2)
    gz, ga, gb = cgd.adapter_linear_backward(go, z, d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    gy, gW, _ = cgd.linear_backward(go, y, _dev(W))
    gx, gw = cgd.rms_norm_backward(gy + cgd.dropout_backward(gz, p, 99, offset=1), s, _dev(w), grad_sum=_dev(G))

    x64, w64, W64, a64, b64 = (v.to(F64).requires_grad_() for v in (c["x"], w, W, c["a"], c["b"]))
    s64 = x64 + r.to(F64)
    rr = 1 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-6)
    y64 = s64 * rr * w64
    z64 = _drop64(y64, p, 99, 1)
    on = (c["idx"] >= 0)[:, None].to(F64)
    j = c["idx"].clamp_min(0)
    k = c["scale"].to(F64)[j][:, None] * on
    h64 = torch.bmm(a64[j], z64[:, :, None])[:, :, 0]
    d64 = k * torch.bmm(b64[j], h64[:, :, None])[:, :, 0]
    out64 = _drop64(y64 @ W64.T + d64, p, 99, 2, s64)
    (out64 * G.to(F64)).sum().backward()
    with torch.no_grad():
        ay, az, ago = y64.abs(), z64.abs(), _drop64(G.to(F64).abs(), p, 99, 2)
        aa, ab, aW = a64.abs(), b64.abs(), W64.abs()
        mh = torch.bmm(aa[j], az[:, :, None])[:, :, 0]
        md = k * torch.bmm(ab[j], mh[:, :, None])[:, :, 0]
        # out: y 1, z 2, delta 1, o 1, itself 1, on the way of o; s: itself
        _within(out, out64, _drop64(ay @ aW.T + md, p, 99, 2, s64.abs()), 6, "out")
        mgh = k * torch.bmm(ab[j].mT, ago[:, :, None])[:, :, 0]
        mga, mgb = torch.zeros_like(aa), torch.zeros_like(ab)
        mga.index_add_(0, j, mgh[:, :, None] * az[:, None, :])
        mgb.index_add_(0, j, (k * ago)[:, :, None] * mh[:, None, :])
        _within(ga, a64.grad, mga, 4, "a")
        _within(gb, b64.grad, mgb, 4, "b")
        _within(gW, W64.grad, ago.T @ ay, 3, "W")
        mgy = ago @ aW + _drop64(torch.bmm(aa[j].mT, mgh[:, :, None])[:, :, 0], p, 99, 1)
        ms = s64.abs()
        t = mgy * w64.abs()
        mgx = rr * (t + ms * rr * rr * (t * ms).mean(1, keepdim=True)) + G.to(F64).abs()
        _within(gx, x64.grad, mgx, 10, "x")
        _within(gw, w64.grad, (mgy * ms * rr).sum(0), 7, "norm weight")


@pytest.mark.parametrize("T,E,K,H,I,align", [(37, 8, 2, 256, 64, 1), (300, 16, 4, 128, 128, 8)])
def test_experts_backward(T, E, K, H, I, align):
    """The way back through combine: rows and weights as the formula has them, and what
    the experts' gradients make of them does not touch the padding."""
    p = _layer(T + E, T, E, K, H, I)
    d = {k: v.to(DEV) for k, v in p.items()}
    G = _bf(_gen(5), T, H).to(DEV)
    logits = cgd.linear(d["x"], d["gate"], out_dtype=F32)
    idx, wts = cgd.route(logits, K)
    (_, _, cnt, _, _), recv, _, handle = cgd.layout_and_dispatch(d["x"], idx, E, 8, expert_alignment=align)
    recv[handle.recv_src_idx < 0] = float("nan")
    h, pre = cgd.grouped_linear(recv, d["w13"], handle, activation="swiglu", counts=cnt, return_preact=True)
    y = cgd.grouped_linear(h, d["w2"], handle, counts=cnt)
    rows = handle.dst_row.long()
    y[handle.recv_src_idx < 0] = float("nan")
    gy, gw = cgd.combine_backward(G, y, handle, wts)
    assert torch.equal(gy[rows.view(-1)], (wts[..., None] * G.float()[:, None, :]).to(BF16).view(T * K, H))
    terms = y[rows].to(F64) * G.to(F64)[:, None, :]
    _near(gw, terms.sum(-1).cpu(), ((H + 2) * U * terms.abs().sum(-1)).cpu(), F32, "weights")
    gy[handle.recv_src_idx < 0] = float("nan")
    gh, gw2, _ = cgd.grouped_linear_backward(gy, h, d["w2"], handle, counts=cnt)
    gr, gw13, _ = cgd.grouped_linear_backward(gh, recv, d["w13"], handle, preact=pre, activation="swiglu", counts=cnt)
    gx = cgd.combine(gr, handle, torch.ones_like(wts))
    gl = cgd.route_backward(gw, logits, idx)
    for v in (gw2, gw13, gx, gl):
        assert v.isfinite().all()


@pytest.mark.parametrize("fmt", [cgd.SCALE_F32, cgd.SCALE_POW2, cgd.SCALE_UE8M0])
def test_fp8_payload(fmt):
    """The norm's FP8 output through dispatch to the experts' FP8 product, its bf16 one to the gate."""
    T, E, K, H, O = 150, 8, 2, 512, 130
    g = _gen(21)
    x, r, w, gate = _bf(g, T, H), _bf(g, T, H), torch.rand(H, generator=g) + 0.5, _bf(g, E, H, scale=2 / math.sqrt(H))
    wq, wd = _fp8_w(g, (E,), O, H)
    (y, payload), s = cgd.rms_norm(_dev(x), _dev(w), residual=_dev(r), cast_fp8=fmt, return_bf16=True)
    idx, _ = cgd.route(cgd.linear(y, _dev(gate), out_dtype=F32), K)
    (q, sc), _, handle = cgd.dispatch(payload, idx, E, 2)
    src = handle.recv_src_idx[:T * K].long()
    assert torch.equal(q.view(torch.uint8)[:T * K], payload[0].view(torch.uint8)[src]) and torch.equal(sc[:T * K], payload[1][src])
    back = cgd.per_token_cast_back(payload, scale_format=fmt)
    _, y64, _, ty = _norm64(x, r, w, 1e-6)
    block = y64.abs().view(T, -1, 128).amax(-1).repeat_interleave(128, 1)
    f = 1.0 if fmt == cgd.SCALE_F32 else 2.0  # a scale that is up to twice as large
    assert ((back.cpu().to(F64) - y64).abs() <= (2.0 ** -4 + STEP) * y64.abs() + f * 2.0 ** -10 * block / 448 * 1.01 + 2 * ty).all()
    out = cgd.grouped_linear((q, sc), tuple(v.to(DEV) for v in wq), handle).cpu()
    f32 = torch.exp2(sc.cpu().to(F64) - 127) if fmt == cgd.SCALE_UE8M0 else sc.cpu().to(F64)
    xd = q.cpu().to(F32).to(F64) * f32.repeat_interleave(128, -1)
    off = handle.expert_offset.cpu()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        v, _, t, _ = _ref(xd[a:b], wd[e], None, None, O, steps=FP8(H))
        _near(out[a:b], v, t, BF16, f"expert {e}")


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------

def _inputs(seed, T, R):
    c = _case(T, 5, R, 256, 128, 0.1, 0 if T < 1000 else 9, seed)
    g = _gen(seed + 100)
    E, K = 16, 4
    recv_idx = torch.rand(T, E, generator=g).topk(K, 1)[1]
    d = {k: _dev(v) for k, v in c.items()}
    d.update(w=torch.rand(256, generator=g).to(DEV), r=_bf(g, T, 256).to(DEV), topk=recv_idx.to(DEV), y=_bf(g, T * K, 256).to(DEV),
             wts=torch.rand(T, K, generator=g).to(DEV), state=torch.tensor([seed, seed * 7], dtype=I64, device=DEV))
    return d


def _step(d):
    (y, (q, sc)), s = cgd.rms_norm(d["x"], d["w"], residual=d["r"], cast_fp8=cgd.SCALE_F32, return_bf16=True)
    z = cgd.dropout(y, 0.3, d["state"], offset=1)
    out, hidden = cgd.adapter_linear(z, d["a"], d["b"], d["idx"], scale=d["scale"], residual=d["res"], return_hidden=True)
    gz, ga, gb = cgd.adapter_linear_backward(d["grad"], z, d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    gx, gw = cgd.rms_norm_backward(cgd.dropout_backward(gz, 0.3, d["state"], offset=1), s, d["w"], grad_sum=d["r"])
    recv, _, h = cgd.low_latency_dispatch(s, d["topk"], 16, 1)[:3]
    gy, gt = cgd.combine_backward(gx, recv, h, d["wts"])
    n = torch.where((h.recv_src_info >= 0)[..., None], gy, 0)
    return y, q.view(torch.uint8), sc, s, z, out, hidden, gz, ga, gb, gx, gw, n, gt


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T,R", [(40, 16), (600, 32), (1300, 64)])
def test_another_stream_and_two_at_once(T, R):
    a, b = _inputs(1, T, R), _inputs(2, T, R)
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


@pytest.mark.parametrize("T,R", [(40, 16), (600, 32), (1300, 64)])
def test_graphs_replayed_with_new_inputs(T, R):
    """Two captured steps, replayed in turn and at once, with eager work in between; the
    tokens' adapters and dropout's numbers change from replay to replay."""
    steps = []
    for seed in (1, 2):
        d = _inputs(seed, T, R)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            _step(d)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            res = _step(d)
        steps.append((d, graph, res))
    for rnd in range(3):
        want = []
        for n, (d, graph, res) in enumerate(steps):
            fresh = _inputs(10 * rnd + n + 3, T, R)
            for k in d:
                d[k].copy_(fresh[k])
            want.append(_step(fresh))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(res, want[n]), (rnd, n)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _, _, res in steps:
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
# Far away, nothing to do, and what is refused
# ---------------------------------------------------------------------------

def test_norm_past_32_bits():
    T, H = 262200, 8192  # 2^31 values and some
    x = torch.ones(T, H, dtype=BF16, device=DEV)
    g = _gen(2)
    tail, w = _bf(g, 3, H), torch.rand(H, generator=g)
    x[-3:] = _dev(tail)
    y, s = cgd.rms_norm(x, _dev(w), residual=x)
    s64, y64, ts, ty = _norm64(tail, tail, w, 1e-6)
    _near(y[-3:], y64, ty, BF16, "y")
    _near(s[-3:], s64, ts, BF16, "sum")
    assert torch.equal(y[0], y[1000])
    gx, _ = cgd.rms_norm_backward(s, x, _dev(w))
    small, _ = cgd.rms_norm_backward(s[-3:].contiguous(), _dev(tail), _dev(w))
    assert torch.equal(gx[-3:], small)


def test_norm_of_many_small_rows():
    """More rows than one launch holds (2^31 work-items)."""
    T = (1 << 28) + 40
    x = torch.ones(T, 8, dtype=BF16, device=DEV)
    x[-50:] = _dev(_bf(_gen(1), 50, 8))
    w = torch.ones(8, device=DEV)
    y = cgd.rms_norm(x, w)
    assert torch.equal(y[-50:], cgd.rms_norm(x[-50:].contiguous(), w)) and (y[:1000] == 1).all() and (y[1 << 27] == 1).all()


def test_dropout_past_32_bits():
    n = (1 << 32) + 4099
    x = torch.ones(n, dtype=BF16, device=DEV)
    y = cgd.dropout(x, 0.5, 7, offset=3, out=x)
    for first in (0, 1 << 28, (1 << 29) - 1, 1 << 29):
        m = min(4096, n - 8 * first)
        keep = torch.from_numpy(kept(m, 7, 3, 32768, first=first))
        assert torch.equal(y[8 * first:8 * first + m].cpu() == 2, keep)
    assert torch.equal(y[-4099:].cpu() == 2, torch.from_numpy(kept(4099, 7, 3, 32768, first=1 << 29)))


def test_adapters_past_32_bits():
    T, I, O = (1 << 19) + 70, 4096, 4096  # x and out of 2^31 values and some
    x = torch.zeros(T, I, dtype=BF16, device=DEV)
    c = _case(70, 3, 8, I, O, 0.2, 0, 4)
    x[-70:] = _dev(c["x"])
    idx = torch.full((T,), -1, dtype=I64, device=DEV)
    idx[-70:] = _dev(c["idx"])
    out, hidden = cgd.adapter_linear(x, _dev(c["a"]), _dev(c["b"]), idx, scale=_dev(c["scale"]), return_hidden=True)
    h, y, th, ty = _adapters64(c, None)
    _near(out[-70:], y, ty, BF16, "out")
    _near(hidden[-70:], h, th, F32, "hidden")
    assert (out[:-70] == 0).all()
    out[-70:] = _dev(c["grad"])
    got = cgd.adapter_linear_backward(out, x, _dev(c["a"]), _dev(c["b"]), idx, hidden, scale=_dev(c["scale"]))
    small = cgd.adapter_linear_backward(_dev(c["grad"]), _dev(c["x"]), _dev(c["a"]), _dev(c["b"]), _dev(c["idx"]), hidden[-70:].contiguous(),
                                        scale=_dev(c["scale"]))
    for a, b in zip((got[0][-70:], *got[1:]), small):  # (sums in another order: half a step apart at most, of the larger terms)
        assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -10 * b.float().abs().max()).all()


def test_combine_backward_far():
    """Rows past 2^31 values; and more tokens than one launch holds."""
    T, K, H = 40000, 8, 7168
    cap = T * K
    dst = torch.arange(cap, dtype=torch.int32, device=DEV).flip(0).view(T, K).contiguous()
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    h = cgd.DispatchHandle(e, e, dst, e, 1, 1, 1, cap)
    y = torch.ones(cap, H, dtype=BF16, device=DEV)
    grad = torch.zeros(T, H, dtype=BF16, device=DEV)
    grad[0], grad[-1] = 2, 3
    w = torch.full((T, K), 0.5, device=DEV)
    gy, gw = cgd.combine_backward(grad, y, h, w)
    assert (gy[-8:] == 1).all() and (gy[:8] == 1.5).all() and (gy[8:-8:999] == 0).all()
    assert (gw[0] == 2 * H).all() and (gw[-1] == 3 * H).all() and (gw[1:-1] == 0).all()
    del y, gy, grad
    T = (1 << 21) + 5
    dst = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
    h = cgd.DispatchHandle(e, e, dst, e, 1, 1, 1, T)
    x = torch.arange(T, device=DEV).to(BF16)[:, None].expand(T, 8).contiguous()
    gy, gw = cgd.combine_backward(x, x, h, torch.full((T, 1), 2.0, device=DEV))
    assert torch.equal(gy, x + x) and torch.equal(gw[:, 0], 8 * x[:, 0].float() ** 2)


def test_no_rows():
    e = lambda *s, **k: torch.empty(*s, dtype=k.get("dtype", BF16), device=DEV)  # noqa: E731
    w = torch.ones(128, device=DEV)
    y, s = cgd.rms_norm(e(0, 128), w, residual=e(0, 128))
    assert y.shape == s.shape == (0, 128)
    q, sc = cgd.rms_norm(e(0, 128), w, cast_fp8=cgd.SCALE_UE8M0)
    assert q.shape == (0, 128) and sc.shape == (0, 1)
    gx, gw = cgd.rms_norm_backward(e(0, 128), e(0, 128), w)
    assert gx.shape == (0, 128) and (gw == 0).all()
    a, b = torch.ones(2, 8, 64, dtype=BF16, device=DEV), torch.ones(2, 24, 8, dtype=BF16, device=DEV)
    out, hid = cgd.adapter_linear(e(0, 64), a, b, e(0, dtype=I64), return_hidden=True)
    assert out.shape == (0, 24) and hid.shape == (0, 8)
    gx, ga, gb = cgd.adapter_linear_backward(e(0, 24), e(0, 64), a, b, e(0, dtype=I64), hid)
    assert gx.shape == (0, 64) and (ga == 0).all() and (gb == 0).all()
    i = e(0, dtype=torch.int32)
    gy, gw = cgd.combine_backward(e(0, 64), e(0, 64), cgd.DispatchHandle(i, i, e(0, 4, dtype=torch.int32), i, 8, 1, 1, 0),
                                  e(0, 4, dtype=F32))
    assert gy.shape == (0, 64) and gw.shape == (0, 4)


def test_refusals():
    x = torch.zeros(8, 128, dtype=BF16, device=DEV)
    w = torch.ones(128, device=DEV)
    idx = torch.zeros(8, dtype=I64, device=DEV)
    a, b = torch.zeros(2, 8, 128, dtype=BF16, device=DEV), torch.zeros(2, 64, 8, dtype=BF16, device=DEV)
    hid = torch.zeros(8, 8, device=DEV)
    go = torch.zeros(8, 64, dtype=BF16, device=DEV)
    room = torch.zeros(9 * 128, dtype=BF16, device=DEV)
    odd = room[4:4 + 8 * 128].view(8, 128)  # not 16-byte aligned
    dst = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    h = cgd.DispatchHandle(e, e, dst, e, 1, 1, 1, 8)
    wt = torch.zeros(8, 2, device=DEV)
    before = room.clone()
    for call in (
            lambda: cgd.rms_norm(x.float(), w), lambda: cgd.rms_norm(x.t(), torch.ones(8, device=DEV)), lambda: cgd.rms_norm(x, w[:64]),
            lambda: cgd.rms_norm(x, w.half()), lambda: cgd.rms_norm(x, w.cpu()), lambda: cgd.rms_norm(odd, w),
            lambda: cgd.rms_norm(x, w, residual=x[:4]), lambda: cgd.rms_norm(x, w, eps=-1.0), lambda: cgd.rms_norm(x, w, sum_out=x),
            lambda: cgd.rms_norm(x, w, return_bf16=True), lambda: cgd.rms_norm(x, w, cast_fp8=3),
            lambda: cgd.rms_norm(x[:, :64].contiguous(), w[:64].contiguous(), cast_fp8=0), lambda: cgd.rms_norm(x[0, 0], w),
            lambda: cgd.rms_norm(x[:, :4].contiguous(), w[:4].contiguous()),
            lambda: cgd.rms_norm(room[:1024].view(8, 128), w, residual=x, sum_out=room[128:].view(8, 128)),
            lambda: cgd.rms_norm_backward(x[:4], x, w), lambda: cgd.rms_norm_backward(x, x, w, grad_sum=x.float()),
            lambda: cgd.rms_norm_backward(odd, x, w),
            lambda: cgd.dropout(x, -0.1, 1), lambda: cgd.dropout(x, 1.5, 1), lambda: cgd.dropout(x, 0.5, -1),
            lambda: cgd.dropout(x, 0.5, 1 << 64), lambda: cgd.dropout(x, 0.5, 1.5), lambda: cgd.dropout(x, 0.5, 1, offset=-1),
            lambda: cgd.dropout(x, 0.5, idx), lambda: cgd.dropout(x, 0.5, torch.zeros(2, dtype=I64)), lambda: cgd.dropout(x.t(), 0.5, 1),
            lambda: cgd.dropout(x, 0.5, 1, residual=x[:4]), lambda: cgd.dropout(odd, 0.5, 1), lambda: cgd.dropout(x.float(), 0.5, 1),
            lambda: cgd.dropout(room[:1024], 0.5, 1, out=room[64:1088]),
            lambda: cgd.adapter_linear(x, a, b, idx.int()), lambda: cgd.adapter_linear(x, a, b, idx[:4]),
            lambda: cgd.adapter_linear(x[:, :64].contiguous(), a, b, idx), lambda: cgd.adapter_linear(x, a, b[:1], idx),
            lambda: cgd.adapter_linear(x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), idx), lambda: cgd.adapter_linear(x, a, b.float(), idx),
            lambda: cgd.adapter_linear(x, a, b.transpose(1, 2), idx), lambda: cgd.adapter_linear(odd, a, b, idx),
            lambda: cgd.adapter_linear(x, a, b, idx, scale=w[:2].half()), lambda: cgd.adapter_linear(x, a, b, idx, residual=x),
            lambda: cgd.adapter_linear(x, a, b, idx, out=x[:, :64]), lambda: cgd.adapter_linear(x, a, b, idx, out=x.view(-1)[:512].view(8, 64)),
            lambda: cgd.adapter_linear_backward(go[:4], x, a, b, idx, hid), lambda: cgd.adapter_linear_backward(go, x, a, b, idx, hid.half()),
            lambda: cgd.adapter_linear_backward(go[:, :60].contiguous(), x, a, b[:, :60].contiguous(), idx, hid),
            lambda: cgd.combine_backward(x, x, dst, wt), lambda: cgd.combine_backward(x[:4], x, h, wt), lambda: cgd.combine_backward(x, x, h, wt.half()),
            lambda: cgd.combine_backward(x, x, h, wt, out=x), lambda: cgd.combine_backward(x, x[None], h, wt), lambda: cgd.combine_backward(odd, x, h, wt)):
        with pytest.raises((ValueError, TypeError, cgd.CgdError)):
            call()
    torch.cuda.synchronize()
    assert torch.equal(room, before)
