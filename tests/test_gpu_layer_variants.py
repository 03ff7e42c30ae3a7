"""Every variant that a size chooses, against the definitions in 64 bits: sizes past the
rules' borders, where the norm takes two rows at a time, or the norm, dropout and combine's
gradient pass the Infinity Cache by; and the C calls with outputs left out. Tolerances are
those of test_gpu_layer.py."""
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from philox import kept
from test_gpu_layer import BF16, F32, F64, I64, U, _adapters64, _adapters_grad64, _bf, _case, _check_fp8, _dev, _gen, _near, _norm64

pytestmark = pytest.mark.gpu

MANY = [(65537, 128), (32769, 256), (16387, 512)]  # two rows of a thread's at a time
FAR = [(200003, 128), (90001, 256), (45001, 512), (22001, 1024), (3001, 7168), (1401, 16384), (1101, 20480)]


def _on_gpu(seed, T, H, n):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(T, H, generator=g, device=DEV).to(BF16) for _ in range(n)] + [torch.rand(H, generator=g, device=DEV) + 0.5]


def _rows_of(T):
    return torch.cat([torch.arange(40), torch.randint(T, (150,), generator=_gen(T)), torch.arange(T - 40, T)])


@pytest.mark.parametrize("T,H", MANY + FAR)
@pytest.mark.parametrize("fmt", [None, cgd.SCALE_F32, cgd.SCALE_UE8M0])
@pytest.mark.parametrize("res", [False, True])
def test_norm_of_many_rows(T, H, fmt, res):
    say(f"norm of many rows T={T} H={H} fmt={fmt} res={res}")
    x, r, w = _on_gpu(T + H, T, H, 2)
    got = cgd.rms_norm(x, w, residual=r if res else None, cast_fp8=fmt, return_bf16=fmt is not None)
    got, total = got if res else (got, None)
    y, q = got if fmt is not None else (got, None)
    at = _rows_of(T)
    s64, y64, ts, ty = _norm64(x[at].cpu(), r[at].cpu() if res else None, w.cpu(), 1e-6)
    _near(y[at], y64, ty, BF16, "y")
    if res:
        _near(total[at], s64, ts, BF16, "sum")
    if q is not None:
        _check_fp8(q[0][at], q[1][at], y64, ty, fmt)
        alone = cgd.rms_norm(x, w, residual=r if res else None, cast_fp8=fmt)
        alone = alone[0] if res else alone
        assert torch.equal(alone[0].view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(alone[1], q[1])
    # every row: few at a time they go through another variant, whose sums have another
    # order; both are rounded once, and off by (H / 2 + 8) u before that
    few = torch.cat([cgd.rms_norm(a, w, residual=b)[0] for a, b in zip(x.split(500), r.split(500))] if res else
                    [cgd.rms_norm(a, w) for a in x.split(500)])
    assert ((y.float() - few.float()).abs() <= (2.0 ** -7 * 1.01 + (H + 32) * U) * few.float().abs()).all()


@pytest.mark.parametrize("T,H", MANY + FAR)
@pytest.mark.parametrize("extra", [False, True])
def test_norm_backward_of_many_rows(T, H, extra):
    say(f"norm backward of many rows T={T} H={H} extra={extra}")
    x, gy, gs, w = _on_gpu(T * 3 + H, T, H, 3)
    gx, gw = cgd.rms_norm_backward(gy, x, w, eps=1e-5, grad_sum=gs if extra else None)
    r = 1 / torch.sqrt(torch.cat([(a.to(F64) ** 2).mean(1, keepdim=True) for a in x.split(1000)]) + 1e-5)
    terms = [(b.to(F64) * a.to(F64) * c) for a, b, c in zip(x.split(1000), gy.split(1000), r.split(1000))]
    _near(gw, sum(t.sum(0) for t in terms).cpu(), ((T + H / 2 + 8) * U * sum(t.abs().sum(0) for t in terms)).cpu(), F32, "grad_weight")
    del terms
    at = _rows_of(T).to(DEV)
    x, gy, gs, r, w = x[at].to(F64), gy[at].to(F64), gs[at].to(F64), r[at], w.to(F64)
    gwx = gy * w * x
    want = r * (gy * w - x * r * r * gwx.mean(1, keepdim=True))
    tol = (2 * H + 16) * U * r * ((gy * w).abs() + x.abs() * r * r * gwx.abs().mean(1, keepdim=True))
    if extra:
        want = want + gs
        tol = tol + 2 * U * (want.abs() + gs.abs())
    _near(gx[at], want.cpu(), tol.cpu(), BF16, "grad_x")


@pytest.mark.parametrize("n,res", [(27962025, True), (27962027, True), (28000003, True), (41943043, False), (41943039, False)])
def test_dropout_past_the_caches(n, res):
    say(f"dropout n={n} res={res}")
    x, r, _ = _on_gpu(n, 1, n, 2)
    x, r = x[0], r[0]
    got = cgd.dropout(x, 0.3, 11, offset=5, residual=r if res else None)
    limit = round(0.3 * 65536)
    scale = 65536 / (65536 - limit)
    add = r.to(F64) if res else torch.zeros((), dtype=F64, device=DEV)
    whole, none = x.to(F64) * scale + add, add.expand(n)
    tol = 3 * U * whole.abs() + U * (whole.abs() + add.abs())
    near = lambda want, t: (got.to(F64) - want).abs() <= t + 2.0 ** -8 * (want.abs() + t) + 2.0 ** -120  # noqa: E731
    is_kept, is_dropped = near(whole, tol), near(none, torch.zeros_like(tol))
    assert (is_kept | is_dropped).all()
    for first in (0, n // 16, n // 8 - 512):
        m = min(4096 + 8, n - 8 * first)
        keep = torch.from_numpy(kept(m, 11, 5, limit, first=first))
        part = slice(8 * first, 8 * first + m)
        assert is_kept[part].cpu()[keep].all() and is_dropped[part].cpu()[~keep].all()


@pytest.mark.parametrize("T,E,K,H", [(580, 64, 8, 7168), (1100, 32, 16, 2056)])
def test_combine_backward_past_the_caches(T, E, K, H):
    say(f"combine backward past the caches T={T} E={E} K={K} H={H}")
    g = _gen(T)
    idx = torch.rand(T, E, generator=g).topk(K, 1)[1]
    idx[torch.rand(T, K, generator=g) < 0.1] = -1
    grad, w = _bf(g, T, H).to(DEV), torch.randn(T, K, generator=g).to(DEV)
    recv, _, handle = cgd.dispatch(grad, _dev(idx), E, 1)
    y, _ = _on_gpu(T, *recv.shape, 1)
    out = torch.full_like(y, 5.0)
    gy, gw = cgd.combine_backward(grad, y, handle, w, out=out)
    dst = handle.dst_row.long()
    t, k = (dst >= 0).nonzero(as_tuple=True)
    rows = dst[t, k]
    assert (gw[dst < 0] == 0).all()
    want = grad[t].to(F64) * y[rows].to(F64)
    _near(gw[t, k], want.sum(1).cpu(), ((H + 2) * U * want.abs().sum(1)).cpu(), F32, "grad_topk_weights")
    want = w[t, k].to(F64)[:, None] * grad[t].to(F64)
    _near(gy[rows], want.cpu(), (U * want.abs()).cpu(), BF16, "grad_expert_out")
    left = torch.ones(len(y), dtype=torch.bool, device=DEV)
    left[rows] = False
    assert (gy[left] == 5).all()


# ---------------------------------------------------------------------------
# Outputs left out: only a C caller can. What is asked for has the bits of the whole call.
# ---------------------------------------------------------------------------

def _call(name, *args):
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(cgd.load(), name)(*args, torch.cuda.current_stream().cuda_stream) == 0, cgd.load().cgd_last_error()
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H", [(3, 64), (40, 256), (9, 1024), (5, 1032), (600, 4096), (3, 20480)])
def test_norm_outputs_left_out(T, H):
    say(f"norm outputs left out T={T} H={H}")
    g = _gen(T + H)
    x, r, gy, w = _bf(g, T, H).to(DEV), _bf(g, T, H).to(DEV), _bf(g, T, H).to(DEV), torch.rand(H, generator=g).to(DEV)
    y, _ = cgd.rms_norm(x, w, residual=r)
    alone = torch.empty_like(y)
    _call("cgd_rms_norm", x, r, w, 1, 1e-6, T, H, alone, None, None, 0, None)  # no sum
    assert torch.equal(alone, y)
    gx, gw = cgd.rms_norm_backward(gy, x, w, grad_sum=r)
    nbytes = cgd.load().cgd_rms_norm_backward_workspace_bytes(T, H)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    gx2, gw2 = torch.empty_like(gx), torch.empty_like(gw)
    _call("cgd_rms_norm_backward", gy, x, w, 1, 1e-6, T, H, r, gx2, None, None, 0)  # which needs no workspace
    _call("cgd_rms_norm_backward", gy, x, w, 1, 1e-6, T, H, r, None, gw2, ws, nbytes)
    assert torch.equal(gx2, gx) and torch.equal(gw2, gw)
    _call("cgd_rms_norm_backward", gy, x, w, 1, 1e-6, T, H, r, None, None, None, 0)


@pytest.mark.parametrize("T,J,R", [(0, 2, 16), (100, 3, 16), (100, 3, 72), (1100, 3, 16), (1100, 5, 72), (1700, 2, 24), (3100, 2, 16), (3100, 2, 40),
                                   (17000, 300, 8)])
def test_adapter_gradients_left_out(T, J, R):
    say(f"adapter gradients left out T={T} J={J} R={R}")
    I, O = 136, 72
    c = _case(T, J, R, I, O, 0.1, 0, T + J + R)
    d = {k: _dev(v) for k, v in c.items()}
    hidden = _adapters64(c, None)[0].to(F32).to(DEV)
    whole = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    want, tol = _adapters_grad64(c, hidden.cpu())
    for v, x, t in zip(whole, want, tol):
        _near(v, x, t, BF16, "whole")
    nbytes = cgd.load().cgd_adapter_linear_backward_workspace_bytes(T, J, R, I, O)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    for asked in range(8):
        out = [torch.full_like(v, 3.0) if asked >> i & 1 else None for i, v in enumerate(whole)]
        _call("cgd_adapter_linear_backward", d["grad"], d["x"] if out[1] is not None else None, d["a"], d["b"], d["scale"], d["idx"],
              hidden if out[2] is not None else None, T, J, R, I, O, *out, ws, nbytes)
        for a, b in zip(out, whole):
            assert a is None or torch.equal(a, b), asked


@pytest.mark.parametrize("T,J,R", [(200, 64, 16), (1100, 32, 16), (4096, 32, 16), (5000, 64, 40), (20000, 512, 8)])
def test_adapters_of_one_request(T, J, R):
    """Many adapters, all tokens of one of them."""
    say(f"adapters of one request T={T} J={J} R={R}")
    c = _case(T, J, R, 136, 72, 0.0, 0, T + J + R)
    c["idx"] = torch.full((T,), J - 2, dtype=I64)
    d = {k: _dev(v) for k, v in c.items()}
    out, hidden = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=d["res"], return_hidden=True)
    h, y, th, ty = _adapters64(c, c["res"])
    _near(hidden, h, th, F32, "hidden")
    _near(out, y, ty, BF16, "out")
    got = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    want, tol = _adapters_grad64(c, hidden.cpu())
    for name, v, x, t in zip(("grad_x", "grad_a", "grad_b"), got, want, tol):
        _near(v, x, t, BF16, name)


# ---------------------------------------------------------------------------
# The largest sizes that are documented
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,J,R,I,O", [(3, 2, 8, 1 << 20, 24), (70, 2, 8, 1 << 20, 72), (3, 2, 16, 72, 1 << 20), (300, 2, 8, 24, 1 << 20), (3, 512, 256, 64, 40),
                                       (300, 512, 256, 40, 64)])
def test_adapters_of_the_largest_sizes(T, J, R, I, O):
    say(f"adapters of the largest sizes T={T} J={J} R={R} I={I} O={O}")
    c = _case(T, J, R, I, O, 0.1, 0, T + R)
    c["idx"][0] = J - 1
    d = {k: _dev(v) for k, v in c.items()}
    out, hidden = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=d["res"], return_hidden=True)
    h, y, th, ty = _adapters64(c, c["res"])
    _near(hidden, h, th, F32, "hidden")
    _near(out, y, ty, BF16, "out")
    got = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    want, tol = _adapters_grad64(c, hidden.cpu())
    for name, v, x, t in zip(("grad_x", "grad_a", "grad_b"), got, want, tol):
        _near(v, x, t, BF16, name)


def test_adapters_of_the_most_tokens():
    """2^26 tokens whose sums are whole numbers below 2^24, so that fp32 holds them."""
    T, J, R, I = 1 << 26, 5, 8, 8
    say(f"adapters of the most tokens T={T}")
    g = torch.Generator(device=DEV).manual_seed(1)
    idx = torch.randint(-1, J, (T,), generator=g, device=DEV)
    place = torch.randint(I, (T,), generator=g, device=DEV)
    x = torch.zeros(T, I, dtype=BF16, device=DEV)
    x.scatter_(1, place[:, None], 1.0)  # one 1 a row
    one = torch.eye(8, device=DEV)
    a = torch.stack([one.roll(j, 0) for j in range(J)]).to(BF16)  # h = x rolled by j
    b = torch.stack([one * (j + 1) for j in range(J)]).to(BF16)
    out, hidden = cgd.adapter_linear(x, a, b, idx, return_hidden=True)
    on = idx >= 0
    for first in range(0, T, 1 << 22):
        part = slice(first, first + (1 << 22))
        j = idx[part].clamp_min(0)
        want = torch.zeros(1 << 22, R, device=DEV).scatter_(1, ((place[part] + j) % R)[:, None], 1.0) * on[part][:, None]
        assert torch.equal(hidden[part], want), first
        assert torch.equal(out[part].float(), want * (j + 1)[:, None]), first
    del out
    gx, ga, gb = cgd.adapter_linear_backward(x, x, a, b, idx, hidden)
    del hidden
    for first in range(0, T, 1 << 22):
        part = slice(first, first + (1 << 22))
        j = idx[part].clamp_min(0)
        want = torch.zeros(1 << 22, I, device=DEV).scatter_(1, ((place[part] - j) % R)[:, None], 1.0) * ((j + 1) * on[part])[:, None]
        assert torch.equal(gx[part].float(), want), first
    count = torch.zeros(J, I, dtype=torch.int64, device=DEV)  # tokens by adapter and place
    count.view(-1).index_add_(0, (idx * I + place)[on], torch.ones(int(on.sum()), dtype=torch.int64, device=DEV))
    assert int(count.max()) * J < 1 << 24
    for j in range(J):
        want_a = torch.diag(count[j].double() * (j + 1))
        want_b = torch.zeros(I, R, dtype=F64, device=DEV)
        want_b[torch.arange(I), (torch.arange(I) + j) % R] = count[j].double()
        assert torch.equal(ga[j], want_a.to(F32).to(BF16)) and torch.equal(gb[j], want_b.to(F32).to(BF16)), j
