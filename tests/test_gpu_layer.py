"""The norm, the adapters, dropout and combine's gradient against plain computations in
64 bits.

Tolerances, derived before the first run (u = 2^-24, half a step of fp32; a result
is off by half a step of its type: bf16 2^-8, e4m3 2^-4 and 2^-10 of a scale below
its normal numbers):
  - an fp32 sum of n terms, in any order, is off by n u of the sum of their sizes;
  - the norm: s = x + residual by u (|x| + |residual|), the mean of squares by
    (n + 2) u of itself (its terms are positive), its root by half of that and 3 u
    more for the root and the division, and each product by u: y by (n / 2 + 8) u
    of itself and what s is off;
  - its gradient: with A = |g w| and B = |x| r^2 mean|g w x| the two terms before
    the factor r, (2 n + 16) u r (A + B) covers both sums, r^3 in the second and the
    products; grad_weight the same for sums over the rows;
  - adapters: h by I u |a||x|, as an operand by 2^-16 of itself (two bf16 parts:
    2^-8 of 2^-8), the second sum by (2 R + 4) u of its terms;
  - gradients of adapters: gh likewise, then sums over R (x) or the tokens (a, b);
  - combine: products by u, the sum over H by H u of its terms."""
import math

import numpy as np
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import DEV, say
from philox import kept

pytestmark = pytest.mark.gpu
BF16, F32, F64, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int64
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: U}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, dtype=F32) * scale).to(BF16)


def _dev(v):
    return None if v is None else v.to(DEV)


def _near(got, want, tol, dtype, what):
    got = got.to(F64).cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol + HALF[dtype] * (want.abs() + tol) + 2.0 ** -120)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {list(i)}: {got[i]} for "
                             f"{want[i]} +- {tol.expand(want.shape)[i]}")


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def _norm64(x, res, w, eps):
    """-> (s, y, tolerances of both)."""
    s = x.to(F64)
    ts = torch.zeros_like(s)
    if res is not None:
        ts = U * (s.abs() + res.to(F64).abs())
        s = s + res.to(F64)
    n = s.shape[-1]
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    y = s * r * w.to(F64)
    # the mean of squares moves with s, too: 2 |s| ts over s^2, at most 2 of the row's relative change
    shift = (s.abs() * ts).sum(-1, keepdim=True) / (s * s).sum(-1, keepdim=True).clamp_min(1e-300)
    return s, y, ts, y.abs() * ((n / 2 + 8) * U + shift) + ts * r * w.to(F64).abs()


WIDTHS = [(1, 8), (5, 16), (33, 128), (7, 136), (3, 256), (9, 264), (4, 512), (2, 520), (17, 1024), (5, 1032), (3, 2048),
          (2, 2056), (1, 4096), (513, 2304), (600, 4096), (1, 7168), (515, 7168), (2, 8192), (513, 8192), (3, 8200),
          (514, 10240), (2, 16384), (1, 16392), (513, 20480), (2, 32768)]


@pytest.mark.parametrize("T,H", WIDTHS)
@pytest.mark.parametrize("res,f32", [(False, False), (True, True), (True, False)])
def test_norm(T, H, res, f32):
    say(f"norm T={T} H={H} res={res} f32={f32}")
    g = _gen(T + H)
    x, r = _bf(g, T, H), _bf(g, T, H, scale=3.0) if res else None
    w = torch.randn(H, generator=g).to(F32 if f32 else BF16)
    got = cgd.rms_norm(_dev(x), _dev(w), eps=1e-5, residual=_dev(r))
    y, total = got if res else (got, None)
    s64, y64, ts, ty = _norm64(x, r, w, 1e-5)
    _near(y, y64, ty, BF16, "y")
    if res:
        _near(total, s64, ts, BF16, "sum")
    else:
        assert isinstance(got, torch.Tensor)


def _check_fp8(q, sc, y64, ty, fmt):
    H = y64.shape[-1]
    blocks = y64.view(-1, H // 128, 128)
    tb = ty.view(-1, H // 128, 128).amax(-1)
    amax = blocks.abs().amax(-1)
    want = amax.clamp_min(1e-4) / 448
    rel = tb / amax.clamp_min(1e-4) + 2 * U
    sc = sc.cpu().view(-1, H // 128)
    s = torch.exp2(sc.to(F64) - 127) if fmt == cgd.SCALE_UE8M0 else sc.to(F64)
    if fmt == cgd.SCALE_F32:
        assert ((s - want).abs() <= want * rel).all()
    else:  # the smallest power of two that is no less
        assert (torch.log2(s) == torch.log2(s).round()).all()
        assert (s >= want * (1 - rel)).all() and (s / 2 < want * (1 + rel)).all()
    v = q.cpu().to(F32).to(F64).view(-1, H // 128, 128)
    tol = 2.0 ** -4 * blocks.abs() + 2.0 ** -10 * s[..., None] + tb[..., None] * 2
    assert v.abs().max() <= 448
    assert ((v * s[..., None] - blocks).abs() <= tol).all()


@pytest.mark.parametrize("T,H", [(1, 128), (9, 256), (3, 384), (5, 640), (2, 1152), (1, 4096), (520, 4096), (3, 7168),
                                 (514, 7168), (2, 16384), (1, 32768)])
@pytest.mark.parametrize("fmt", [cgd.SCALE_F32, cgd.SCALE_POW2, cgd.SCALE_UE8M0])
@pytest.mark.parametrize("res", [False, True])
def test_norm_fp8(T, H, fmt, res):
    say(f"norm fp8 T={T} H={H} fmt={fmt} res={res}")
    g = _gen(T * 3 + H)
    x, r = _bf(g, T, H), _bf(g, T, H) if res else None
    w = torch.rand(H, generator=g) + 0.5
    w[:64] *= 30
    w[128:256] = 0  # a block of zeros keeps a positive scale
    got = cgd.rms_norm(_dev(x), _dev(w), residual=_dev(r), cast_fp8=fmt, return_bf16=True)
    (y, (q, sc)), total = got if res else (got, None)
    s64, y64, ts, ty = _norm64(x, r, w, 1e-6)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (T, H) and sc.shape == (T, H // 128)
    assert sc.dtype == (torch.uint8 if fmt == cgd.SCALE_UE8M0 else F32)
    _near(y, y64, ty, BF16, "y")
    _check_fp8(q, sc, y64, ty, fmt)
    if res:
        _near(total, s64, ts, BF16, "sum")
    alone = cgd.rms_norm(_dev(x), _dev(w), residual=_dev(r), cast_fp8=fmt)
    q2, sc2 = alone[0] if res else alone
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)


def test_norm_shapes_and_in_place():
    g = _gen(4)
    x, r, w = _bf(g, 3, 5, 256), _bf(g, 3, 5, 256), torch.rand(256, generator=g)
    y, s = cgd.rms_norm(_dev(x), _dev(w), residual=_dev(r))
    assert y.shape == s.shape == (3, 5, 256)
    q, sc = cgd.rms_norm(_dev(x), _dev(w), cast_fp8=cgd.SCALE_F32)
    assert q.shape == (3, 5, 256) and sc.shape == (3, 5, 2)
    one = cgd.rms_norm(_dev(x)[0, 0], _dev(w))
    assert one.shape == (256,) and torch.equal(one, cgd.rms_norm(_dev(x), _dev(w))[0, 0])
    for H in (64, 256, 2048, 7168, 16384):  # the stream written over itself, or over the other term
        x, r, w = _dev(_bf(g, 600, H)), _dev(_bf(g, 600, H)), _dev(torch.rand(H, generator=g))
        y, s = cgd.rms_norm(x, w, residual=r)
        a = r.clone()
        y2, a2 = cgd.rms_norm(x, w, residual=a, sum_out=a)
        assert a2 is a and torch.equal(a, s) and torch.equal(y2, y)
        b = x.clone()
        y2, _ = cgd.rms_norm(b, w, residual=r, sum_out=b)
        assert torch.equal(b, s) and torch.equal(y2, y)


def test_norm_special_values():
    """A row that holds NaN or an infinity spoils itself alone; a row of zeros gives zeros."""
    g = _gen(9)
    for H in (128, 1024, 7168):
        x, w = _bf(g, 8, H), torch.rand(H, generator=g)
        x[2] = 0
        x[4, H // 2] = float("nan")
        x[6, 3] = float("inf")
        big = torch.full((1, H), 1e30, dtype=BF16, device=DEV)  # its squares are more than float32 holds
        assert (cgd.rms_norm(big, _dev(w)) == 0).all()
        y = cgd.rms_norm(_dev(x), _dev(w)).cpu()
        _, y64, _, ty = _norm64(x, None, w, 1e-6)
        ok = [0, 1, 2, 3, 5, 7]
        _near(y[ok], y64[ok], ty[ok], BF16, "rows")
        assert (y[2] == 0).all() and y[4].isnan().all() and y[6, 3].isnan()
        gr = _bf(g, 8, H)
        dx, _ = cgd.rms_norm_backward(_dev(gr), _dev(x), _dev(w))
        dx = dx.cpu()
        assert dx[ok].isfinite().all() and dx[4].isnan().all()


@pytest.mark.parametrize("T,H", WIDTHS + [(2000, 64), (3000, 128), (1100, 512), (5000, 1024)])
@pytest.mark.parametrize("extra,f32", [(False, False), (True, True)])
def test_norm_backward(T, H, extra, f32):
    say(f"norm backward T={T} H={H} extra={extra} f32={f32}")
    g = _gen(T * 5 + H)
    x, gy = _bf(g, T, H), _bf(g, T, H)
    gs = _bf(g, T, H) if extra else None
    w = torch.randn(H, generator=g).to(F32 if f32 else BF16)
    gx, gw = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w), eps=1e-5, grad_sum=_dev(gs))
    again = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w), eps=1e-5, grad_sum=_dev(gs))
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1]) and gw.dtype == w.dtype
    x, gy, w64 = x.to(F64), gy.to(F64), w.to(F64)
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5)
    gwx = gy * w64 * x
    want = r * (gy * w64 - x * r * r * gwx.mean(1, keepdim=True))
    tol = (2 * H + 16) * U * r * ((gy * w64).abs() + x.abs() * r * r * gwx.abs().mean(1, keepdim=True))
    if extra:
        want = want + gs.to(F64)
        tol = tol + 2 * U * (want.abs() + gs.to(F64).abs())
    _near(gx, want, tol, BF16, "grad_x")
    _near(gw, (gy * x * r).sum(0), (T + H / 2 + 8) * U * (gy * x * r).abs().sum(0), w.dtype, "grad_weight")


@pytest.mark.parametrize("H", [64, 520, 2304])
def test_norm_gradient_against_differences(H):
    """Along one direction, by central differences in 64 bits."""
    g = _gen(H)
    x, gy, w = _bf(g, 6, H), _bf(g, 6, H), torch.rand(H, generator=g) + 0.5
    gx, gw = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w))
    d, e = torch.randn(6, H, generator=g, dtype=F64), torch.randn(H, generator=g, dtype=F64)

    def value(h):
        return (_norm64(x.to(F64) + h * d, None, w.to(F64) + h * e, 1e-6)[1] * gy.to(F64)).sum()
    want = (value(1e-4) - value(-1e-4)) / 2e-4
    got = (gx.cpu().to(F64) * d).sum() + (gw.cpu().to(F64) * e).sum()
    size = (gx.cpu().to(F64) * d).abs().sum() + (gw.cpu().to(F64) * e).abs().sum()
    assert (got - want).abs() <= (2.0 ** -8 + 1e-5) * size


# ---------------------------------------------------------------------------
# Adapters
# ---------------------------------------------------------------------------

def _case(T, J, R, I, O, none, runs, seed, scaled=True):
    g = _gen(seed)
    n = runs or T
    idx = torch.randint(J, (n,), generator=g)
    idx[torch.rand(n, generator=g) < none] = -1
    if runs:
        edge = torch.sort(torch.randint(T + 1, (runs - 1,), generator=g))[0]
        idx = idx[torch.bucketize(torch.arange(T), edge, right=True)]
    return dict(x=_bf(g, T, I), a=_bf(g, J, R, I, scale=1 / math.sqrt(I)), b=_bf(g, J, O, R, scale=1 / math.sqrt(R)), idx=idx,
                scale=torch.rand(J, generator=g) + 0.25 if scaled else None, res=_bf(g, T, O), grad=_bf(g, T, O))


def _adapters64(c, res):
    """-> (hidden, out, tolerances of both)."""
    T, I = c["x"].shape
    J, O, R = c["b"].shape
    h, th = torch.zeros(T, R, dtype=F64), torch.zeros(T, R, dtype=F64)
    y = torch.zeros(T, O, dtype=F64) if res is None else res.to(F64).clone()
    ty = 2 * U * y.abs()
    for j in range(J):
        t = (c["idx"] == j).nonzero()[:, 0]
        if not len(t):
            continue
        x, a, b = c["x"][t].to(F64), c["a"][j].to(F64), c["b"][j].to(F64)
        k = 1.0 if c["scale"] is None else float(c["scale"][j])
        h[t], th[t] = x @ a.T, I * U * (x.abs() @ a.abs().T)
        d, size = k * h[t] @ b.T, k * h[t].abs() @ b.abs().T
        y[t] += d
        ty[t] += k * (th[t] + h[t].abs() * (2.0 ** -16 + 2 * U)) @ b.abs().T + (2 * R + 4) * U * size
    return h, y, th, ty


SHAPES = [  # T, J, R, I, O, none, runs
    (1, 1, 8, 8, 1, 0.0, 0), (1, 5, 64, 4096, 7168, 0.0, 0), (2, 3, 16, 72, 24, 0.0, 0), (16, 1, 8, 264, 130, 0.0, 0),
    (17, 4, 24, 320, 63, 0.3, 0), (31, 2, 16, 1000, 257, 0.0, 1), (64, 64, 32, 512, 512, 0.1, 0),
    (128, 32, 16, 7168, 256, 0.1, 0), (100, 512, 8, 128, 96, 0.0, 0), (130, 3, 40, 640, 320, 0.5, 7),
    (255, 20, 24, 136, 264, 0.2, 0), (256, 300, 16, 264, 72, 0.1, 0), (256, 2, 32, 128, 128, 0.0, 2), (257, 9, 8, 72, 136, 0.1, 0),
    (1023, 3, 16, 136, 64, 0.1, 8), (1024, 40, 32, 64, 200, 0.0, 0), (300, 8, 64, 1032, 515, 0.1, 9), (513, 2, 128, 264, 264, 0.0, 3), (600, 5, 72, 136, 1003, 0.2, 0),
    (1030, 7, 16, 2304, 136, 0.1, 0), (1500, 1, 256, 256, 300, 0.0, 1), (2100, 16, 32, 200, 520, 0.05, 30),
    (2500, 3, 136, 328, 72, 0.1, 5), (4093, 8, 64, 448, 264, 0.1, 24),
    # many tokens: their order by chunks
    (8193, 40, 8, 16, 24, 0.1, 0), (16384, 3, 8, 72, 24, 0.1, 0), (16385, 512, 8, 24, 16, 0.1, 0), (20000, 1, 8, 64, 8, 0.3, 0),
    (33000, 512, 16, 16, 8, 0.9, 40), (70001, 64, 16, 24, 40, 0.05, 500), (300000, 2, 8, 8, 8, 0.5, 0)]


@pytest.mark.parametrize("T,J,R,I,O,none,runs", SHAPES)
@pytest.mark.parametrize("res,scaled", [(False, True), (True, False)])
def test_adapters(T, J, R, I, O, none, runs, res, scaled):
    say(f"adapters T={T} J={J} R={R} I={I} O={O} none={none} runs={runs} res={res} scaled={scaled}")
    c = _case(T, J, R, I, O, none, runs, T + J + R + I + O, scaled)
    d = {k: _dev(v) for k, v in c.items()}
    r = c["res"] if res else None
    out, hidden = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=_dev(r), return_hidden=True)
    alone = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=_dev(r))
    torch.cuda.synchronize()
    h, y, th, ty = _adapters64(c, r)
    assert out.dtype == BF16 and hidden.dtype == F32
    _near(hidden, h, th, F32, "hidden")
    _near(out, y, ty, BF16, "out")
    assert torch.equal(out, alone)
    if res:  # over the residual itself
        over = d["res"].clone()
        cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=over, out=over)
        assert torch.equal(over, out)


def _adapters_grad64(c, hidden):
    T, I = c["x"].shape
    J, O, R = c["b"].shape
    gx, tx = torch.zeros(T, I, dtype=F64), torch.zeros(T, I, dtype=F64)
    ga, ta = torch.zeros(J, R, I, dtype=F64), torch.zeros(J, R, I, dtype=F64)
    gb, tb = torch.zeros(J, O, R, dtype=F64), torch.zeros(J, O, R, dtype=F64)
    for j in range(J):
        t = (c["idx"] == j).nonzero()[:, 0]
        if not len(t):
            continue
        x, a, b, g = c["x"][t].to(F64), c["a"][j].to(F64), c["b"][j].to(F64), c["grad"][t].to(F64)
        k = 1.0 if c["scale"] is None else float(c["scale"][j])
        gh = k * g @ b
        th = k * (O + 2) * U * (g.abs() @ b.abs()) + 2.0 ** -16 * gh.abs()  # as an operand
        h = k * hidden[t].to(F64)
        n = len(t)
        gx[t], tx[t] = gh @ a, th @ a.abs() + (2 * R + 4) * U * gh.abs() @ a.abs()
        ga[j], ta[j] = gh.T @ x, th.T @ x.abs() + (2 * n + 4) * U * gh.abs().T @ x.abs()
        gb[j], tb[j] = g.T @ h, (2.0 ** -16 + (2 * n + 4) * U) * g.abs().T @ h.abs()
    return (gx, ga, gb), (tx, ta, tb)


@pytest.mark.parametrize("T,J,R,I,O,none,runs", [s for s in SHAPES if s[4] % 8 == 0] +
                         [(1, 1, 8, 8, 8, 0.0, 0), (40, 3, 16, 136, 264, 1.0, 0), (33, 2, 8, 64, 72, 0.0, 1),
                          (700, 2, 64, 264, 136, 0.0, 2), (1025, 1, 16, 128, 128, 0.0, 1),
                          # the tokens of few adapters in shares
                          (1535, 1, 16, 128, 64, 0.0, 1), (1536, 1, 24, 136, 72, 0.2, 0), (3100, 2, 40, 264, 136, 0.1, 0),
                          (4000, 2, 16, 72, 8, 1.0, 0), (5000, 3, 8, 24, 264, 0.0, 2)])
@pytest.mark.parametrize("scaled", [True, False])
def test_adapters_backward(T, J, R, I, O, none, runs, scaled):
    say(f"adapters backward T={T} J={J} R={R} I={I} O={O} none={none} runs={runs} scaled={scaled}")
    c = _case(T, J, R, I, O, none, runs, T * 2 + J + R + I + O, scaled)
    hidden = _adapters64(c, None)[0].to(F32)
    hidden[c["idx"] < 0] = float("nan")  # nobody reads the rows of tokens without an adapter
    d = {k: _dev(v) for k, v in c.items()}
    call = lambda: cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], _dev(hidden), scale=d["scale"])  # noqa: E731
    got, again = call(), call()
    torch.cuda.synchronize()
    want, tol = _adapters_grad64(c, hidden)
    for name, a, b, t, e in zip(("grad_x", "grad_a", "grad_b"), got, want, tol, again):
        _near(a, b, t, BF16, name)
        assert torch.equal(a, e), name


def test_adapter_gradients_against_differences():
    c = _case(37, 3, 16, 64, 48, 0.2, 0, 5)
    d = {k: _dev(v) for k, v in c.items()}
    _, hidden = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], return_hidden=True)
    got = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    g = _gen(6)
    way = [torch.randn(c[k].shape, generator=g, dtype=F64) for k in ("x", "a", "b")]

    def value(h):
        m = dict(c, **{k: c[k].to(F64) + h * w for k, w in zip(("x", "a", "b"), way)})
        return (_adapters64(m, None)[1] * c["grad"].to(F64)).sum()
    want = (value(1e-4) - value(-1e-4)) / 2e-4
    parts = [(a.cpu().to(F64) * w) for a, w in zip(got, way)]
    assert (sum(p.sum() for p in parts) - want).abs() <= (2.0 ** -8 + 1e-5) * sum(p.abs().sum() for p in parts)


def test_adapters_special_values():
    """NaN and infinities in one token, in an adapter that no token has, and in a
    token without an adapter stay where they are."""
    c = _case(70, 4, 16, 128, 96, 0.0, 0, 11)
    c["idx"][c["idx"] == 2] = 1
    c["idx"][5], c["idx"][6], c["idx"][7] = -1, 0, 4  # 4: no adapter
    c["idx"][8], c["idx"][9] = -(1 << 40), 1 << 40
    c["a"][2], c["b"][2] = float("nan"), float("inf")
    c["x"][5], c["x"][6, 3] = float("nan"), float("inf")
    d = {k: _dev(v) for k, v in c.items()}
    out = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=d["res"]).cpu()
    clean = dict(c, x=c["x"].clone())
    clean["x"][6] = 0
    _, y, _, ty = _adapters64(clean, c["res"])
    keep = [i for i in range(70) if i != 6]
    _near(out[keep], y[keep], ty[keep], BF16, "others")
    assert not out[6].isfinite().any()
    for i in (5, 7, 8, 9):
        assert torch.equal(out[i], c["res"][i])
    c["x"][6] = 1
    hidden = _adapters64(dict(c, x=clean["x"]), None)[0].to(F32)
    d["x"] = _dev(c["x"])
    gx, ga, gb = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], _dev(hidden), scale=d["scale"])
    assert (gx[[5, 7, 8, 9]] == 0).all() and (ga[2] == 0).all() and (gb[2] == 0).all()
    assert gx.isfinite().all() and ga.isfinite().all() and gb.isfinite().all()


@pytest.mark.parametrize("T,R", [(5, 8), (5, 40), (100, 16), (300, 24), (1100, 8), (1100, 72), (4000, 8)])
def test_adapters_infinite_scale(T, R):
    """Of positive values an infinite scale makes infinities and no NaN: what a tile is
    padded with does not meet it. An adapter without tokens has zero gradients all the same."""
    g = _gen(12)
    pos = lambda *shape: _dev((torch.rand(shape, generator=g) + 0.5).to(BF16))
    x, a, b, grad, res = pos(T, 136), pos(3, R, 136), pos(3, 72, R), pos(T, 72), pos(T, 72)
    idx = torch.randint(2, (T,), generator=g)
    idx[0] = 0
    idx[3] = -1
    idx, inf = _dev(idx), float("inf")
    runs = []
    for scale in ([inf, 0.5, inf], [1.0, 0.5, 1.0]):
        scale = torch.tensor(scale, device=DEV)
        out, hidden = cgd.adapter_linear(x, a, b, idx, scale=scale, residual=res, return_hidden=True)
        runs.append((out, hidden, *cgd.adapter_linear_backward(grad, x, a, b, idx, hidden, scale=scale)))
    (out, hidden, gx, ga, gb), (out1, hidden1, gx1, ga1, gb1) = runs
    first = idx == 0
    assert torch.equal(hidden, hidden1) and hidden.isfinite().all()
    assert (out[first] == inf).all() and torch.equal(out[~first], out1[~first])
    assert (gx[first] == inf).all() and torch.equal(gx[~first], gx1[~first])
    assert (ga[0] == inf).all() and torch.equal(ga[1:], ga1[1:])
    assert (gb[0] == inf).all() and torch.equal(gb[1:], gb1[1:])


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 7, 8, 9, 100, 4096, 4097, 777 * 1003, 1 << 20])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99, 1.0])
@pytest.mark.parametrize("res", [False, True])
def test_dropout(n, p, res):
    say(f"dropout n={n} p={p} res={res}")
    g = _gen(n)
    x, r = _bf(g, n), _bf(g, n) if res else None
    seed, offset = (n * 0x9E3779B97F4A7C15 + 3) % 2 ** 64, (n << 31) + 17
    got = cgd.dropout(_dev(x), p, seed, offset=offset, residual=_dev(r))
    limit = round(p * 65536)
    keep = torch.from_numpy(kept(n, seed, offset, limit))
    y = torch.where(keep, x.to(F64) * (65536 / max(1, 65536 - limit)), 0.0)
    tol = 3 * U * y.abs()
    if res:
        y = y + r.to(F64)
        tol = tol + U * (y.abs() + r.to(F64).abs())
    _near(got, y, tol, BF16, "dropout")
    if p == 0.0 and not res:
        assert torch.equal(got.cpu(), x)
    if not res:  # the gradient drops the same elements, and the state's numbers are added to the others
        ones = torch.ones(n, dtype=BF16, device=DEV)
        assert torch.equal(cgd.dropout_backward(ones, p, seed, offset=offset).cpu() != 0, keep)
        signed = (seed + 2 ** 63) % 2 ** 64 - 2 ** 63
        state = torch.tensor([signed, offset - 5], device=DEV)
        assert torch.equal(cgd.dropout(_dev(x), p, state, offset=5), got)


def test_dropout_in_place_and_special_values():
    g = _gen(3)
    x = _bf(g, 5, 333)
    x[0, ::2], x[1, ::2], x[2, ::2] = float("nan"), float("inf"), -float("inf")
    r = _bf(g, 5, 333)
    out = cgd.dropout(_dev(x), 0.5, 42, residual=_dev(r))
    keep = torch.from_numpy(kept(5 * 333, 42, 0, 32768)).view(5, 333)
    assert torch.equal(out.cpu()[~keep], r[~keep])
    for over in ("x", "r"):
        a, b = _dev(x).clone(), _dev(r).clone()
        res = cgd.dropout(a, 0.5, 42, residual=b, out=a if over == "x" else b)
        assert torch.equal(res.nan_to_num(7.0), out.nan_to_num(7.0)) and res is (a if over == "x" else b)
    a = torch.empty(0, 64, dtype=BF16, device=DEV)
    assert cgd.dropout(a, 0.5, 1).shape == (0, 64)


# ---------------------------------------------------------------------------
# Combine's gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,K,H,align,none", [(1, 1, 1, 8, 1, 0.0), (3, 8, 2, 64, 4, 0.0), (129, 256, 8, 7168, 1, 0.0),
                                                (127, 512, 16, 4096, 1, 0.1), (300, 20, 5, 520, 8, 0.3), (17, 16, 3, 2056, 1, 1.0),
                                                (64, 4, 3, 16384, 1, 0.0), (2000, 32, 4, 128, 16, 0.05)])
def test_combine_backward(T, E, K, H, align, none):
    say(f"combine backward T={T} E={E} K={K} H={H} align={align} none={none}")
    g = _gen(T + E + K + H)
    idx = torch.rand(T, E, generator=g).topk(K, 1)[1]
    idx[torch.rand(T, K, generator=g) < none] = -1
    x = _bf(g, T, H)
    recv, _, handle = cgd.dispatch(_dev(x), _dev(idx), E, 1, expert_alignment=align)
    y = _bf(g, recv.shape[0], H)
    dst = handle.dst_row.cpu().long()
    used = dst >= 0
    assert torch.equal(used, idx >= 0)
    rows = torch.zeros(recv.shape[0], dtype=torch.bool)
    rows[dst[used]] = True
    y[~rows] = float("nan")  # nobody reads them
    w, grad = torch.randn(T, K, generator=g), _bf(g, T, H)
    out = torch.full((recv.shape[0], H), 5.0, dtype=BF16, device=DEV)
    gy, gw = cgd.combine_backward(_dev(grad), _dev(y), handle, _dev(w), out=out)
    assert gy is out
    _, gw2 = cgd.combine_backward(_dev(grad), _dev(y), handle, _dev(w))
    assert torch.equal(gw, gw2)
    gy = gy.cpu()
    assert (gy[~rows] == 5).all()
    terms = torch.where(used[..., None], grad.to(F64)[:, None, :] * y.to(F64)[dst.clamp_min(0)], 0.0)
    _near(gw, terms.sum(-1), (H + 2) * U * terms.abs().sum(-1), F32, "grad_topk_weights")
    t, k = used.nonzero(as_tuple=True)
    want = w[t, k].to(F64)[:, None] * grad[t].to(F64)
    _near(gy[dst[t, k]], want, U * want.abs(), BF16, "grad_expert_out")


def test_combine_backward_packed_and_cut():
    """The packed layout with slots that found no room; rows behind a cut receive buffer."""
    g = _gen(8)
    T, E, K, H, cap = 90, 8, 3, 256, 20
    idx = torch.rand(T, E, generator=g).topk(K, 1)[1]
    x, grad, w = _bf(g, T, H), _bf(g, T, H), torch.randn(T, K, generator=g)
    _, counts, handle = cgd.low_latency_dispatch(_dev(x), _dev(idx), E, 1, expert_capacity=cap)
    dst = handle.dst_row.cpu().long()
    assert (dst < 0).any()
    y = _bf(g, E, cap, H)
    gy, gw = cgd.combine_backward(_dev(grad), _dev(y), handle, _dev(w))
    assert gy.shape == (E, cap, H)
    t, k = (dst >= 0).nonzero(as_tuple=True)
    want = w[t, k].to(F64)[:, None] * grad[t].to(F64)
    _near(gy.view(-1, H).cpu()[dst[t, k]], want, U * want.abs(), BF16, "grad_expert_out")
    terms = torch.where((dst >= 0)[..., None], grad.to(F64)[:, None, :] * y.view(-1, H).to(F64)[dst.clamp_min(0)], 0.0)
    _near(gw, terms.sum(-1), (H + 2) * U * terms.abs().sum(-1), F32, "grad_topk_weights")
    # as combine: a slot whose row the buffer does not have is no slot
    recv, _, h = cgd.dispatch(_dev(x), _dev(idx), E, 1)
    y = _bf(g, 100, H)
    gy, gw = cgd.combine_backward(_dev(grad), _dev(y), h, _dev(w))
    dst = h.dst_row.cpu().long()
    assert (gw.cpu()[dst >= 100] == 0).all() and (gw.cpu()[dst < 100] != 0).all()
