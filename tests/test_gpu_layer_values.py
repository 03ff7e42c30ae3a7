"""The layer's operators at the edges of their number formats, against the definitions in
64 bits: infinite operands of the adapters, values next to the largest number, and rows
whose squares are too small or too large for fp32. What is finite is held to the tolerances of
test_gpu_layer.py; what is infinite or NaN by the definition has to be so."""
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from gpu_util import say
from test_gpu_layer import BF16, F32, F64, U, _adapters64, _adapters_grad64, _check_fp8, _dev, _gen, _near, _norm64

pytestmark = pytest.mark.gpu
INF = float("inf")


def _as_defined(got, want, tol, dtype, what):
    """Finite values by their tolerance, the others as they are."""
    got, finite = got.cpu(), want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: {int((got.isnan() != want.isnan()).sum())} of {got.numel()} wrongly NaN or not"
    inf = want.isinf()
    assert torch.equal(got[inf].double(), want[inf]), f"{what}: infinities"
    _near(got[finite], want[finite], tol.expand(want.shape)[finite], dtype, what)


def _positive(T, J, R, I, O, seed):
    """Positive values: every sum's sign is known, so an infinity comes out as one."""
    g = _gen(seed)
    pos = lambda *shape: (torch.rand(shape, generator=g) + 0.5).to(BF16)  # noqa: E731
    c = dict(x=pos(T, I), a=pos(J, R, I), b=pos(J, O, R), idx=torch.randint(J, (T,), generator=g), scale=torch.rand(J, generator=g) + 0.25,
             res=pos(T, O), grad=pos(T, O))
    c["idx"][T // 2], c["idx"][0] = -1, 0
    c["x"][0], c["x"][0, 0] = 0, 1  # hidden values that bf16 holds: their second part is 0
    c["grad"][0], c["grad"][0, 0] = 0, 1
    c["scale"][0] = 1
    return c


@pytest.mark.parametrize("T,J,R,I,O", [(1, 1, 8, 64, 40), (70, 3, 16, 136, 72), (100, 2, 40, 72, 128), (300, 3, 24, 136, 72), (520, 2, 136, 64, 64),
                                       (1100, 3, 8, 72, 136), (1500, 2, 64, 136, 72), (1100, 2, 72, 64, 136), (1200, 2, 200, 72, 72), (3300, 2, 16, 64, 72)])
def test_adapters_infinite_operands(T, J, R, I, O):
    """An infinity in b, a, x or grad_out: each is the other operand of values that go into
    a product in two parts, the second of them 0 or of the other sign."""
    say(f"adapters infinite operands T={T} J={J} R={R} I={I} O={O}")
    clean = _positive(T, J, R, I, O, T + R)
    if T == 1:
        clean["idx"][0] = 0
    hidden = _adapters64(clean, None)[0].to(F32)

    def forward(c):
        d = {k: _dev(v) for k, v in c.items()}
        out, h = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], residual=d["res"], return_hidden=True)
        h64, y64, th, ty = _adapters64(c, c["res"])
        _as_defined(h, h64, th, F32, "hidden")
        _as_defined(out, y64, ty, BF16, "out")
        return y64

    def backward(c):
        d = {k: _dev(v) for k, v in c.items()}
        got = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], _dev(hidden), scale=d["scale"])
        want, tol = _adapters_grad64(c, hidden)
        for name, v, w, t in zip(("grad_x", "grad_a", "grad_b"), got, want, tol):
            _as_defined(v, w, t, BF16, name)
        return want

    def with_infinity(name, at, value):
        c = dict(clean, **{name: clean[name].clone()})
        c[name][at] = value
        return c

    assert forward(with_infinity("b", (0, O - 1, R - 1), -INF)).isinf().any()
    both = with_infinity("b", (0, 3, 0), INF)
    both["b"][0, 3, R // 2] = -INF  # of both signs: NaN
    assert forward(both).isnan().any()
    assert backward(with_infinity("a", (0, R - 1, 5), INF))[0].isinf().any()
    if T > 1:
        t = int((clean["idx"] == 0).nonzero()[-1])
        assert backward(with_infinity("x", (t, I - 1), -INF))[1].isinf().any()
        assert backward(with_infinity("grad", (t, O // 2), INF))[2].isinf().any()


@pytest.mark.parametrize("T,R", [(3, 8), (70, 24), (300, 64), (1100, 8), (1300, 72), (3300, 16)])
def test_adapters_next_to_the_largest_number(T, R):
    """Scaled hidden values of 3.4e38, which bf16 would round to an infinity: the results,
    some 2^-10 of them and less, are finite."""
    say(f"adapters next to the largest number T={T} R={R}")
    J, I, O = 2, 72, 136
    g = _gen(T + R)
    small = lambda *shape: ((torch.rand(shape, generator=g) + 0.5) * 2.0 ** -30).to(BF16)  # noqa: E731
    c = dict(x=small(T, I), a=small(J, R, I), b=small(J, O, R), idx=torch.randint(J, (T,), generator=g),
             scale=torch.tensor([3.4e38, -3.4e38]), res=small(T, O), grad=small(T, O))
    c["x"][:, 0], c["a"][:, :, 0], c["b"][:, 0], c["grad"][:, 0] = 2.0 ** 10, 2.0 ** -10, 2.0 ** -10, 2.0 ** 10
    d = {k: _dev(v) for k, v in c.items()}
    out, hidden = cgd.adapter_linear(d["x"], d["a"], d["b"], d["idx"], scale=d["scale"], return_hidden=True)
    assert (hidden == 1).all()
    _, y64, _, ty = _adapters64(c, None)
    _near(out, y64, ty, BF16, "out")
    gx, ga, gb = cgd.adapter_linear_backward(d["grad"], d["x"], d["a"], d["b"], d["idx"], hidden, scale=d["scale"])
    want, tol = _adapters_grad64(c, hidden.cpu())
    _near(gx, want[0], tol[0], BF16, "grad_x")
    # (the first columns of x and grad are 2^10: their products are past the largest number)
    _near(ga[:, :, 1:], want[1][:, :, 1:], tol[1][:, :, 1:], BF16, "grad_a")
    _near(gb[:, 1:], want[2][:, 1:], tol[2][:, 1:], BF16, "grad_b")


FAINT = [(5, 64), (7, 200), (9, 256), (3, 512), (5, 1024), (4, 1032), (3, 7168), (600, 4096), (515, 8200), (3, 20480), (65600, 64)]


def _faint(T, H, scale, seed):
    """Rows of `scale`, one in three of ordinary size among them; -> x, residual, weight."""
    g = _gen(seed)
    x, r = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    size = torch.full((T, 1), scale)
    size[2::3] = 1
    return (x * size).to(BF16), (r * size).to(BF16), torch.rand(H, generator=g) + 0.5


@pytest.mark.parametrize("T,H", FAINT)
@pytest.mark.parametrize("scale", [1e-15, 1e-22, 1e-30, 2.0 ** -130])
def test_norm_of_rows_whose_squares_vanish(T, H, scale):
    """Without eps, or with one that is as small, a row's size does not matter."""
    say(f"norm of faint rows T={T} H={H} scale={scale}")
    x, r, w = _faint(T, H, scale, T + H)
    for eps in (0.0, 1e-40) if T < 10000 else (0.0,):
        eps64 = torch.tensor(eps, dtype=F32).to(F64).item()
        y = cgd.rms_norm(_dev(x), _dev(w), eps=eps)
        _, y64, _, ty = _norm64(x, None, w, eps64)
        _near(y, y64, ty, BF16, "y alone")
        fp8 = cgd.SCALE_F32 if H % 128 == 0 else None
        got, total = cgd.rms_norm(_dev(x), _dev(w), eps=eps, residual=_dev(r), cast_fp8=fp8, return_bf16=fp8 is not None)
        s64, y64, _, ty = _norm64(x, r, w, eps64)
        y, q = got if fp8 is not None else (got, None)
        _near(y, y64, ty, BF16, "y")
        assert torch.equal(total.cpu(), (x.float() + r.float()).to(BF16))
        if q:
            _check_fp8(*q, y64, ty, fp8)


def _check_norm_backward(x, gy, w, eps):
    T, H = x.shape
    gx, gw = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w), eps=eps)
    x, gy, w64 = x.to(F64), gy.to(F64), w.to(F64)
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    gwx = gy * w64 * x
    want = r * (gy * w64 - x * r * r * gwx.mean(1, keepdim=True))
    tol = (2 * H + 16) * U * r * ((gy * w64).abs() + x.abs() * r * r * gwx.abs().mean(1, keepdim=True))
    _near(gx, want, tol, BF16, "grad_x")
    _near(gw, (gy * x * r).sum(0), (T + H / 2 + 8) * U * (gy * x * r).abs().sum(0), F32, "grad_weight")


@pytest.mark.parametrize("T,H", FAINT)
def test_norm_of_rows_whose_squares_vanish_in_place(T, H):
    x, r, w = map(_dev, _faint(T, H, 1e-30, T - H))
    y, total = cgd.rms_norm(x, w, eps=0.0, residual=r)
    for over in (0, 1):
        terms = [x.clone(), r.clone()]
        y2, s2 = cgd.rms_norm(terms[0], w, eps=0.0, residual=terms[1], sum_out=terms[over])
        assert s2 is terms[over] and torch.equal(s2, total) and torch.equal(y2, y)


@pytest.mark.parametrize("T,H", FAINT)
@pytest.mark.parametrize("scale", [1e-15, 1e-22, 1e-30, 2.0 ** -130])
def test_norm_backward_of_rows_whose_squares_vanish(T, H, scale):
    say(f"norm backward of faint rows T={T} H={H} scale={scale}")
    x, _, w = _faint(T, H, scale, T * 3 + H)
    gy = (torch.randn(T, H, generator=_gen(1)) * 2.0 ** -20).to(BF16)  # (2^130 times 1 would be infinite)
    _check_norm_backward(x, gy, w, 0.0)


@pytest.mark.parametrize("T,H", FAINT)
@pytest.mark.parametrize("scale", [1e18, 1e30, 3e37])
def test_norm_backward_of_rows_whose_squares_overflow(T, H, scale):
    """Rows that the norm gives zeros for, and ordinary ones: grad_y of 2^100 makes the
    gradients large enough to see, and g x overflow as well."""
    say(f"norm backward of large rows T={T} H={H} scale={scale}")
    x, _, w = _faint(T, H, scale, T * 5 + H)
    x = x.clamp(-3e38, 3e38)
    gy = torch.randn(T, H, generator=_gen(2)).to(BF16)
    gy[::2] *= 2.0 ** 100
    _check_norm_backward(x, gy, w, 1e-6)


def test_norm_of_zeros_without_eps():
    """0 / 0."""
    x, w = torch.zeros(2, 256, dtype=BF16), torch.ones(256)
    x[1] = 1e-30
    y = cgd.rms_norm(_dev(x), _dev(w), eps=0.0)
    assert y[0].isnan().all() and (y[1] == 1).all()


@pytest.mark.parametrize("T,H", [(5, 64), (9, 256), (3, 512), (5, 1032), (600, 4096), (515, 8200), (3, 20480)])
def test_norm_backward_of_an_infinite_gradient(T, H):
    """It spoils its own row, and its own column of grad_weight, which is infinite. (That
    row's other terms are added to grad_weight behind those of the other rows: an fp32
    sum in another order, off by the same bound.)"""
    say(f"norm backward of an infinite gradient T={T} H={H}")
    g = _gen(T + H)
    x, gy, w = torch.randn(T, H, generator=g).to(BF16), torch.randn(T, H, generator=g).to(BF16), torch.rand(H, generator=g) + 0.5
    x[1, 3] = 1
    clean = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w))
    gy[1, 3] = INF
    size = x[:, 3:4].to(F64) ** 2
    gx, gw = cgd.rms_norm_backward(_dev(gy), _dev(x), _dev(w))
    rows, columns = torch.arange(T) != 1, torch.arange(H) != 3
    assert not gx[1].isfinite().any() and torch.equal(gx[rows], clean[0][rows])
    assert gw[3] == INF
    x, gy = x[:, columns].to(F64), gy[:, columns].to(F64)
    terms = gy * x / torch.sqrt(((x * x).sum(1, keepdim=True) + size) / H + 1e-6)
    _near(gw.cpu()[columns], terms.sum(0), (T + H / 2 + 8) * U * terms.abs().sum(0), F32, "grad_weight")
