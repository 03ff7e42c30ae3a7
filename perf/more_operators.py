"""Cases for measuring the operators that a layer needs beside its router, moves and
products: the root-mean-square norm with the residual's addition (and the FP8
payload as its output), low-rank adapters of many requests beside a shared
projection, dropout whose mask is never stored, and the gradient of combine.

`run` computes a case in plain torch operations, or with `own` set through the
package's entry points. Sizes are those of the repository's workloads (hidden 7168
and 4096, top-8 of 256 experts, 128 and 4096 tokens)."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's norm between two layers of a decode step: latency
        dict(name="norm_token", op="norm", T=1, H=4096, residual=True, out="bf16", wide=False),
        # ahead of a prefill batch's layer: bf16 for the gate, FP8 for dispatch, the residual stream updated
        dict(name="norm_prefill_fp8", op="norm", T=4096, H=7168, residual=True, out="both", wide=False),
        # the norm of each head's query: many short rows, fp32 weights
        dict(name="norm_heads", op="norm", T=131040, H=128, residual=False, out="bf16", wide=True),
        # training: the norm's gradient, with the one that comes down the residual stream
        dict(name="norm_grad", op="norm_grad", T=4095, H=7168, residual=True, wide=False),
        # one request alone, adapters of a large rank
        dict(name="adapters_token", op="adapters", T=1, J=8, R=64, I=4096, O=7168, requests=0, none=0.0, scaled=True,
             residual=True, shared=False),
        # a decode batch: every token another request's, some without an adapter, beside the shared projection
        dict(name="adapters_decode", op="adapters", T=128, J=32, R=16, I=7168, O=4096, requests=0, none=0.1,
             scaled=True, residual=False, shared=True),
        # a prefill batch of 24 requests, an odd number of tokens
        dict(name="adapters_prefill", op="adapters", T=4093, J=8, R=64, I=7168, O=4096, requests=24, none=0.1,
             scaled=True, residual=True, shared=False),
        # training 16 adapters at once
        dict(name="adapters_grad", op="adapters_grad", T=4095, J=16, R=16, I=4096, O=7168, requests=40, none=0.05,
             scaled=True),
        # the layer's output on its way to the residual stream in training
        dict(name="dropout_residual", op="dropout", T=4096, H=7168, p=0.1, residual=True, grad=False),
        # the gradient at an adapter's input, odd sizes
        dict(name="dropout_grad_odd", op="dropout", T=777, H=1003, p=0.25, residual=False, grad=True),
        # the gradient of a prefill batch's combine
        dict(name="combine_grad", op="combine_grad", T=4096, E=256, K=8, H=7168, masked=0.0),
        # a small step, top-16, some slots not selected
        dict(name="combine_grad_masked", op="combine_grad", T=127, E=512, K=16, H=4096, masked=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log_int(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "adapters", "adapters", "adapters_grad", "dropout", "combine_grad"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8", "both"])
        H = _mult(rng, 64, 16384, 8 if out == "bf16" else 128)
        return dict(op=op, T=_log_int(rng, 1, min(200000, 29000000 // H)), H=H, residual=rng.random() < 0.6, out=out,
                    wide=rng.random() < 0.5)
    if op == "norm_grad":
        H = _mult(rng, 64, 16384, 8)
        return dict(op=op, T=_log_int(rng, 1, min(200000, 29000000 // H)), H=H, residual=rng.random() < 0.6,
                    wide=rng.random() < 0.5)
    if op == "adapters":
        shared = rng.random() < 0.3
        c = dict(op=op, T=_log_int(rng, 1, 1024 if shared else 4096), J=_log_int(rng, 1, 64), R=rng.choice([8, 16, 32, 64, 128]),
                 I=_mult(rng, 64, 7168, 8), O=_log_int(rng, 16, 4096), none=rng.choice([0.0, 0.1, 0.9]),
                 scaled=rng.random() < 0.7, residual=not shared and rng.random() < 0.5, shared=shared)
        return dict(c, requests=rng.choice([0, 1, _log_int(rng, 1, 64)]))
    if op == "adapters_grad":
        return dict(op=op, T=_log_int(rng, 1, 4096), J=_log_int(rng, 1, 32), R=rng.choice([8, 16, 32, 64]),
                    I=_mult(rng, 64, 4096, 8), O=_mult(rng, 64, 4096, 8), requests=rng.choice([0, 1, _log_int(rng, 1, 64)]),
                    none=rng.choice([0.0, 0.1]), scaled=rng.random() < 0.7)
    if op == "dropout":
        H = _log_int(rng, 1, 16384)
        return dict(op=op, T=_log_int(rng, 1, min(100000, 29000000 // H)), H=H, p=rng.choice([0.0, 0.05, 0.1, 0.5, 0.9]),
                    residual=rng.random() < 0.5, grad=False)
    E = rng.choice([1, 8, 64, 256, 512])
    K = rng.randint(1, min(16, E))
    H = _mult(rng, 64, 7168, 8)
    return dict(op=op, T=_log_int(rng, 1, min(32768, 230000000 // (K * H))), E=E, K=K, H=H, masked=rng.choice([0.0, 0.1]))


def work(case):
    op = case["op"]
    T = case["T"]
    if op in ("norm", "norm_grad"):
        n, w = T * case["H"], case["H"] * (4 if case["wide"] else 2)
        if op == "norm_grad":
            return {"bytes": n * (8 if case["residual"] else 6) + 2 * w, "flops": 10 * n}
        out = {"bf16": 2.0, "fp8": 1 + 4 / 128, "both": 3 + 4 / 128}[case["out"]]
        return {"bytes": n * ((6 if case["residual"] else 2) + out) + w, "flops": 5 * n}
    if op == "dropout":
        return {"bytes": T * case["H"] * (6 if case["residual"] else 4), "flops": 4 * T * case["H"]}
    if op == "combine_grad":
        K, H = case["K"], case["H"]
        rows = T * K * (1 - case["masked"])
        return {"bytes": T * H * 2 + rows * H * 4 + T * K * 12, "flops": 3 * rows * H}
    I, O, R = case["I"], case["O"], case["R"]
    used = case["J"] * (1 - (1 - 1 / case["J"]) ** (case["requests"] or T))  # adapters that some token has
    rows = T * (1 - case["none"])
    if op == "adapters_grad":
        b = T * (2 * I + 2 * I + 2 * O + 4 * R + 8) + used * R * (I + O) * 2 + case["J"] * R * (I + O) * 2
        return {"bytes": b, "flops": 4 * rows * R * (I + O)}
    b = T * (2 * I + 2 * O + 8 + (2 * O if case["residual"] else 0)) + used * R * (I + O) * 2
    f = 2 * rows * R * (I + O)
    if case["shared"]:
        b, f = b + I * O * 2, f + 2 * T * I * O
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=BF16, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(scale)


def _adapter_of(g, case):
    """The adapter of each token: of `requests` runs of tokens, or (0) of each token by itself."""
    T, n = case["T"], case["requests"] or case["T"]
    j = torch.randint(case["J"], (n,), generator=g, device=DEV)
    j[torch.rand(n, generator=g, device=DEV) < case["none"]] = -1
    if not case["requests"]:
        return j
    share = torch.rand(n, generator=g, device=DEV, dtype=F64).add_(0.1)
    edge = torch.cumsum(share, 0) / share.sum() * T
    run = torch.searchsorted(edge, torch.arange(T, device=DEV, dtype=F64), right=True)
    return j[run.clamp_max(n - 1)]


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        H = case["H"]
        s["x"] = _randn(g, T, H)
        s["w"] = torch.rand(H, generator=g, device=DEV).add_(0.5).to(F32 if case["wide"] else BF16)
        if op == "norm":
            s["res"] = _randn(g, T, H, scale=2.0) if case["residual"] else None
        else:
            s["grad"] = _randn(g, T, H)
            s["gsum"] = _randn(g, T, H) if case["residual"] else None
        return s
    if op == "dropout":
        s["x"] = _randn(g, T, case["H"])
        s["res"] = _randn(g, T, case["H"]) if case["residual"] else None
        s["seed"], s["offset"] = seed * 7919 + 12345678901, seed % 977
        return s
    if op == "combine_grad":
        E, K, H = case["E"], case["K"], case["H"]
        idx = torch.rand(T, E, generator=g, device=DEV).topk(K, 1)[1]
        off = torch.rand(T, K, generator=g, device=DEV) < case["masked"]
        flat = idx.masked_fill(off, E).view(-1)  # a stable order by expert: the rows of the receive buffer
        order = torch.argsort(flat, stable=True)
        dst = torch.empty(T * K, dtype=torch.int32, device=DEV)
        dst[order] = torch.arange(T * K, dtype=torch.int32, device=DEV)
        s["dst"] = dst.view(T, K).masked_fill(off, -1)
        count = torch.bincount(flat, minlength=E + 1)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), count[:E].cumsum(0)]).to(torch.int32)
        s["counts"] = count[:E].to(torch.int32)
        s["src"] = torch.where(flat[order] < E, order // K, -1).to(torch.int32)
        s["grad"] = _randn(g, T, H)
        s["y"] = _randn(g, T * K, H)
        w = torch.rand(T, K, generator=g, device=DEV).add_(0.05)
        s["wts"] = (w / w.sum(1, keepdim=True)).masked_fill_(off, 0.0)
        s["out"] = torch.zeros(T * K, H, dtype=BF16, device=DEV)  # rows without data are left as they were
        return s
    J, R, I, O = case["J"], case["R"], case["I"], case["O"]
    s["idx"] = _adapter_of(g, case)
    s["x"] = _randn(g, T, I)
    s["a"] = _randn(g, J, R, I, scale=1 / math.sqrt(I))
    s["b"] = _randn(g, J, O, R, scale=1 / math.sqrt(R))
    s["scale"] = torch.rand(J, generator=g, device=DEV).add_(0.5) if case["scaled"] else None
    if op == "adapters_grad":
        s["grad"] = _randn(g, T, O)
        # the hidden values that the forward call gave: a x in fp32, nothing for a token without an adapter
        every = s["x"].to(F32) @ s["a"].to(F32).view(J * R, I).t()
        s["hidden"] = every.view(T, J, R)[torch.arange(T, device=DEV), s["idx"].clamp_min(0)]
        s["hidden"].masked_fill_((s["idx"] < 0)[:, None], 0.0)
        return s
    s["w"] = _randn(g, O, I, scale=1 / math.sqrt(I)) if case["shared"] else None
    s["res"] = _randn(g, T, O) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_norm(s):
    c = s["case"]
    v = s["x"].to(F32)
    if s["res"] is not None:
        v = v + s["res"].to(F32)
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["w"].to(F32)
    out = {}
    if c["out"] != "bf16":
        b = y.view(c["T"], c["H"] // 128, 128)
        amax = b.abs().amax(2).clamp_min(1e-4)
        out["codes"] = (b * (448.0 / amax)[:, :, None]).clamp(-448, 448).to(FP8).view(c["T"], c["H"])
        out["scales"] = amax / 448.0
    if c["out"] != "fp8":
        out["y"] = y.to(BF16)
    if s["res"] is not None:
        out["sum"] = v.to(BF16)
    return out


def _plain_norm_grad(s):
    v, g, w = s["x"].to(F32), s["grad"].to(F32), s["w"].to(F32)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    xh = v * r
    gw = g * w
    dx = (gw - xh * (gw * xh).mean(1, keepdim=True)) * r
    if s["gsum"] is not None:
        dx = dx + s["gsum"].to(F32)
    return dx.to(BF16), (g * xh).sum(0).to(s["w"].dtype)


def _words(n, seed, offset):
    """Philox4x32-10 of the counters (i, offset) for i < n under the key `seed`: [n, 4] words of 32 bits."""
    low = 0xFFFFFFFF
    i = torch.arange(n, device=DEV, dtype=torch.int64)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):  # a product of two 32-bit numbers keeps its 64 bits in an int64, sign or not
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (q >> 32 & low) ^ c1 ^ k0, q & low, (p >> 32 & low) ^ c3 ^ k1, p & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return torch.stack([c0, c1, c2, c3], 1)


def _plain_dropout(s):
    c = s["case"]
    n = s["x"].numel()
    w = _words(-(-n // 8), s["seed"], s["offset"])
    u = torch.stack([w & 0xFFFF, w >> 16], 2).view(-1)[:n].view(c["T"], c["H"])
    limit = round(c["p"] * 65536)
    y = torch.where(u >= limit, s["x"].to(F32) * (65536 / max(1, 65536 - limit)), 0.0)
    return (y if s["res"] is None else y + s["res"].to(F32)).to(BF16)


def _one_of(s):
    """[T, J * R]: 1 where a column belongs to the token's adapter, times the adapter's scale."""
    c = s["case"]
    at = (s["idx"][:, None] == torch.arange(c["J"], device=DEV)[None, :]).to(F32)
    scaled = at if s["scale"] is None else at * s["scale"][None, :]
    return at.repeat_interleave(c["R"], 1), scaled.repeat_interleave(c["R"], 1)


def _flat(s):
    """All adapters as one: a [J * R, I] and b [O, J * R]."""
    c = s["case"]
    n = c["J"] * c["R"]
    return s["a"].to(F32).view(n, c["I"]), s["b"].to(F32).transpose(0, 1).reshape(c["O"], n)


def _plain_adapters(s):
    a, b = _flat(s)
    x = s["x"].to(F32)
    y = (x @ a.t() * _one_of(s)[1]) @ b.t()
    if s["w"] is not None:
        y = x @ s["w"].to(F32).t() + y
    return (y if s["res"] is None else y + s["res"].to(F32)).to(BF16)


def _plain_adapters_grad(s):
    c = s["case"]
    a, b = _flat(s)
    x, g = s["x"].to(F32), s["grad"].to(F32)
    at, scaled = _one_of(s)
    gh = g @ b * scaled
    h = s["hidden"].repeat(1, c["J"]) * scaled
    da = (gh.t() @ x).view(c["J"], c["R"], c["I"])
    db = (g.t() @ h).view(c["O"], c["J"], c["R"]).transpose(0, 1)
    return (gh @ a).to(BF16), da.to(BF16), db.to(BF16).contiguous()


def _plain_combine_grad(s):
    g, dst = s["grad"].to(F32), s["dst"].long()
    used = dst >= 0
    rows = s["y"].to(F32)[dst.clamp_min(0)]
    dw = torch.where(used, (rows * g[:, None, :]).sum(2), 0.0)
    slot = torch.full((s["y"].shape[0] + 1,), -1, dtype=torch.int64, device=DEV)
    slot[torch.where(used, dst, s["y"].shape[0]).view(-1)] = torch.arange(dst.numel(), device=DEV)
    slot = slot[:-1]
    dy = g[(slot.clamp_min(0) // dst.shape[1])] * s["wts"].view(-1)[slot.clamp_min(0)][:, None]
    s["out"].copy_(torch.where((slot >= 0)[:, None], dy, s["out"]))
    return s["out"], dw


def _plain(s):
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dropout": _plain_dropout, "adapters": _plain_adapters,
            "adapters_grad": _plain_adapters_grad, "combine_grad": _plain_combine_grad}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import combine_get_dispatch_06_amd as cgd
    s, c = state, state["case"]
    op = c["op"]
    if op == "norm":
        fp8 = c["out"] != "bf16"
        r = cgd.rms_norm(s["x"], s["w"], eps=EPS, residual=s["res"], cast_fp8=cgd.SCALE_F32 if fp8 else None,
                         return_bf16=c["out"] == "both")
        y, total = (r, None) if s["res"] is None else r
        out = {} if total is None else {"sum": total}
        if c["out"] == "both":
            y, (out["codes"], out["scales"]) = y
        elif fp8:
            out["codes"], out["scales"] = y
        if c["out"] != "fp8":
            out["y"] = y
        return out
    if op == "norm_grad":
        return cgd.rms_norm_backward(s["grad"], s["x"], s["w"], eps=EPS, grad_sum=s["gsum"])
    if op == "dropout":
        if c["grad"]:
            return cgd.dropout_backward(s["x"], c["p"], s["seed"], offset=s["offset"])
        return cgd.dropout(s["x"], c["p"], s["seed"], offset=s["offset"], residual=s["res"])
    if op == "combine_grad":
        n = s["y"].shape[0]
        handle = cgd.DispatchHandle(s["offsets"], s["src"], s["dst"], s["counts"], c["E"], 1, 1, n)
        return cgd.combine_backward(s["grad"], s["y"], handle, s["wts"], out=s["out"])
    if op == "adapters_grad":
        return cgd.adapter_linear_backward(s["grad"], s["x"], s["a"], s["b"], s["idx"], s["hidden"], scale=s["scale"])
    delta = cgd.adapter_linear(s["x"], s["a"], s["b"], s["idx"], scale=s["scale"], residual=s["res"])
    return cgd.linear(s["x"], s["w"], residual=delta) if c["shared"] else delta


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(s):
    c = s["case"]
    v = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    n = torch.linalg.vector_norm(v, dim=1)
    y = s["w"].double()[None, :] * v / torch.sqrt(n * n / c["H"] + EPS)[:, None]
    out = {}
    if c["out"] != "bf16":
        top = torch.maximum(y.unflatten(1, (-1, 128)).abs().max(2)[0], torch.tensor(1e-4, dtype=F64, device=DEV))
        out["scales"] = top / 448
        out["codes"] = y / out["scales"].repeat_interleave(128, 1)
    if c["out"] != "fp8":
        out["y"] = y
    if s["res"] is not None:
        out["sum"] = v
    return out


def _exact_norm_grad(s):
    """The derivative of the formula itself."""
    with torch.enable_grad():
        v, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w
        dv, dw = torch.autograd.grad(y, (v, w), s["grad"].double())
    return dv if s["gsum"] is None else dv + s["gsum"].double(), dw


def _kept(n, seed, offset, limit):
    """Which of n elements stay, by the generator in unsigned 64-bit numbers on the host."""
    word = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    ctr = [np.arange(-(-n // 8), dtype=np.uint64)]
    ctr = [ctr[0] & word, ctr[0] >> half, np.full_like(ctr[0], offset & 0xFFFFFFFF), np.full_like(ctr[0], offset >> 32)]
    for r in range(10):
        key = [np.uint64(((seed & 0xFFFFFFFF) + r * 0x9E3779B9) % 2 ** 32),
               np.uint64(((seed >> 32 & 0xFFFFFFFF) + r * 0xBB67AE85) % 2 ** 32)]
        a, b = np.uint64(0xD2511F53) * ctr[0], np.uint64(0xCD9E8D57) * ctr[2]
        ctr = [(b >> half) ^ ctr[1] ^ key[0], b & word, (a >> half) ^ ctr[3] ^ key[1], a & word]
    out = np.empty((ctr[0].size, 8), dtype=np.int32)
    for i in range(4):
        out[:, 2 * i] = (ctr[i] & np.uint64(0xFFFF)).astype(np.int32)
        out[:, 2 * i + 1] = (ctr[i] >> np.uint64(16)).astype(np.int32)
    return torch.from_numpy(out.reshape(-1)[:n] >= limit).to(DEV)


def _exact_dropout(s):
    c = s["case"]
    limit = int(math.floor(c["p"] * 65536 + 0.5))
    keep = _kept(c["T"] * c["H"], s["seed"], s["offset"], limit).view(c["T"], c["H"])
    y = torch.zeros(c["T"], c["H"], dtype=F64, device=DEV)
    y[keep] = s["x"].double()[keep] / (1 - limit / 65536)
    return y if s["res"] is None else y + s["res"].double()


def _exact_adapters(s):
    """Adapter by adapter."""
    c = s["case"]
    y = torch.zeros(c["T"], c["O"], dtype=F64, device=DEV)
    if s["w"] is not None:
        y += torch.matmul(s["x"].double(), s["w"].double().t())
    if s["res"] is not None:
        y += s["res"].double()
    for j in range(c["J"]):
        t = (s["idx"] == j).nonzero()[:, 0]
        k = 1.0 if s["scale"] is None else s["scale"][j].double()
        y[t] += k * torch.matmul(torch.matmul(s["x"][t].double(), s["a"][j].double().t()), s["b"][j].double().t())
    return y


def _exact_adapters_grad(s):
    c = s["case"]
    dx = torch.zeros(c["T"], c["I"], dtype=F64, device=DEV)
    da, db = torch.zeros(s["a"].shape, dtype=F64, device=DEV), torch.zeros(s["b"].shape, dtype=F64, device=DEV)
    for j in range(c["J"]):
        t = (s["idx"] == j).nonzero()[:, 0]
        k = 1.0 if s["scale"] is None else s["scale"][j].double()
        g, a = k * s["grad"][t].double(), s["a"][j].double()
        gh = torch.matmul(g, s["b"][j].double())
        dx[t] = torch.matmul(gh, a)
        da[j] = torch.matmul(gh.t(), s["x"][t].double())
        db[j] = torch.matmul(g.t(), s["hidden"][t].double())
    return dx, da, db


def _exact_combine_grad(s):
    """Slot by slot."""
    dy = s["out"].double()
    dw = torch.zeros(s["wts"].shape, dtype=F64, device=DEV)
    for k in range(s["case"]["K"]):
        t = (s["dst"][:, k] >= 0).nonzero()[:, 0]
        r = s["dst"][t, k].long()
        g = s["grad"][t].double()
        dw[t, k] = torch.linalg.vecdot(g, s["y"][r].double())
        dy[r] = s["wts"][t, k].double()[:, None] * g
    return dy, dw


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "dropout": _exact_dropout, "adapters": _exact_adapters,
            "adapters_grad": _exact_adapters_grad, "combine_grad": _exact_combine_grad}[case["op"]](s)
