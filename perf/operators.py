"""Cases for measuring the operators around the expert-parallel path: the router
that makes topk_idx and topk_weights, the experts' grouped products over the rows
that dispatch delivers, and the dense product with its epilogue (gate, shared expert).

`run` computes a case in plain torch operations, or with `own` set through the
package's entry points. Sizes are those of the repository's workloads (hidden 7168
and 4096, top-8 of 256 experts, top-16 of 512) with an expert width of 2048."""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step's routing: sigmoid scores, a selection bias that balances the experts, 4 of 8 groups
        dict(name="route_decode", op="route", T=128, E=256, K=8, scoring="sigmoid", biased=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=0.0),
        # the largest routing of the layer's limits: top-16 of 512
        dict(name="route_top16", op="route", T=32768, E=512, K=16, scoring="softmax", biased=False, groups=1,
             topk_groups=1, group_top=1, renorm=True, scale=1.0, dtype="f32", masked=0.0),
        # a training step's routing gradient, an odd number of tokens, some experts masked out
        dict(name="route_grad", op="route_grad", T=8191, E=256, K=8, scoring="softmax", renorm=False, scale=1.0,
             dtype="bf16", masked=0.02),
        # the gate of a decode step: few rows, a long reduction, scores in fp32
        dict(name="gate_decode", op="linear", T=128, I=7168, O=256, act="", bias=False, residual=False, out="f32",
             fp8=False),
        # the shared expert's second product on a prefill batch, added to the combined rows
        dict(name="shared_down", op="linear", T=4096, I=2048, O=7168, act="", bias=False, residual=True, out="bf16",
             fp8=False),
        # a small dense block with everything in its epilogue, odd sizes
        dict(name="dense_gelu_odd", op="linear", T=777, I=4104, O=1003, act="gelu", bias=True, residual=True,
             out="bf16", fp8=False),
        # training the shared expert's first product
        dict(name="shared_up_grad", op="linear_grad", T=4095, I=4096, O=2048, act="swiglu", bias=True),
        # one rank's experts at decode: 16 experts, some 64 rows each; the weights are what is read
        dict(name="experts_up_decode", op="grouped", G=16, rows=1024, skew=0.5, I=7168, O=2048, act="swiglu",
             bias=False, fp8=False),
        # one rank's experts on prefill: 32 experts, 32768 rows unevenly spread
        dict(name="experts_up_prefill", op="grouped", G=32, rows=32768, skew=0.6, I=7168, O=2048, act="swiglu",
             bias=False, fp8=False),
        # the same rank's second product with the FP8 payload
        dict(name="experts_down_fp8", op="grouped", G=32, rows=32768, skew=0.6, I=2048, O=7168, act="", bias=False,
             fp8=True),
        # the packed low-latency layout with the FP8 payload: fixed buffers, few rows in each, some experts empty
        dict(name="experts_packed_fp8", op="packed", G=16, cap=128, fill=0.5, I=7168, O=2048, act="swiglu",
             bias=False, fp8=True),
        # training the experts' second product: ragged rows, one expert without any
        dict(name="experts_grad", op="grouped_grad", G=32, rows=16384, skew=0.6, I=2048, O=4096, act="", bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log_int(rng, lo, hi) // m * m)


def _width(rng, act, fp8, most):
    """Output features; FP8 SwiGLU has whole scale blocks of gate and of up rows."""
    return _mult(rng, 128, most, 128) if fp8 and act == "swiglu" else _log_int(rng, 16, most)


def draw(rng):
    op = rng.choice(["route", "route_grad", "linear", "linear_grad", "grouped", "grouped", "packed", "grouped_grad"])
    if op == "route" or op == "route_grad":
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        E = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        group_top = rng.choice([1, 2])
        c = dict(op=op, T=_log_int(rng, 1, 32768), E=E, K=rng.randint(1, min(16, E // groups * keep)),
                 scoring=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                 scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.02]))
        if op == "route":
            c.update(biased=rng.random() < 0.5, groups=groups, topk_groups=keep, group_top=group_top)
        return c
    act = rng.choice(["", "relu", "silu", "gelu", "swiglu"])
    if op == "linear":
        fp8 = rng.random() < 0.25
        return dict(op=op, T=_log_int(rng, 1, 4096), I=_mult(rng, 128, 7168, 128 if fp8 else 8),
                    O=_width(rng, act, fp8, 4096), act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    out="bf16" if fp8 else rng.choice(["bf16", "f32"]), fp8=fp8)
    if op == "linear_grad":
        return dict(op=op, T=_log_int(rng, 1, 4096), I=_mult(rng, 64, 4096, 8), O=_log_int(rng, 16, 2048), act=act,
                    bias=rng.random() < 0.5)
    if op == "grouped_grad":
        return dict(op=op, G=_log_int(rng, 1, 32), rows=_log_int(rng, 1, 8192), skew=rng.uniform(0, 1),
                    I=_mult(rng, 64, 2048, 8), O=_log_int(rng, 16, 2048), act=act, bias=rng.random() < 0.5)
    fp8 = rng.random() < 0.5
    c = dict(op=op, G=_log_int(rng, 1, 48), I=_mult(rng, 128, 4096, 128 if fp8 else 8), O=_width(rng, act, fp8, 2048),
             act=act, bias=rng.random() < 0.5, fp8=fp8)
    if op == "packed":
        c.update(cap=_log_int(rng, 1, 256), fill=rng.uniform(0.05, 1.0))
    else:
        c.update(rows=_log_int(rng, 1, 16384), skew=rng.uniform(0, 1))
    return c


def _wide(case):
    """Weight rows of a product with O outputs (SwiGLU: gate rows, then up rows)."""
    return case["O"] * (2 if case["act"] == "swiglu" else 1)


def _rows(case):
    """Rows that hold data, on average over the seeds."""
    if case["op"] == "packed":
        return case["G"] * max(1.0, case["cap"] * case["fill"] * 0.5)
    return case["T"] if "T" in case else case["rows"]


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, K = case["T"], case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * K * 12, "flops": T * E * 4}
        return {"bytes": 2 * T * E * size + T * K * 12, "flops": T * E * 6}
    rows, I, O, W = _rows(case), case["I"], case["O"], _wide(case)
    groups = case.get("G", 1)
    groups = min(groups, rows)
    if op.endswith("_grad"):
        pre = rows * W * 2 if case["act"] else 0
        b = rows * I * 2 * 2 + rows * O * 2 + pre + 2 * case.get("G", 1) * W * I * 2
        return {"bytes": b, "flops": 4 * rows * W * I}
    size = 1 if case["fp8"] else 2
    out = 4 if case.get("out") == "f32" else 2
    b = rows * I * size + groups * W * I * size + rows * O * out + (rows * O * 2 if case.get("residual") else 0)
    return {"bytes": b, "flops": 2 * rows * W * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=F32, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32 if dtype != BF16 else BF16).mul_(scale).to(dtype)


def _counts(g, groups, rows, skew):
    """Rows of each group: an uneven share for each, whole numbers that add up to `rows`."""
    share = torch.exp(skew * torch.randn(groups, generator=g, device=DEV, dtype=F64))
    edge = torch.round(torch.cumsum(share, 0) / share.sum() * rows).to(torch.int64)
    edge[-1] = rows
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), edge])
    return off


def _fp8(g, lead, I):
    """FP8 codes of normal values and one fp32 scale for 128 values of a row, as the per-token cast gives them."""
    q = (torch.randn(*lead, I, generator=g, device=DEV, dtype=BF16).clamp_(-4, 4) * 112).to(torch.float8_e4m3fn)
    sc = torch.rand(*lead, I // 128, generator=g, device=DEV, dtype=F32).add_(0.5).mul_(1 / 112)
    return q, sc


def _fp8_weight(g, lead, O, I):
    """FP8 codes of a weight and one fp32 scale for each block of 128 x 128."""
    q = (torch.randn(*lead, O, I, generator=g, device=DEV, dtype=BF16).clamp_(-4, 4) * 112).to(torch.float8_e4m3fn)
    sc = torch.rand(*lead, -(-O // 128), I // 128, generator=g, device=DEV, dtype=F32).add_(0.5)
    return q, sc.mul_(1 / (112 * math.sqrt(I)))


def _logits(g, case):
    x = _randn(g, case["T"], case["E"], scale=1.5)
    if case["masked"]:  # experts that are out of service, by token
        x[torch.rand(x.shape, generator=g, device=DEV) < case["masked"]] = -math.inf
        x[case["T"] // 2] = -math.inf  # a token that may go nowhere
    return x.to(F32 if case["dtype"] == "f32" else BF16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("route", "route_grad"):
        s["logits"] = _logits(g, case)
        T, E, K = case["T"], case["E"], case["K"]
        if op == "route":
            s["bias"] = _randn(g, E, scale=0.1) if case["biased"] else None
        else:
            key = torch.rand(T, E, generator=g, device=DEV).masked_fill_(torch.isinf(s["logits"]), -1.0)
            v, i = torch.topk(key, K, dim=1)
            s["idx"] = torch.where(v < 0, -1, i)
            s["grad"] = _randn(g, T, K)
        return s
    I, O, W = case["I"], case["O"], _wide(case)
    grad = op.endswith("_grad")
    if op.startswith("linear"):
        lead, rows, G = (), (case["T"],), 1
    else:
        G = case["G"]
        lead = (G,)
        if op == "packed":
            rows = (G, case["cap"])
            n = torch.rand(G, generator=g, device=DEV).mul_(case["fill"] * case["cap"] + 1).to(torch.int32)
            s["counts"] = n.clamp_(0, case["cap"])
        else:
            rows = (case["rows"],)
            off = _counts(g, G, case["rows"], case["skew"])
            if grad and G > 2:
                off[G // 2 + 1] = off[G // 2]  # an expert that no token chose
            s["offsets"] = off.to(torch.int32)
            s["edges"] = off.tolist()  # the plan a host keeps
    if case.get("fp8"):
        s["x"] = _fp8(g, rows, I)
        s["w"] = _fp8_weight(g, lead, W, I)
    else:
        s["x"] = _randn(g, *rows, I, dtype=BF16)
        s["w"] = _randn(g, *lead, W, I, dtype=BF16, scale=1 / math.sqrt(I))
    s["b"] = _randn(g, *lead, W, dtype=BF16, scale=0.5) if case["bias"] else None
    if grad:
        s["grad"] = _randn(g, *rows, O, dtype=BF16)
        s["pre"] = _randn(g, *rows, W, dtype=BF16) if case["act"] else None
    elif case.get("residual"):
        s["res"] = _randn(g, *rows, O, dtype=BF16)
    if op == "packed":  # rows past a count are left as they were
        s["out"] = torch.zeros(*rows, O, dtype=BF16, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_route(s):
    c = s["case"]
    l = s["logits"].to(F64)
    p = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    v = l if s["bias"] is None and c["group_top"] == 1 else p + (0 if s["bias"] is None else s["bias"].to(F64))
    v = v.masked_fill(torch.isinf(l), -math.inf)
    if c["groups"] > 1:
        T, E = l.shape
        vg = v.view(T, c["groups"], E // c["groups"])
        top = torch.sort(vg, dim=2, descending=True)[0][:, :, :c["group_top"]]
        # the second of a group with one selectable expert adds nothing
        score = torch.where(torch.isinf(top[:, :, :1]), -math.inf, torch.where(torch.isinf(top), 0.0, top).sum(2, True))
        order = torch.sort(score[:, :, 0], dim=1, descending=True, stable=True)[1]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=l.device)
        keep.scatter_(1, order[:, :c["topk_groups"]], True)
        v = vg.masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    val, idx = torch.sort(v, dim=1, descending=True, stable=True)
    val, idx = val[:, :c["K"]], idx[:, :c["K"]]
    w = torch.gather(p, 1, idx).masked_fill(torch.isinf(val), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(torch.isinf(val), -1, idx), (w * c["scale"]).to(F32)


def _plain_route_grad(s):
    c = s["case"]
    l, idx, g = s["logits"].to(F32), s["idx"], s["grad"] * c["scale"]
    sel = idx >= 0
    at = idx.clamp_min(0)
    g = g * sel
    p = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    ps = torch.gather(p, 1, at) * sel
    if c["renorm"]:
        total = ps.sum(1, keepdim=True)
        inv = torch.where(total > 0, 1 / total, 0.0)
        g = (g - (g * ps * inv).sum(1, keepdim=True)) * inv * sel
    full = torch.zeros_like(p).scatter_add_(1, at, g)
    if c["scoring"] == "sigmoid":
        out = full * p * (1 - p)
    else:
        out = p * (full - (full * p).sum(1, keepdim=True))
    return out.to(s["logits"].dtype)


def _act(pre, act, O):
    if act == "relu":
        return pre.clamp_min(0)
    if act == "silu":
        return pre * torch.sigmoid(pre)
    if act == "gelu":
        return 0.5 * pre * (1 + torch.erf(pre * math.sqrt(0.5)))
    if act == "swiglu":
        gate = pre[..., :O]
        return gate * torch.sigmoid(gate) * pre[..., O:]
    return pre


def _act_grad(g, pre, act, O):
    if act == "relu":
        return g * (pre > 0)
    if act == "silu":
        s = torch.sigmoid(pre)
        return g * (s + pre * s * (1 - s))
    if act == "gelu":
        return g * (0.5 * (1 + torch.erf(pre * math.sqrt(0.5))) +
                    pre * torch.exp(-0.5 * pre * pre) * (1 / math.sqrt(2 * math.pi)))
    if act == "swiglu":
        gate, up = pre[..., :O], pre[..., O:]
        s = torch.sigmoid(gate)
        return torch.cat([g * up * (s + gate * s * (1 - s)), g * gate * s], -1)
    return g


def _plain_x(x):
    if isinstance(x, tuple):
        q, sc = x
        return (q.to(F32).view(*sc.shape, 128) * sc[..., None]).view(q.shape)
    return x.to(F32)


def _plain_w(w):
    if isinstance(w, tuple):
        q, sc = w
        full = sc.repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)
        return q.to(F32) * full
    return w.to(F32)


def _pick(v, a, b=None):
    """Rows a..b of an input, or entry a; of both parts where it is a (codes, scales) pair."""
    if v is None:
        return None
    if isinstance(v, tuple):
        return tuple(_pick(t, a, b) for t in v)
    return v[a] if b is None else v[a:b]


def _product(x, w, b, c):
    pre = _plain_x(x) @ _plain_w(w).mT
    if b is not None:
        pre = pre + b.to(F32).unsqueeze(-2)
    return _act(pre, c["act"], c["O"])


def _product_grad(grad, x, w, pre, c):
    d = grad.to(F32)
    if c["act"]:
        d = _act_grad(d, pre.to(F32), c["act"], c["O"])
    return (d @ w.to(F32)).to(BF16), (d.mT @ x.to(F32)).to(BF16), d.sum(-2).to(BF16) if c["bias"] else None


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_grad":
        return _plain_route_grad(s)
    if op == "linear":
        y = _product(s["x"], s["w"], s["b"], c)
        if c["residual"]:
            y = y + s["res"].to(F32)
        return y.to(F32 if c["out"] == "f32" else BF16)
    if op == "linear_grad":
        return _product_grad(s["grad"], s["x"], s["w"], s["pre"], c)
    if op == "packed":
        y = _product(s["x"], s["w"], s["b"], c)
        valid = torch.arange(c["cap"], device=y.device)[None, :] < s["counts"][:, None]
        s["out"].copy_(torch.where(valid[:, :, None], y, s["out"]))
        return s["out"]
    edges = s["edges"]
    if op == "grouped":  # ragged: one product for each expert
        y = torch.empty(c["rows"], c["O"], dtype=BF16, device=DEV)
        for e, (a, b) in enumerate(zip(edges, edges[1:])):
            if b > a:
                y[a:b] = _product(_pick(s["x"], a, b), _pick(s["w"], e), _pick(s["b"], e), c)
        return y
    gx = torch.empty_like(s["x"])
    gw = torch.empty_like(s["w"])
    gb = torch.empty(s["w"].shape[:2], dtype=BF16, device=DEV) if c["bias"] else None
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        gx[a:b], gw[e], db = _product_grad(s["grad"][a:b], s["x"][a:b], s["w"][e], _pick(s["pre"], a, b), c)
        if gb is not None:
            gb[e] = db
    return gx, gw, gb


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import combine_get_dispatch_06_amd as cgd
    s, c = state, state["case"]
    op = c["op"]
    if op == "route":
        return cgd.route(s["logits"], c["K"], scoring=c["scoring"], bias=s["bias"], num_groups=c["groups"],
                         num_topk_groups=c["topk_groups"], group_score_topk=c["group_top"], renormalize=c["renorm"],
                         scale=c["scale"])
    if op == "route_grad":
        return cgd.route_backward(s["grad"], s["logits"], s["idx"], scoring=c["scoring"], renormalize=c["renorm"],
                                  scale=c["scale"])
    act = c["act"] or None
    if op == "linear":
        return cgd.linear(s["x"], s["w"], bias=s["b"], activation=act, residual=s.get("res"),
                          out_dtype=F32 if c["out"] == "f32" else BF16)
    if op == "linear_grad":
        return cgd.linear_backward(s["grad"], s["x"], s["w"], preact=s["pre"], activation=act, bias_grad=c["bias"])
    if op == "grouped":
        return cgd.grouped_linear(s["x"], s["w"], s["offsets"], bias=s["b"], activation=act)
    if op == "packed":
        return cgd.grouped_linear(s["x"], s["w"], s["counts"], bias=s["b"], activation=act, out=s["out"])
    return cgd.grouped_linear_backward(s["grad"], s["x"], s["w"], s["offsets"], preact=s["pre"], activation=act,
                                       bias_grad=c["bias"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_route(s):
    """By repeated selection: the best group K' times, then the best expert K times."""
    c = s["case"]
    l = s["logits"].double()
    T, E = l.shape
    off = l == -math.inf
    top = l.masked_fill(off, -1e300).amax(1, keepdim=True)
    ex = torch.exp(l - top).masked_fill(off, 0.0)
    score = ex / ex.sum(1, keepdim=True).clamp_min(1e-300) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-l))
    choice = l if s["bias"] is None and c["group_top"] == 1 else score + (0.0 if s["bias"] is None else s["bias"].double())
    choice = torch.where(off, -math.inf, choice)
    n = E // c["groups"]
    if c["groups"] > 1:
        a = choice.view(T, c["groups"], n)
        best = a.amax(2)
        if c["group_top"] == 2 and n > 1:
            rest = a.scatter(2, a.argmax(2, keepdim=True), -math.inf).amax(2)
            best = torch.where(torch.isinf(rest), best, best + rest)
        allowed = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(c["topk_groups"]):
            m = best.amax(1, keepdim=True)
            first = ((best == m) & ~allowed).long().argmax(1, keepdim=True)
            allowed.scatter_(1, first, True)
            best = best.scatter(1, first, -math.inf)
        choice = choice.masked_fill(~allowed.repeat_interleave(n, 1), -math.inf)
    idx, wts = [], []
    for _ in range(c["K"]):
        m = choice.amax(1, keepdim=True)
        first = (choice == m).long().argmax(1, keepdim=True)
        none = m == -math.inf
        idx.append(torch.where(none, -1, first))
        wts.append(torch.where(none, 0.0, score.gather(1, first)))
        choice = choice.scatter(1, first, -math.inf)
    idx, wts = torch.cat(idx, 1), torch.cat(wts, 1)
    if c["renorm"]:
        total = wts.sum(1, keepdim=True)
        wts = torch.where(total > 0, wts / total, 0.0)
    return idx, wts * c["scale"]


def _exact_route_grad(s):
    """The Jacobian of the weights, slot by slot."""
    c = s["case"]
    l = s["logits"].double()
    off = l == -math.inf
    if c["scoring"] == "softmax":
        ex = torch.exp(l - l.masked_fill(off, -1e300).amax(1, keepdim=True)).masked_fill(off, 0.0)
        p = ex / ex.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1 / (1 + torch.exp(-l))
    idx, grad = s["idx"], s["grad"].double()
    total = sum(torch.where(idx[:, k] >= 0, p.gather(1, idx[:, k:k + 1].clamp_min(0))[:, 0], 0.0)
                for k in range(c["K"]))
    dp = torch.zeros_like(p)
    for k in range(c["K"]):
        at = idx[:, k:k + 1].clamp_min(0)
        use = idx[:, k] >= 0
        g = torch.where(use, grad[:, k] * c["scale"], 0.0)
        if not c["renorm"]:
            dp.scatter_add_(1, at, g[:, None])
            continue
        ok = total > 0  # w = p_k / total
        t = torch.where(ok, total, 1.0)
        pk = p.gather(1, at)[:, 0]
        dp.scatter_add_(1, at, torch.where(ok, g / t, 0.0)[:, None])
        for j in range(c["K"]):
            use_j = (idx[:, j] >= 0) & ok
            dp.scatter_add_(1, idx[:, j:j + 1].clamp_min(0), torch.where(use_j, -g * pk / t / t, 0.0)[:, None])
    if c["scoring"] == "sigmoid":
        return dp * p * (1 - p)
    return p * dp - p * (p * dp).sum(1, keepdim=True)


def _decoded(v, weight):
    if not isinstance(v, tuple):
        return v.double()
    q, sc = v
    out = q.float().double()
    for k in range(sc.shape[-1]):
        col = sc[..., k].double()
        if weight:
            col = col[..., torch.arange(q.shape[-2], device=DEV) // 128]
        out[..., k * 128:(k + 1) * 128] *= col[..., None]
    return out


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_rows(x, w, b, c):
    z = torch.matmul(_decoded(x, False), _decoded(w, True).transpose(-1, -2))
    if b is not None:
        z = z + b.double()
    O = c["O"]
    if c["act"] == "swiglu":
        return _silu64(z[:, :O]) * z[:, O:]
    return {"": lambda v: v, "relu": torch.relu, "silu": _silu64,
            "gelu": lambda v: v * 0.5 * torch.erfc(-v / math.sqrt(2.0))}[c["act"]](z)


def _exact_grads(grad, x, w, pre, c):
    d = grad.double()
    if c["act"]:
        with torch.enable_grad():  # the derivative of the formula itself
            z = pre.double().requires_grad_(True)
            O = c["O"]
            y = {"relu": torch.relu, "silu": _silu64, "gelu": lambda v: v * 0.5 * torch.erfc(-v / math.sqrt(2.0)),
                 "swiglu": lambda v: _silu64(v[:, :O]) * v[:, O:]}[c["act"]](z)
            d = torch.autograd.grad(y, z, d)[0]
    return torch.matmul(d, w.double()), torch.matmul(d.t(), x.double()), d.sum(0) if c["bias"] else None


def exact(case, seed):
    s = prepare(case, seed)
    op, c = case["op"], case
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "linear":
        y = _exact_rows(s["x"], s["w"], s["b"], c)
        return y + s["res"].double() if c["residual"] else y
    if op == "linear_grad":
        return _exact_grads(s["grad"], s["x"], s["w"], s["pre"], c)
    if op == "packed":
        out = s["out"].double()
        for e, n in enumerate(s["counts"].tolist()):
            out[e, :n] = _exact_rows(_pick(_pick(s["x"], e), 0, n), _pick(s["w"], e), _pick(s["b"], e), c)
        return out
    edges = s["edges"]
    parts = []
    for e in range(c["G"]):
        a, b = edges[e], edges[e + 1]
        if op == "grouped":
            parts.append(_exact_rows(_pick(s["x"], a, b), _pick(s["w"], e), _pick(s["b"], e), c))
        else:
            parts.append(_exact_grads(s["grad"][a:b], s["x"][a:b], s["w"][e], _pick(s["pre"], a, b), c))
    if op == "grouped":
        return torch.cat(parts)
    return (torch.cat([p[0] for p in parts]), torch.stack([p[1] for p in parts]),
            torch.stack([p[2] for p in parts]) if c["bias"] else None)
