"""Measured cases of the operators around the dispatch: the gate, the row
quantisation and the experts' product.

- ``gate``: router logits to ``topk_idx`` / ``topk_weights`` (softmax or
  sigmoid scores, ties to the lowest expert); a training step also gives the
  per-expert counts, the balance loss and the gradient of the logits.
- ``quantize``: bf16 rows to fp8 (e4m3) with one fp32 scale per row and block
  of 128 channels; ``swiglu``: the same of SwiGLU(h), h = [gate | up];
  ``swiglu_grad``: the same of SwiGLU's gradient with respect to h.
- ``product``: expert-major fp8 rows times each expert's fp8 weights
  [N, K] (one scale per 128 x 128 block) to bf16; ``experts``: an expert layer,
  the product with 2I gate and up channels, SwiGLU and the quantisation of its
  result, then the product back to K channels in bf16.

``own`` False computes the plain form in fp32 torch operations; ``own`` True
makes the calls of the framework. ``exact`` is the definition in float64.
"""

import math

import torch

own = False

FP8_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
BLOCK = 128
ZIPF_S = 1.2


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------- cases


def _gate(name, tokens, experts, topk, dtype, scoring, train, mask=0.0, bias=False):
    c = {"op": "gate", "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype, "scoring": scoring,
         "train": train, "mask": mask, "bias": bias}
    return dict(c, name=name) if name else c


def _rows(name, op, rows, width):
    c = {"op": op, "rows": rows, "width": width}
    return dict(c, name=name) if name else c


def _product(name, op, rows, experts, k, n, align, routing):
    c = {"op": op, "rows": rows, "experts": experts, "k": k, "n": n, "align": align, "routing": routing}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One decoded token: the router of a 256-expert layer with a selection bias.
        _gate("gate_one_token", 1, 256, 8, "bf16", "sigmoid", False, bias=True),
        # A ragged decode batch on the 128-expert layer.
        _gate("gate_decode_333", 333, 128, 8, "fp32", "softmax", False),
        # A training step on the 4096-token batch, 5 % of the tokens padding.
        _gate("gate_train_4096", 4096, 256, 8, "bf16", "sigmoid", True, mask=0.05, bias=True),
        # A training step on the largest batch, fp32 logits.
        _gate("gate_train_65536", 65536, 256, 8, "fp32", "softmax", True),
        # The 4096 x 7168 batch on its way into the fp8 dispatch.
        _rows("quantize_4096", "quantize", 4096, 7168),
        # Between the products while decoding: 8 routed rows.
        _rows("swiglu_8_rows", "swiglu", 8, 2048),
        # The gradient on its way back through the activation, 32768 routed rows and some.
        _rows("swiglu_grad_32777", "swiglu_grad", 32777, 2048),
        # One token's 8 experts of the 32 on this GPU.
        _product("experts_one_token", "experts", 8, 32, 7168, 2048, 1, "uniform"),
        # 64 decoded tokens, down projection, buckets unaligned.
        _product("product_512_rows", "product", 512, 32, 2048, 7168, 1, "uniform"),
        # A skewed prefill on 8 experts of width 4096.
        _product("product_zipf_8191", "product", 8191, 8, 4096, 4096, 16, "zipf"),
        # The 4096-token batch, buckets of 128.
        _product("experts_32768", "experts", 32768, 32, 7168, 2048, 128, "uniform"),
        # Its input gradient through the down projection: the product with transposed weights.
        _product("product_grad_32768", "product", 32768, 32, 7168, 2048, 128, "uniform"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "quantize", "swiglu", "swiglu_grad", "product", "product", "experts", "experts"])
    if op == "gate":
        experts = _log_int(rng, 6, 512)
        tokens = _log_int(rng, 1, min(65536, 65536 * 256 // experts))
        scoring = rng.choice(["softmax", "sigmoid"])
        return _gate(None, tokens, experts, rng.randint(1, min(12, experts)), rng.choice(["bf16", "fp32"]), scoring,
                     rng.random() < 0.6, rng.choice([0.0, 0.05, 0.3]), scoring == "sigmoid" and rng.random() < 0.7)
    if op == "quantize":
        width = 16 * _log_int(rng, 8, 512)
        return _rows(None, op, _log_int(rng, 1, 65536 * 4096 // width), width)
    if op in ("swiglu", "swiglu_grad"):
        width = BLOCK * _log_int(rng, 1, 32)
        return _rows(None, op, _log_int(rng, 1, 32768 * 2048 // width), width)
    while True:
        experts = _log_int(rng, 2, 64)
        k = 16 * _log_int(rng, 16, 448)
        n = BLOCK * _log_int(rng, 2, 16) if op == "experts" else 8 * _log_int(rng, 32, 896)
        routing = rng.choice(["uniform", "uniform", "zipf"])
        rows = _log_int(rng, 1, 32768)
        wide = 3 * n if op == "experts" else n
        cap = 1.9e12 if routing == "uniform" else 0.4e12
        if experts * wide * k <= 1400e6 and 2.0 * rows * wide * k <= cap and 3072 not in (k, n, rows):
            return _product(None, op, rows, experts, k, n, rng.choice([1, 16, 128]), routing)


# -------------------------------------------------------------------- inputs


def _generator(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + stream)
    return g


def _normal(shape, seed, stream, dtype=torch.float32):
    return torch.randn(shape, generator=_generator(seed, stream), device="cuda", dtype=dtype)


def _expert_probability(case):
    e = case["experts"]
    if case["routing"] == "uniform":
        return [1.0 / e] * e
    w = [(i + 1.0) ** -ZIPF_S for i in range(e)]
    return [v / sum(w) for v in w]


def _to_blocks(w):
    """[E, N, K] weights as fp8 with one fp32 scale per 128 x 128 block."""
    e, n, k = w.shape
    nb, kb = _ceil(n, BLOCK), _ceil(k, BLOCK)
    full = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    blocks = full.view(e, nb, BLOCK, kb, BLOCK)
    amax = blocks.abs().amax(dim=(2, 4)).float().clamp_min(AMAX_FLOOR)
    q = (blocks * (FP8_MAX / amax)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(e, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous(), amax / FP8_MAX


def _inputs(case, seed):
    op = case["op"]
    s = {"case": case}
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = (1.5 * _normal((t, e), seed, 0)).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["bias"] = 0.1 * _normal((e,), seed, 1) if case["bias"] else None
        s["mask"] = None
        if case["mask"]:
            s["mask"] = torch.rand((t,), generator=_generator(seed, 2), device="cuda") >= case["mask"]
        if case["train"]:
            s["grad_weights"] = _normal((t, k), seed, 3)
            s["grad_loss"] = 0.5 + torch.rand((1,), generator=_generator(seed, 4), device="cuda")
        s["normalize"], s["scale"], s["coef"] = True, 2.5, 0.01
        return s
    if op in ("quantize", "swiglu", "swiglu_grad"):
        r, w = case["rows"], case["width"]
        s["x"] = _normal((r, w if op == "quantize" else 2 * w), seed, 0, torch.bfloat16)
        if op == "swiglu_grad":
            s["grad"] = _normal((r, w), seed, 1, torch.bfloat16)
        return s
    rows, e, k, n, a = case["rows"], case["experts"], case["k"], case["n"], case["align"]
    p = torch.tensor(_expert_probability(case), device="cuda")
    owner = torch.multinomial(p, rows, replacement=True, generator=_generator(seed, 0))
    count = torch.bincount(owner, minlength=e)
    psum = torch.zeros((e + 1,), dtype=torch.int64, device="cuda")
    psum[1:] = torch.cumsum((count + a - 1) // a * a, 0)
    capacity = rows + e * (a - 1)  # the worst case, as a program that does not read the totals back allocates
    s["count"], s["psum"] = count.to(torch.int32), psum.to(torch.int32)
    s["host_count"], s["host_psum"], s["capacity"] = count.tolist(), psum.tolist(), capacity
    s["active"] = torch.nonzero(count).view(-1)
    s["most"] = max(s["host_count"])
    place = torch.repeat_interleave(psum[:-1] - (torch.cumsum(count, 0) - count), count) + torch.arange(rows, device="cuda")
    x = torch.zeros((capacity, k), dtype=torch.float32, device="cuda")
    x[place] = _normal((rows, k), seed, 1)
    q, sf = _quantize_plain(x)
    sf[torch.ones(capacity, dtype=torch.bool, device="cuda").index_fill_(0, place, False)] = 0.0  # pad rows, as dispatched
    s["x"], s["x_sf"] = q, sf
    wide = 2 * n if op == "experts" else n
    s["w"], s["w_sf"] = _to_blocks(_normal((e, wide, k), seed, 2, torch.bfloat16) * (k ** -0.5))
    if op == "experts":
        s["down"], s["down_sf"] = _to_blocks(_normal((e, k, n), seed, 3, torch.bfloat16) * (n ** -0.5))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    new = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "gate":
        if own:
            import moe_token_dispatch_amd as M

            p = M.make_gate_problem(case["tokens"], case["experts"], case["topk"],
                                    M.GATE_SOFTMAX if case["scoring"] == "softmax" else M.GATE_SIGMOID,
                                    logits_dtype=s["logits"].dtype, normalize=s["normalize"], route_scale=s["scale"],
                                    loss_coef=s["coef"])
            s["out"] = M.alloc_gate(p, "cuda", balance=case["train"])
            s["plan"] = M.GatePlan(p, s["logits"], s["out"], M.alloc_gate_workspace(p, "cuda"), select_bias=s["bias"],
                                   token_mask=s["mask"])
            if case["train"]:
                s["grad_logits"] = torch.empty_like(s["logits"])
                s["back"] = M.GateBackwardPlan(p, s["logits"], s["out"], s["grad_weights"], s["grad_loss"],
                                               s["grad_logits"], token_mask=s["mask"])
        return s
    if op in ("quantize", "swiglu", "swiglu_grad"):
        r, w = case["rows"], case["width"] * (2 if op == "swiglu_grad" else 1)
        s["q"], s["q_sf"] = new((r, w), torch.float8_e4m3fn), new((r, _ceil(w, BLOCK)), torch.float32)
        if own:
            import moe_token_dispatch_amd as M

            if op == "quantize":
                s["plan"] = M.QuantizePlan(s["x"], s["q"], s["q_sf"])
            elif op == "swiglu":
                s["plan"] = M.SwigluQuantizePlan(s["x"], s["q"], s["q_sf"])
            else:
                s["plan"] = M.SwigluBackwardQuantizePlan(s["x"], s["grad"], s["q"], s["q_sf"])
        return s
    n, k = case["n"], case["k"]
    s["out"] = new((s["capacity"], n if op == "product" else k), torch.bfloat16)
    if own:
        import moe_token_dispatch_amd as M

        layout = (s["psum"], s["count"])
        if op == "product":
            p = M.make_expert_problem(case["experts"], k, n, s["capacity"], case["rows"])
            s["plan"] = M.ExpertProductPlan(p, *layout, s["x"], s["x_sf"], s["w"], s["w_sf"], s["out"])
        else:
            a, a_sf = new((s["capacity"], n), torch.float8_e4m3fn), new((s["capacity"], n // BLOCK), torch.float32)
            up = M.make_expert_problem(case["experts"], k, 2 * n, s["capacity"], case["rows"])
            down = M.make_expert_problem(case["experts"], n, k, s["capacity"], case["rows"])
            s["up"] = M.ExpertSwigluPlan(up, *layout, s["x"], s["x_sf"], s["w"], s["w_sf"], a, a_sf)
            s["plan"] = M.ExpertProductPlan(down, *layout, a, a_sf, s["down"], s["down_sf"], s["out"])
    return s


# --------------------------------------------------------------- plain forms


def _scores(s):
    z = s["logits"].float()
    if s["case"]["scoring"] == "softmax":
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
        return z, score, score
    score = 1.0 / (1.0 + torch.exp(-z))
    choice = score if s["bias"] is None else score + s["bias"]
    return choice, score, score / score.sum(dim=1, keepdim=True)


def _gate_plain(s):
    case = s["case"]
    t, e, k = case["tokens"], case["experts"], case["topk"]
    choice, score, prob = _scores(s)
    idx = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    picked = torch.gather(score, 1, idx)
    total = picked.sum(dim=1, keepdim=True)
    weights = s["scale"] * picked / total
    live = torch.ones((t,), dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    out_idx = torch.where(live[:, None], idx, -1)
    out_weights = torch.where(live[:, None], weights, 0.0)
    if not case["train"]:
        return {"topk_idx": out_idx, "topk_weights": out_weights}
    chosen = torch.zeros((t, e), dtype=torch.float32, device="cuda").scatter_(1, idx, 1.0) * live[:, None]
    count = chosen.sum(dim=0)
    prob_sum = (prob * live[:, None]).sum(dim=0)
    n = live.sum().float().clamp_min(1.0)
    unit = s["coef"] * e / (k * n * n)
    loss = unit * (count * prob_sum).sum()
    # Gradients: of the weights to the picked scores, of the loss to the probabilities.
    dw = s["grad_weights"]
    d_picked = s["scale"] / total * (dw - (dw * picked / total).sum(dim=1, keepdim=True))
    d_score = torch.zeros((t, e), dtype=torch.float32, device="cuda").scatter_(1, idx, d_picked)
    d_prob = s["grad_loss"] * unit * count
    if case["scoring"] == "softmax":
        d = d_score + d_prob
        dz = score * (d - (score * d).sum(dim=1, keepdim=True))
    else:
        d = d_score + (d_prob - (prob * d_prob).sum(dim=1, keepdim=True)) / score.sum(dim=1, keepdim=True)
        dz = d * score * (1.0 - score)
    return {"topk_idx": out_idx, "topk_weights": out_weights, "expert_count": count.to(torch.int32), "prob_sum": prob_sum,
            "loss": loss.view(1), "grad_logits": torch.where(live[:, None], dz, 0.0).to(s["logits"].dtype)}


def _quantize_plain(x):
    """fp32 [R, W] rows to fp8 and one scale per row and block of 128 channels (the last one may be short)."""
    r, w = x.shape
    nb = _ceil(w, BLOCK)
    full = x if nb * BLOCK == w else torch.nn.functional.pad(x, (0, nb * BLOCK - w))
    blocks = full.view(r, nb, BLOCK)
    amax = blocks.abs().amax(dim=2).clamp_min(AMAX_FLOOR)
    q = (blocks * (FP8_MAX / amax)[:, :, None]).view(r, nb * BLOCK)[:, :w].to(torch.float8_e4m3fn)
    return q, amax / FP8_MAX


def _swiglu_plain(h):
    g, u = torch.chunk(h, 2, dim=1)
    return g / (1.0 + torch.exp(-g)) * u


def _swiglu_grad_plain(h, da):
    g, u = torch.chunk(h, 2, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-g))
    return torch.cat([da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig], dim=1)


def _wide_scales(sf, dim, size):
    return torch.repeat_interleave(sf, BLOCK, dim=dim).narrow(dim, 0, size)


def _place_plain(s):
    """[active experts, longest] rows of the buffer, and which of them are live."""
    count, first = s["count"].long()[s["active"]], s["psum"].long()[:-1][s["active"]]
    at = torch.arange(s["most"], device="cuda")
    live = at[None, :] < count[:, None]
    return torch.where(live, first[:, None] + at[None, :], 0), live


def _product_plain(x, x_sf, w, w_sf, active):
    """fp32 products of each active expert's rows x [active, longest, K]."""
    n, k = w.shape[1:]
    x = x.float() * _wide_scales(x_sf, 2, k)
    w = w.view(torch.uint8)[active].view(torch.float8_e4m3fn).float()
    w = w * _wide_scales(_wide_scales(w_sf[active], 2, k), 1, n)
    return torch.bmm(x, w.transpose(1, 2).contiguous())


def run(s):
    op = s["case"]["op"]
    if op == "gate":
        if not own:
            return _gate_plain(s)
        s["plan"]()
        out = s["out"]
        if not s["case"]["train"]:
            return {"topk_idx": out.topk_idx, "topk_weights": out.topk_weights}
        s["back"]()
        return {"topk_idx": out.topk_idx, "topk_weights": out.topk_weights, "expert_count": out.expert_count,
                "prob_sum": out.prob_sum, "loss": out.loss, "grad_logits": s["grad_logits"]}
    if op in ("quantize", "swiglu", "swiglu_grad"):
        if own:
            s["plan"]()
            return {"q": s["q"], "sf": s["q_sf"]}
        x = s["x"].float()
        if op == "swiglu":
            x = _swiglu_plain(x)
        elif op == "swiglu_grad":
            x = _swiglu_grad_plain(x, s["grad"].float())
        q, sf = _quantize_plain(x)
        return {"q": q, "sf": sf}
    if own:
        if op == "experts":
            s["up"]()
        s["plan"]()
        return {"out": s["out"]}
    place, live = _place_plain(s)
    x = s["x"].view(torch.uint8)[place].view(torch.float8_e4m3fn)
    y = _product_plain(x, s["x_sf"][place], s["w"], s["w_sf"], s["active"])
    if op == "experts":
        q, sf = _quantize_plain(_swiglu_plain(y.view(-1, y.shape[2])))
        y = _product_plain(q.view(*live.shape, -1), sf.view(*live.shape, -1), s["down"], s["down_sf"], s["active"])
    s["out"][place[live]] = y[live].to(torch.bfloat16)
    return {"out": s["out"]}


# --------------------------------------------------------------------- exact


def _exact_gate(s):
    case = s["case"]
    t, e, k = case["tokens"], case["experts"], case["topk"]
    z = s["logits"].double()
    if case["scoring"] == "softmax":
        score = torch.softmax(z, dim=1)
        order = z
    else:
        score = torch.sigmoid(z)
        order = score if s["bias"] is None else score + s["bias"].double()
    denom = score.sum(1, keepdim=True)
    prob = score / denom
    # An expert's place in its token's order; the k first are taken.
    place = torch.argsort(torch.argsort(order, dim=1, descending=True, stable=True), dim=1)
    taken = place < k
    idx = torch.argsort(place, dim=1)[:, :k]
    live = s["mask"] if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device="cuda")
    picked = score.gather(1, idx)
    weights = s["scale"] * picked / picked.sum(1, keepdim=True) * live[:, None]
    if not case["train"]:
        return {"topk_idx": None, "topk_weights": weights}
    count = taken[live].sum(0).double()
    n = float(live.sum())
    prob_sum = prob[live].sum(0)
    unit = s["coef"] * e / (k * n * n) if n else 0.0
    # The gradient from the Jacobians: weights = scale * picked / sum(picked), prob = score / sum(score).
    dw = s["grad_weights"].double() * s["scale"]
    psum = picked.sum(1, keepdim=True)
    d_score = torch.zeros_like(z)
    d_score.scatter_(1, idx, dw / psum - (dw * picked).sum(1, keepdim=True) / psum ** 2)
    dp = s["grad_loss"].double() * unit * count
    if case["scoring"] == "softmax":
        total = d_score + dp
        dz = score * total - score * (score * total).sum(1, keepdim=True)
    else:
        total = d_score + dp / denom - (score * dp).sum(1, keepdim=True) / denom ** 2
        dz = total * score * (1 - score)
    return {"topk_idx": None, "topk_weights": weights, "expert_count": None, "prob_sum": prob_sum,
            "loss": (unit * (count * prob_sum).sum()).view(1), "grad_logits": dz * live[:, None]}


def _exact_rows(x):
    """The rows' values over their scales, and the scales; the 8-bit values are the nearest ones to those."""
    r, w = x.shape
    nb = _ceil(w, BLOCK)
    block = torch.arange(w, device=x.device) // BLOCK
    top = torch.zeros((r, nb), dtype=torch.float64, device=x.device)
    top.scatter_reduce_(1, block.expand(r, w), x.abs(), "amax")
    sf = top.clamp_min(AMAX_FLOOR) / FP8_MAX
    v = x / sf[:, block]
    # e4m3: 3 bits behind the leading one, exponents from -6 on.
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step, sf


def _exact_product(x, w, w_sf):
    n, k = w.shape
    w = w.double() * w_sf.double()[torch.arange(n, device="cuda") // BLOCK][:, torch.arange(k, device="cuda") // BLOCK]
    return x @ w.t()


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(s)
    if op in ("quantize", "swiglu", "swiglu_grad"):
        x = s["x"].double()
        if op != "quantize":
            w = case["width"]
            g, u = x[:, :w], x[:, w:]
            sig = torch.sigmoid(g)
            if op == "swiglu":
                x = g * sig * u
            else:
                d = s["grad"].double()
                x = torch.cat([d * u * (sig + g * sig * torch.sigmoid(-g)), d * g * sig], 1)
        q, sf = _exact_rows(x)
        return {"q": q, "sf": sf}
    n, k = case["n"], case["k"]
    out = torch.zeros((s["capacity"], n if op == "product" else k), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, c = s["host_psum"][e], s["host_count"][e]
        if not c:
            continue
        x = s["x"][lo:lo + c].double() * s["x_sf"][lo:lo + c].double()[:, torch.arange(k, device="cuda") // BLOCK]
        y = _exact_product(x, s["w"][e], s["w_sf"][e])
        if op == "experts":
            q, sf = _exact_rows(y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:])
            y = _exact_product(q * sf[:, torch.arange(n, device="cuda") // BLOCK], s["down"][e], s["down_sf"][e])
        out[lo:lo + c] = y
    return {"out": out}


# ---------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        table = t * e * (2 if case["dtype"] == "bf16" else 4)
        small = t * k * 12 + (4 * e if case["bias"] else 0) + (t if case["mask"] else 0)
        if not case["train"]:
            return {"bytes": table + small, "flops": 8 * t * e}
        return {"bytes": 2 * table + small + 4 * t * k + 8 * e + 8, "flops": 20 * t * e}
    if op in ("quantize", "swiglu", "swiglu_grad"):
        r, w = case["rows"], case["width"]
        if op == "quantize":
            return {"bytes": r * (3 * w + 4 * _ceil(w, BLOCK)), "flops": 3 * r * w}
        if op == "swiglu":
            return {"bytes": r * (5 * w + 4 * _ceil(w, BLOCK)), "flops": 9 * r * w}
        return {"bytes": r * (8 * w + 4 * _ceil(2 * w, BLOCK)), "flops": 20 * r * w}
    rows, k, n = case["rows"], case["k"], case["n"]
    kb, nb = _ceil(k, BLOCK), _ceil(n, BLOCK)
    active = sum(1.0 - (1.0 - p) ** rows for p in _expert_probability(case))
    if op == "product":
        weights, values, out = n * k + 4 * nb * kb, n * k, n
    else:
        weights, values, out = 3 * (n * k + 4 * nb * kb), 3 * n * k, k
    return {"bytes": rows * (k + 4 * kb + 2 * out) + active * weights + 8 * case["experts"] + 4,
            "flops": 2.0 * rows * values}
