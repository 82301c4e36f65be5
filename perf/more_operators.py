"""Measured cases of the operators that stand before and behind an expert
layer: the gate with expert groups, the RMS norm, and the combine's gradient.

- ``gate``: router logits to ``topk_idx`` / ``topk_weights`` where a token's
  experts come from its few best groups of experts (those a rank or a node
  holds), ties to the lowest group and expert; a training step also gives the
  counts, the balance loss and the gradient of the logits.
- ``norm``: h = x + residual (bf16), y = h / sqrt(mean h^2 + eps) * weight to
  bf16 rows, to fp8 rows with one fp32 scale per 128 channels, or to both;
  ``norm_grad``: the gradients of h and of the weight.
- ``combine_grad``: the combine's gradient: of each top-k weight, and of each
  expert-major row, in bf16 or in fp8 with its scales.

``own`` False computes the plain form in fp32 torch operations; ``own`` True
makes the calls of the framework. ``exact`` is the definition in float64.
"""

import math

import torch

own = False

FP8_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
BLOCK = 128
EPS = 1e-6


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------- cases


def _gate(name, tokens, experts, groups, groups_taken, topk, dtype, scoring, train, mask=0.0, bias=False):
    """Sigmoid groups go by the sum of their two largest choices, softmax groups by their largest one."""
    c = {"op": "gate", "tokens": tokens, "experts": experts, "groups": groups, "groups_taken": groups_taken, "topk": topk,
         "dtype": dtype, "scoring": scoring, "train": train, "mask": mask, "bias": bias}
    return dict(c, name=name) if name else c


def _norm(name, rows, width, out, residual, weight):
    c = {"op": "norm", "rows": rows, "width": width, "out": out, "residual": residual, "weight": weight}
    return dict(c, name=name) if name else c


def _norm_grad(name, rows, width, residual, weight):
    c = {"op": "norm_grad", "rows": rows, "width": width, "residual": residual, "weight": weight}
    return dict(c, name=name) if name else c


def _combine_grad(name, tokens, topk, width, experts, align, out, mask=0.0):
    c = {"op": "combine_grad", "tokens": tokens, "topk": topk, "width": width, "experts": experts, "align": align, "out": out,
         "mask": mask}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One decoded token: 256 experts on 8 ranks, at most 4 of them for a token.
        _gate("gate_one_token", 1, 256, 8, 4, 8, "bf16", "sigmoid", False, bias=True),
        # A ragged decode batch, 160 experts in groups of 20.
        _gate("gate_decode_333", 333, 160, 8, 3, 6, "fp32", "softmax", False),
        # A prefill of 16384 tokens.
        _gate("gate_prefill_16384", 16384, 256, 8, 4, 8, "bf16", "sigmoid", False, bias=True),
        # A training step on the largest batch, 5 % of the tokens padding.
        _gate("gate_train_65536", 65536, 256, 8, 4, 8, "fp32", "softmax", True, mask=0.05),
        # One decoded token between two layers: residual, rows for the router and fp8 rows for the dispatch.
        _norm("norm_one_token", 1, 7168, "both", True, "bf16"),
        # A ragged decode batch of a narrower model, straight to fp8.
        _norm("norm_333_fp8", 333, 4096, "fp8", True, "bf16"),
        # The 4096 x 7168 batch on its way into the layer.
        _norm("norm_4096", 4096, 7168, "both", True, "bf16"),
        # Its gradient, with the one that comes along the residual.
        _norm_grad("norm_grad_4096", 4096, 7168, True, "bf16"),
        # A ragged batch of an odd width, fp32 weights, nothing beside the norm.
        _norm_grad("norm_grad_8191", 8191, 2064, False, "fp32"),
        # A ragged micro-batch of 64 tokens less one on 32 experts.
        _combine_grad("combine_grad_63", 63, 8, 7168, 32, 1, "bf16"),
        # The 4096 x 7168 batch into the fp8 product of the down projection's gradient.
        _combine_grad("combine_grad_4096", 4096, 8, 7168, 256, 128, "fp8", mask=0.05),
        # A narrower, longer batch, bf16 rows.
        _combine_grad("combine_grad_8191", 8191, 6, 4096, 64, 16, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate", "norm", "norm", "norm_grad", "norm_grad", "combine_grad", "combine_grad"])
    if op == "gate":
        groups = rng.choice([2, 4, 8, 8, 16, 20])
        size = _log_int(rng, 2, 512 // groups)
        experts, taken = groups * size, rng.randint(1, max(1, groups // 2))
        tokens = _log_int(rng, 1, min(65536, 65536 * 256 // experts))
        scoring = rng.choice(["softmax", "sigmoid"])
        return _gate(None, tokens, experts, groups, taken, rng.randint(1, min(12, taken * size)), rng.choice(["bf16", "fp32"]),
                     scoring, rng.random() < 0.5, rng.choice([0.0, 0.05, 0.3]), scoring == "sigmoid" and rng.random() < 0.7)
    if op in ("norm", "norm_grad"):
        width = 16 * _log_int(rng, 8, 512)
        rows = _log_int(rng, 1, 4096 * 7168 // width)
        residual, weight = rng.random() < 0.7, rng.choice(["bf16", "bf16", "fp32"])
        if op == "norm":
            return _norm(None, rows, width, rng.choice(["bf16", "fp8", "both"]), residual, weight)
        return _norm_grad(None, rows, width, residual, weight)
    width, topk = 16 * _log_int(rng, 16, 448), rng.randint(1, 8)
    tokens = _log_int(rng, 1, min(16384, 4096 * 8 * 7168 // (width * topk)))
    return _combine_grad(None, tokens, topk, width, _log_int(rng, topk, 256), rng.choice([1, 16, 128]), rng.choice(["bf16", "fp8"]),
                         rng.choice([0.0, 0.05, 0.3]))


# -------------------------------------------------------------------- inputs


def _generator(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + stream)
    return g


def _normal(shape, seed, stream, dtype=torch.float32):
    return torch.randn(shape, generator=_generator(seed, stream), device="cuda", dtype=dtype)


def _uniform(shape, seed, stream):
    return torch.rand(shape, generator=_generator(seed, stream), device="cuda")


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(case, seed):
    op = case["op"]
    s = {"case": case}
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = (1.5 * _normal((t, e), seed, 0)).to(_type(case["dtype"]))
        s["bias"] = 0.1 * _normal((e,), seed, 1) if case["bias"] else None
        s["mask"] = _uniform((t,), seed, 2) >= case["mask"] if case["mask"] else None
        if case["train"]:
            s["grad_weights"] = _normal((t, k), seed, 3)
            s["grad_loss"] = 0.5 + _uniform((1,), seed, 4)
        s["scale"], s["coef"] = 2.5, 0.01
        return s
    if op in ("norm", "norm_grad"):
        r, w = case["rows"], case["width"]
        s["weight"] = (1.0 + 0.2 * _normal((w,), seed, 0)).to(_type(case["weight"]))
        # The residual stream grows with depth and has channels that stand out.
        spread = 2.0 * torch.exp(0.5 * _normal((w,), seed, 1))
        if op == "norm":
            s["x"] = _normal((r, w), seed, 2, torch.bfloat16)
            s["residual"] = (spread * _normal((r, w), seed, 3)).to(torch.bfloat16) if case["residual"] else None
        else:
            s["h"] = (spread * _normal((r, w), seed, 2)).to(torch.bfloat16)
            s["grad_y"] = _normal((r, w), seed, 3, torch.bfloat16)
            s["grad_h"] = _normal((r, w), seed, 4, torch.bfloat16) if case["residual"] else None
        return s
    t, k, w, e, a = case["tokens"], case["topk"], case["width"], case["experts"], case["align"]
    owner = torch.argsort(_uniform((t, e), seed, 0), dim=1)[:, :k].reshape(-1)
    if case["mask"]:
        owner = torch.where((_uniform((t,), seed, 1) >= case["mask"]).repeat_interleave(k), owner, e)
    count = torch.bincount(owner, minlength=e + 1)[:e]
    first = torch.cumsum((count + a - 1) // a * a, 0) - (count + a - 1) // a * a
    order = torch.argsort(owner, stable=True)
    before = torch.cumsum(count, 0) - count
    live = int(count.sum())
    of = owner[order[:live]]
    slot = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
    slot[order[:live]] = (first[of] + torch.arange(live, device="cuda") - before[of]).to(torch.int32)
    s["slot"], s["capacity"] = slot.view(t, k), t * k + e * (a - 1)
    score = torch.exp(_normal((t, k), seed, 2))
    s["weights"] = score / score.sum(1, keepdim=True)
    s["y"] = _normal((s["capacity"], w), seed, 3, torch.bfloat16)
    s["grad_out"] = _normal((t, w), seed, 4, torch.bfloat16)
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
                                    logits_dtype=s["logits"].dtype, route_scale=s["scale"], loss_coef=s["coef"])
            groups = M.make_gate_groups(case["groups"], case["groups_taken"], 1 if case["scoring"] == "softmax" else 2)
            s["out"] = M.alloc_gate(p, "cuda", balance=case["train"])
            s["plan"] = M.GroupedGatePlan(p, groups, s["logits"], s["out"], M.alloc_gate_workspace(p, "cuda"),
                                          select_bias=s["bias"], token_mask=s["mask"])
            if case["train"]:
                s["grad_logits"] = torch.empty_like(s["logits"])
                s["back"] = M.GateBackwardPlan(p, s["logits"], s["out"], s["grad_weights"], s["grad_loss"],
                                               s["grad_logits"], token_mask=s["mask"])
        return s
    if op == "norm":
        r, w = case["rows"], case["width"]
        s["h"] = new((r, w), torch.bfloat16) if case["residual"] else None
        s["y"] = new((r, w), torch.bfloat16) if case["out"] != "fp8" else None
        s["q"] = new((r, w), torch.float8_e4m3fn) if case["out"] != "bf16" else None
        s["sf"] = new((r, _ceil(w, BLOCK)), torch.float32) if case["out"] != "bf16" else None
        if own:
            import moe_token_dispatch_amd as M

            s["plan"] = M.RmsNormPlan(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], y=s["y"], q=s["q"], sf=s["sf"])
        return s
    if op == "norm_grad":
        r, w = case["rows"], case["width"]
        s["grad_x"], s["grad_weight"] = new((r, w), torch.bfloat16), new((w,), torch.float32)
        if own:
            import moe_token_dispatch_amd as M

            s["plan"] = M.RmsNormBackwardPlan(s["h"], s["weight"], s["grad_y"], EPS, s["grad_x"], grad_h=s["grad_h"],
                                              grad_weight=s["grad_weight"], workspace=M.alloc_rms_norm_workspace(r, w, "cuda"))
        return s
    t, k, w, rows = case["tokens"], case["topk"], case["width"], s["capacity"]
    s["grad_weights"] = new((t, k), torch.float32)
    s["grad_y"] = new((rows, w), torch.bfloat16) if case["out"] == "bf16" else None
    s["grad_q"] = new((rows, w), torch.float8_e4m3fn) if case["out"] == "fp8" else None
    s["grad_sf"] = new((rows, _ceil(w, BLOCK)), torch.float32) if case["out"] == "fp8" else None
    if own:
        import moe_token_dispatch_amd as M

        s["plan"] = M.CombineBackwardPlan(s["slot"], s["weights"], s["y"], s["grad_out"], grad_weights=s["grad_weights"],
                                          grad_y=s["grad_y"], grad_q=s["grad_q"], grad_sf=s["grad_sf"])
    return s


# --------------------------------------------------------------- plain forms


def _gate_plain(s):
    case = s["case"]
    t, e, k, groups = case["tokens"], case["experts"], case["topk"], case["groups"]
    z = s["logits"].float()
    if case["scoring"] == "softmax":
        x = torch.exp(z - z.amax(dim=1, keepdim=True))
        choice, score = z, x / x.sum(dim=1, keepdim=True)
        prob = score
        of_group = choice.view(t, groups, -1).amax(dim=2)
    else:
        score = 1.0 / (1.0 + torch.exp(-z))
        choice = score if s["bias"] is None else score + s["bias"]
        prob = score / score.sum(dim=1, keepdim=True)
        of_group = torch.topk(choice.view(t, groups, -1), 2, dim=2)[0].sum(dim=2)
    best = torch.sort(of_group, dim=1, descending=True, stable=True)[1][:, :case["groups_taken"]]
    taken = torch.zeros((t, groups), dtype=torch.bool, device="cuda").scatter_(1, best, True)
    choice = torch.where(torch.repeat_interleave(taken, e // groups, dim=1), choice, -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    picked = torch.gather(score, 1, idx)
    total = picked.sum(dim=1, keepdim=True)
    live = torch.ones((t,), dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    out_idx = torch.where(live[:, None], idx, -1)
    out_weights = torch.where(live[:, None], s["scale"] * picked / total, 0.0)
    if not case["train"]:
        return {"topk_idx": out_idx, "topk_weights": out_weights}
    count = (torch.zeros((t, e), dtype=torch.float32, device="cuda").scatter_(1, idx, 1.0) * live[:, None]).sum(dim=0)
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


def _norm_plain(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
    x = h.float()
    y = x * (1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)) * s["weight"].float()
    out = {"h": h} if s["residual"] is not None else {}
    if s["y"] is not None:
        out["y"] = y.to(torch.bfloat16)
    if s["q"] is not None:
        out["q"], out["sf"] = _quantize_plain(y)
    return out


def _norm_grad_plain(s):
    x, dy = s["h"].float(), s["grad_y"].float()
    r = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    unit, g = x * r, dy * s["weight"].float()
    dx = r * (g - unit * (g * unit).mean(dim=1, keepdim=True))
    if s["grad_h"] is not None:
        dx = dx + s["grad_h"].float()
    return {"grad_x": dx.to(torch.bfloat16), "grad_weight": (dy * unit).sum(dim=0)}


def _combine_grad_plain(s):
    slot = s["slot"].long()
    live, at = slot >= 0, slot.clamp_min(0)
    d = s["grad_out"].float()[:, None, :]
    dw = torch.where(live, (d * s["y"][at].float()).sum(dim=2), 0.0)
    rows = (s["weights"][:, :, None] * d)[live]
    if s["grad_y"] is not None:
        s["grad_y"][slot[live]] = rows.to(torch.bfloat16)
        return {"grad_weights": dw, "grad_y": s["grad_y"]}
    q, sf = _quantize_plain(rows)
    s["grad_q"].view(torch.uint8)[slot[live]] = q.view(torch.uint8)
    s["grad_sf"][slot[live]] = sf
    return {"grad_weights": dw, "grad_q": s["grad_q"], "grad_sf": s["grad_sf"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"gate": _gate_plain, "norm": _norm_plain, "norm_grad": _norm_grad_plain, "combine_grad": _combine_grad_plain}[op](s)
    s["plan"]()
    if op == "gate":
        out = s["out"]
        if not s["case"]["train"]:
            return {"topk_idx": out.topk_idx, "topk_weights": out.topk_weights}
        s["back"]()
        return {"topk_idx": out.topk_idx, "topk_weights": out.topk_weights, "expert_count": out.expert_count,
                "prob_sum": out.prob_sum, "loss": out.loss, "grad_logits": s["grad_logits"]}
    names = {"norm": ("h", "y", "q", "sf"), "norm_grad": ("grad_x", "grad_weight"),
             "combine_grad": ("grad_weights", "grad_y", "grad_q", "grad_sf")}[op]
    return {name: s[name] for name in names if s[name] is not None}


# --------------------------------------------------------------------- exact


def _order(values):
    """Each value's place in its row, largest first, of equal ones the lowest index first."""
    return torch.argsort(torch.argsort(values, dim=1, descending=True, stable=True), dim=1)


def _exact_gate(s):
    case = s["case"]
    t, e, k, groups = case["tokens"], case["experts"], case["topk"], case["groups"]
    size = e // groups
    z = s["logits"].double()
    # The choice is defined on fp32 values: the logits, or the sigmoid and its sums rounded to fp32.
    choice = s["logits"].float()
    if case["scoring"] == "sigmoid":
        choice = torch.sigmoid(choice)
        if s["bias"] is not None:
            choice = choice + s["bias"]
    score = torch.softmax(z, dim=1) if case["scoring"] == "softmax" else torch.sigmoid(z)
    group_score = torch.empty((t, groups), dtype=torch.float32, device="cuda")
    for g in range(groups):
        part = torch.sort(choice[:, g * size:(g + 1) * size], dim=1, descending=True)[0]
        group_score[:, g] = part[:, 0] if case["scoring"] == "softmax" else part[:, 0] + part[:, 1]
    open_group = _order(group_score) < case["groups_taken"]
    choice = choice.masked_fill(~open_group[:, torch.arange(e, device="cuda") // size], -math.inf)
    idx = torch.argsort(_order(choice), dim=1)[:, :k]
    denom = score.sum(1, keepdim=True)
    prob = score / denom
    live = s["mask"] if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device="cuda")
    picked = score.gather(1, idx)
    weights = s["scale"] * picked / picked.sum(1, keepdim=True) * live[:, None]
    if not case["train"]:
        return {"topk_idx": None, "topk_weights": weights}
    count = torch.bincount(idx[live].reshape(-1), minlength=e).double()
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


def _exact_scaled(x):
    """float64 rows over their scales, not rounded to 8 bits, and the scales."""
    r, w = x.shape
    block = torch.arange(w, device=x.device) // BLOCK
    top = torch.zeros((r, _ceil(w, BLOCK)), dtype=torch.float64, device=x.device)
    top.scatter_reduce_(1, block.expand(r, w), x.abs(), "amax")
    sf = top.clamp_min(AMAX_FLOOR) / FP8_MAX
    return x / sf[:, block], sf


def _exact_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.double() + s["residual"].double()).float().to(torch.bfloat16)  # defined on the rounded sum
    x = h.double()
    y = x * torch.rsqrt(x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS) * s["weight"].double()
    out = {}
    if s["residual"] is not None:
        out["h"] = s["x"].double() + s["residual"].double()
    if s["case"]["out"] != "fp8":
        out["y"] = y
    if s["case"]["out"] != "bf16":
        out["q"], out["sf"] = _exact_scaled(y)
    return out


def _exact_norm_grad(s):
    # dx_i = sum_j (dy_j w_j) d(x_j r)/dx_i, r = (sum x^2 / W + eps)^(-1/2), dr/dx_i = -r^3 x_i / W.
    x, dy = s["h"].double(), s["grad_y"].double()
    r = (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS) ** -0.5
    along = (dy * s["weight"].double() * x).sum(1, keepdim=True)
    dx = dy * s["weight"].double() * r - x * (r ** 3 * along / x.shape[1])
    if s["grad_h"] is not None:
        dx += s["grad_h"].double()
    return {"grad_x": dx, "grad_weight": (dy * x * r).sum(0)}


def _exact_combine_grad(s):
    case = s["case"]
    t, k, w = case["tokens"], case["topk"], case["width"]
    d = s["grad_out"].double()
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    fp8 = case["out"] == "fp8"
    rows = torch.zeros((s["capacity"], w), dtype=torch.float64, device="cuda")
    sf = torch.zeros((s["capacity"], _ceil(w, BLOCK)), dtype=torch.float64, device="cuda")
    for j in range(k):
        token = torch.nonzero(s["slot"][:, j] >= 0).view(-1)
        slot = s["slot"][token, j].long()
        dw[token, j] = torch.linalg.vecdot(d[token], s["y"][slot].double())
        row = s["weights"][token, j].double()[:, None] * d[token]
        if fp8:
            rows[slot], sf[slot] = _exact_scaled(row)
        else:
            rows[slot] = row
    return {"grad_weights": dw, "grad_q": rows, "grad_sf": sf} if fp8 else {"grad_weights": dw, "grad_y": rows}


def exact(case, seed):
    """The values that run() rounds to its outputs' types (8-bit ones in units of their scales)."""
    return {"gate": _exact_gate, "norm": _exact_norm, "norm_grad": _exact_norm_grad,
            "combine_grad": _exact_combine_grad}[case["op"]](_inputs(case, seed))


# ---------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        table = t * e * (2 if case["dtype"] == "bf16" else 4)
        small = t * k * 12 + (4 * e if case["bias"] else 0) + (t if case["mask"] else 0)
        if not case["train"]:
            return {"bytes": table + small, "flops": 10 * t * e}
        return {"bytes": 2 * table + small + 4 * t * k + 8 * e + 8, "flops": 22 * t * e}
    if op in ("norm", "norm_grad"):
        r, w = case["rows"], case["width"]
        weight = w * (2 if case["weight"] == "bf16" else 4)
        if op == "norm":
            a_row = 2 * w + (4 * w if case["residual"] else 0)
            a_row += {"bf16": 2 * w, "fp8": w + 4 * _ceil(w, BLOCK), "both": 3 * w + 4 * _ceil(w, BLOCK)}[case["out"]]
            return {"bytes": r * a_row + weight, "flops": 8 * r * w}
        return {"bytes": r * (6 * w + (2 * w if case["residual"] else 0)) + weight + 4 * w, "flops": 12 * r * w}
    t, k, w = case["tokens"], case["topk"], case["width"]
    live = (1.0 - case["mask"]) * t * k
    a_row = 2 * w + (2 * w if case["out"] == "bf16" else w + 4 * _ceil(w, BLOCK))
    return {"bytes": (1.0 - case["mask"]) * t * 2 * w + live * a_row + 12 * t * k, "flops": live * 4 * w}
