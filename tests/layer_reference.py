"""The gate, the quantisation and the experts' product from their definitions,
in float64 on the CPU. Test infrastructure; shares no code with the product."""

from __future__ import annotations

import math

import torch

FP8 = torch.float8_e4m3fn
AMAX_FLOOR = 2.0 ** -100


# ---------------------------------------------------------------------- gate


def gate(z, topk, sigmoid, normalize, scale, coef, bias=None, mask=None):
    """Per token, in float64: the choice, weights, shares, counts and loss."""
    z = z.double()
    t, e = z.shape
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    nothing = torch.isneginf(z)
    if sigmoid:
        score = torch.where(nothing, 0.0, torch.sigmoid(z))
        order = score + (0.0 if bias is None else bias.double())
        order = torch.where(nothing, -math.inf, order)
    else:
        score = torch.where(nothing.all(1, keepdim=True), 0.0, torch.softmax(z, dim=1))
        order = z.clone()
    order = torch.where(torch.isnan(order), -math.inf, order)
    idx = torch.full((t, topk), -1, dtype=torch.long)
    picked = torch.zeros((t, topk), dtype=torch.float64)
    for i in range(t):
        if not live[i]:
            continue
        left = sorted((x for x in range(e) if order[i, x] != -math.inf), key=lambda x: (-float(order[i, x]), x))[:topk]
        for j, x in enumerate(left):
            idx[i, j] = x
            picked[i, j] = score[i, x]
    total = picked.sum(1, keepdim=True)
    weights = scale * picked
    if normalize:
        weights = torch.where(total == 0, 0.0, weights / torch.where(total == 0, 1.0, total))
    denom = score.sum(1, keepdim=True)
    share = torch.where(denom == 0, 0.0, score / torch.where(denom == 0, 1.0, denom))
    n = int(live.sum())
    prob_sum = share[live].sum(0) if n else torch.zeros(e, dtype=torch.float64)
    count = torch.bincount(idx[idx >= 0], minlength=e)
    loss = coef * e / (topk * n * n) * float((count.double() * prob_sum).sum()) if n else 0.0
    return dict(idx=idx, weights=weights, prob_sum=prob_sum, count=count, live=n, loss=loss, order=order)


def gate_table(z, topk, sigmoid, normalize, scale, coef, bias=None, mask=None):
    """gate() for many tokens at once: a stable sort in place of a loop over them."""
    z = z.double()
    t, e = z.shape
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    nothing = torch.isneginf(z)
    if sigmoid:
        score = torch.where(nothing, 0.0, torch.sigmoid(z))
        order = torch.where(nothing, -math.inf, score + (0.0 if bias is None else bias.double()))
    else:
        score = torch.where(nothing.all(1, keepdim=True), 0.0, torch.softmax(z, dim=1))
        order = z.clone()
    order = torch.where(torch.isnan(order), -math.inf, order)
    best, idx = (x[:, :topk] for x in torch.sort(order, dim=1, descending=True, stable=True))
    idx = torch.where(torch.isneginf(best) | ~live[:, None], -1, idx)
    picked = torch.where(idx >= 0, score.gather(1, idx.clamp_min(0)), 0.0)
    total = picked.sum(1, keepdim=True)
    weights = scale * picked
    if normalize:
        weights = torch.where(total == 0, 0.0, weights / torch.where(total == 0, 1.0, total))
    denom = score.sum(1, keepdim=True)
    share = torch.where(denom == 0, 0.0, score / torch.where(denom == 0, 1.0, denom))
    n = int(live.sum())
    prob_sum = share[live].sum(0)
    count = torch.bincount(idx[idx >= 0], minlength=e)
    loss = coef * e / (topk * n * n) * float((count.double() * prob_sum).sum()) if n else 0.0
    return dict(idx=idx, weights=weights, prob_sum=prob_sum, count=count, live=n, loss=loss, order=order)


def gate_gradient(z, idx, count, sigmoid, normalize, scale, coef, dw, dloss, mask=None):
    """By automatic differentiation of the definition, the choice and the counts fixed."""
    z = z.double().clone().requires_grad_(True)
    t, e = z.shape
    k = idx.shape[1]
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    n = int(live.sum())
    total = torch.zeros((), dtype=torch.float64)
    for i in range(t):
        if not live[i] or bool(torch.isneginf(z[i]).all()):
            continue
        s = torch.sigmoid(z[i]) if sigmoid else torch.softmax(z[i], 0)
        took = idx[i] >= 0
        p = s[idx[i][took]]
        w = scale * (p / p.sum() if normalize else p)
        if dw is not None:
            total = total + (w * dw[i][took].double()).sum()
        if dloss is not None:
            share = s / s.sum() if e > 1 else torch.ones(1, dtype=torch.float64)  # a lone expert's share is constant
            total = total + float(dloss) * coef * e / (k * n * n) * (count.double() * share).sum()
    if not total.requires_grad:
        return torch.zeros_like(z)
    total.backward()
    return z.grad


# -------------------------------------------------------------- quantisation


def e4m3(v):
    """float64 values rounded to the nearest e4m3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def quantize(x):
    """float64 rows to (values in units of their scale before rounding, scales [R, blocks])."""
    r, w = x.shape
    nb = -(-w // 128)
    sf = torch.zeros((r, nb), dtype=torch.float64)
    v = torch.zeros_like(x)
    for b in range(nb):
        part = x[:, 128 * b:128 * b + 128]
        sf[:, b] = part.abs().amax(1).clamp_min(AMAX_FLOOR) / 448.0
        v[:, 128 * b:128 * b + 128] = part / sf[:, b:b + 1]
    return v, sf


def swiglu(h):
    g, u = torch.chunk(h.double(), 2, dim=1)
    return g * torch.sigmoid(g) * u


def swiglu_gradient(h, grad):
    h = h.double().clone().requires_grad_(True)
    swiglu(h).backward(grad.double())
    return h.grad


def assert_quantised(q, sf, x, rel):
    """fp8 values and fp32 scales of float64 rows x whose fp32 values the kernel
    had within `rel` of the block's largest magnitude: the scale within rel,
    each value within half an e4m3 step of the exact quotient, widened by rel
    of 448 for the value and of the quotient for the scale."""
    v, want_sf = quantize(x)
    got_sf = sf.double()
    assert torch.all((got_sf - want_sf).abs() <= rel * want_sf), "scales"
    got = q.double()
    half = torch.exp2(torch.floor(torch.log2(torch.maximum(v.abs(), got.abs()).clamp_min(2.0 ** -6))) - 3) / 2
    slack = rel * 448.0 + 2 * rel * v.abs()
    assert torch.all((got - v).abs() <= half + slack), "values"


# ------------------------------------------------------------------- product


def product(x, x_sf, w, w_sf, psum, count):
    """float64 [rows, N] with NaN in the rows no expert owns, the sum of
    magnitudes of each, and the sum over blocks of (x's largest) * (w's largest)."""
    rows, k = x.shape
    e, n, _ = w.shape
    kb = torch.arange(k) // 128
    nb = torch.arange(n) // 128
    out = torch.full((rows, n), math.nan, dtype=torch.float64)
    mag, top = torch.zeros((rows, n), dtype=torch.float64), torch.zeros((rows, n), dtype=torch.float64)
    for i in range(e):
        lo, c = int(psum[i]), int(count[i])
        if c == 0:
            continue
        xd = x[lo:lo + c].double() * x_sf[lo:lo + c].double()[:, kb]
        wd = w[i].double() * w_sf[i].double()[nb][:, kb]
        out[lo:lo + c] = xd @ wd.t()
        mag[lo:lo + c] = xd.abs() @ wd.abs().t()
        for b in range(-(-k // 128)):
            part = slice(128 * b, 128 * b + 128)
            top[lo:lo + c] += xd[:, part].abs().amax(1, keepdim=True) * wd[:, part].abs().amax(1)
    return out, mag, top
