"""The gate with expert groups, the RMS norm and the combine's gradient from
their definitions, in float64 on the CPU. Test infrastructure; shares no code
with the product."""

from __future__ import annotations

import math

import torch


# ---------------------------------------------------------------------- gate

# Choices below 2 in magnitude: a sigmoid within 2 units of 2^-24, the bias's
# addition and the pair's sum half a unit of 2^-23 each. What is further apart
# than this is in the same order in fp32.
NEAR = 8 * 2.0 ** -23


def grouped_choice(z, groups, taken, topk, sigmoid, pairs, bias=None, mask=None):
    """(idx [T, K], near [T]): the choice, -1 where nothing is left; whether fp32
    scores may decide it otherwise (two values that it compares are within NEAR
    and not of the same logits and biases). Equal sums of other operands count:
    (x + b) + y and x + (y + b) are one number, but round to two in fp32, each
    addition by up to 2^-24 of its result."""
    t, e = z.shape
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    choice = z.double()
    if sigmoid:
        choice = torch.where(torch.isneginf(choice), -math.inf, torch.sigmoid(choice))
        choice = choice + (0.0 if bias is None else bias.double())
    choice = torch.where(torch.isnan(choice), -math.inf, choice)
    made = torch.stack((z.double(), (z.new_zeros(e) if bias is None else bias).double().expand(t, e)), 2)  # of what
    made = torch.nan_to_num(made, nan=1e30)
    best, first = torch.sort(choice.view(t, groups, e // groups), dim=2, descending=True, stable=True)
    first = first[:, :, :2 if pairs else 1] + e // groups * torch.arange(groups)[:, None]
    parts = made.gather(1, first.flatten(1)[:, :, None].expand(-1, -1, 2)).view(t, groups, 2 * first.shape[2])
    marks = best[:, :, 0].clone()
    if pairs and best.shape[2] > 1:
        second = best[:, :, 1]
        marks = torch.where(torch.isneginf(second), marks, marks + second)
    value, order = torch.sort(marks, dim=1, descending=True, stable=True)
    opened = torch.zeros((t, groups), dtype=torch.bool)
    opened.scatter_(1, order[:, :taken], ~torch.isneginf(value[:, :taken]))
    inner = torch.where(opened.repeat_interleave(e // groups, 1), choice, -math.inf)
    most, full = torch.sort(inner, dim=1, descending=True, stable=True)
    idx = torch.where(torch.isneginf(most[:, :topk]) | ~live[:, None], -1, full[:, :topk])
    near = torch.zeros(t, dtype=torch.bool)
    if sigmoid:
        # (Of what is taken against all that is left: between a value and another's
        # there may be equals of the first.)
        gap = lambda a, b, of, to: ((of != to).any(-1) & ((a - b).abs() <= NEAR)).any(1)  # noqa: E731
        if taken < groups:
            rank = parts.gather(1, order[:, :, None].expand_as(parts))
            cut = slice(taken - 1, taken), slice(taken, taken + 1)
            near |= gap(value[:, cut[0]], value[:, taken:], rank[:, cut[0]], rank[:, taken:])
            near |= gap(value[:, :taken], value[:, cut[1]], rank[:, :taken], rank[:, cut[1]])
        rank = made.gather(1, full[:, :, None].expand_as(made))
        near |= gap(most[:, :topk - 1], most[:, 1:topk], rank[:, :topk - 1], rank[:, 1:topk])
        near |= gap(most[:, topk - 1:topk], most[:, topk:], rank[:, topk - 1:topk], rank[:, topk:])
    return idx, near & live


def gate_outputs(z, idx, sigmoid, normalize, scale, coef, mask=None):
    """Weights, probability sums, counts and loss of a choice."""
    z = z.double()
    t, e = z.shape
    k = idx.shape[1]
    live = torch.ones(t, dtype=torch.bool) if mask is None else mask.bool()
    nothing = torch.isneginf(z)
    if sigmoid:
        score = torch.where(nothing, 0.0, torch.sigmoid(z))
    else:
        score = torch.where(nothing.all(1, keepdim=True), 0.0, torch.softmax(z, dim=1))
    picked = torch.where(idx >= 0, score.gather(1, idx.clamp_min(0)), 0.0)
    weights = scale * picked
    if normalize:
        total = picked.sum(1, keepdim=True)
        weights = torch.where(total == 0, 0.0, weights / torch.where(total == 0, 1.0, total))
    denom = score.sum(1, keepdim=True)
    share = torch.where(denom == 0, 0.0, score / torch.where(denom == 0, 1.0, denom))
    n = int(live.sum())
    prob_sum = share[live].sum(0)
    count = torch.bincount(idx[idx >= 0], minlength=e)
    loss = coef * e / (k * n * n) * float((count.double() * prob_sum).sum()) if n else 0.0
    return dict(weights=weights, prob_sum=prob_sum, count=count, live=n, loss=loss)


# ------------------------------------------------------------------ RMS norm


def rounded_sum(x, residual):
    """bf16 h of bf16 rows: the sum in fp32, rounded once more."""
    return x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)


def rms_norm(h, weight, eps):
    h = h.double()
    return h * (h.pow(2).mean(1, keepdim=True) + eps).rsqrt() * weight.double()


def rms_norm_gradient(h, weight, grad_y, eps, grad_h=None):
    """(grad_x, grad_weight) by automatic differentiation of the definition."""
    h, w = h.double().clone().requires_grad_(True), weight.double().clone().requires_grad_(True)
    (rms_norm(h, w, eps) * grad_y.double()).sum().backward()
    return h.grad + (0.0 if grad_h is None else grad_h.double()), w.grad


# ------------------------------------------------------- combine's gradient


def combine_gradient(slot, weights, y, grad_out):
    """(grad_weights [T, K], the sums of their terms' magnitudes, grad_y [rows, H] with NaN in the rows no entry has)."""
    t, k = slot.shape
    rows, width = y.shape
    dw, size = torch.zeros((t, k), dtype=torch.float64), torch.zeros((t, k), dtype=torch.float64)
    dy = torch.full((rows, width), math.nan, dtype=torch.float64)
    for i in range(t):
        for j in range(k):
            s = int(slot[i, j])
            if not 0 <= s < rows:
                continue
            terms = grad_out[i].double() * y[s].double()
            dw[i, j], size[i, j] = terms.sum(), terms.abs().sum()
            dy[s] = float(weights[i, j]) * grad_out[i].double()
    return dw, size, dy
