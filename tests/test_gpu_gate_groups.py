"""The gate with expert groups against its definition in float64."""

import math

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import block_reference as R
from tests import layer_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# As the gate's: exp, a division and sums of up to 4096 terms, a few dozen roundings of 2^-24.
REL = 64 * 2.0 ** -24
FIELDS = ("topk_idx", "topk_weights", "expert_count", "prob_sum", "live_tokens", "loss")


def _logits(t, e, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((t, e), generator=g)).to(dtype)


def _run(z, groups, taken, topk, sigmoid, pairs, normalize=True, scale=1.0, coef=0.01, bias=None, mask=None, idx_bytes=8,
         balance=True):
    p = M.make_gate_problem(*z.shape, topk, M.GATE_SIGMOID if sigmoid else M.GATE_SOFTMAX, z.dtype, normalize, scale, coef,
                            idx_bytes)
    out = M.alloc_gate(p, DEV, balance=balance)
    for f in FIELDS:
        if getattr(out, f) is not None:
            getattr(out, f).fill_(77)
    ws = M.alloc_gate_workspace(p, DEV)
    ws.fill_(0xA5)
    to = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    M.dispatch_gate_grouped(p, M.make_gate_groups(groups, taken, 2 if pairs else 1), to(z), out, ws, select_bias=to(bias),
                            token_mask=to(mask))
    torch.cuda.synchronize()
    return p, out


def _check(z, groups, taken, topk, sigmoid, pairs, normalize=True, scale=1.0, coef=0.01, bias=None, mask=None, **kw):
    """The choice, and what follows from the choice that was made."""
    p, out = _run(z, groups, taken, topk, sigmoid, pairs, normalize, scale, coef, bias, mask, **kw)
    idx = out.topk_idx.cpu().long()
    want, near = R.grouped_choice(z, groups, taken, topk, sigmoid, pairs, bias, mask)
    assert torch.equal(idx[~near], want[~near])
    assert int(near.sum()) <= 1 + z.shape[0] // 50  # (they say nothing: few are left out)
    took = idx >= 0
    assert torch.equal(took, want >= 0)
    assert torch.all(torch.sort(torch.where(took, idx, -1 - torch.arange(topk)), dim=1)[0].diff(dim=1) != 0)  # no expert twice
    of = torch.where(took, idx.clamp_min(0) // (z.shape[1] // groups), 0)
    used = torch.zeros((z.shape[0], groups)).scatter_add_(1, of, took.float())
    assert torch.all((used > 0).sum(1) <= taken)
    ref = R.gate_outputs(z, idx, sigmoid, normalize, scale, coef, mask)
    w = out.topk_weights.cpu().double()
    assert torch.all((w - ref["weights"]).abs() <= REL * (ref["weights"].abs() + abs(scale) * 2.0 ** -20))
    if out.loss is not None:
        assert torch.equal(out.expert_count.cpu().long(), ref["count"]) and int(out.live_tokens) == ref["live"]
        assert torch.all((out.prob_sum.cpu().double() - ref["prob_sum"]).abs() <= REL * (ref["prob_sum"] + 2.0 ** -60))
        assert abs(float(out.loss) - ref["loss"]) <= 2 * REL * abs(ref["loss"])
    return p, out


# Tokens, experts, groups, groups taken, entries: every number of registers per lane, groups of one
# expert and of many, odd sizes, as many entries as the taken groups have experts, batches either
# side of each form's.
SHAPES = [(1, 256, 8, 4, 8), (33, 160, 8, 3, 6), (257, 72, 8, 2, 5), (40, 4096, 64, 5, 32), (64, 1000, 20, 3, 12),
          (50, 7, 7, 3, 3), (40, 64, 2, 1, 8), (20, 2048, 16, 4, 8), (31, 600, 3, 2, 1), (100, 63, 21, 2, 6),
          (64, 96, 6, 1, 16), (17, 130, 2, 1, 9), (48, 1026, 54, 7, 8), (9, 64, 64, 6, 6), (70, 252, 63, 62, 8),
          (300, 200, 5, 2, 8), (8192, 256, 8, 4, 8), (8193, 132, 33, 5, 6), (16385, 65, 5, 2, 4), (20000, 256, 64, 9, 7),
          (8200, 128, 16, 1, 8), (8200, 250, 10, 4, 8), (8192, 160, 8, 3, 6), (8192, 252, 9, 4, 1), (8195, 192, 3, 2, 2),
          (8193, 180, 15, 6, 8), (8194, 200, 5, 1, 7), (8197, 256, 2, 1, 8), (8191, 256, 16, 7, 8), (8192, 68, 17, 5, 4),
          (8201, 72, 6, 5, 3), (8199, 76, 1, 1, 8), (8192, 64, 8, 3, 8), (8200, 32, 8, 3, 4), (8193, 16, 4, 2, 8),
          (8195, 8, 2, 1, 4), (8200, 60, 15, 4, 8), (8201, 48, 12, 6, 1), (9000, 20, 5, 2, 8), (8192, 64, 2, 1, 9),
          (8192, 64, 16, 9, 8), (8197, 12, 3, 2, 8), (16384, 512, 16, 4, 8), (16387, 260, 13, 4, 4),
          (16390, 384, 8, 3, 5), (16385, 264, 3, 2, 6), (16384, 508, 1, 1, 7), (16384, 500, 5, 1, 8)]


@pytest.mark.parametrize("t,e,groups,taken,topk", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "pairs"])
def test_shapes(t, e, groups, taken, topk, scoring):
    for dtype in (torch.bfloat16, torch.float32):
        z = _logits(t, e, dtype, t + e)
        bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(e)) if scoring == "pairs" else None
        mask = torch.rand(t, generator=torch.Generator().manual_seed(t)) > 0.1
        mask = mask if dtype == torch.float32 else None
        _check(z, groups, taken, topk, scoring != "softmax", scoring == "pairs", scale=2.5, bias=bias, mask=mask)


@pytest.mark.parametrize("t", [0, 1, 2, 3, 33, 5000])
@pytest.mark.parametrize("balance", [False, True])
def test_token_counts(t, balance):
    z = _logits(t, 64, torch.bfloat16, 5 + t)
    _check(z, 4, 2, 6, True, True, normalize=False, idx_bytes=4, balance=balance)


@pytest.mark.parametrize("t", [8200, 16400])
@pytest.mark.parametrize("balance", [False, True])
def test_large_batches_in_every_output(t, balance):
    z = _logits(t, 120, torch.float32, t)
    mask = torch.ones(t, dtype=torch.bool)
    mask[5:8000] = False
    for groups, taken, topk in ((6, 2, 8), (24, 3, 12), (40, 30, 3)):
        _check(z, groups, taken, topk, True, True, normalize=False, scale=-1.5, idx_bytes=4, balance=balance, mask=mask)
        _, out = _run(z, groups, taken, topk, False, False, mask=torch.zeros(t, dtype=torch.bool), balance=balance)
        assert torch.all(out.topk_idx == -1) and torch.all(out.topk_weights == 0)


@pytest.mark.parametrize("t", [8191, 8195, 16384])
@pytest.mark.parametrize("e,groups,taken,topk", [(512, 16, 4, 8), (260, 13, 3, 4), (384, 8, 4, 6), (320, 4, 1, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "pairs"])
def test_many_experts_with_ties_and_nothing_to_take(t, e, groups, taken, topk, scoring):
    z = (2.0 * _logits(t, e, torch.float32, t + e)).round() / 2.0
    z[0] = -math.inf
    z[1, e // groups:] = -math.inf
    z[2, :e - 1] = -math.inf
    z[3] = 0.0
    z[4, ::3] = -math.inf
    bias = None
    if scoring == "pairs":
        bias = (0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e))).round(decimals=1)
        bias[e // groups + 1] = -math.inf
    mask = torch.arange(t) % 7 != 6
    for balance in (False, True):
        _, out = _check(z, groups, taken, topk, scoring != "softmax", scoring == "pairs", scale=2.5, bias=bias, mask=mask,
                        balance=balance)
        idx = out.topk_idx.cpu()
        assert torch.all(idx[0] == -1) and idx[2, 0] == e - 1 and torch.all(idx[2, 1:] == -1) and torch.all(idx[6] == -1)


@pytest.mark.parametrize("t", [300, 9000])
def test_ties_go_to_the_lowest_group_and_expert(t):
    # Logits from a handful of values: groups and experts tie in every row.
    z = torch.randint(-2, 3, (t, 96), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    z[0] = 0.0
    for groups, taken in ((8, 3), (24, 5), (48, 4)):
        for sigmoid, pairs in ((False, False), (True, False), (True, True)):
            _, out = _check(z, groups, taken, 5, sigmoid, pairs)
            assert out.topk_idx[0].tolist() == [0, 1, 2, 3, 4]
    # The sums of two pairs of different values never tie here; the best pair may be two equal ones.
    z[1], z[1, 7], z[1, 8:10] = -5.0, 2.0, 1.0
    _, out = _run(z, 12, 1, 5, True, True)
    assert out.topk_idx[1].tolist() == [8, 9, 10, 11, 12]
    _, out = _run(z, 12, 1, 5, True, False)
    assert out.topk_idx[1].tolist() == [7, 0, 1, 2, 3]


@pytest.mark.parametrize("t", [40, 8200])
def test_rows_and_groups_with_nothing_to_take(t):
    z = _logits(t, 80, torch.float32, 17)
    z[0] = -math.inf
    z[1, 10:] = -math.inf          # one group of eight
    z[2, :79] = -math.inf          # a lone expert
    z[3, ::10] = -math.inf
    z[4] = torch.finfo(torch.float32).min
    z[5, 11:], z[5, 1:10] = -math.inf, -math.inf   # two lone experts in two groups
    for sigmoid, pairs in ((False, False), (True, False), (True, True)):
        _, out = _check(z, 8, 3, 6, sigmoid, pairs)
        idx = out.topk_idx.cpu()
        assert torch.all(idx[0] == -1) and torch.all(idx[1] < 10) and idx[2].tolist() == [79] + [-1] * 5
        assert sorted(idx[5].tolist()) == [-1, -1, -1, -1, 0, 10]
        assert torch.all(torch.isfinite(out.topk_weights)) and math.isfinite(float(out.loss))


@pytest.mark.parametrize("t", [24, 8200])
def test_bias_closes_experts_and_groups(t):
    z = _logits(t, 64, torch.float32, 19)
    bias = torch.zeros(64)
    bias[8:16] = -math.inf     # a group of eight that is gone
    bias[20] = math.nan
    bias[32:40] = 3.0          # one that is always taken
    _, out = _check(z, 8, 2, 8, True, True, bias=bias)
    idx = out.topk_idx.cpu()
    assert not torch.any((idx >= 8) & (idx < 16)) and not torch.any(idx == 20)
    assert torch.all((idx[:, 0] >= 32) & (idx[:, 0] < 40))
    # Sums past fp32's range: -inf is still something to take, +inf the most there is.
    bias = torch.full((64,), -3e38)
    _, out = _run(z, 8, 2, 8, True, True, bias=bias)
    assert torch.all(out.topk_idx >= 0) and torch.all(out.topk_idx < 16)  # all groups alike
    bias[40:48] = 3e38
    _, out = _run(z, 8, 1, 8, True, True, bias=bias)
    assert torch.all((out.topk_idx >= 40) & (out.topk_idx < 48))


@pytest.mark.parametrize("t", [6, 8200])
def test_nan_and_infinite_logits(t):
    z = _logits(t, 64, torch.float32, 23)
    z[1, 5] = math.nan
    z[2] = math.nan
    z[3, 50] = math.inf
    for sigmoid, pairs in ((False, False), (True, False), (True, True)):
        _, out = _run(z, 8, 2, 6, sigmoid, pairs)
        idx = out.topk_idx.cpu()
        assert not torch.any(idx[1] == 5) and torch.all(idx[1] >= 0) and torch.all(idx[2] == -1)
        assert math.isnan(float(out.loss)) and torch.all(torch.isfinite(out.topk_weights[0]))
        if not sigmoid:
            assert int(idx[3, 0]) == 50


@pytest.mark.parametrize("t,e,k", [(50, 96, 7), (8192, 256, 8), (16384, 128, 5)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_all_groups_are_the_gate(t, e, k, sigmoid):
    z = _logits(t, e, torch.float32, 29).to(DEV)
    bias = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(1)).to(DEV) if sigmoid else None
    p = M.make_gate_problem(t, e, k, M.GATE_SIGMOID if sigmoid else M.GATE_SOFTMAX, z.dtype, loss_coef=0.5)
    a, b, ws = M.alloc_gate(p, DEV), M.alloc_gate(p, DEV), M.alloc_gate_workspace(p, DEV)
    M.dispatch_gate(p, z, a, ws, select_bias=bias)
    for groups in (1, 4, 32):
        M.dispatch_gate_grouped(p, M.make_gate_groups(groups, groups), z, b, ws, select_bias=bias)
        assert all(torch.equal(getattr(a, f), getattr(b, f)) for f in FIELDS)


@pytest.mark.parametrize("t,e,groups,taken,k", [(64, 256, 8, 4, 8), (9000, 256, 8, 4, 8), (9000, 72, 6, 2, 4),
                                                 (17000, 512, 16, 4, 8), (17000, 272, 4, 2, 4)])
@pytest.mark.parametrize("pairs", [False, True])
def test_forms_agree(t, e, groups, taken, k, pairs):
    """Rows choose alike in batches of every form, with and without balance outputs, and every time."""
    z = _logits(t, e, torch.bfloat16, 31)
    bias = (0.05 * torch.randn(e, generator=torch.Generator().manual_seed(2))).round(decimals=2) if pairs else None
    _, a = _run(z, groups, taken, k, pairs, pairs, bias=bias)
    for balance in (True, False):
        _, b = _run(z, groups, taken, k, pairs, pairs, bias=bias, balance=balance)
        assert torch.equal(a.topk_idx, b.topk_idx)
        if balance:
            assert all(torch.equal(getattr(a, f), getattr(b, f)) for f in FIELDS)
    few = torch.arange(0, t, t // 60)
    _, b = _run(z[few], groups, taken, k, pairs, pairs, bias=bias)
    assert torch.equal(a.topk_idx.cpu()[few], b.topk_idx.cpu())


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient(sigmoid):
    """dispatch_gate_backward takes the grouped gate's outputs."""
    t, e, k = 40, 48, 5
    z = _logits(t, e, torch.float32, 37)
    p, out = _run(z, 6, 2, k, sigmoid, sigmoid, True, 2.0, 0.5)
    g = torch.Generator().manual_seed(4)
    dw, dloss = torch.randn((t, k), generator=g), torch.tensor([1.3])
    dz = torch.empty_like(z, device=DEV)
    M.dispatch_gate_backward(p, z.to(DEV), out, dw.to(DEV), dloss.to(DEV), dz)
    want = layer_reference.gate_gradient(z, out.topk_idx.cpu(), out.expert_count.cpu(), sigmoid, True, 2.0, 0.5, dw, dloss)
    size = 2.0 * dw.abs().amax() + want.abs().amax()
    assert torch.all((dz.cpu().double() - want).abs() <= REL * want.abs() + 8 * REL * size)


def test_unaligned_rows_and_what_lies_beside():
    t, e = 19, 255
    z = torch.randint(-3, 4, (t, e), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    flat = torch.full((t * e + 2,), math.nan, dtype=z.dtype, device=DEV)
    flat[1:-1] = z.view(-1).to(DEV)
    p = M.make_gate_problem(t, e, 8, M.GATE_SOFTMAX, z.dtype)
    out = M.alloc_gate(p, DEV)
    idx = torch.full((t + 2, 8), 99, dtype=torch.int64, device=DEV)
    out.topk_idx = idx[1:-1]
    M.dispatch_gate_grouped(p, M.make_gate_groups(17, 4), flat[1:-1].view(t, e), out, M.alloc_gate_workspace(p, DEV))
    want, _ = R.grouped_choice(z, 17, 4, 8, False, False)
    assert torch.equal(out.topk_idx.cpu(), want)
    assert torch.all(idx[0] == 99) and torch.all(idx[-1] == 99)


def test_plans_streams_and_a_graph():
    t, e, k = 300, 160, 6
    groups = M.make_gate_groups(8, 3)
    p = M.make_gate_problem(t, e, k, M.GATE_SOFTMAX, torch.float32, loss_coef=0.1)
    batches = [_logits(t, e, torch.float32, 50 + i).to(DEV) for i in range(4)]
    eager = []
    for z in batches:
        out = M.alloc_gate(p, DEV)
        M.dispatch_gate_grouped(p, groups, z, out, M.alloc_gate_workspace(p, DEV))
        eager.append(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # Two calls at once, each with its own outputs and workspace.
    outs = [M.alloc_gate(p, DEV) for _ in range(2)]
    M.GroupedGatePlan(p, groups, batches[0], outs[0], M.alloc_gate_workspace(p, DEV))()
    M.GroupedGatePlan(p, groups, batches[1], outs[1], M.alloc_gate_workspace(p, DEV), stream=side)()
    torch.cuda.synchronize()
    for a, b in zip(outs, eager):
        assert all(torch.equal(getattr(a, f), getattr(b, f)) for f in FIELDS)
    with torch.cuda.stream(side):
        z, out = batches[0].clone(), M.alloc_gate(p, DEV)
        plan = M.GroupedGatePlan(p, groups, z, out, M.alloc_gate_workspace(p, DEV))
        graph = torch.cuda.CUDAGraph()
        plan()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            plan()
    for _ in range(2):
        for batch, want in zip(batches, eager):
            z.copy_(batch)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(getattr(out, f), getattr(want, f)) for f in FIELDS)
            M.dispatch_gate_grouped(p, groups, batches[0], outs[0], M.alloc_gate_workspace(p, DEV))  # eager work in between


def test_binding_refuses_wrong_tensors():
    p = M.make_gate_problem(10, 20, 4, M.GATE_SIGMOID, torch.float32, loss_coef=1.0)
    z, out, ws = torch.zeros((10, 20), device=DEV), M.alloc_gate(p, DEV), M.alloc_gate_workspace(p, DEV)
    good = M.make_gate_groups(4, 2)
    for bad in (z.cpu(), z.to(torch.bfloat16), z[:9], z.t()):
        with pytest.raises(ValueError, match="logits"):
            M.dispatch_gate_grouped(p, good, bad, out, ws)
    with pytest.raises(ValueError, match="select_bias"):
        M.dispatch_gate_grouped(p, good, z, out, ws, select_bias=torch.zeros(19, device=DEV))
    for groups in (M.make_gate_groups(3, 1), M.make_gate_groups(10, 1), M.make_gate_groups(4, 5)):
        with pytest.raises(M.DispatchError):
            M.dispatch_gate_grouped(p, groups, z, out, ws)
    with pytest.raises(M.DispatchError):
        M.dispatch_gate_grouped(p, good, z, out, ws[:256])


# Four tokens per wavefront with two groups a lane, and entries past the eighth in live rows of every scoring.
@pytest.mark.parametrize("t,e,groups,taken,topk", [(8193, 40, 20, 7, 2), (8200, 60, 20, 5, 12), (8195, 32, 32, 9, 6),
                                                   (8200, 128, 8, 3, 12)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "pairs"])
def test_many_groups_and_entries_of_few_experts(t, e, groups, taken, topk, scoring):
    test_shapes(t, e, groups, taken, topk, scoring)
