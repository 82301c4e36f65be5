"""The gate and its gradient against their definitions in float64."""

import math

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import layer_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# fp32 arithmetic: exp, a division and sums of up to 4096 terms leave a
# relative error of a few dozen roundings of 2^-24.
REL = 64 * 2.0 ** -24
# A bf16 result adds half a unit of its 8 bits.
BF16 = 2.0 ** -8


def _logits(t, e, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((t, e), generator=g)).to(dtype)


def _run(z, topk, sigmoid, normalize=True, scale=1.0, coef=0.01, bias=None, mask=None, idx_bytes=8, balance=True):
    t, e = z.shape
    p = M.make_gate_problem(t, e, topk, M.GATE_SIGMOID if sigmoid else M.GATE_SOFTMAX, z.dtype, normalize, scale, coef,
                            idx_bytes)
    out = M.alloc_gate(p, DEV, balance=balance)
    for v in (out.topk_idx, out.topk_weights, out.expert_count, out.prob_sum, out.live_tokens, out.loss):
        if v is not None:
            v.fill_(77)
    ws = M.alloc_gate_workspace(p, DEV)
    ws.fill_(0xA5)
    to = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    M.dispatch_gate(p, to(z), out, ws, select_bias=to(bias), token_mask=to(mask))
    torch.cuda.synchronize()
    return p, out


def _check(z, topk, sigmoid, normalize=True, scale=1.0, coef=0.01, bias=None, mask=None, idx_bytes=8, exact_choice=True):
    p, out = _run(z, topk, sigmoid, normalize, scale, coef, bias, mask, idx_bytes)
    ref = R.gate(z, topk, sigmoid, normalize, scale, coef, bias, mask)
    idx = out.topk_idx.cpu().long()
    if exact_choice:
        assert torch.equal(idx, ref["idx"])
    else:
        # fp32 scores may order two experts otherwise only where they are
        # within the scores' rounding of each other.
        a = torch.where(idx >= 0, ref["order"].gather(1, idx.clamp_min(0)), 0.0)
        b = torch.where(ref["idx"] >= 0, ref["order"].gather(1, ref["idx"].clamp_min(0)), 0.0)
        assert torch.equal(idx < 0, ref["idx"] < 0)
        assert torch.all((a - b).abs() <= 8 * 2.0 ** -24 * (1 + b.abs()))
        for row in idx.tolist():
            took = [x for x in row if x >= 0]
            assert len(set(took)) == len(took)
    w = out.topk_weights.cpu().double()
    assert torch.all((w - ref["weights"]).abs() <= REL * (ref["weights"].abs() + scale * 2.0 ** -20))
    if exact_choice:
        assert torch.equal(out.expert_count.cpu().long(), ref["count"])
    assert int(out.expert_count.sum()) == int((idx >= 0).sum())
    assert int(out.live_tokens) == ref["live"]
    assert torch.all((out.prob_sum.cpu().double() - ref["prob_sum"]).abs() <= REL * (ref["prob_sum"] + 2.0 ** -60))
    assert abs(float(out.loss) - ref["loss"]) <= 2 * REL * abs(ref["loss"]) + (0 if exact_choice else 1e-3 * ref["loss"])
    return p, out, ref


# Experts: one, fewer than a wavefront, either side of each step of the
# registers per lane; tokens either side of a workgroup's wavefronts.
@pytest.mark.parametrize("e", [1, 5, 63, 64, 65, 128, 129, 256, 257, 600, 1025, 4096])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_every_expert_count(e, sigmoid):
    k = min(e, 8)
    z = _logits(33, e, torch.float32, 100 + e)
    _check(z, k, sigmoid, exact_choice=not sigmoid)


@pytest.mark.parametrize("t", [0, 1, 2, 15, 16, 17, 257, 5000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_token_count(t, dtype):
    z = _logits(t, 64, dtype, 7 + t)
    p, out, ref = _check(z, 4, False, idx_bytes=4, scale=2.5)
    if t == 0:
        assert float(out.loss) == 0.0 and int(out.live_tokens) == 0


@pytest.mark.parametrize("k", [1, 2, 31, 32])
@pytest.mark.parametrize("normalize", [True, False])
def test_topk_widths(k, normalize):
    z = _logits(40, 32, torch.float32, 3)
    _check(z, k, False, normalize=normalize, scale=1.5)
    _check(z, k, True, normalize=normalize, scale=1.5, exact_choice=False)


def test_ties_go_to_the_lowest_expert():
    # bf16 logits from a handful of values: every row is full of ties.
    g = torch.Generator().manual_seed(5)
    z = torch.randint(-2, 3, (200, 300), generator=g).to(torch.bfloat16)
    z[0] = 0.0
    z[1, ::2] = -0.0  # equal to 0
    z[1, 1::2] = 0.0
    _check(z, 8, False)
    _check(z, 8, True)


def test_selection_bias_moves_the_choice_only():
    z = _logits(64, 96, torch.float32, 9)
    bias = torch.zeros(96)
    bias[10] = 5.0
    bias[20] = -math.inf  # never taken
    bias[30] = math.nan   # never taken
    p, out, ref = _check(z, 6, True, bias=bias, exact_choice=False)
    idx = out.topk_idx.cpu()
    assert torch.all(idx[:, 0] == 10)
    assert not torch.any((idx == 20) | (idx == 30))


def test_masked_tokens_count_nowhere():
    z = _logits(100, 40, torch.bfloat16, 11)
    mask = torch.rand(100, generator=torch.Generator().manual_seed(1)) > 0.4
    mask[:3] = torch.tensor([False, True, False])
    for m in (mask, mask.to(torch.uint8)):
        _check(z, 4, False, mask=m)
        _check(z, 4, True, mask=m, exact_choice=False)
    p, out, _ = _check(z, 4, False, mask=torch.zeros(100, dtype=torch.bool))
    assert float(out.loss) == 0.0 and int(out.live_tokens) == 0 and torch.all(out.topk_idx == -1)


def test_masked_experts():
    """-inf logits are never taken; what is left over of a token is -1 with weight 0."""
    z = _logits(20, 70, torch.float32, 13)
    z[0] = -math.inf
    z[1, 3:] = -math.inf
    z[2, :] = -math.inf
    z[2, 69] = 1.0
    z[3, ::2] = -math.inf
    low = torch.finfo(torch.float32).min
    z[4] = low              # the type's lowest value is a value: an even row
    z[5, 2:] = low
    for sigmoid in (False, True):
        for normalize in (False, True):
            p, out, ref = _check(z, 5, sigmoid, normalize=normalize, exact_choice=not sigmoid)
            idx = out.topk_idx.cpu()
            assert torch.all(idx[0] == -1) and torch.all(idx[1] >= -1) and int((idx[1] >= 0).sum()) == 3
            assert idx[2].tolist() == [69, -1, -1, -1, -1]
            assert torch.all(torch.isfinite(out.topk_weights)) and math.isfinite(float(out.loss))


def test_nan_shows_and_is_never_taken():
    z = _logits(4, 70, torch.float32, 17)
    z[1, 5] = math.nan
    z[2] = math.nan
    for sigmoid in (False, True):
        p, out = _run(z, 4, sigmoid)
        idx = out.topk_idx.cpu()
        assert not torch.any(idx[1] == 5) and torch.all(idx[1] >= 0) and torch.all(idx[2] == -1)
        assert math.isnan(float(out.loss))
        assert torch.all(torch.isfinite(out.topk_weights[0])) and torch.all(torch.isfinite(out.topk_weights[3]))
        if not sigmoid:
            assert torch.all(torch.isnan(out.topk_weights[1]))


def test_without_balance_outputs_the_same_table():
    z = _logits(777, 200, torch.bfloat16, 19)
    _, a = _run(z, 8, True)
    _, b = _run(z, 8, True, balance=False)
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)


def test_results_repeat_bit_for_bit():
    z = _logits(20000, 256, torch.float32, 23)
    first = None
    for _ in range(3):
        _, out = _run(z, 8, True)
        got = [out.topk_idx.clone(), out.topk_weights.clone(), out.prob_sum.clone(), out.loss.clone()]
        if first is not None:
            assert all(torch.equal(x, y) for x, y in zip(first, got))
        first = got


def test_sigmoid_scores_equal_torch_elementwise():
    """The score that the choice compares is torch's 1 / (1 + exp(-z)) for every bf16 logit."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    z = z[: z.numel() // 32 * 32].view(-1, 32)
    _, out = _run(z, 32, True, normalize=False, balance=False)
    want = 1.0 / (1.0 + torch.exp(-z.to(DEV).float()))
    assert torch.equal(out.topk_weights, want.gather(1, out.topk_idx))


def _gradient(p, z, out, dw, dloss, mask=None):
    dz = torch.full(z.shape, 77.0, dtype=z.dtype, device=DEV)
    to = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    M.dispatch_gate_backward(p, to(z), out, to(dw), to(dloss), dz, token_mask=to(mask))
    torch.cuda.synchronize()
    return dz.cpu().double()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e,k", [(1, 1), (7, 3), (64, 8), (130, 6), (300, 32)])
def test_gradient_matches_the_definition(sigmoid, normalize, dtype, e, k):
    t = 21
    z = _logits(t, e, dtype, 31 + e)
    z[3, e // 2:] = -math.inf if e > 1 else 0.0
    mask = torch.ones(t, dtype=torch.bool)
    mask[5] = False
    p, out = _run(z, k, sigmoid, normalize, 2.0, 0.5, None, mask)
    g = torch.Generator().manual_seed(2)
    dw = torch.randn((t, k), generator=g)
    dloss = torch.tensor([1.7])
    idx, count = out.topk_idx.cpu(), out.expert_count.cpu()
    rel = REL + (BF16 if dtype == torch.bfloat16 else 0)
    for a, b in ((dw, dloss), (dw, None), (None, dloss), (None, None)):
        want = R.gate_gradient(z, idx, count, sigmoid, normalize, 2.0, 0.5, a, b, mask)
        got = _gradient(p, z, out, a, b, mask)
        # Terms of the size of the weights' gradient cancel in a row.
        size = (2.0 * dw.abs().amax() if a is not None else 0.0) + (want.abs().amax() if b is not None else 0.0)
        assert torch.all((got - want).abs() <= rel * want.abs() + 8 * REL * size), (got - want).abs().max()


def test_gradient_against_differences():
    """The loss's change under small changes of single logits, the forward pass in float64."""
    t, e, k = 6, 12, 3
    z = _logits(t, e, torch.float32, 41)
    for sigmoid in (False, True):
        p, out = _run(z, k, sigmoid, True, 2.0, 0.5)
        idx, count = out.topk_idx.cpu(), out.expert_count.cpu()
        dw = torch.randn((t, k), generator=torch.Generator().manual_seed(3))
        got = _gradient(p, z, out, dw, torch.tensor([1.0]))

        def value(zz):
            s = torch.sigmoid(zz) if sigmoid else torch.softmax(zz, 1)
            picked = s.gather(1, idx)
            w = 2.0 * picked / picked.sum(1, keepdim=True)
            share = s / s.sum(1, keepdim=True)
            return float((w * dw.double()).sum() + 0.5 * e / (k * t * t) * (count.double() * share.sum(0)).sum())

        h = 1e-5  # central differences: error h^2 times a third derivative of order 10
        for i, j in ((0, 0), (1, 5), (2, int(idx[2, 0])), (3, int(idx[3, 2])), (5, 11)):
            up, down = z.double().clone(), z.double().clone()
            up[i, j] += h
            down[i, j] -= h
            assert abs((value(up) - value(down)) / (2 * h) - float(got[i, j])) <= 1e-5


def test_gradient_of_empty_rows_and_stray_entries():
    z = _logits(5, 70, torch.float32, 43)
    z[2] = -math.inf
    p, out = _run(z, 4, False)
    dw = torch.ones((5, 4))
    assert torch.all(_gradient(p, z, out, dw, torch.tensor([1.0]))[2] == 0)
    out.topk_idx[0, 1] = 70   # outside: skipped
    out.topk_idx[0, 2] = -5
    assert torch.all(torch.isfinite(_gradient(p, z, out, dw, None)))


def test_plans_and_streams():
    z = _logits(300, 128, torch.bfloat16, 47).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = M.make_gate_problem(300, 128, 8, M.GATE_SOFTMAX, loss_coef=0.1)
    a, b = M.alloc_gate(p, DEV), M.alloc_gate(p, DEV)
    ws_a, ws_b = M.alloc_gate_workspace(p, DEV), M.alloc_gate_workspace(p, DEV)
    M.dispatch_gate(p, z, a, ws_a)
    M.GatePlan(p, z, b, ws_b, stream=side)()
    dw, dl = torch.ones((300, 8), device=DEV), torch.ones(1, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    da, db = torch.empty_like(z), torch.empty_like(z)
    M.dispatch_gate_backward(p, z, a, dw, dl, da)
    M.GateBackwardPlan(p, z, b, dw, dl, db, stream=side)()
    torch.cuda.synchronize()
    for f in ("topk_idx", "topk_weights", "expert_count", "prob_sum", "live_tokens", "loss"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(da, db)


def test_binding_refuses_wrong_tensors():
    p = M.make_gate_problem(10, 20, 4, M.GATE_SIGMOID, torch.float32, loss_coef=1.0)
    z = torch.zeros((10, 20), device=DEV)
    out, ws = M.alloc_gate(p, DEV), M.alloc_gate_workspace(p, DEV)
    for bad in (z.cpu(), z.to(torch.bfloat16), z[:9], z.t()):
        with pytest.raises(ValueError, match="logits"):
            M.dispatch_gate(p, bad, out, ws)
    with pytest.raises(ValueError, match="select_bias"):
        M.dispatch_gate(p, z, out, ws, select_bias=torch.zeros(19, device=DEV))
    with pytest.raises(ValueError, match="token_mask"):
        M.dispatch_gate(p, z, out, ws, token_mask=torch.ones(9, dtype=torch.bool, device=DEV))
    with pytest.raises(M.DispatchError):
        M.dispatch_gate(p, z, out, None)
    with pytest.raises(M.DispatchError):
        M.dispatch_gate(p, z, out, ws[:256])
    with pytest.raises(ValueError, match="grad_weights"):
        M.dispatch_gate_backward(p, z, out, torch.zeros((10, 3), device=DEV), None, z.clone())
    with pytest.raises(ValueError, match="grad_logits"):
        M.dispatch_gate_backward(p, z, out, None, None, z[:9])
    soft = M.make_gate_problem(10, 20, 4, M.GATE_SOFTMAX, torch.float32)
    with pytest.raises(M.DispatchError):
        M.dispatch_gate(soft, z, out, ws, select_bias=torch.zeros(20, device=DEV))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        M.make_gate_problem(1, 2, 1, logits_dtype=torch.float16)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e", [63, 65, 127, 129, 255, 257, 511, 999, 2047, 2049])
def test_odd_expert_counts_at_any_alignment(sigmoid, dtype, e):
    """Rows of an odd length, their first element one past an aligned address; nothing beside them is written."""
    t, k = 19, 8
    g = torch.Generator().manual_seed(e)
    z = torch.randint(-3, 4, (t, e), generator=g).to(dtype)  # many ties
    z[4, : e - 1] = -math.inf   # one expert, the last
    z[5, 0] = z[5, e - 1] = 9.0
    p = M.make_gate_problem(t, e, k, M.GATE_SIGMOID if sigmoid else M.GATE_SOFTMAX, dtype, True, 2.0, 0.5, 8)
    out = M.alloc_gate(p, DEV)
    flat = torch.full((t * e + 2,), math.nan, dtype=dtype, device=DEV)
    rows = flat[1:-1].view(t, e)
    rows.copy_(z)
    M.dispatch_gate(p, rows, out, M.alloc_gate_workspace(p, DEV))
    torch.cuda.synchronize()
    ref = R.gate(z, k, sigmoid, True, 2.0, 0.5, None, None)
    idx, count = out.topk_idx.cpu().long(), out.expert_count.cpu()
    assert torch.equal(idx, ref["idx"]) and torch.equal(count.long(), ref["count"])
    assert torch.all((out.topk_weights.cpu().double() - ref["weights"]).abs() <= REL * (ref["weights"] + 2.0 ** -20))
    assert torch.all((out.prob_sum.cpu().double() - ref["prob_sum"]).abs() <= REL * (ref["prob_sum"] + 2.0 ** -60))
    dw = torch.randn((t, k), generator=g)
    dloss = torch.tensor([1.7])
    grad = torch.full((t * e + 2,), 77.0, dtype=dtype, device=DEV)
    M.dispatch_gate_backward(p, rows, out, dw.to(DEV), dloss.to(DEV), grad[1:-1].view(t, e))
    torch.cuda.synchronize()
    grad = grad.cpu().double()
    assert grad[0] == 77 and grad[-1] == 77
    want = R.gate_gradient(z, idx, count, sigmoid, True, 2.0, 0.5, dw, dloss, None)
    rel = REL + (BF16 if dtype == torch.bfloat16 else 0)
    size = 2.0 * dw.abs().amax() + want.abs().amax()
    got = grad[1:-1].view(t, e)
    assert torch.all((got - want).abs() <= rel * want.abs() + 8 * REL * size), (got - want).abs().max()


def _many(t, e, k, dtype, sigmoid, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randint(-3, 4, (t, e), generator=g).to(dtype) if ties else _logits(t, e, dtype, seed)
    z[1] = -math.inf                      # nothing to take
    z[2, 3:] = -math.inf                  # three of k
    z[3, : e - 1] = -math.inf             # the last alone
    z[4] = 0.0                            # all equal
    z[4, ::2] = -0.0
    z[t - 1] = torch.arange(e).to(dtype) / 16
    mask = torch.rand((t,), generator=g) > 0.1
    mask[:5] = True
    mask[t - 1] = True
    return z, mask


@pytest.mark.parametrize("e,k", [(65, 4), (66, 8), (67, 5), (97, 8), (128, 8), (129, 6), (130, 8), (191, 7), (255, 8), (256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens(e, k, sigmoid, dtype, monkeypatch):
    monkeypatch.setattr(R, "gate", R.gate_table)
    t = 8192 + e  # not a multiple of a wavefront's or a workgroup's tokens
    z, mask = _many(t, e, k, dtype, sigmoid, e, ties=True)
    # (The last row's largest sigmoids are equal in fp32, though not in fp64.)
    _, out, _ = _check(z, k, sigmoid, scale=2.5, mask=mask, exact_choice=not sigmoid)
    if sigmoid:
        fp32 = 1.0 / (1.0 + torch.exp(-z.to(DEV).float()))
        want = torch.sort(fp32, dim=1, descending=True, stable=True).indices[:, :k]
        rows = mask.to(DEV)
        rows[:4] = False  # (rows with fewer than k to take)
        assert torch.equal(out.topk_idx[rows], want[rows])
    z, mask = _many(t, e, k, dtype, sigmoid, e + 1)
    bias = torch.randn((e,), generator=torch.Generator().manual_seed(e)) if sigmoid else None
    _check(z, k, sigmoid, normalize=False, mask=mask, bias=bias, idx_bytes=4, exact_choice=not sigmoid)


@pytest.mark.parametrize("t", [8191, 8192, 8195, 65539])
def test_many_tokens_at_any_alignment(t):
    """The choice on both sides of the change of form and past one pass, from rows at odd addresses; without balance alike."""
    e, k = 129, 8
    z, mask = _many(t, e, k, torch.bfloat16, False, t, ties=True)
    flat = torch.full((t * e + 2,), math.nan, dtype=torch.bfloat16, device=DEV)
    rows = flat[1:-1].view(t, e)
    rows.copy_(z)
    p = M.make_gate_problem(t, e, k, M.GATE_SOFTMAX, torch.bfloat16, True, 1.0, 0.5, 8)
    ref = R.gate_table(z, k, False, True, 1.0, 0.5, None, mask)
    tables = []
    for balance in (True, False, True):
        out = M.alloc_gate(p, DEV, balance=balance)
        M.dispatch_gate(p, rows, out, M.alloc_gate_workspace(p, DEV), token_mask=mask.to(DEV))
        torch.cuda.synchronize()
        assert torch.equal(out.topk_idx.cpu().long(), ref["idx"])
        if balance:
            assert torch.equal(out.expert_count.cpu().long(), ref["count"]) and int(out.live_tokens) == ref["live"]
        tables.append(out)
    assert torch.equal(tables[0].topk_weights, tables[1].topk_weights)
    for name in ("topk_weights", "prob_sum", "loss"):
        assert torch.equal(getattr(tables[0], name), getattr(tables[2], name))  # bit for bit


@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_tokens_nan_and_infinity(sigmoid):
    t, e, k = 8200, 200, 8
    z, _ = _many(t, e, k, torch.float32, sigmoid, 11)
    z[10, 5] = math.nan
    z[11] = math.nan
    z[12, 7] = math.inf
    few, many = z[:64].contiguous(), z
    _, a = _run(few, k, sigmoid)
    _, b = _run(many, k, sigmoid)
    # The same choice as in the form of few tokens; NaN shows in the same places.
    assert torch.equal(a.topk_idx, b.topk_idx[:64])
    wa, wb = a.topk_weights, b.topk_weights[:64]
    assert torch.equal(torch.isnan(wa), torch.isnan(wb))
    assert torch.all(((wa - wb).abs() <= REL * wa.abs()) | torch.isnan(wa))
    assert not torch.any(b.topk_idx[10] == 5) and torch.all(b.topk_idx[11] == -1)


@pytest.mark.parametrize("e", [7, 65, 256, 600, 2049])
@pytest.mark.parametrize("t", [1, 2, 8, 9, 16, 17, 31, 32, 33, 64, 65])
def test_balance_of_few_tokens(t, e):
    """Either side of the batches that one workgroup finishes alone."""
    mask = torch.rand((t,), generator=torch.Generator().manual_seed(t)) > 0.3
    _check(_logits(t, e, torch.float32, t + e), min(e, 8), False, mask=mask, coef=0.5)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_lone_weight_has_no_gradient(sigmoid):
    """One entry, normalised: its weight is constant, and only the loss has a gradient."""
    t, e = 300, 40
    z = _logits(t, e, torch.float32, 3)
    p, out = _run(z, 1, sigmoid, True, 2.5, 0.01)
    dw = 10 * torch.randn((t, 1), generator=torch.Generator().manual_seed(4))
    assert torch.all(_gradient(p, z, out, dw, None) == 0)
    loss = torch.tensor([1.0])
    assert torch.equal(_gradient(p, z, out, dw, loss), _gradient(p, z, out, None, loss))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_beside_a_large_one_of_a_small_share(dtype):
    """A selection bias puts an expert of a tiny score first; its weight's gradient is large, and tiny in all others'."""
    t, e, k = 33, 20, 4
    z = _logits(t, e, torch.float32, 71, 0.5)
    z[:, 7] = -20.0
    z = z.to(dtype)
    bias = torch.zeros(e)
    bias[7] = 5.0
    p, out = _run(z, k, True, True, 2.0, 0.5, bias)
    idx, count = out.topk_idx.cpu(), out.expert_count.cpu()
    assert torch.all(idx[:, 0] == 7)
    dw = torch.randn((t, k), generator=torch.Generator().manual_seed(5))
    dw[:, 0] *= 1e6
    got = _gradient(p, z, out, dw, None)
    want = R.gate_gradient(z, idx, count, True, True, 2.0, 0.5, dw, None)
    # A weight's gradient and the mean of all, each with a few roundings of
    # what it is added up from: shares times gradients, no more.
    score = torch.sigmoid(z.double()).gather(1, idx)
    share = score / score.sum(1, keepdim=True)
    mean = (share * dw.double().abs()).sum(1, keepdim=True)
    bound = torch.zeros_like(want).scatter_(1, idx, REL * 2.0 * share * (dw.double().abs() + mean))
    assert torch.all((got - want).abs() <= bound + (BF16 if dtype == torch.bfloat16 else 0) * want.abs())


def _smallest(t, e):
    """fp32 sigmoid logits whose scores are 2^-115 to 2^-128, the smallest that are not 0: all of a row's, or one alone."""
    z = -88.7228 + 9.0 * torch.rand((t, e), generator=torch.Generator().manual_seed(t + e))
    z[1] = -88.72283  # the last fp32 number whose exp(-z) is finite
    z[2] = -math.inf
    z[2, e // 2] = -88.72283
    return z


# A score of 2^-128 has 21 bits: half a unit of them, and as much again from exp,
# in a share, its sum and the products that they enter.
SMALLEST = 8 * 2.0 ** -21


@pytest.mark.parametrize("e,k", [(1, 1), (7, 1), (7, 3), (70, 8)])
@pytest.mark.parametrize("scale", [2.5, 1e-3])
def test_smallest_sigmoid_scores(e, k, scale):
    """Shares of scores whose reciprocals are past fp32's range, in the weights, the loss and both gradients."""
    t = 33
    z = _smallest(t, e)
    p, out = _run(z, k, True, True, scale, 0.5)
    idx, count = out.topk_idx.cpu(), out.expert_count.cpu()
    took = idx >= 0
    score = torch.sigmoid(z.double())
    picked = torch.where(took, score.gather(1, idx.clamp_min(0)), 0.0)
    share = picked / picked.sum(1, keepdim=True)
    got = out.topk_weights.cpu().double()
    assert torch.all((got - scale * share).abs() <= SMALLEST * scale * share)
    prob_sum = (score / score.sum(1, keepdim=True)).sum(0)
    assert torch.all((out.prob_sum.cpu().double() - prob_sum).abs() <= SMALLEST * prob_sum)
    loss = 0.5 * e / (k * t * t) * float((count.double() * prob_sum).sum())
    assert abs(float(out.loss) - loss) <= SMALLEST * loss
    dw, dloss = torch.randn((t, k), generator=torch.Generator().manual_seed(6)), torch.tensor([1.7])
    for a, b in ((dw, None), (None, dloss), (dw, dloss)):
        want = R.gate_gradient(z, idx, count, True, True, scale, 0.5, a, b)
        # Each gradient's terms: an entry's share times its own and the mean gradient, the same of the shares of all.
        size = (scale * dw.abs().max() if a is not None else 0.0) + \
            (2 * 1.7 * 0.5 * e / (k * t * t) * float(count.max()) if b is not None else 0.0)
        assert torch.all((_gradient(p, z, out, a, b) - want).abs() <= 2 * SMALLEST * size)
    # Not normalised, the weights' gradient is in fp32's smallest numbers, the loss's as before.
    p, out = _run(z, k, True, False, scale, 0.5)
    got = _gradient(p, z, out, dw, None)
    want = R.gate_gradient(z, idx, count, True, False, scale, 0.5, dw, None)
    assert torch.all((got - want).abs() <= SMALLEST * want.abs() + 2.0 ** -147)


def test_smallest_sigmoid_scores_of_many_tokens():
    t, e, k = 8229, 130, 8
    z = _smallest(t, e)
    p, out = _run(z, k, True, True, 2.5, 0.5)
    few, b = _run(z[:64].contiguous(), k, True, True, 2.5, 0.5)
    assert torch.equal(out.topk_idx[:64], b.topk_idx)
    assert torch.all((out.topk_weights[:64] - b.topk_weights).abs() <= SMALLEST * b.topk_weights)
    score = torch.sigmoid(z.double())
    prob_sum = (score / score.sum(1, keepdim=True)).sum(0)
    assert torch.all((out.prob_sum.cpu().double() - prob_sum).abs() <= SMALLEST * prob_sum)


# Tokens past one for each wavefront of the gradient's grid (512 workgroups of
# 16, 8 and 4 wavefronts, by the number of experts), not a multiple of anything.
@pytest.mark.parametrize("t,e,k", [(8192 + 37, 64, 8), (20011, 129, 8), (8192 + 37, 512, 5), (4096 + 45, 601, 8),
                                   (2048 + 77, 1100, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_many_tokens(t, e, k, sigmoid, dtype):
    """A wavefront's later tokens: the same rows in calls of at most 300, with the same counts, have the same bits."""
    z, mask = _many(t, e, k, dtype, sigmoid, e)
    p, out = _run(z, k, sigmoid, True, 2.5, 0.5, None, mask)
    g = torch.Generator().manual_seed(t)
    dw, dloss = torch.randn((t, k), generator=g).to(DEV), torch.tensor([1.7], device=DEV)
    zd, md = z.to(DEV), mask.to(DEV)
    for a, b, m in ((dw, dloss, md), (None, dloss, md), (dw, None, None)):
        got = torch.full_like(zd, 77.0)
        M.dispatch_gate_backward(p, zd, out, a, b, got, token_mask=m)
        want = torch.full_like(zd, 78.0)
        for first in range(0, t, 300):
            part = slice(first, min(first + 300, t))
            n = part.stop - first
            few = M.make_gate_problem(n, e, k, M.GATE_SIGMOID if sigmoid else M.GATE_SOFTMAX, dtype, True, 2.5, 0.5)
            rows = M.GateTensors(out.topk_idx[part], out.topk_weights[part], out.expert_count, out.prob_sum,
                                 out.live_tokens, out.loss)
            M.dispatch_gate_backward(few, zd[part], rows, None if a is None else a[part], b, want[part],
                                     token_mask=None if m is None else m[part])
        bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
        assert torch.equal(got.view(bits), want.view(bits))
        assert m is None or torch.all(got[~md] == 0)


@pytest.mark.parametrize("e,k", [(65, 4), (67, 5), (128, 5), (129, 4), (256, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens_of_four_and_five_sigmoids(e, k, dtype, monkeypatch):
    """Either side of the batch from which few sigmoid entries take the form of many tokens."""
    monkeypatch.setattr(R, "gate", R.gate_table)
    for t in (2 * 8192 - 1, 2 * 8192 + e):
        z, mask = _many(t, e, k, dtype, True, e, ties=True)
        _, out, _ = _check(z, k, True, scale=2.5, mask=mask, exact_choice=False)
        fp32 = 1.0 / (1.0 + torch.exp(-z.to(DEV).float()))
        want = torch.sort(fp32, dim=1, descending=True, stable=True).indices[:, :k]
        rows = mask.to(DEV)
        rows[:4] = False  # (rows with fewer than k to take)
        assert torch.equal(out.topk_idx[rows], want[rows])
        z, mask = _many(t, e, k, dtype, True, e + 1)
        bias = torch.randn((e,), generator=torch.Generator().manual_seed(e))
        _check(z, k, True, normalize=False, mask=mask, bias=bias, idx_bytes=4, exact_choice=False)


def test_sigmoid_scores_that_are_all_zero():
    """Logits below -88.7: experts are taken, with weights, shares and gradients of 0."""
    t, e, k = 20, 70, 4
    z = torch.full((t, e), -1000.0)
    z[::2] = -89.0
    z[5] = torch.finfo(torch.float32).min
    p, out = _run(z, k, True, True, 2.5, 0.5)
    assert torch.equal(out.topk_idx.cpu(), torch.arange(k).expand(t, k))
    assert torch.all(out.topk_weights == 0) and torch.all(out.prob_sum == 0) and float(out.loss) == 0.0
    dw = torch.randn((t, k), generator=torch.Generator().manual_seed(8))
    assert torch.all(_gradient(p, z, out, dw, torch.tensor([1.0])) == 0)
