"""The combine's gradient against its definition in float64."""

import math

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import block_reference as R
from tests import layer_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -24
BF16 = 2.0 ** -8
FILL = 0x5A


def _inputs(t, k, width, rows, seed, mask=0.1):
    """Every entry a slot of its own, some of them masked; more rows than entries."""
    g = torch.Generator().manual_seed(seed)
    slot = torch.randperm(rows, generator=g)[: t * k].to(torch.int32).view(t, k)
    slot[torch.rand((t, k), generator=g) < mask] = -1
    weights = torch.randn((t, k), generator=g)
    y = torch.randn((rows, width), generator=g).to(torch.bfloat16)
    d = torch.randn((t, width), generator=g).to(torch.bfloat16)
    return slot, weights, y, d


def _run(slot, weights, y, d, form, want_weights=True):
    t, k = slot.shape
    rows, width = y.shape
    dw = torch.full((t, k), -7.0, device=DEV) if want_weights else None
    dy = torch.full((rows, width), -7.0, dtype=torch.bfloat16, device=DEV) if form == "bf16" else None
    dq = torch.full((rows, width), FILL, dtype=torch.uint8, device=DEV) if form == "fp8" else None
    dsf = torch.full((rows, -(-width // 128)), -7.0, device=DEV) if form == "fp8" else None
    M.dispatch_combine_backward(slot.to(DEV), weights.to(DEV), y.to(DEV), d.to(DEV), dw, dy, dq, dsf)
    torch.cuda.synchronize()
    return dw, dy, dq, dsf


def _check(slot, weights, y, d, form):
    dw, dy, dq, dsf = _run(slot, weights, y, d, form)
    want_w, size, want_y = R.combine_gradient(slot, weights, y, d)
    # A lane adds width / 64 products over up to 16 wavefronts, then 6 steps and 16 wavefronts.
    chain = 8 * math.ceil(y.shape[1] / (8 * 64)) + 22
    assert torch.all((dw.cpu().double() - want_w).abs() <= chain * ULP * size + 2.0 ** -140)
    mine = ~torch.isnan(want_y).all(1)
    if form == "bf16":
        got = dy.cpu()
        assert torch.all(got[~mine] == -7)
        err = (got[mine].double() - want_y[mine]).abs()
        assert torch.all(err <= (BF16 + 2 * ULP) * want_y[mine].abs() + 2.0 ** -134)
    elif form == "fp8":
        assert torch.all(dq.cpu()[~mine] == FILL) and torch.all(dsf.cpu()[~mine] == -7)
        layer_reference.assert_quantised(dq.cpu()[mine].view(torch.float8_e4m3fn).float(), dsf.cpu()[mine], want_y[mine], 6 * ULP)
    return dw


@pytest.mark.parametrize("width", [8, 16, 24, 136, 512, 520, 528, 2064, 7168, 8192, 8208, 20000])
@pytest.mark.parametrize("form", ["bf16", "fp8", "none"])
def test_widths(width, form):
    if form == "fp8" and width % 16:
        width += 8
    _check(*_inputs(5, 3, width, 19, width), form)


@pytest.mark.parametrize("t,k", [(0, 4), (1, 1), (1, 8), (63, 8), (40, 9), (21, 32), (300, 2), (17, 16),
                                 (255, 8), (256, 9), (300, 32), (128, 3), (100, 17)])
@pytest.mark.parametrize("form", ["bf16", "fp8", "none"])
def test_tokens_and_entries(t, k, form):
    _check(*_inputs(t, k, 272, t * k + 5, 100 * t + k), form)


@pytest.mark.parametrize("form", ["bf16", "fp8"])
def test_weights_gradient_left_out(form):
    args = _inputs(20, 6, 528, 130, 3)
    full = _run(*args, form)
    less = _run(*args, form, want_weights=False)
    assert less[0] is None
    for a, b in zip(full[1:], less[1:]):
        assert a is None or torch.equal(a, b)
    # y is not read then: any rows give its shape.
    slot, w, y, d = (x.to(DEV) for x in args)
    if form == "bf16":
        dy = torch.full(y.shape, -7.0, dtype=torch.bfloat16, device=DEV)
        M.dispatch_combine_backward(slot, w, None, d, grad_y=dy)
        assert torch.equal(dy, full[1])


def test_masked_tokens_and_slots_outside():
    slot, w, y, d = _inputs(12, 4, 144, 60, 5, mask=0.0)
    slot[3] = -1
    slot[4, 1], slot[5, 2], slot[6, 0] = 60, 2 ** 31 - 1, -2 ** 31
    d[3] = math.nan  # of a token with no entry: read by nothing
    for form in ("bf16", "fp8"):
        dw = _check(slot, w, y, d, form)
        assert torch.all(dw[3] == 0) and dw[4, 1] == 0 and dw[5, 2] == 0 and dw[6, 0] == 0


def test_special_values():
    slot, w, y, d = _inputs(6, 2, 256, 12, 7, mask=0.0)
    w[0] = 0.0
    d[1] = 0.0
    d[2, 5], d[3, 200] = math.nan, math.inf
    w[4] = 2.0 ** -120   # rows below the floor of the scales
    w[5] = -3.0
    dw, dy, _, _ = _run(slot, w, y, d, "bf16")
    _, _, dq, dsf = _run(slot, w, y, d, "fp8")
    want = w[:, :, None] * d.float()[:, None, :]
    got = dy.cpu()[slot.long()]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = torch.isfinite(want)
    assert torch.equal(got[fine], want.to(torch.bfloat16)[fine])
    # The same rows quantised from fp32: as dispatch_quantize does bf16 rows that hold them exactly.
    w1 = torch.full_like(w, 2.0)
    _, rows2, _, _ = _run(slot, w1, y, d, "bf16")
    _, _, q2, sf2 = _run(slot, w1, y, d, "fp8")
    q = torch.full_like(q2, FILL)
    sf = torch.full_like(sf2, -7.0)
    M.dispatch_quantize(rows2, q, sf)
    torch.cuda.synchronize()
    at = slot.long().view(-1).to(DEV)
    assert torch.equal(torch.nan_to_num(sf[at], 3.0), torch.nan_to_num(sf2[at], 3.0)) and torch.equal(q[at], q2[at])
    v, s = dq.cpu().view(torch.float8_e4m3fn).float()[slot.long()], dsf.cpu()[slot.long()]
    assert torch.all(v[0] == 0) and torch.all(v[1] == 0) and torch.all(s[0] == 2.0 ** -100 / torch.tensor(448.0))
    assert torch.all(torch.isnan(s[2, :, 0])) and torch.all(torch.isinf(s[3, :, 1])) and torch.all(torch.isfinite(s[2, :, 1]))
    assert torch.all(s[4] == 2.0 ** -100 / torch.tensor(448.0))


def test_gradient_against_differences():
    """The change of sum(out dout) under small changes of single weights and values, the combine in float64."""
    slot, w, y, d = _inputs(5, 3, 64, 20, 11)
    dw, dy, _, _ = _run(slot, w, y, d, "bf16")

    def value(ww, yy):
        rows = torch.where((slot >= 0)[:, :, None], ww.double()[:, :, None] * yy.double()[slot.long().clamp_min(0)], 0.0)
        return float((rows.sum(1) * d.double()).sum())

    for i, j in ((0, 0), (2, 1), (4, 2)):
        up, down = w.double().clone(), w.double().clone()
        up[i, j] += 0.5   # (linear: the difference is exact)
        down[i, j] -= 0.5
        want = value(up, y) - value(down, y)
        assert abs(float(dw[i, j]) - want) <= 1e-5 * (1 + abs(want))
        s = int(slot[i, j])
        if s >= 0:
            up, down = y.double().clone(), y.double().clone()
            up[s, 7] += 0.5
            down[s, 7] -= 0.5
            want = value(w, up) - value(w, down)
            assert abs(float(dy[s, 7]) - want) <= BF16 * abs(want) + 1e-6


@pytest.mark.parametrize("form", ["bf16", "fp8"])
def test_rows_beyond_32_bit_offsets(form):
    rows, width = 300200, 7168
    assert rows * width > 2 ** 31
    y = torch.zeros((rows, width), dtype=torch.bfloat16, device=DEV)
    slot, w, some, d = _inputs(3, 2, width, 6, 13, mask=0.0)
    at = rows - 1 - 100 * slot.long()  # near the end
    y[at.view(-1).to(DEV)] = some[slot.long().view(-1)].to(DEV)
    want_w, size, want_y = R.combine_gradient(slot, w, some, d)
    dw = torch.empty((3, 2), device=DEV)
    outs = {}
    if form == "bf16":
        outs["grad_y"] = torch.full((rows, width), -7.0, dtype=torch.bfloat16, device=DEV)
    else:
        outs["grad_q"] = torch.full((rows, width), FILL, dtype=torch.uint8, device=DEV)
        outs["grad_sf"] = torch.full((rows, 56), -7.0, device=DEV)
    M.dispatch_combine_backward(at.to(torch.int32).to(DEV), w.to(DEV), y, d.to(DEV), dw, **outs)
    torch.cuda.synchronize()
    assert torch.all((dw.cpu().double() - want_w).abs() <= 200 * ULP * size)
    want = want_y[slot.long().view(-1)]
    if form == "bf16":
        got = outs["grad_y"][at.view(-1).to(DEV)].cpu().double()
        assert torch.all((got - want).abs() <= (BF16 + 2 * ULP) * want.abs())
    else:
        pick = lambda x: x[at.view(-1).to(DEV)].cpu()  # noqa: E731
        layer_reference.assert_quantised(pick(outs["grad_q"]).view(torch.float8_e4m3fn).float(), pick(outs["grad_sf"]), want, 6 * ULP)


def test_many_tokens():
    t, k, width = 3000, 4, 512
    slot, w, y, d = (x.to(DEV) for x in _inputs(t, k, width, t * k + 77, 17))
    dw, dy = torch.empty((t, k), device=DEV), torch.zeros_like(y)
    M.dispatch_combine_backward(slot, w, y, d, dw, dy)
    live, at = slot >= 0, slot.long().clamp_min(0)
    terms = d.double()[:, None, :] * y[at].double()
    want = torch.where(live, terms.sum(2), 0.0)
    assert torch.all((dw.double() - want).abs() <= 40 * ULP * terms.abs().sum(2))
    rows = (w[:, :, None] * d.float()[:, None, :])[live].to(torch.bfloat16)
    full = torch.zeros_like(y)
    full[at[live]] = rows
    assert torch.equal(dy, full)


@pytest.mark.parametrize("form", ["bf16", "fp8"])
def test_more_tokens_than_the_grid_holds(form):
    t, width = 1060000, 16
    rows = t + 5
    g = torch.Generator(device=DEV).manual_seed(3)
    slot = torch.randperm(rows, generator=g, device=DEV)[:t].to(torch.int32).view(t, 1)
    w = torch.randn((t, 1), generator=g, device=DEV)
    y = torch.randn((rows, width), generator=g, device=DEV).to(torch.bfloat16)
    d = torch.randn((t, width), generator=g, device=DEV).to(torch.bfloat16)
    dw = torch.empty((t, 1), device=DEV)
    rows_of = (w * d.float())
    at = slot.long().view(-1)
    if form == "bf16":
        dy = torch.zeros_like(y)
        M.dispatch_combine_backward(slot, w, y, d, dw, dy)
        assert torch.equal(dy[at], rows_of.to(torch.bfloat16))
    else:
        q, sf = torch.zeros((rows, width), dtype=torch.uint8, device=DEV), torch.zeros((rows, 1), device=DEV)
        M.dispatch_combine_backward(slot, w, y, d, dw, None, q, sf)
        amax = rows_of.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
        top = torch.full_like(amax, 448.0)
        assert torch.equal(sf[at], amax / top)
        assert torch.equal(q[at], (rows_of * (top / amax)).to(torch.float8_e4m3fn).view(torch.uint8))
    terms = d.double() * y[at].double()
    assert torch.all((dw.double().view(-1) - terms.sum(1)).abs() <= 30 * ULP * terms.abs().sum(1))


def test_weights_gradient_of_a_large_batch_alone():
    slot, w, y, d = _inputs(5000, 4, 4096, 20100, 31)
    dw, _, _, _ = _run(slot, w, y, d, "none")
    at = slot.long().clamp_min(0).to(DEV)
    terms = d.to(DEV).float()[:, None, :] * y.to(DEV)[at].float()
    want = torch.where((slot >= 0).to(DEV), terms.double().sum(2), 0.0)
    assert torch.all((dw.double() - want).abs() <= 100 * ULP * terms.double().abs().sum(2))


def test_plans_streams_and_a_graph():
    t, k, width, rows = 60, 8, 1040, 600
    batches = [tuple(x.to(DEV) for x in _inputs(t, k, width, rows, 20 + i)) for i in range(3)]
    new = lambda: (torch.zeros((t, k), device=DEV), torch.zeros((rows, width), dtype=torch.uint8, device=DEV),  # noqa: E731
                   torch.zeros((rows, 9), device=DEV))
    eager = []
    for b in batches:
        dw, q, sf = new()
        M.dispatch_combine_backward(*b, dw, None, q, sf)
        eager.append((dw, q, sf))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a, b = new(), new()
    side.wait_stream(torch.cuda.current_stream())
    M.CombineBackwardPlan(*batches[0], a[0], None, a[1], a[2])()
    M.CombineBackwardPlan(*batches[1], b[0], None, b[1], b[2], stream=side)()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for got, want in ((a, eager[0]), (b, eager[1])) for x, y in zip(got, want))
    ins = tuple(x.clone() for x in batches[0])
    plan = M.CombineBackwardPlan(*ins, a[0], None, a[1], a[2], stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        plan()
    for _ in range(2):
        for batch, want in zip(batches, eager):
            for x, y in zip(ins, batch):
                x.copy_(y)
            a[1].zero_()
            a[2].zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a, want))
            M.dispatch_combine_backward(*batches[0], b[0], None, b[1], b[2])  # eager work in between


def test_binding_refuses_wrong_tensors():
    slot, w, y, d = (x.to(DEV) for x in _inputs(4, 2, 64, 10, 1))
    dw, dy = torch.empty((4, 2), device=DEV), torch.empty_like(y)
    q, sf = torch.empty((10, 64), dtype=torch.uint8, device=DEV), torch.empty((10, 1), device=DEV)
    for bad in ((slot.long(), w, y, d), (slot, w.double(), y, d), (slot, w, y.float(), d), (slot, w, y, d.float()),
                (slot, w[:3], y, d), (slot, w, y, d[:, :32].contiguous()), (slot, w, None, d), (slot[0], w, y, d),
                (slot, w, y.cpu(), d)):
        with pytest.raises(ValueError):
            M.dispatch_combine_backward(*bad, dw, None if bad[2] is None else dy)
    with pytest.raises(ValueError, match="line up"):
        M.dispatch_combine_backward(slot, w, y, d, dw, dy[:9])
    with pytest.raises(ValueError, match="grad_weights"):
        M.dispatch_combine_backward(slot, w, y, d, dw[:3], dy)
    with pytest.raises(ValueError, match="grad_sf"):
        M.dispatch_combine_backward(slot, w, y, d, dw, None, q, sf[:9])
    for kw in (dict(grad_y=dy, grad_q=q, grad_sf=sf), dict(grad_q=q), dict()):
        with pytest.raises(M.DispatchError):
            M.dispatch_combine_backward(slot, w, y, d, **kw)


@pytest.mark.parametrize("form", ["bf16", "fp8", "none"])
@pytest.mark.parametrize("want_weights", [True, False])
def test_no_expert_rows(form, want_weights):
    """A buffer of no rows: every slot is outside it, the weights' gradient is 0."""
    if form == "none" and not want_weights:
        return
    slot, w, y, d = _inputs(5, 3, 272, 19, 23)
    dw, dy, dq, dsf = _run(slot, w, y[:0], d, form, want_weights)
    assert dw is None or torch.all(dw == 0)
    assert all(x is None or x.numel() == 0 for x in (dy, dq, dsf))
