"""The RMS norm and its gradient against their definitions in float64."""

import math

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import block_reference as R
from tests import layer_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -24   # half a step of fp32
BF16 = 2.0 ** -8   # half a step of bf16
# The sum of squares: a lane adds up to 64 of them, 6 steps over the wavefront and up to 16 wavefronts:
# 86 roundings, of positive terms. The root halves that; with the mean, eps, the root and the division
# (4), r is within 47 roundings, and h r w within 49.
REL = 49 * ULP
FILL = 0x5A
WIDTHS = [16, 32, 112, 128, 144, 496, 512, 528, 1040, 2064, 4096, 7168, 8192, 8208, 16384, 16400, 40000, 65536]


def _bf16(shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def _weight(w, dtype, seed=1):
    return (1.0 + 0.2 * torch.randn(w, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _on(x):
    return None if x is None else x.to(DEV)


def _forward(x, weight, eps=1e-6, residual=None, outs="both", valid=None):
    r, w = x.shape
    rows = lambda: torch.full((r, w), -7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h = rows() if residual is not None else None
    y = rows() if outs != "fp8" else None
    q = torch.full((r, w), FILL, dtype=torch.uint8, device=DEV) if outs != "bf16" else None
    sf = torch.full((r, -(-w // 128)), -7.0, device=DEV) if outs != "bf16" else None
    M.dispatch_rms_norm(_on(x), _on(weight), eps, residual=_on(residual), h=h, y=y, q=q, sf=sf, num_valid_rows=_on(valid))
    torch.cuda.synchronize()
    return h, y, q, sf


def _close_bf16(got, want, rel):
    got = got.cpu().double()
    assert torch.all((got - want).abs() <= (BF16 + 2 * rel) * want.abs() + 2.0 ** -134), (got - want).abs().max()


def _check(x, weight, residual=None, outs="both", eps=1e-6, rel=REL):
    h, y, q, sf = _forward(x, weight, eps, residual, outs)
    want_h = R.rounded_sum(x, residual)
    if residual is not None:
        assert torch.equal(h.cpu(), want_h)
    want = R.rms_norm(want_h, weight, eps)
    if y is not None:
        _close_bf16(y, want, rel)
    if q is not None:
        layer_reference.assert_quantised(q.view(torch.float8_e4m3fn).float().cpu(), sf.cpu(), want, rel + 4 * ULP)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 2, 5])
def test_widths(rows, width):
    for i, (res, outs, dtype) in enumerate([(True, "both", torch.bfloat16), (False, "bf16", torch.float32),
                                            (True, "fp8", torch.float32), (False, "fp8", torch.bfloat16)]):
        x = _bf16((rows, width), 10 * width + i)
        _check(x, _weight(width, dtype), _bf16((rows, width), 7 + i, 4.0) if res else None, outs)


@pytest.mark.parametrize("rows,width", [(0, 128), (333, 4096), (511, 272), (512, 272), (513, 1024), (1030, 144), (4097, 16),
                                        (700, 7168), (512, 16400), (2048, 256), (4097, 128), (5003, 176), (4099, 112),
                                        (2047, 144)])
@pytest.mark.parametrize("outs", ["both", "bf16", "fp8"])
def test_rows(rows, width, outs):
    _check(_bf16((rows, width), rows), _weight(width, torch.bfloat16), _bf16((rows, width), 3, 4.0), outs)
    _check(_bf16((rows, width), rows), _weight(width, torch.float32), None, outs)


def test_single_outputs_are_those_of_both():
    x, res, w = _bf16((600, 1040), 1), _bf16((600, 1040), 2), _weight(1040, torch.bfloat16)
    h, y, q, sf = _forward(x, w, residual=res)
    _, y1, _, _ = _forward(x, w, residual=res, outs="bf16")
    _, _, q1, sf1 = _forward(x, w, residual=res, outs="fp8")
    assert torch.equal(y, y1) and torch.equal(q, q1) and torch.equal(sf, sf1)
    # What is quantised is the fp32 row, as dispatch_quantize would of one that bf16 holds.
    _, y2, q2, sf2 = _forward(torch.ones((3, 256), dtype=torch.bfloat16), torch.ones(256), eps=3.0)
    assert torch.all(y2 == 0.5) and torch.all(q2.view(torch.float8_e4m3fn).float() == 448.0)
    assert torch.all(sf2 == torch.tensor(0.5, device=DEV) / torch.tensor(448.0, device=DEV))


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("rows", [3, 600])
def test_sum_in_place(target, rows):
    x, res, w = _bf16((rows, 2064), 1).to(DEV), _bf16((rows, 2064), 2).to(DEV), _weight(2064, torch.float32).to(DEV)
    want_h, want_y, _, _ = _forward(x, w, residual=res, outs="bf16")
    y = torch.empty_like(x)
    h = x if target == "x" else res
    M.dispatch_rms_norm(x, w, 1e-6, residual=res, h=h, y=y)
    assert torch.equal(h, want_h) and torch.equal(y, want_y)


@pytest.mark.parametrize("valid", [-3, 0, 1, 5, 9, 100])
@pytest.mark.parametrize("width", [48, 2064])
def test_rows_past_the_valid_ones_are_not_touched(valid, width):
    rows = 9
    n = max(0, min(valid, rows))
    x, res, w = _bf16((rows, width), 1), _bf16((rows, width), 2), _weight(width, torch.bfloat16)
    x[n:], res[n:] = math.nan, math.nan
    h, y, q, sf = _forward(x, w, residual=res, valid=torch.tensor([valid], dtype=torch.int32))
    assert torch.all(h[n:] == -7) and torch.all(y[n:] == -7) and torch.all(q[n:] == FILL) and torch.all(sf[n:] == -7)
    _close_bf16(y[:n], R.rms_norm(R.rounded_sum(x[:n], res[:n]), w, 1e-6), REL)
    dy = _bf16((rows, width), 3)
    dy[n:] = math.nan
    dx, dw = _backward(x, w, dy, res, valid=torch.tensor([valid], dtype=torch.int32))
    assert torch.all(dx[n:] == -7) and torch.all(torch.isfinite(dx[:n])) and torch.all(torch.isfinite(dw))
    if n == 0:
        assert torch.all(dw == 0)


def test_ends_of_the_range():
    w = torch.ones(256)
    x = torch.zeros((8, 256), dtype=torch.bfloat16)
    x[1] = 2.0 ** -120                # far below eps
    x[2, 0] = 2.0 ** 60               # one channel has it all
    x[3] = 2.0 ** 59                  # the sum of squares is 2^126
    x[4] = torch.finfo(torch.bfloat16).max
    x[5, 3], x[6, 7] = math.inf, math.nan
    x[7] = 1.0
    h, y, q, sf = _forward(x, w)
    y, q = y.float().cpu(), q.view(torch.float8_e4m3fn).float().cpu()
    assert torch.all(y[0] == 0) and torch.all(q[0] == 0)
    _close_bf16(y[1].bfloat16(), R.rms_norm(x[1:2], w, 1e-6)[0], REL)
    assert y[2, 0] == 16.0 and torch.all(y[2, 1:] == 0) and torch.all(y[3] == 1.0)
    assert torch.all(y[4] == 0)       # the squares pass fp32's range: r is 0
    assert math.isnan(float(y[5, 3])) and torch.all(torch.isnan(y[6]))
    assert torch.all(y[7] == 1.0) and torch.all(q[7] == 448.0)  # (1 + eps rounds to 1 after the root)


def _backward(h, weight, dy, dh=None, eps=1e-6, want_weight=True, valid=None):
    r, w = h.shape
    dx = torch.full((r, w), -7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((w,), -7.0, device=DEV) if want_weight else None
    ws = None
    if want_weight:
        ws = M.alloc_rms_norm_workspace(r, w, DEV)
        ws.fill_(0xFF)
    M.dispatch_rms_norm_backward(_on(h), _on(weight), _on(dy), eps, dx, grad_h=_on(dh), grad_weight=dw, workspace=ws,
                                 num_valid_rows=_on(valid))
    torch.cuda.synchronize()
    return dx, dw


def _check_backward(h, weight, dy, dh, eps=1e-6):
    dx, dw = _backward(h, weight, dy, dh, eps)
    want_x, want_w = R.rms_norm_gradient(h, weight, dy, eps, dh)
    x, d, w = h.double(), dy.double(), weight.double()
    r = (x.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    # r g - r u mean(g u) + dh: each part within REL of its size, the mean's terms of either sign
    # within REL of the sum of their magnitudes; then bf16.
    size = (r * d * w).abs() + (r * x * r) .abs() * (d * w * x * r).abs().mean(1, keepdim=True)
    if dh is not None:
        size = size + dh.double().abs()
    err = (dx.cpu().double() - want_x).abs()
    assert torch.all(err <= BF16 * want_x.abs() + 2 * REL * size + 2.0 ** -134), (err / (size + 2.0 ** -134)).max()
    # The rows' terms, each within REL, added in any order.
    terms = (d * x * r).abs().sum(0)
    assert torch.all((dw.cpu().double() - want_w).abs() <= (REL + h.shape[0] * ULP) * terms + 2.0 ** -140)
    dx2, _ = _backward(h, weight, dy, dh, eps, want_weight=False)
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 2, 5])
def test_gradient_widths(rows, width):
    for i, (dtype, res) in enumerate([(torch.bfloat16, True), (torch.float32, False)]):
        _check_backward(_bf16((rows, width), width + i, 3.0), _weight(width, dtype), _bf16((rows, width), 5 + i),
                        _bf16((rows, width), 9) if res else None)


@pytest.mark.parametrize("rows,width", [(333, 4096), (511, 272), (512, 272), (513, 1024), (1030, 144), (4097, 16), (700, 7168),
                                        (520, 16400), (2100, 128), (1100, 512), (8192, 256), (8191, 176), (8213, 208),
                                        (16385, 128), (16384, 16), (20001, 80), (30001, 240)])
def test_gradient_rows(rows, width):
    _check_backward(_bf16((rows, width), 1, 3.0), _weight(width, torch.bfloat16), _bf16((rows, width), 2),
                    _bf16((rows, width), 3))


def test_gradient_of_no_rows():
    none = torch.zeros((0, 144), dtype=torch.bfloat16)
    _, dw = _backward(none, _weight(144, torch.float32), none)
    assert torch.all(dw == 0)


def test_gradient_of_empty_and_tiny_rows():
    h = torch.zeros((4, 128), dtype=torch.bfloat16)
    h[1] = 2.0 ** -100
    h[2, 5] = 1.0
    dy = _bf16((4, 128), 3)
    _check_backward(h, _weight(128, torch.float32), dy, None)


def test_gradient_against_differences():
    """The change of sum(y dy) under small changes of single values, the forward pass in float64."""
    h, w, dy = _bf16((3, 48), 1, 2.0), _weight(48, torch.float32), _bf16((3, 48), 2)
    dx, dw = _backward(h, w, dy)
    value = lambda hh, ww: float((R.rms_norm(hh, ww, 1e-6) * dy.double()).sum())  # noqa: E731
    step = 1e-5  # central differences: error step^2 times a third derivative of order 10
    for i, j in ((0, 0), (1, 17), (2, 47)):
        up, down = h.double().clone(), h.double().clone()
        up[i, j] += step
        down[i, j] -= step
        want = (value(up, w) - value(down, w)) / (2 * step)
        assert abs(float(dx[i, j]) - want) <= BF16 * abs(want) + 1e-5
        up, down = w.double().clone(), w.double().clone()
        up[j] += step
        down[j] -= step
        want = (value(h, up) - value(h, down)) / (2 * step)
        assert abs(float(dw[j]) - want) <= 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("target", ["grad_y", "grad_h"])
def test_gradient_in_place(target):
    h, w = _bf16((600, 2064), 1).to(DEV), _weight(2064, torch.float32).to(DEV)
    grads = {"grad_y": _bf16((600, 2064), 2).to(DEV), "grad_h": _bf16((600, 2064), 3).to(DEV)}
    want, _ = _backward(h, w, grads["grad_y"], grads["grad_h"])
    M.dispatch_rms_norm_backward(h, w, grads["grad_y"], 1e-6, grads[target], grad_h=grads["grad_h"])
    assert torch.equal(grads[target], want)


def test_results_repeat_bit_for_bit():
    h, w, dy = _bf16((3000, 2064), 1), _weight(2064, torch.bfloat16), _bf16((3000, 2064), 2)
    first = _backward(h, w, dy)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, _backward(h, w, dy)))


def test_rows_beyond_32_bit_offsets():
    rows, width = 33000, 65536
    assert rows * width > 2 ** 31
    x = torch.empty((rows, width), dtype=torch.bfloat16, device=DEV)
    x.fill_(1.0)
    tail = _bf16((3, width), 4)
    x[-3:] = tail.to(DEV)
    w = _weight(width, torch.bfloat16)
    y, q = torch.empty_like(x), torch.empty((rows, width), dtype=torch.uint8, device=DEV)
    sf = torch.empty((rows, width // 128), device=DEV)
    M.dispatch_rms_norm(x, w.to(DEV), 1e-6, y=y, q=q, sf=sf)
    want = R.rms_norm(tail, w, 1e-6)
    _close_bf16(y[-3:], want, REL)
    layer_reference.assert_quantised(q[-3:].view(torch.float8_e4m3fn).float().cpu(), sf[-3:].cpu(), want, REL + 4 * ULP)
    dy = torch.zeros_like(x)
    dtail = _bf16((3, width), 5)
    dy[-3:] = dtail.to(DEV)
    dw = torch.empty(width, device=DEV)
    M.dispatch_rms_norm_backward(x, w.to(DEV), dy, 1e-6, y, grad_weight=dw,
                                 workspace=M.alloc_rms_norm_workspace(rows, width, DEV))
    want_x, want_w = R.rms_norm_gradient(tail, w, dtail, 1e-6)
    size = dtail.double().abs() * w.double() + tail.double().abs() * (dtail.double() * w.double() * tail.double()).abs().mean(1, keepdim=True)
    assert torch.all((y[-3:].cpu().double() - want_x).abs() <= BF16 * want_x.abs() + 4 * REL * size)
    assert torch.all((dw.cpu().double() - want_w).abs() <= 2 * REL * (dtail.double() * tail.double()).abs().sum(0))


@pytest.mark.parametrize("rows,width", [(4300000, 16), (2100200, 1040)])
def test_more_rows_than_the_grid_holds(rows, width):
    """The same 100 rows again and again: every repetition gives the same bits."""
    some = _bf16((100, width), 6).to(DEV)
    x = some.repeat(rows // 100, 1)
    w = _weight(width, torch.bfloat16).to(DEV)
    y = torch.empty_like(x)
    M.dispatch_rms_norm(x, w, 1e-6, y=y)
    _close_bf16(y[:100], R.rms_norm(some.cpu(), w.cpu(), 1e-6), REL)
    assert torch.all(y.view(-1, 100, width) == y[:100])
    dx = y
    M.dispatch_rms_norm_backward(x, w, x, 1e-6, dx)
    want, _ = R.rms_norm_gradient(some.cpu(), w.cpu(), some.cpu(), 1e-6)
    size = some.cpu().double().abs() * 2 + some.cpu().double().abs() * some.cpu().double().pow(2).mean(1, keepdim=True) * 2
    assert torch.all((dx[:100].cpu().double() - want).abs() <= BF16 * want.abs() + 4 * REL * size)
    assert torch.all(dx.view(-1, 100, width) == dx[:100])


@pytest.mark.parametrize("rows,width,valid", [(600, 16400, 300), (700, 7168, 511), (3000, 528, 1), (2000, 40000, 1999),
                                              (9000, 176, 8201), (20000, 112, 5), (16384, 128, 16381), (8192, 256, 0)])
def test_valid_rows_of_large_batches(rows, width, valid):
    x, w = _bf16((rows, width), 1).to(DEV), _weight(width, torch.float32).to(DEV)
    n = torch.tensor([valid], dtype=torch.int32, device=DEV)
    y, dx = torch.full_like(x, -7.0), torch.full_like(x, -7.0)
    dw, short = torch.empty(width, device=DEV), torch.empty(width, device=DEV)
    M.dispatch_rms_norm(x, w, 1e-6, y=y, num_valid_rows=n)
    M.dispatch_rms_norm_backward(x, w, x, 1e-6, dx, grad_weight=dw, num_valid_rows=n,
                                 workspace=M.alloc_rms_norm_workspace(rows, width, DEV))
    assert torch.all(y[valid:] == -7) and torch.all(dx[valid:] == -7)
    want_y, want_x = torch.empty_like(x[:valid]), torch.empty_like(x[:valid])
    M.dispatch_rms_norm(x[:valid], w, 1e-6, y=want_y)
    M.dispatch_rms_norm_backward(x[:valid], w, x[:valid], 1e-6, want_x, grad_weight=short,
                                 workspace=M.alloc_rms_norm_workspace(valid, width, DEV))
    # (Fewer rows may be cut otherwise: their sums are added in another order, and a bf16 rounding may turn.)
    near = lambda a, b: torch.all((a.double() - b.double()).abs() <= 2 * BF16 * b.double().abs() + 1e-5)  # noqa: E731
    assert near(y[:valid], want_y) and near(dx[:valid], want_x)
    terms = (x[:valid].double().pow(2) * (x[:valid].double().pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()).sum(0)
    assert torch.all((dw.double() - short.double()).abs() <= 2 * (REL + valid * ULP) * terms)


def test_plans_streams_and_a_graph():
    rows, width = 200, 1040
    w = _weight(width, torch.bfloat16).to(DEV)
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731

    def plans(stream=None):
        b = dict(x=new(rows, width), res=new(rows, width), h=new(rows, width), y=new(rows, width),
                 q=new(rows, width, dtype=torch.uint8), sf=new(rows, 9, dtype=torch.float32), dy=new(rows, width),
                 dx=new(rows, width), dw=new(width, dtype=torch.float32), ws=M.alloc_rms_norm_workspace(rows, width, DEV))
        return b, (M.RmsNormPlan(b["x"], w, 1e-6, residual=b["res"], h=b["h"], y=b["y"], q=b["q"], sf=b["sf"], stream=stream),
                   M.RmsNormBackwardPlan(b["h"], w, b["dy"], 1e-6, b["dx"], grad_h=b["y"], grad_weight=b["dw"],
                                         workspace=b["ws"], stream=stream))

    names, ins = ("h", "y", "q", "sf", "dx", "dw"), ("x", "res", "dy")
    batches = [{k: _bf16((rows, width), 10 * i + j).to(DEV) for j, k in enumerate(ins)} for i in range(3)]
    eager = []
    for batch in batches:
        b, steps = plans()
        for k in ins:
            b[k].copy_(batch[k])
        for step in steps:
            step()
        eager.append({k: b[k].clone() for k in names})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    here, there = plans(), plans(side)
    for k in ins:
        here[0][k].copy_(batches[0][k])
        there[0][k].copy_(batches[1][k])
    side.wait_stream(torch.cuda.current_stream())
    for a, b in zip(here[1], there[1]):  # two calls at once
        a()
        b()
    torch.cuda.synchronize()
    for b, want in ((here[0], eager[0]), (there[0], eager[1])):
        assert all(torch.equal(b[k], want[k]) for k in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        for step in there[1]:
            step()
    for _ in range(2):
        for batch, want in zip(batches, eager):
            for k in ins:
                there[0][k].copy_(batch[k])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(there[0][k], want[k]) for k in names)
            here[1][0]()  # eager work in between


def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV), torch.ones(256, device=DEV)
    y, sf = torch.empty_like(x), torch.empty((4, 2), device=DEV)
    q = torch.empty((4, 256), dtype=torch.uint8, device=DEV)
    for bad in (x.float(), x.t(), x[0], x.cpu()):
        with pytest.raises(ValueError, match="x must be"):
            M.dispatch_rms_norm(bad, w, 1e-6, y=y)
    for kw, match in ((dict(weight=w[:255]), "weight"), (dict(weight=w.half()), "weight"), (dict(y=y[:3]), "y holds"),
                      (dict(q=q[:3], sf=sf), "q holds"), (dict(q=q, sf=sf[:3]), "sf holds"), (dict(y=y.float()), "y must be"),
                      (dict(y=y, residual=x[:3], h=x), "residual"), (dict(y=y, num_valid_rows=torch.ones(1, device=DEV)), "num_valid")):
        args = dict(dict(weight=w, eps=1e-6, y=None), **kw)
        with pytest.raises(ValueError, match=match):
            M.dispatch_rms_norm(x, **args)
    for kw in (dict(), dict(y=y, residual=x), dict(y=y, h=x), dict(q=q), dict(y=y, eps=0.0)):
        with pytest.raises(M.DispatchError):
            M.dispatch_rms_norm(x, w, **dict(dict(eps=1e-6), **kw))
    with pytest.raises(M.DispatchError):
        M.dispatch_rms_norm_backward(x, w, x, 1e-6, y, grad_weight=torch.empty(256, device=DEV))
    with pytest.raises(ValueError, match="grad_x"):
        M.dispatch_rms_norm_backward(x, w, x, 1e-6, y[:3])


@pytest.mark.parametrize("rows,width", [(6, 256), (6, 2064), (6, 16400), (16800, 128), (8400, 256), (1200, 4096)])
@pytest.mark.parametrize("same", [True, False])
def test_gradient_at_the_ends_of_the_range(rows, width, same):
    """A row whose squares pass fp32's range has r = 0: what comes along the residual goes on as it is, whether
    the sum of grad_y w h is infinite too (same signs) or has no value (either sign)."""
    top = torch.finfo(torch.bfloat16).max
    h = torch.zeros((6, width), dtype=torch.bfloat16)
    h[1] = 2.0 ** -120
    h[2, 5] = 2.0 ** 60
    h[3] = 2.0 ** 48
    h[4], h[5] = top, -1.0
    h = h.repeat(rows // 6, 1)
    past = torch.arange(rows) % 6 == 4
    dy = torch.ones((rows, width), dtype=torch.bfloat16) if same else _bf16((rows, width), 2)
    dh, w = _bf16((rows, width), 3), torch.ones(width)
    for add in (None, dh):
        dx, dw = _backward(h, w, dy, add)
        dx, dw = dx.cpu(), dw.cpu().double()
        assert torch.all(dx[past] == (0.0 if add is None else dh[past]))
        x, d = h[~past].double(), dy[~past].double()
        want_x, want_w = R.rms_norm_gradient(h[~past], w, dy[~past], 1e-6, None if add is None else dh[~past])
        r = (x.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
        # As in _check_backward.
        size = (r * d).abs() + (r * x * r).abs() * (d * x * r).abs().mean(1, keepdim=True)
        size = size + (0.0 if add is None else dh[~past].double().abs())
        assert torch.all((dx[~past].double() - want_x).abs() <= BF16 * want_x.abs() + 2 * REL * size + 2.0 ** -134)
        assert torch.all((dw - want_w).abs() <= (REL + h.shape[0] * ULP) * (d * x * r).abs().sum(0) + 2.0 ** -140)
    # What is no number stays one.
    h[3, 3], h[5, 7], dy[4, 9] = math.inf, math.nan, math.nan
    dx, dw = _backward(h, w, dy, dh)
    dx = dx.cpu()
    assert math.isnan(float(dx[3, 3])) and torch.all(torch.isnan(dx[5])) and math.isnan(float(dx[4, 9]))
    assert all(math.isnan(float(dw[i])) for i in (3, 7, 9))


def _weight_gradient(h, dy, eps=1e-6):
    """(the weight's gradient in float64, the sums of its terms' magnitudes) of device rows."""
    x, d = h.double(), dy.double()
    terms = d * x * (x.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    return terms.sum(0), terms.abs().sum(0)


# Up to 8 rows a lane, 2 joins of a wavefront's rows, 16 wavefronts or rows of a workgroup, then the rows of
# sums: up to 6 for each of 128 groups of threads, 3 joins and 16 wavefronts: 51 additions in a row.
CHAIN = 51 * ULP


# 16, 32 and 64 lanes a row and several wavefronts, for each a shape whose last row is alone in its round of the grid.
@pytest.mark.parametrize("rows,width,valid", [(16385, 128, None), (16384, 16, None), (20001, 80, None), (8193, 240, None),
                                              (30001, 240, None), (4097, 512, None), (8213, 208, None), (3073, 1040, None),
                                              (1025, 4096, None), (769, 2064, None), (513, 7168, None), (257, 16400, None),
                                              (9000, 176, 8201), (16384, 128, 16381), (600, 4096, 513)])
def test_gradient_of_the_weight_has_every_row(rows, width, valid):
    h, dy = (_bf16((rows, width), seed).to(DEV) for seed in (1, 2))
    w, last = _weight(width, torch.bfloat16), (valid or rows) - 1
    n = None if valid is None else torch.tensor([valid], dtype=torch.int32)
    _, dw = _backward(h, w, dy, valid=n)
    want, size = _weight_gradient(h[:last + 1], dy[:last + 1])
    bound = (REL + CHAIN) * size
    assert torch.all((dw.double() - want).abs() <= bound)
    # The bound sees any one row that is left out.
    for row in (0, last // 2, last):
        less = want - _weight_gradient(h[row:row + 1], dy[row:row + 1])[0]
        assert torch.any((less - want).abs() > 4 * bound)
    # And of nothing but that row.
    for row in (0, last // 2, last):
        one = torch.zeros_like(dy)
        one[row] = dy[row]
        _, dw = _backward(h, w, one, valid=n)
        want_one, size_one = _weight_gradient(h[row:row + 1], dy[row:row + 1])
        assert torch.all((dw.double() - want_one).abs() <= REL * size_one)


# 16 and 32 lanes a row, and a wavefront a row: 1050000, 1050000 and 1075000 workgroups' rows for a grid of 2^20.
@pytest.mark.parametrize("rows,width", [(16800000, 16), (8400000, 144), (4300000, 272)])
def test_more_narrow_rows_than_the_grid_holds(rows, width):
    test_more_rows_than_the_grid_holds(rows, width)


# Four vectors a lane and eight, which the gradient loads again for its second look.
@pytest.mark.parametrize("rows,width", [(3, 16400), (520, 16400), (3, 40000), (300, 40000)])
def test_wide_rows_in_place(rows, width):
    a, b, c = (_bf16((rows, width), seed).to(DEV) for seed in (1, 2, 3))
    w = _weight(width, torch.float32).to(DEV)
    want_h, want_y, _, _ = _forward(a, w, residual=b, outs="bf16")
    want_x, want_w = _backward(a, w, b, c)
    for target in (0, 1):
        x, res, y = a.clone(), b.clone(), torch.empty_like(a)
        h = (x, res)[target]
        M.dispatch_rms_norm(x, w, 1e-6, residual=res, h=h, y=y)
        assert torch.equal(h, want_h) and torch.equal(y, want_y)
        dy, dh, dw = b.clone(), c.clone(), torch.empty(width, device=DEV)
        dx = (dy, dh)[target]
        M.dispatch_rms_norm_backward(a, w, dy, 1e-6, dx, grad_h=dh, grad_weight=dw,
                                     workspace=M.alloc_rms_norm_workspace(rows, width, DEV))
        assert torch.equal(dx, want_x) and torch.equal(dw, want_w)
