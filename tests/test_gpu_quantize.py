"""Quantisation to fp8 with block scales, of rows, of SwiGLU and of its gradient."""

import math

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import layer_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 2.0 ** -24


def _rows(r, w, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((r, w), generator=g)).to(torch.bfloat16)


def _out(r, w):
    q = torch.full((max(r, 1), w), 0x5A, dtype=torch.uint8, device=DEV)[:r]
    sf = torch.full((max(r, 1), -(-w // 128)), -7.0, device=DEV)[:r]
    return q, sf


def _values(q):
    return q.view(R.FP8).float().cpu()


@pytest.mark.parametrize("r", [0, 1, 2, 17, 300])
@pytest.mark.parametrize("w", [16, 112, 128, 144, 512, 2880, 7168])
def test_rows(r, w):
    x = _rows(r, w, 10 * r + w)
    q, sf = _out(r, w)
    M.dispatch_quantize(x.to(DEV), q, sf)
    # bf16 inputs are exact; the scale and the quotient round a few times.
    R.assert_quantised(_values(q), sf.cpu(), x.double(), 4 * EPS)


def test_rows_equal_the_fp32_formula_bit_for_bit():
    x = _rows(500, 1024, 3, 5.0).to(DEV)
    q, sf = _out(500, 1024)
    M.dispatch_quantize(x, q, sf)
    blocks = x.float().view(500, 8, 128)
    amax = blocks.abs().amax(2).clamp_min(2.0 ** -100)
    top = torch.full_like(amax, 448.0)  # (torch turns a division by a number into a product)
    assert torch.equal(sf, amax / top)
    want = (blocks * (top / amax)[:, :, None]).view(500, 1024).to(R.FP8)
    assert torch.equal(q, want.view(torch.uint8))


def test_edges_of_the_range():
    x = torch.zeros((8, 256), dtype=torch.bfloat16)
    x[1] = 2.0 ** -130                       # below the floor
    x[2, 0], x[2, 1:] = 2.0 ** 100, 1.0      # all but one value vanish
    x[3] = torch.finfo(torch.bfloat16).max
    x[4, ::2] = -torch.finfo(torch.bfloat16).max
    x[5, 7] = math.inf
    x[6, 200] = math.nan
    x[7, 128:] = -3.0
    q, sf = _out(8, 256)
    M.dispatch_quantize(x.to(DEV), q, sf)
    v, s = _values(q), sf.cpu()
    keep = [0, 1, 2, 3, 4, 7]
    R.assert_quantised(v[keep], s[keep], x[keep].double(), 4 * EPS)
    assert torch.all(s[0] == torch.tensor(2.0 ** -100) / 448.0) and torch.all(v[0] == 0)
    assert math.isinf(float(s[5, 0])) and math.isnan(float(v[5, 7])) and math.isfinite(float(s[5, 1]))
    assert math.isnan(float(s[6, 1])) and torch.all(torch.isnan(v[6, 128:])) and math.isfinite(float(s[6, 0]))


@pytest.mark.parametrize("r,w", [(1, 128), (3, 256), (37, 2048), (260, 384)])
def test_swiglu(r, w):
    h = _rows(r, 2 * w, r + w, 2.0)
    q, sf = _out(r, w)
    M.dispatch_swiglu_quantize(h.to(DEV), q, sf)
    # exp to about an ulp, a division and two products: a few roundings.
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu(h), 16 * EPS)


@pytest.mark.parametrize("r,w", [(1, 128), (3, 256), (37, 2048), (260, 384)])
def test_swiglu_gradient(r, w):
    h, d = _rows(r, 2 * w, r + w, 2.0), _rows(r, w, r + w + 1)
    q, sf = _out(r, 2 * w)
    M.dispatch_swiglu_backward_quantize(h.to(DEV), d.to(DEV), q, sf)
    # 1 + g (1 - s) cancels near g = -1.28: its roundings count against |g|.
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu_gradient(h, d), 64 * EPS)


def test_swiglu_gradient_against_differences():
    h, d = _rows(2, 256, 5), _rows(2, 128, 6)
    q, sf = _out(2, 256)
    M.dispatch_swiglu_backward_quantize(h.to(DEV), d.to(DEV), q, sf)
    got = _values(q).double() * sf.cpu().double().repeat_interleave(128, 1)
    step = 1e-5
    for i, j in ((0, 0), (0, 130), (1, 77), (1, 255)):
        up, down = h.double().clone(), h.double().clone()
        up[i, j] += step
        down[i, j] -= step
        slope = float(((R.swiglu(up) - R.swiglu(down)) * d.double()).sum()) / (2 * step)
        # e4m3 keeps 4 bits, and subnormals below 2^-6 of the scale.
        bound = max(abs(slope) / 16, float(sf[i, j // 128]) * 2.0 ** -10) + 1e-8
        assert abs(float(got[i, j]) - slope) <= bound


def test_far_arguments_of_swiglu():
    h = torch.zeros((1, 256), dtype=torch.bfloat16)
    h[0, :6] = torch.tensor([-1000.0, -100.0, -60.0, 60.0, 100.0, 1000.0])
    h[0, 128:] = 1.0
    q, sf = _out(1, 128)
    M.dispatch_swiglu_quantize(h.to(DEV), q, sf)
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu(h), 16 * EPS)
    d = torch.ones((1, 128), dtype=torch.bfloat16)
    q, sf = _out(1, 256)
    M.dispatch_swiglu_backward_quantize(h.to(DEV), d.to(DEV), q, sf)
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu_gradient(h, d), 64 * EPS)


@pytest.mark.parametrize("valid", [-3, 0, 1, 5, 9, 100])
def test_rows_past_the_valid_ones_are_not_touched(valid):
    r, w = 9, 256
    n = torch.tensor([valid], dtype=torch.int32, device=DEV)
    live = max(0, min(valid, r))
    x, h, d = (t.to(DEV) for t in (_rows(r, w, 1), _rows(r, 2 * w, 2), _rows(r, w, 3)))
    for call, width, full in (
            (lambda q, sf, n: M.dispatch_quantize(x, q, sf, n), w, x),
            (lambda q, sf, n: M.dispatch_swiglu_quantize(h, q, sf, n), w, h),
            (lambda q, sf, n: M.dispatch_swiglu_backward_quantize(h, d, q, sf, n), 2 * w, h)):
        q0, sf0 = _out(r, width)
        call(q0, sf0, None)
        q, sf = _out(r, width)
        call(q, sf, n)
        assert torch.equal(q[:live], q0[:live]) and torch.equal(sf[:live], sf0[:live])
        assert torch.all(q[live:] == 0x5A) and torch.all(sf[live:] == -7.0)


def test_rows_beyond_32_bit_offsets():
    """The last rows of a buffer of more than 2^32 bytes."""
    w = 8192
    r = (1 << 32) // (2 * w) + 3
    x = torch.zeros((r, w), dtype=torch.bfloat16, device=DEV)
    tail = _rows(5, w, 9)
    x[-5:] = tail.to(DEV)
    q, sf = torch.empty((r, w), dtype=torch.uint8, device=DEV), torch.empty((r, w // 128), device=DEV)
    M.dispatch_quantize(x, q, sf)
    R.assert_quantised(_values(q[-5:]), sf[-5:].cpu(), tail.double(), 4 * EPS)
    assert torch.all(q[:7] == 0)


def test_plans_and_streams():
    x, h, d = (t.to(DEV) for t in (_rows(50, 512, 1), _rows(50, 1024, 2), _rows(50, 512, 3)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for direct, plan, w in (
            (lambda q, s: M.dispatch_quantize(x, q, s), lambda q, s: M.QuantizePlan(x, q, s, stream=side), 512),
            (lambda q, s: M.dispatch_swiglu_quantize(h, q, s), lambda q, s: M.SwigluQuantizePlan(h, q, s, stream=side), 512),
            (lambda q, s: M.dispatch_swiglu_backward_quantize(h, d, q, s),
             lambda q, s: M.SwigluBackwardQuantizePlan(h, d, q, s, stream=side), 1024)):
        (q0, s0), (q1, s1) = _out(50, w), _out(50, w)
        side.wait_stream(torch.cuda.current_stream())
        direct(q0, s0)
        plan(q1, s1)()
        torch.cuda.synchronize()
        assert torch.equal(q0, q1) and torch.equal(s0, s1)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    q, sf = _out(4, 256)
    with pytest.raises(ValueError, match="x must be"):
        M.dispatch_quantize(x.float(), q, sf)
    with pytest.raises(ValueError, match="contiguous"):
        M.dispatch_quantize(x[:, ::2], q, sf)
    with pytest.raises(ValueError, match="q holds"):
        M.dispatch_quantize(x, q[:3], sf)
    with pytest.raises(ValueError, match="sf holds"):
        M.dispatch_quantize(x, q, sf[:3])
    with pytest.raises(ValueError, match="grad"):
        M.dispatch_swiglu_backward_quantize(x, x[:, :128], q, sf)
    with pytest.raises(M.DispatchError):
        M.dispatch_quantize(x[:, :8].contiguous(), q, sf)         # not a multiple of 16
    with pytest.raises(M.DispatchError):
        M.dispatch_swiglu_quantize(x[:, :96].contiguous(), q, sf)  # halves of 48


def _every_gate():
    """Every finite bf16 value once as the first channel of a block whose other gates are -2..2, the up values 1."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    h = torch.ones((z.numel(), 256), dtype=torch.bfloat16)
    h[:, :128] = torch.linspace(-2, 2, 128).to(torch.bfloat16)
    h[:, 0] = z
    return h


def test_swiglu_of_every_finite_gate():
    """The sigmoid is 0 or 1 far out, whatever the size of z; nothing finite becomes NaN."""
    h = _every_gate()
    q, sf = _out(h.shape[0], 128)
    M.dispatch_swiglu_quantize(h.to(DEV), q, sf)
    # As test_swiglu; the values of gates below -87 are under 2^-119, the floor of a block is 2^-100.
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu(h), 16 * EPS)


def test_swiglu_gradient_of_every_finite_gate():
    h = _every_gate()
    d = torch.ones((h.shape[0], 128), dtype=torch.bfloat16)
    q, sf = _out(h.shape[0], 256)
    M.dispatch_swiglu_backward_quantize(h.to(DEV), d.to(DEV), q, sf)
    # g (1 - s) has up to 17.3 times the sigmoid's error of 3 units (from there on s is 1), and a few roundings.
    R.assert_quantised(_values(q), sf.cpu(), R.swiglu_gradient(h, d), 64 * EPS)


def test_swiglu_of_infinite_gates():
    """g / (1 + exp(-g)): infinity stays, -infinity has no value; other blocks keep theirs."""
    h = torch.ones((2, 512), dtype=torch.bfloat16)
    h[0, 3], h[1, 3] = math.inf, -math.inf
    q, sf = _out(2, 256)
    M.dispatch_swiglu_quantize(h.to(DEV), q, sf)
    v, s = _values(q), sf.cpu()
    assert math.isinf(float(s[0, 0])) and math.isnan(float(v[0, 3])) and math.isnan(float(s[1, 0]))
    R.assert_quantised(v[:, 128:], s[:, 1:], R.swiglu(h)[:, 128:], 16 * EPS)


def test_swiglu_gradient_needs_a_gradient():
    h = torch.zeros((4, 512), dtype=torch.bfloat16, device=DEV)
    q, sf = _out(4, 512)
    for call in (M.dispatch_swiglu_backward_quantize, M.SwigluBackwardQuantizePlan):
        with pytest.raises(ValueError, match="grad"):
            call(h, None, q, sf)


# Buffers past the Infinity Cache (256 MB read and written) take another form of
# the kernel: its first, middle and last rows against the same rows by themselves.
@pytest.mark.parametrize("name,r,w", [("rows", 12500, 7168), ("swiglu", 26300, 2048), ("swiglu_gradient", 16500, 2048)])
def test_large_buffers(name, r, w):
    g = torch.Generator(device=DEV).manual_seed(r)
    normal = lambda width: torch.randn((r, width), generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    ins = {"rows": [w], "swiglu": [2 * w], "swiglu_gradient": [2 * w, w]}[name]
    ins = [normal(width) for width in ins]
    call, width, channel_bytes = {"rows": (M.dispatch_quantize, w, 3), "swiglu": (M.dispatch_swiglu_quantize, w, 5),
                                  "swiglu_gradient": (M.dispatch_swiglu_backward_quantize, 2 * w, 8)}[name]
    assert r * w * channel_bytes > 1 << 28
    q, sf = _out(r, width)
    call(*ins, q, sf)
    assert not torch.any(sf == -7.0)
    for first in (0, r // 2, r - 100):
        part = slice(first, first + 100)
        few_q, few_sf = _out(100, width)
        call(*[x[part] for x in ins], few_q, few_sf)
        assert torch.equal(q[part], few_q) and torch.equal(sf[part], few_sf)
    n = torch.tensor([r - 50], dtype=torch.int32, device=DEV)
    q2, sf2 = _out(r, width)
    call(*ins, q2, sf2, n)
    assert torch.equal(q2[:-50], q[:-50]) and torch.equal(sf2[:-50], sf[:-50])
    assert torch.all(q2[-50:] == 0x5A) and torch.all(sf2[-50:] == -7.0)
