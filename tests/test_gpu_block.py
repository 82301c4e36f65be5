"""The norm, the gate by groups, the dispatch, the experts' products and the
combine run together as a block (examples/moe_layer.py), forward and backward,
against the block in float64, and captured into a HIP graph."""

import importlib.util
import os

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import block_reference as R
from tests.test_gpu_moe_layer import _off, _reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
L = importlib.util.module_from_spec(spec)
spec.loader.exec_module(L)

EPS = 1e-6
# Tokens, hidden, inter, experts, entries, groups, groups taken.
SHAPES = [(64, 256, 128, 8, 2, 4, 2), (300, 512, 256, 16, 4, 4, 2), (1, 384, 128, 6, 3, 2, 1)]


def _inputs(tokens, hidden, seed, count=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16) for _ in range(count)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,groups,taken", SHAPES)
def test_block_and_its_gradients(tokens, hidden, inter, experts, topk, groups, taken):
    block = L.MoeBlock(tokens, hidden, inter, experts, topk, groups=(groups, taken))
    block.norm_weight.copy_(1.0 + 0.2 * torch.randn(hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)))
    x, residual, dout, dh = _inputs(tokens, hidden, 1)
    out, h = block.forward(x, residual)
    dx, dw = block.backward(dout, dh)
    torch.cuda.synchronize()
    assert int(block.lay.status) == 0
    assert torch.equal(h, R.rounded_sum(x, residual))
    idx = block.route.topk_idx
    want_idx, _ = R.grouped_choice(block.logits.cpu(), groups, taken, topk, False, False)
    assert torch.equal(idx.cpu(), want_idx)
    hr, wr = h.double().requires_grad_(True), block.norm_weight.double().requires_grad_(True)
    y = R.rms_norm(hr, wr, EPS)
    logits = y @ block.router.double().t()
    want, loss = _reference(block, y, logits, idx)
    ((want * dout.double()).sum() + loss + (hr * dh.double()).sum()).backward()
    # Two quantisations to e4m3 on the way forward (2.6 % each, up to 5 % through
    # SwiGLU), two more on the way back; the gradient of h has dh, exact, beside.
    assert _off(out, want.detach()) < 0.06
    assert _off(dx, hr.grad) < 0.09
    assert _off(dw, wr.grad) < 0.09
    # The norm's own gradient from the rows' gradient that the block had: bf16 at the end alone.
    want_x, want_w = R.rms_norm_gradient(h, block.norm_weight, block.dy, EPS, dh)
    assert _off(dx, want_x) < 2.0 ** -8
    assert _off(dw, want_w) < 1e-5
    # The combine's gradient: the weights' from the rows that the block had.
    slot = block.lay.expert_slot.view(tokens, topk)
    want_dw = (dout.double()[:, None, :] * block.y.double()[slot.long()]).sum(2)
    assert _off(block.dweights, want_dw) < 1e-5


def test_block_in_a_graph():
    """Forward and backward captured once and replayed on other rows, eager work in between."""
    shape = (40, 512, 256, 8, 2)
    block = L.MoeBlock(*shape, groups=(4, 2))
    batches = [_inputs(40, 512, 20 + i) for i in range(3)]
    names = ("out", "h", "dx_in", "dnorm_weight", "dlogits")
    eager = []
    for x, residual, dout, dh in batches:
        block.forward(x, residual)
        block.backward(dout, dh)
        eager.append([getattr(block, n).clone() for n in names])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = L.MoeBlock(*shape, groups=(4, 2))  # plans on this stream

        def parts():
            first = [other.norm]
            second = other.steps + other.back
            return first, second

        first, second = parts()
        for step in first + second:
            step()
        side.synchronize()
        graphs = [torch.cuda.CUDAGraph() for _ in range(3)]
        for graph, steps in zip(graphs, (first, second, [other.norm_back])):
            with torch.cuda.graph(graph, stream=side):
                for step in steps:
                    step()
    torch.cuda.synchronize()
    for _ in range(2):
        for (x, residual, dout, dh), want in zip(batches, eager):
            for to, value in ((other.x_in, x), (other.residual, residual), (other.dout, dout), (other.dh, dh)):
                to.copy_(value)
            torch.cuda.synchronize()
            graphs[0].replay()
            torch.cuda.synchronize()
            torch.matmul(other.x, other.router.t(), out=other.logits)
            torch.cuda.synchronize()
            graphs[1].replay()
            torch.cuda.synchronize()
            torch.addmm(other.dx, other.dlogits, other.router, out=other.dy)
            torch.cuda.synchronize()
            graphs[2].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(getattr(other, n), w) for n, w in zip(names, want))
            block.forward(x, residual)  # eager work between the replays


def test_a_token_reaches_few_ranks():
    """With a group for each rank the dispatch sends a token to at most as many ranks as groups are taken."""
    tokens, experts, ranks, taken, topk = 500, 64, 8, 3, 6
    z = torch.randn((tokens, experts), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(torch.bfloat16)
    p = M.make_gate_problem(tokens, experts, topk, M.GATE_SIGMOID)
    route = M.alloc_gate(p, "cuda")
    M.dispatch_gate_grouped(p, M.make_gate_groups(ranks, taken, 2), z, route, M.alloc_gate_workspace(p, "cuda"))
    prob = M.make_problem(tokens, topk, experts, ranks, 1, row_bytes=64)
    lay = M.alloc_layout(prob, "cuda")
    M.dispatch_layout(prob, route.topk_idx, lay, M.alloc_workspace(prob, "cuda"))
    torch.cuda.synchronize()
    assert int(lay.status) == 0 and torch.equal(lay.expert_count, route.expert_count)
    ranks_of = (lay.rank_slot.view(tokens, topk) >= 0).sum(1)
    assert int(ranks_of.max()) <= taken and int(lay.rank_psum[-1]) == int(ranks_of.sum())


def test_command_runs_the_block(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--tokens", "16", "--hidden", "256", "--inter", "128", "--experts", "8",
                                     "--topk", "2", "--steps", "2", "--groups", "4", "--topk-groups", "2", "--norm"])
    L.main()
    assert "us a layer" in capsys.readouterr().out
