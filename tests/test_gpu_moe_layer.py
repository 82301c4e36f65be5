"""The gate, the fp8 dispatch, the experts' products and the combine run
together (examples/moe_layer.py) against the layer in float64, its gradients
against automatic differentiation, and captured into a HIP graph."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
L = importlib.util.module_from_spec(spec)
spec.loader.exec_module(L)

SHAPES = [(64, 256, 128, 8, 2), (300, 512, 256, 16, 4), (1, 384, 128, 6, 3)]


def _wide(q, sf):
    n, k = q.shape[1:]
    block = lambda size: torch.arange(size, device=q.device) // 128  # noqa: E731
    return q.double() * sf.double()[:, block(n)][:, :, block(k)]


def _reference(layer, x, logits, idx):
    """The layer in float64 for the choice idx, differentiable in x and logits."""
    up, down = _wide(layer.up, layer.up_sf), _wide(layer.down, layer.down_sf)
    t, k = idx.shape
    e = logits.shape[1]
    p = torch.softmax(logits, 1)
    picked = p.gather(1, idx)
    weights = picked / picked.sum(1, keepdim=True)
    h = torch.bmm(up[idx.reshape(-1)], x.repeat_interleave(k, 0)[:, :, None]).squeeze(2)
    g, u = torch.chunk(h, 2, 1)
    y = torch.bmm(down[idx.reshape(-1)], (g * torch.sigmoid(g) * u)[:, :, None]).squeeze(2).view(t, k, -1)
    count = torch.bincount(idx.reshape(-1), minlength=e).double()
    return (weights[:, :, None] * y).sum(1), 0.01 * e / (k * t * t) * (count * p.sum(0)).sum()


def _off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", SHAPES)
def test_layer_and_its_gradients(tokens, hidden, inter, experts, topk):
    layer = L.MoeLayer(tokens, hidden, inter, experts, topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16)
    out = layer.forward(x)
    dx, dlogits = layer.backward(dout)
    torch.cuda.synchronize()
    assert int(layer.lay.status) == 0
    idx = layer.route.topk_idx
    xr, zr = x.double().requires_grad_(True), layer.logits.double().requires_grad_(True)
    want, loss = _reference(layer, xr, zr, idx)
    ((want * dout.double()).sum() + loss).backward()
    # Each quantisation to e4m3 leaves a relative error of about 2^-4 / sqrt(6)
    # = 2.6 % rms of the values: two on the way forward (x and the activation)
    # give 3.6 %, and through SwiGLU's two factors up to 5 %; the gradients see
    # those and two of their own.
    assert _off(out, want.detach()) < 0.06
    assert _off(dx, xr.grad) < 0.09
    # The logits' gradient from the weights' gradient that the layer had: no
    # 8-bit value in between, bf16 at the end.
    z = layer.logits.double().requires_grad_(True)
    p = torch.softmax(z, 1)
    picked = p.gather(1, idx)
    _, loss_z = _reference(layer, x.double(), z, idx)
    ((picked / picked.sum(1, keepdim=True) * layer.dweights.double()).sum() + loss_z).backward()
    assert _off(dlogits, z.grad) < 2.0 ** -8
    assert abs(float(layer.route.loss) - float(loss)) <= 1e-5 * float(loss)


def test_layer_in_a_graph():
    """Captured once and replayed on other rows, the program's own eager work in between."""
    tokens, hidden, inter, experts, topk = 40, 512, 256, 8, 2
    layer = L.MoeLayer(tokens, hidden, inter, experts, topk, training=False)
    g = torch.Generator(device="cuda").manual_seed(2)
    batches = [torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    eager = [(layer.forward(x).clone(), layer.route.loss.clone(), layer.route.topk_idx.clone()) for x in batches]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = L.MoeLayer(tokens, hidden, inter, experts, topk, training=False)  # plans on this stream
        graph = torch.cuda.CUDAGraph()
        for step in other.steps:
            step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            for step in other.steps:
                step()
    torch.cuda.synchronize()
    for turn in range(2):
        for x, (out, loss, idx) in zip(batches, eager):
            other.x.copy_(x)
            torch.matmul(other.x, other.router.t(), out=other.logits)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(other.route.topk_idx, idx)
            assert torch.equal(other.out, out) and torch.equal(other.route.loss, loss)
            layer.forward(batches[turn])  # eager work between the replays


def test_step_times_shape(capsys, monkeypatch):
    """The example's command runs."""
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--tokens", "16", "--hidden", "256", "--inter", "128", "--experts",
                                     "8", "--topk", "2", "--steps", "2"])
    L.main()
    assert "us a layer" in capsys.readouterr().out
