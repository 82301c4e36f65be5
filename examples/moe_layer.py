"""An expert layer on one GPU: gate, fp8 dispatch, the experts' products, combine.

    python examples/moe_layer.py [--tokens 4096] [--hidden 7168] [--inter 2048] [--experts 32] [--topk 8]

forward():  logits -> dispatch_gate -> topk_idx, topk_weights (and the balance loss)
            x -> dispatch_quantize -> dispatch_layout_and_scatter -> expert-major fp8 rows
            -> dispatch_expert_product_swiglu -> dispatch_expert_product -> dispatch_combine
backward(): the gradients of the layer's input and of the logits, the experts'
            weights fixed: the same products with the weights laid out
            transposed, SwiGLU's gradient from the up product kept in bf16, and
            dispatch_gate_backward. (The combine's own gradient is a gather and
            a product of rows, in torch.)

Every call is prepared once; a step is one C call each.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_token_dispatch_amd as M  # noqa: E402

FP8 = torch.float8_e4m3fn
BLOCK = M.SF_BLOCK


def quantise_weights(w):
    """[E, N, K] weights to fp8 with one fp32 scale per 128 x 128 block."""
    e, n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    full = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(e, nb, BLOCK, kb, BLOCK).float()
    amax = full.abs().amax(dim=(2, 4)).clamp_min(2.0 ** -100)
    q = (full * (448.0 / amax)[:, :, None, :, None]).to(FP8).view(e, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous()
    return q, amax / 448.0


def transposed(q, sf):
    """The weights for the rows' gradient."""
    return q.view(torch.uint8).transpose(1, 2).contiguous().view(FP8), sf.transpose(1, 2).contiguous()


class MoeLayer:
    def __init__(self, tokens, hidden, inter, experts, topk, device="cuda", alignment=16, seed=0, loss_coef=0.01,
                 training=True):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
        self.up, self.up_sf = quantise_weights(normal(experts, 2 * inter, hidden) * hidden ** -0.5)
        self.down, self.down_sf = quantise_weights(normal(experts, hidden, inter) * inter ** -0.5)
        self.router = (normal(experts, hidden) * hidden ** -0.5).to(torch.bfloat16)

        new = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        self.x, self.x_q = new((tokens, hidden), torch.bfloat16), new((tokens, hidden), FP8)
        self.x_sf = new((tokens, -(-hidden // BLOCK)), torch.float32)
        self.logits, self.out = new((tokens, experts), torch.bfloat16), new((tokens, hidden), torch.bfloat16)

        gate = M.make_gate_problem(tokens, experts, topk, M.GATE_SOFTMAX, self.logits.dtype, loss_coef=loss_coef)
        self.route = M.alloc_gate(gate, device)
        self.prob = M.make_problem(tokens, topk, experts, 1, alignment, row_bytes=hidden, sf_per_token=self.x_sf.shape[1],
                                   flags=M.EXPERT_MAJOR | M.ZERO_PAD)
        self.lay, ws, self.rows = (M.alloc_layout(self.prob, device), M.alloc_workspace(self.prob, device),
                                   M.alloc_rows(self.prob, device))
        cap = self.prob.recv_capacity_rows
        a, a_sf = new((cap, inter), FP8), new((cap, inter // BLOCK), torch.float32)
        self.y = new((cap, hidden), torch.bfloat16)
        layout = (self.lay.expert_psum, self.lay.expert_count)
        rows = (self.rows.recv_x, self.rows.recv_sf)
        pairs = tokens * topk
        up = M.make_expert_problem(experts, hidden, 2 * inter, cap, pairs)
        down = M.make_expert_problem(experts, inter, hidden, cap, pairs)
        self.steps = [
            M.GatePlan(gate, self.logits, self.route, M.alloc_gate_workspace(gate, device)),
            M.QuantizePlan(self.x, self.x_q, self.x_sf),
            M.Plan(self.prob, self.route.topk_idx, self.lay, ws, self.x_q.view(torch.uint8), self.x_sf, self.rows),
            M.ExpertSwigluPlan(up, *layout, *rows, self.up, self.up_sf, a, a_sf),
            M.ExpertProductPlan(down, *layout, a, a_sf, self.down, self.down_sf, self.y),
            M.CombinePlan(self.lay.expert_slot, self.route.topk_weights, self.y, self.out),
        ]
        if not training:
            return
        # Backward: dy -> da (down transposed) -> dh (SwiGLU) -> dx of each row (up transposed) -> dx of each token.
        total = self.lay.expert_psum[-1:]
        self.dy = new((cap, hidden), torch.bfloat16)
        dy_q, dy_sf = new((cap, hidden), FP8), new((cap, self.x_sf.shape[1]), torch.float32)
        h, da = new((cap, 2 * inter), torch.bfloat16), new((cap, inter), torch.bfloat16)
        dh_q, dh_sf = new((cap, 2 * inter), FP8), new((cap, 2 * inter // BLOCK), torch.float32)
        row_dx, self.dx = new((cap, hidden), torch.bfloat16), new((tokens, hidden), torch.bfloat16)
        self.dweights, self.dloss = new((tokens, topk), torch.float32), torch.ones(1, device=device)
        self.dlogits, ones = torch.zeros_like(self.logits), torch.ones((tokens, topk), device=device)
        up_t, down_t = transposed(self.up, self.up_sf), transposed(self.down, self.down_sf)
        self.back = [
            M.QuantizePlan(self.dy, dy_q, dy_sf, num_valid_rows=total),
            M.ExpertProductPlan(M.make_expert_problem(experts, hidden, inter, cap, pairs), *layout, dy_q, dy_sf, *down_t, da),
            M.ExpertProductPlan(up, *layout, *rows, self.up, self.up_sf, h),
            M.SwigluBackwardQuantizePlan(h, da, dh_q, dh_sf, num_valid_rows=total),
            M.ExpertProductPlan(M.make_expert_problem(experts, 2 * inter, hidden, cap, pairs), *layout, dh_q, dh_sf, *up_t,
                                row_dx),
            M.CombinePlan(self.lay.expert_slot, ones, row_dx, self.dx),
            M.GateBackwardPlan(gate, self.logits, self.route, self.dweights, self.dloss, self.dlogits),
        ]

    def forward(self, x):
        """x [T, H] bf16 -> out [T, H] bf16; the balance loss is self.route.loss."""
        self.x.copy_(x)
        torch.matmul(self.x, self.router.t(), out=self.logits)
        for step in self.steps:
            step()
        return self.out

    def backward(self, dout):
        """dout [T, H] -> gradients of x through the experts and of the logits (weights, and the loss with gradient 1)."""
        slot = self.lay.expert_slot.long()
        live = slot >= 0
        at = slot.clamp_min(0)
        d = dout.float()[:, None, :].expand(-1, slot.shape[1], -1)
        self.dweights.copy_(torch.where(live, (d * self.y[at].float()).sum(-1), 0.0))
        self.dy[slot[live]] = (self.route.topk_weights[:, :, None] * d)[live].to(torch.bfloat16)
        for step in self.back:
            step()
        return self.dx, self.dlogits


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 7168), ("inter", 2048), ("experts", 32), ("topk", 8), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer = MoeLayer(a.tokens, a.hidden, a.inter, a.experts, a.topk, training=False)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    for _ in range(3):
        layer.forward(x)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        layer.forward(x)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / a.steps * 1e6
    flops = 6.0 * a.tokens * a.topk * a.hidden * a.inter
    print(f"{a.tokens} tokens x {a.hidden}, top-{a.topk} of {a.experts} experts of width {a.inter}: {us:.1f} us a layer, "
          f"{flops / us / 1e6:.0f} TFLOP/s of expert products, balance loss {float(layer.route.loss):.5f}")


if __name__ == "__main__":
    main()
