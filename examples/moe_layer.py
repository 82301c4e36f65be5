"""An expert layer on one GPU: gate, fp8 dispatch, the experts' products, combine.

    python examples/moe_layer.py [--tokens 4096] [--hidden 7168] [--inter 2048] [--experts 32] [--topk 8]
                                 [--groups 8 --topk-groups 4] [--norm]

forward():  logits -> dispatch_gate -> topk_idx, topk_weights (and the balance loss)
            x -> dispatch_quantize -> dispatch_layout_and_scatter -> expert-major fp8 rows
            -> dispatch_expert_product_swiglu -> dispatch_expert_product -> dispatch_combine
backward(): the gradients of the layer's input and of the logits, the experts'
            weights fixed: the same products with the weights laid out
            transposed, SwiGLU's gradient from the up product kept in bf16,
            dispatch_combine_backward before them and dispatch_gate_backward.

MoeBlock is the layer behind its norm: dispatch_rms_norm adds the residual and
gives the router its bf16 rows and the dispatch its fp8 rows, in place of
dispatch_quantize; dispatch_rms_norm_backward takes the gradient back.

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
                 training=True, groups=None):
        """groups: (groups of experts, groups that a token's experts come from), or None."""
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
        gate_ws = M.alloc_gate_workspace(gate, device)
        self.steps = [
            M.GatePlan(gate, self.logits, self.route, gate_ws) if groups is None else
            M.GroupedGatePlan(gate, M.make_gate_groups(*groups), self.logits, self.route, gate_ws),
            M.QuantizePlan(self.x, self.x_q, self.x_sf),
            M.Plan(self.prob, self.route.topk_idx, self.lay, ws, self.x_q.view(torch.uint8), self.x_sf, self.rows),
            M.ExpertSwigluPlan(up, *layout, *rows, self.up, self.up_sf, a, a_sf),
            M.ExpertProductPlan(down, *layout, a, a_sf, self.down, self.down_sf, self.y),
            M.CombinePlan(self.lay.expert_slot, self.route.topk_weights, self.y, self.out),
        ]
        if not training:
            return
        # Backward: dout -> dy of each row -> da (down transposed) -> dh (SwiGLU) -> dx of each row (up transposed)
        # -> dx of each token.
        total = self.lay.expert_psum[-1:]
        self.dout = new((tokens, hidden), torch.bfloat16)
        dy_q, dy_sf = new((cap, hidden), FP8), new((cap, self.x_sf.shape[1]), torch.float32)
        h, da = new((cap, 2 * inter), torch.bfloat16), new((cap, inter), torch.bfloat16)
        dh_q, dh_sf = new((cap, 2 * inter), FP8), new((cap, 2 * inter // BLOCK), torch.float32)
        row_dx, self.dx = new((cap, hidden), torch.bfloat16), new((tokens, hidden), torch.bfloat16)
        self.dweights, self.dloss = new((tokens, topk), torch.float32), torch.ones(1, device=device)
        self.dlogits, ones = torch.zeros_like(self.logits), torch.ones((tokens, topk), device=device)
        up_t, down_t = transposed(self.up, self.up_sf), transposed(self.down, self.down_sf)
        self.back = [
            M.CombineBackwardPlan(self.lay.expert_slot.view(tokens, topk), self.route.topk_weights, self.y, self.dout,
                                  grad_weights=self.dweights, grad_q=dy_q, grad_sf=dy_sf),
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
        self.dout.copy_(dout)
        for step in self.back:
            step()
        return self.dx, self.dlogits


class MoeBlock(MoeLayer):
    """The layer behind its norm: h = x + residual, out = layer(norm(h)); h goes on along the residual."""

    def __init__(self, tokens, hidden, *args, device="cuda", eps=1e-6, training=True, **kw):
        super().__init__(tokens, hidden, *args, device=device, training=training, **kw)
        new = lambda shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        self.x_in, self.residual, self.h = (new((tokens, hidden)) for _ in range(3))
        self.norm_weight = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.steps[1] = None  # the rows come quantised from the norm
        self.norm = M.RmsNormPlan(self.x_in, self.norm_weight, eps, residual=self.residual, h=self.h, y=self.x, q=self.x_q,
                                  sf=self.x_sf)
        self.steps = [step for step in self.steps if step is not None]
        if training:
            self.dy, self.dh, self.dx_in = (new((tokens, hidden)) for _ in range(3))
            self.dnorm_weight = new(hidden, torch.float32)
            self.norm_back = M.RmsNormBackwardPlan(self.h, self.norm_weight, self.dy, eps, self.dx_in, grad_h=self.dh,
                                                   grad_weight=self.dnorm_weight,
                                                   workspace=M.alloc_rms_norm_workspace(tokens, hidden, device))

    def forward(self, x, residual):
        """x, residual [T, H] bf16 -> out [T, H] and h [T, H] bf16."""
        self.x_in.copy_(x)
        self.residual.copy_(residual)
        self.norm()
        torch.matmul(self.x, self.router.t(), out=self.logits)
        for step in self.steps:
            step()
        return self.out, self.h

    def backward(self, dout, dh):
        """dout, dh [T, H] -> gradients of h (x's and the residual's) and of the norm's weight."""
        dx, dlogits = super().backward(dout)
        self.dh.copy_(dh)
        torch.addmm(dx, dlogits, self.router, out=self.dy)
        self.norm_back()
        return self.dx_in, self.dnorm_weight


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 7168), ("inter", 2048), ("experts", 32), ("topk", 8), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--groups", type=int, help="a token's experts come from --topk-groups groups of them")
    ap.add_argument("--topk-groups", type=int, default=1)
    ap.add_argument("--norm", action="store_true", help="the layer behind its residual and norm")
    a = ap.parse_args()
    groups = (a.groups, a.topk_groups) if a.groups else None
    layer = (MoeBlock if a.norm else MoeLayer)(a.tokens, a.hidden, a.inter, a.experts, a.topk, training=False, groups=groups)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    inputs = (x, x) if a.norm else (x,)
    for _ in range(3):
        layer.forward(*inputs)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        layer.forward(*inputs)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / a.steps * 1e6
    flops = 6.0 * a.tokens * a.topk * a.hidden * a.inter
    print(f"{a.tokens} tokens x {a.hidden}, top-{a.topk} of {a.experts} experts of width {a.inter}: {us:.1f} us a layer, "
          f"{flops / us / 1e6:.0f} TFLOP/s of expert products, balance loss {float(layer.route.loss):.5f}")


if __name__ == "__main__":
    main()
