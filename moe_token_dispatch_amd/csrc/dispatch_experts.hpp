// Launchers of the gate, the quantisation and the experts' product, called by
// the C ABI after its host checks, and what sizes their workspaces and grids.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_dispatch.h"

namespace moe_dispatch {

constexpr int kGateMaxGroups = 512;  // workgroups of a gate forward with balance outputs

// Workgroups of a gate forward with balance outputs: each leaves one partial
// row of E probability sums, E counts and its live tokens.
inline int gate_groups(int64_t num_tokens, int waves) {
    // One workgroup up to two tokens per wavefront: it needs no second kernel
    // (256 experts: 16 tokens 6.2 us, 32 8.9, against 10.0; 48 would take 11.8).
    // One token per wavefront up to 256 workgroups, one per CU; a second one
    // per CU (better hidden latencies, but twice the partial rows) where each
    // wavefront still gets two tokens.
    if (num_tokens <= 2 * waves) return 1;
    const int64_t g = (num_tokens + waves - 1) / waves;
    if (g <= kGateMaxGroups / 2) return (int)g;
    return g < 2 * kGateMaxGroups ? kGateMaxGroups / 2 : kGateMaxGroups;
}
inline size_t gate_partial_words(int32_t num_experts) { return 2 * (size_t)num_experts + 1; }
// Workspace: the partial rows, then the parts of the loss (one double for
// each 16 experts) and the ticket of the workgroups that add them.
struct GateWorkspace {
    size_t loss_part, ticket, bytes;
};
inline GateWorkspace gate_workspace(int32_t num_experts) {
    GateWorkspace w;
    w.loss_part = (kGateMaxGroups * gate_partial_words(num_experts) * 4 + 255) & ~size_t(255);
    w.ticket = w.loss_part + DISPATCH_MAX_EXPERTS / 16 * sizeof(double);
    w.bytes = w.ticket + 256;
    return w;
}
inline size_t gate_workspace_bytes(int32_t num_experts) { return gate_workspace(num_experts).bytes; }

hipError_t launch_gate(const dispatch_gate_problem_t& p, const void* logits, const float* select_bias,
                       const uint8_t* token_mask, const dispatch_gate_out_t& out, void* workspace,
                       hipStream_t stream);
hipError_t launch_gate_backward(const dispatch_gate_problem_t& p, const void* logits, const uint8_t* token_mask,
                                const void* topk_idx, const float* grad_weights, const int32_t* expert_count,
                                const int32_t* live_tokens, const float* grad_loss, void* grad_logits,
                                hipStream_t stream);

enum class QuantizeSource { kRows, kSwiglu, kSwigluGrad };
hipError_t launch_quantize(QuantizeSource source, const dispatch_quantize_problem_t& p, const void* x,
                           const void* grad, const int32_t* num_valid_rows, void* q, float* sf, hipStream_t stream);

// out_sf: not NULL for the product with the SwiGLU and quantisation behind it.
// workspace: NULL or of expert_workspace_bytes.
size_t expert_workspace_bytes(const dispatch_expert_problem_t& p);
hipError_t launch_expert_product(const dispatch_expert_problem_t& p, const int32_t* expert_psum,
                                 const int32_t* expert_count, const void* x, const float* x_sf, const void* w,
                                 const float* w_sf, void* out, float* out_sf, void* workspace, hipStream_t stream);

}  // namespace moe_dispatch
