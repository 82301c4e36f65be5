// C ABI of the gate, the norm, the quantisation, the experts' product and the
// combine's gradient: argument checks, then the launches. As in dispatch_api.cpp, every check runs on the
// host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "dispatch_experts.hpp"
#include "moe_dispatch.h"

namespace {

bool aligned_to(const void* ptr, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(ptr) % bytes) == 0; }

int status_of(hipError_t err) { return err == hipSuccess ? DISPATCH_OK : DISPATCH_ERR_HIP; }

int check_gate(const dispatch_gate_problem_t* p) {
    if (p == nullptr) return DISPATCH_ERR_NULL;
    if (p->num_experts < 1 || p->num_experts > DISPATCH_MAX_EXPERTS) return DISPATCH_ERR_ARG;
    if (p->num_topk < 1 || p->num_topk > DISPATCH_MAX_TOPK || p->num_topk > p->num_experts) return DISPATCH_ERR_ARG;
    if (p->num_tokens < 0 || p->num_tokens > INT32_MAX || p->num_tokens * p->num_topk > INT32_MAX)
        return DISPATCH_ERR_ARG;
    if (p->scoring != DISPATCH_GATE_SOFTMAX && p->scoring != DISPATCH_GATE_SIGMOID) return DISPATCH_ERR_ARG;
    if (p->logits_bytes != 2 && p->logits_bytes != 4) return DISPATCH_ERR_ARG;
    if (p->topk_idx_bytes != 4 && p->topk_idx_bytes != 8) return DISPATCH_ERR_ARG;
    if ((p->flags & ~uint32_t(DISPATCH_GATE_NORMALIZE)) != 0) return DISPATCH_ERR_ARG;
    if (!std::isfinite(p->route_scale) || !std::isfinite(p->loss_coef)) return DISPATCH_ERR_ARG;
    return DISPATCH_OK;
}

int check_rms_norm(const dispatch_rms_norm_problem_t* problem) {
    if (problem == nullptr) return DISPATCH_ERR_NULL;
    const dispatch_rms_norm_problem_t& p = *problem;
    if (p.num_rows < 0 || p.num_rows > INT32_MAX || p.width < 16 || p.width > DISPATCH_MAX_NORM_WIDTH)
        return DISPATCH_ERR_ARG;
    if (p.weight_bytes != 2 && p.weight_bytes != 4) return DISPATCH_ERR_ARG;
    if (!std::isfinite(p.eps) || p.eps < FLT_MIN) return DISPATCH_ERR_ARG;
    if (p.width % 16 != 0) return DISPATCH_ERR_ALIGN;
    return DISPATCH_OK;
}

int check_quantize(const dispatch_quantize_problem_t* p, bool swiglu, int64_t sf_per_block, const void* x,
                   const void* grad, bool wants_grad, const int32_t* num_valid_rows, const void* q,
                   const float* sf) {
    if (p == nullptr) return DISPATCH_ERR_NULL;
    if (p->num_rows < 0 || p->num_rows > INT32_MAX || p->width < 16 || p->width > (int64_t(1) << 30))
        return DISPATCH_ERR_ARG;
    if (p->width % (swiglu ? DISPATCH_SF_BLOCK : 16) != 0) return DISPATCH_ERR_ALIGN;
    const int64_t blocks = (p->width + DISPATCH_SF_BLOCK - 1) / DISPATCH_SF_BLOCK * sf_per_block;
    if (p->num_rows * blocks > INT32_MAX) return DISPATCH_ERR_ARG;
    if (p->num_rows > 0 && (!x || !q || !sf || (wants_grad && !grad))) return DISPATCH_ERR_NULL;
    const void* rows[] = {x, grad, q};
    for (const void* r : rows)
        if (r && !aligned_to(r, 16)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {num_valid_rows, sf};
    for (const void* w : words)
        if (w && !aligned_to(w, 4)) return DISPATCH_ERR_ALIGN;
    return DISPATCH_OK;
}

int check_experts(const dispatch_expert_problem_t* problem, bool swiglu) {
    if (problem == nullptr) return DISPATCH_ERR_NULL;
    const dispatch_expert_problem_t& p = *problem;
    if (p.num_experts < 1 || p.num_experts > DISPATCH_MAX_EXPERTS || p.reserved != 0) return DISPATCH_ERR_ARG;
    if (p.in_features < 16 || p.in_features > (int64_t(1) << 20) || p.out_features < 8 ||
        p.out_features > (int64_t(1) << 20))
        return DISPATCH_ERR_ARG;
    if (p.expert_rows < 0 || p.expert_rows > INT32_MAX || p.max_routed_rows < 0) return DISPATCH_ERR_ARG;
    if (p.in_features % 16 != 0 || p.out_features % (swiglu ? 2 * DISPATCH_SF_BLOCK : 8) != 0)
        return DISPATCH_ERR_ALIGN;
    // Tiles (at least 16 rows x 256 channels each) are counted in 32 bits.
    if ((p.expert_rows / 16 + p.num_experts) * ((p.out_features + 255) / 256) > INT32_MAX) return DISPATCH_ERR_ARG;
    return DISPATCH_OK;
}

int expert_product(const dispatch_expert_problem_t* problem, const int32_t* expert_psum, const int32_t* expert_count,
                   const void* x, const float* x_sf, const void* w, const float* w_sf, void* out, float* out_sf,
                   bool swiglu, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int rc = check_experts(problem, swiglu);
    if (rc != DISPATCH_OK) return rc;
    const dispatch_expert_problem_t& p = *problem;
    if (!expert_psum || !expert_count || !w || !w_sf) return DISPATCH_ERR_NULL;
    if (p.expert_rows > 0 && (!x || !x_sf || !out || (swiglu && !out_sf))) return DISPATCH_ERR_NULL;
    const void* rows[] = {x, w, out};
    for (const void* r : rows)
        if (r && !aligned_to(r, 16)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {expert_psum, expert_count, x_sf, w_sf, out_sf};
    for (const void* q : words)
        if (q && !aligned_to(q, 4)) return DISPATCH_ERR_ALIGN;
    if (workspace != nullptr &&
        (!aligned_to(workspace, 256) || workspace_bytes < moe_dispatch::expert_workspace_bytes(p)))
        return DISPATCH_ERR_WORKSPACE;
    return status_of(moe_dispatch::launch_expert_product(p, expert_psum, expert_count, x, x_sf, w, w_sf, out,
                                                         swiglu ? out_sf : nullptr, workspace, stream));
}

int gate(const dispatch_gate_problem_t* problem, const dispatch_gate_groups_t* groups, const void* logits,
         const float* select_bias, const uint8_t* token_mask, const dispatch_gate_out_t* out, void* workspace,
         size_t workspace_bytes, hipStream_t stream) {
    const int rc = check_gate(problem);
    if (rc != DISPATCH_OK) return rc;
    const dispatch_gate_problem_t& p = *problem;
    if (out == nullptr) return DISPATCH_ERR_NULL;
    if (p.num_tokens > 0 && (!logits || !out->topk_idx || !out->topk_weights)) return DISPATCH_ERR_NULL;
    if (select_bias && p.scoring != DISPATCH_GATE_SIGMOID) return DISPATCH_ERR_ARG;
    const bool balance = out->expert_count || out->prob_sum || out->live_tokens || out->loss;
    if (balance && (!out->expert_count || !out->prob_sum || !out->live_tokens || !out->loss))
        return DISPATCH_ERR_NULL;
    if (logits && !aligned_to(logits, p.logits_bytes)) return DISPATCH_ERR_ALIGN;
    if (out->topk_idx && !aligned_to(out->topk_idx, p.topk_idx_bytes)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {select_bias, out->topk_weights, out->expert_count, out->prob_sum, out->live_tokens,
                           out->loss};
    for (const void* q : words)
        if (q && !aligned_to(q, 4)) return DISPATCH_ERR_ALIGN;
    if (balance && (workspace == nullptr || !aligned_to(workspace, 256) ||
                    workspace_bytes < moe_dispatch::gate_workspace_bytes(p.num_experts)))
        return DISPATCH_ERR_WORKSPACE;
    return status_of(moe_dispatch::launch_gate(p, groups, logits, select_bias, token_mask, *out, workspace, stream));
}

}  // namespace

extern "C" {

int dispatch_gate_workspace_size(const dispatch_gate_problem_t* problem, size_t* bytes) {
    const int rc = check_gate(problem);
    if (rc != DISPATCH_OK) return rc;
    if (bytes == nullptr) return DISPATCH_ERR_NULL;
    *bytes = moe_dispatch::gate_workspace_bytes(problem->num_experts);
    return DISPATCH_OK;
}

int dispatch_gate(const dispatch_gate_problem_t* problem, const void* logits, const float* select_bias,
                  const uint8_t* token_mask, const dispatch_gate_out_t* out, void* workspace,
                  size_t workspace_bytes, hipStream_t stream) {
    return gate(problem, nullptr, logits, select_bias, token_mask, out, workspace, workspace_bytes, stream);
}

int dispatch_gate_grouped(const dispatch_gate_problem_t* problem, const dispatch_gate_groups_t* groups,
                          const void* logits, const float* select_bias, const uint8_t* token_mask,
                          const dispatch_gate_out_t* out, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    if (problem == nullptr || groups == nullptr) return DISPATCH_ERR_NULL;
    const dispatch_gate_groups_t& g = *groups;
    if (g.num_groups < 1 || g.num_groups > DISPATCH_MAX_GATE_GROUPS || problem->num_experts % g.num_groups != 0 ||
        g.reserved != 0)
        return DISPATCH_ERR_ARG;
    if (g.topk_groups < 1 || g.topk_groups > g.num_groups ||
        problem->num_topk > (int64_t)g.topk_groups * (problem->num_experts / g.num_groups))
        return DISPATCH_ERR_ARG;
    if (g.score_experts != 1 && (g.score_experts != 2 || problem->scoring != DISPATCH_GATE_SIGMOID))
        return DISPATCH_ERR_ARG;
    return gate(problem, groups, logits, select_bias, token_mask, out, workspace, workspace_bytes, stream);
}

int dispatch_gate_backward(const dispatch_gate_problem_t* problem, const void* logits, const uint8_t* token_mask,
                           const void* topk_idx, const float* grad_weights, const int32_t* expert_count,
                           const int32_t* live_tokens, const float* grad_loss, void* grad_logits,
                           hipStream_t stream) {
    const int rc = check_gate(problem);
    if (rc != DISPATCH_OK) return rc;
    const dispatch_gate_problem_t& p = *problem;
    if (p.num_tokens > 0 && (!logits || !grad_logits || (grad_weights && !topk_idx))) return DISPATCH_ERR_NULL;
    if (grad_loss && (!expert_count || !live_tokens)) return DISPATCH_ERR_NULL;
    if ((logits && !aligned_to(logits, p.logits_bytes)) || (grad_logits && !aligned_to(grad_logits, p.logits_bytes)))
        return DISPATCH_ERR_ALIGN;
    if (topk_idx && !aligned_to(topk_idx, p.topk_idx_bytes)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {grad_weights, expert_count, live_tokens, grad_loss};
    for (const void* q : words)
        if (q && !aligned_to(q, 4)) return DISPATCH_ERR_ALIGN;
    return status_of(moe_dispatch::launch_gate_backward(p, logits, token_mask, topk_idx, grad_weights, expert_count,
                                                        live_tokens, grad_loss, grad_logits, stream));
}

int dispatch_quantize(const dispatch_quantize_problem_t* problem, const void* x, const int32_t* num_valid_rows,
                      void* q, float* sf, hipStream_t stream) {
    const int rc = check_quantize(problem, false, 1, x, nullptr, false, num_valid_rows, q, sf);
    if (rc != DISPATCH_OK) return rc;
    return status_of(moe_dispatch::launch_quantize(moe_dispatch::QuantizeSource::kRows, *problem, x, nullptr,
                                                   num_valid_rows, q, sf, stream));
}

int dispatch_swiglu_quantize(const dispatch_quantize_problem_t* problem, const void* h,
                             const int32_t* num_valid_rows, void* q, float* sf, hipStream_t stream) {
    const int rc = check_quantize(problem, true, 1, h, nullptr, false, num_valid_rows, q, sf);
    if (rc != DISPATCH_OK) return rc;
    return status_of(moe_dispatch::launch_quantize(moe_dispatch::QuantizeSource::kSwiglu, *problem, h, nullptr,
                                                   num_valid_rows, q, sf, stream));
}

int dispatch_swiglu_backward_quantize(const dispatch_quantize_problem_t* problem, const void* h, const void* grad,
                                      const int32_t* num_valid_rows, void* q, float* sf, hipStream_t stream) {
    const int rc = check_quantize(problem, true, 2, h, grad, true, num_valid_rows, q, sf);
    if (rc != DISPATCH_OK) return rc;
    return status_of(moe_dispatch::launch_quantize(moe_dispatch::QuantizeSource::kSwigluGrad, *problem, h, grad,
                                                   num_valid_rows, q, sf, stream));
}

int dispatch_expert_workspace_size(const dispatch_expert_problem_t* problem, size_t* bytes) {
    const int rc = check_experts(problem, false);
    if (rc != DISPATCH_OK) return rc;
    if (bytes == nullptr) return DISPATCH_ERR_NULL;
    *bytes = moe_dispatch::expert_workspace_bytes(*problem);
    return DISPATCH_OK;
}

int dispatch_expert_product(const dispatch_expert_problem_t* problem, const int32_t* expert_psum,
                            const int32_t* expert_count, const void* x, const float* x_sf, const void* w,
                            const float* w_sf, void* out, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    return expert_product(problem, expert_psum, expert_count, x, x_sf, w, w_sf, out, nullptr, false, workspace,
                          workspace_bytes, stream);
}

int dispatch_expert_product_swiglu(const dispatch_expert_problem_t* problem, const int32_t* expert_psum,
                                   const int32_t* expert_count, const void* x, const float* x_sf, const void* w,
                                   const float* w_sf, void* out_q, float* out_sf, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    return expert_product(problem, expert_psum, expert_count, x, x_sf, w, w_sf, out_q, out_sf, true, workspace,
                          workspace_bytes, stream);
}

int dispatch_rms_norm(const dispatch_rms_norm_problem_t* problem, const void* x, const void* residual,
                      const void* weight, const int32_t* num_valid_rows, void* h, void* y, void* q, float* sf,
                      hipStream_t stream) {
    const int rc = check_rms_norm(problem);
    if (rc != DISPATCH_OK) return rc;
    if (!weight || (problem->num_rows > 0 && !x)) return DISPATCH_ERR_NULL;
    if (problem->num_rows > 0 && ((residual == nullptr) != (h == nullptr) || (q == nullptr) != (sf == nullptr) ||
                                  (!y && !q)))
        return DISPATCH_ERR_NULL;
    const void* rows[] = {x, residual, weight, h, y, q};
    for (const void* r : rows)
        if (r && !aligned_to(r, 16)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {num_valid_rows, sf};
    for (const void* w : words)
        if (w && !aligned_to(w, 4)) return DISPATCH_ERR_ALIGN;
    return status_of(moe_dispatch::launch_rms_norm(*problem, x, residual, weight, num_valid_rows, h, y, q, sf, stream));
}

int dispatch_rms_norm_workspace_size(const dispatch_rms_norm_problem_t* problem, size_t* bytes) {
    const int rc = check_rms_norm(problem);
    if (rc != DISPATCH_OK) return rc;
    if (bytes == nullptr) return DISPATCH_ERR_NULL;
    *bytes = moe_dispatch::rms_norm_workspace_bytes(*problem);
    return DISPATCH_OK;
}

int dispatch_rms_norm_backward(const dispatch_rms_norm_problem_t* problem, const void* h, const void* weight,
                               const void* grad_y, const void* grad_h, const int32_t* num_valid_rows, void* grad_x,
                               float* grad_weight, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int rc = check_rms_norm(problem);
    if (rc != DISPATCH_OK) return rc;
    if (!weight || (problem->num_rows > 0 && (!h || !grad_y || !grad_x))) return DISPATCH_ERR_NULL;
    const void* rows[] = {h, weight, grad_y, grad_h, grad_x, grad_weight};
    for (const void* r : rows)
        if (r && !aligned_to(r, 16)) return DISPATCH_ERR_ALIGN;
    if (num_valid_rows && !aligned_to(num_valid_rows, 4)) return DISPATCH_ERR_ALIGN;
    if (grad_weight && (workspace == nullptr || !aligned_to(workspace, 256) ||
                        workspace_bytes < moe_dispatch::rms_norm_workspace_bytes(*problem)))
        return DISPATCH_ERR_WORKSPACE;
    return status_of(moe_dispatch::launch_rms_norm_backward(*problem, h, weight, grad_y, grad_h, num_valid_rows,
                                                            grad_x, grad_weight, workspace, stream));
}

int dispatch_combine_backward(const dispatch_combine_problem_t* problem, const int32_t* expert_slot,
                              const float* topk_weights, const void* y, const void* grad_out, float* grad_weights,
                              void* grad_y, void* grad_q, float* grad_sf, hipStream_t stream) {
    if (problem == nullptr) return DISPATCH_ERR_NULL;
    const dispatch_combine_problem_t& p = *problem;
    if (p.num_tokens < 0 || p.num_tokens > INT32_MAX || p.num_topk < 1 || p.num_topk > DISPATCH_MAX_TOPK ||
        p.reserved != 0 || p.expert_rows < 0 || p.hidden < 8 || p.hidden > (int64_t(1) << 30) - 8)
        return DISPATCH_ERR_ARG;
    if (grad_y && (grad_q || grad_sf)) return DISPATCH_ERR_ARG;
    if (p.hidden % 8 != 0 || (grad_q && p.hidden % 16 != 0)) return DISPATCH_ERR_ALIGN;
    if (p.num_tokens > 0) {
        if (!expert_slot || !topk_weights || !grad_out) return DISPATCH_ERR_NULL;
        if (p.expert_rows > 0 && !grad_weights && !grad_y && !grad_q) return DISPATCH_ERR_NULL;
        if (grad_weights && p.expert_rows > 0 && !y) return DISPATCH_ERR_NULL;
        if ((grad_q == nullptr) != (grad_sf == nullptr)) return DISPATCH_ERR_NULL;
    }
    const void* rows[] = {y, grad_out, grad_y, grad_q};
    for (const void* r : rows)
        if (r && !aligned_to(r, 16)) return DISPATCH_ERR_ALIGN;
    const void* words[] = {expert_slot, topk_weights, grad_weights, grad_sf};
    for (const void* w : words)
        if (w && !aligned_to(w, 4)) return DISPATCH_ERR_ALIGN;
    return status_of(moe_dispatch::launch_combine_backward(p, expert_slot, topk_weights, y, grad_out, grad_weights,
                                                           grad_y, grad_q, grad_sf, stream));
}

}  // extern "C"
