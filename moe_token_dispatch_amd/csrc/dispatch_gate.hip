// The gate on gfx950: router logits to the routing table and its weights, the
// per-expert counts and the balance loss, and the gradient of the logits.
//
// One wavefront per token. Lane l holds the logits of experts l, l + 64, ...,
// V = ceil(E / 64) of them in registers, so a row is read once, and a row of
// scores, its sums and its choice never leave the wavefront.
//
// Choice: K rounds of a wave maximum over what is left. Selection compares
// the fp32 values themselves (for softmax the logits, whose order the scores
// share), so ties are exact ties and go to the lowest expert. They are
// compared as unsigned integers that order as the values do: an integer
// maximum takes one instruction where a float maximum also has to quiet NaN.
//
// Balance: a wavefront keeps prob_sum of its lanes' experts in registers over
// all its tokens; a workgroup adds its wavefronts in order and leaves one
// partial row; a second kernel adds the partial rows in order. No float goes
// through an atomic, so the sums do not depend on timing (the counts are
// integers and do go through LDS atomics).
#include "dispatch_common.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

constexpr float kNone = -__builtin_inff();

struct GateParams {
    const void* logits;
    const float* bias;
    const uint8_t* mask;
    void* topk_idx;
    float* topk_weights;
    float* partial;    // [groups][2E + 1]: prob sums, counts and live tokens (as integer bits)
    uint32_t* ticket;  // cleared here for the kernel that adds the partial rows
    int64_t num_tokens;
    int32_t num_experts;
    int32_t num_topk;
    int32_t logits_bytes;
    int32_t idx_bytes;
    uint32_t flags;
    float route_scale;
};

// Wavefronts per workgroup that leave each enough registers for its V
// experts per lane.
template <int V>
constexpr int kGateWaves = V <= 8 ? 16 : (V == 16 ? 8 : 4);

// Lane's logits of row t, -inf past the last expert.
template <int V>
__device__ __forceinline__ void load_row(const void* logits, int32_t bytes, int64_t t, int32_t E, int lane,
                                         float (&z)[V]) {
    if (bytes == 2) {
        const uint16_t* row = static_cast<const uint16_t*>(logits) + t * E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * kWave + lane;
            z[v] = e < E ? bf16_low(row[e]) : kNone;
        }
    } else {
        const float* row = static_cast<const float*>(logits) + t * E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * kWave + lane;
            z[v] = e < E ? row[e] : kNone;
        }
    }
}

// A value as an unsigned integer of the same order, both zeros alike. What is
// never taken, NaN and -inf, gets kNoKey, below every other value's.
constexpr uint32_t kNoKey = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float c) {
    const uint32_t u = __float_as_uint(fmaxf(c, kNone) + 0.f);  // (fmaxf drops NaN)
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// exp(x) for x <= 0 from the hardware's exp2: the argument's rounding leaves a
// relative error of |x| 2^-24, far from where exp(x) counts in a sum with 1.
__device__ __forceinline__ float exp_nonpositive(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// A row's sum of scores (before softmax divides by it) and its reciprocal, 0
// for a row whose scores are all 0.
struct RowSum {
    float sum, inv;
    // s / sum, the product's rounding corrected: a lone score's share is 1, so
    // that its gradient cancels exactly.
    __device__ __forceinline__ float share(float s) const {
        const float p = s * inv;
        return __builtin_fmaf(__builtin_fmaf(-p, sum, s), inv, p);
    }
};

// Scores of a row in place of its logits (softmax scores are shares already).
template <int V, bool kSigmoid>
__device__ __forceinline__ RowSum scores(float (&z)[V]) {
    float sum = 0.f;
    if (kSigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = z[v] == kNone ? 0.f : sigmoid(z[v]);
            sum += z[v];
        }
        sum = wave_sum(sum);
        return {sum, sum == 0.f ? 0.f : 1.f / sum};
    }
    float top = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, z[v]);
    top = wave_max(top);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        z[v] = z[v] == kNone ? 0.f : exp_nonpositive(z[v] - top);
        sum += z[v];
    }
    sum = wave_sum(sum);
    const RowSum r{sum, sum == 0.f ? 0.f : 1.f / sum};
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] *= r.inv;
    return r;
}

template <int V, bool kSigmoid, bool kBalance>
__global__ void __launch_bounds__(kGateWaves<V> * kWave) gate_kernel(GateParams p) {
    // A row of scores per wavefront, then with kBalance the workgroup's
    // counts [E] and live tokens [1].
    extern __shared__ float lds[];
    const int W = blockDim.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int E = p.num_experts, K = p.num_topk;
    float* const score_row = lds + wave * V * kWave;
    int* const counts = reinterpret_cast<int*>(lds + W * V * kWave);
    float prob_sum[V];
    int live = 0;
    if (kBalance) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
        for (int i = threadIdx.x; i < E + 1; i += W * kWave) counts[i] = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) prob_sum[v] = 0.f;
        __syncthreads();
    }
    const int64_t stride = (int64_t)gridDim.x * W;
    int64_t t = (int64_t)blockIdx.x * W + wave;
    // The next token's row is loaded while this one's is worked on.
    float next[V];
    if (t < p.num_tokens) load_row<V>(p.logits, p.logits_bytes, t, E, lane, next);
    for (; t < p.num_tokens; t += stride) {
        int picked = -1;     // lane k: entry k's expert
        float weight = 0.f;  // lane k: its score
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = next[v];
        if (t + stride < p.num_tokens) load_row<V>(p.logits, p.logits_bytes, t + stride, E, lane, next);
        if (p.mask == nullptr || p.mask[t] != 0) {
            uint32_t c[V];
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = order_key(s[v]);
            const RowSum row_sum = scores<V, kSigmoid>(s);
            if (kSigmoid) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e = v * kWave + lane;
                    const float b = p.bias != nullptr && e < E ? p.bias[e] : 0.f;
                    c[v] = c[v] == kNoKey ? kNoKey : order_key(s[v] + b);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) score_row[v * kWave + lane] = s[v];
            for (int k = 0; k < K; ++k) {
                uint32_t m = c[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = m > c[v] ? m : c[v];
                m = wave_max(m);
                if (m == kNoKey) break;
                int e = -1;
#pragma unroll
                for (int v = V - 1; v >= 0; --v) {
                    const uint64_t hit = __ballot(c[v] == m);
                    if (hit != 0) e = v * kWave + __builtin_ctzll(hit);
                }
                const bool here = lane == (e & (kWave - 1));
#pragma unroll
                for (int v = 0; v < V; ++v) c[v] = here && (e / kWave) == v ? kNoKey : c[v];
                picked = lane == k ? e : picked;
            }
            __builtin_amdgcn_wave_barrier();
            if (picked >= 0) weight = score_row[picked];
            __builtin_amdgcn_wave_barrier();
            if (p.flags & DISPATCH_GATE_NORMALIZE) {
                const float total = wave_sum(weight);
                weight = total == 0.f ? 0.f : p.route_scale * weight / total;
            } else {
                weight *= p.route_scale;
            }
            if (kBalance) {
#pragma unroll
                for (int v = 0; v < V; ++v) prob_sum[v] += kSigmoid ? row_sum.share(s[v]) : s[v];
                ++live;
                if (picked >= 0) atomicAdd(counts + picked, 1);
            }
        }
        if (lane < K) {
            const int64_t at = t * K + lane;
            if (p.idx_bytes == 8)
                static_cast<int64_t*>(p.topk_idx)[at] = picked;
            else
                static_cast<int32_t*>(p.topk_idx)[at] = picked;
            p.topk_weights[at] = weight;
        }
    }
    if (!kBalance) return;
    // Each wavefront leaves its sums in its row; a thread adds an expert's
    // over the rows, in order.
#pragma unroll
    for (int v = 0; v < V; ++v) score_row[v * kWave + lane] = prob_sum[v];
    if (lane == 0) atomicAdd(counts + E, live);
    __syncthreads();
    float* const out = p.partial + (int64_t)blockIdx.x * (2 * E + 1);
    for (int i = threadIdx.x; i < 2 * E + 1; i += W * kWave) {
        float x = __int_as_float(counts[i - E < 0 ? 0 : i - E]);
        if (i < E) {
            x = lds[i];
            for (int w = 1; w < W; ++w) x += lds[w * V * kWave + i];
        }
        out[i] = x;
    }
}

// Adds the partial rows. A workgroup takes 16 experts: its 64 groups of 16
// threads add every 64th row, then the groups are added in order. Its part of
// the loss goes to the workspace, and the workgroup that finds itself the last
// adds those, in order too. One workgroup for all experts took 22.8 us for
// 256 rows of 256 experts, this form 6.6.
constexpr int kSumThreads = 1024;
constexpr int kSumExperts = 16;
constexpr int kSumGroups = kSumThreads / kSumExperts;

__global__ void __launch_bounds__(kSumThreads)
gate_sum_kernel(const float* partial, int groups, int E, int K, float loss_coef, int32_t* expert_count,
                float* prob_sum, int32_t* live_tokens, float* loss, double* loss_part, uint32_t* ticket) {
    constexpr int kWaves = kSumThreads / kWave;
    __shared__ float part_sum[kWaves][kSumExperts];
    __shared__ int part_count[kWaves][kSumExperts];
    const int64_t stride = 2 * (int64_t)E + 1;
    const int g0 = threadIdx.x / kSumExperts, e0 = threadIdx.x % kSumExperts;
    const int e = blockIdx.x * kSumExperts + e0;
    float s = 0.f;
    int n = 0;
    if (e < E) {
        for (int g = g0; g < groups; g += kSumGroups) {
            s += partial[g * stride + e];
            n += __float_as_int(partial[g * stride + E + e]);
        }
    }
    // The four groups of a wavefront, then the wavefronts in order.
    s += __shfl_xor(s, 16);
    n += __shfl_xor(n, 16);
    s += __shfl_xor(s, 32);
    n += __shfl_xor(n, 32);
    const int lane = threadIdx.x & (kWave - 1);
    if (lane < kSumExperts) {
        part_sum[threadIdx.x / kWave][lane] = s;
        part_count[threadIdx.x / kWave][lane] = n;
    }
    // The first wavefront also adds the live tokens of all rows (only the last
    // workgroup needs them, but it would wait for them).
    int live = 0;
    if (threadIdx.x < kWave) {
        for (int g = lane; g < groups; g += kWave) live += __float_as_int(partial[g * stride + 2 * E]);
        for (int step = kWave / 2; step > 0; step /= 2) live += __shfl_xor(live, step);
    }
    __syncthreads();
    if (threadIdx.x >= kWave) return;
    double mine = 0.0;
    if (lane < kSumExperts && e < E) {
        s = part_sum[0][lane];
        n = part_count[0][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            s += part_sum[w][lane];
            n += part_count[w][lane];
        }
        prob_sum[e] = s;
        expert_count[e] = n;
        mine = (double)n * (double)s;
    }
    for (int step = kSumExperts / 2; step > 0; step /= 2) mine += __shfl_xor(mine, step);
    if (threadIdx.x != 0) return;
    // The part goes past the caches that XCDs do not share, and has arrived
    // before the ticket is taken: no cache has to be written back for it.
    __hip_atomic_store(loss_part + blockIdx.x, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t before = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before != gridDim.x - 1) return;
    double total = 0.0;
    for (unsigned i = 0; i < gridDim.x; ++i)
        total += __hip_atomic_load(loss_part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *live_tokens = live;
    *loss = live == 0 ? 0.f : (float)((double)loss_coef * E / ((double)K * live * live) * total);
}

struct GateBackwardParams {
    const void* logits;
    const uint8_t* mask;
    const void* topk_idx;
    const float* grad_weights;
    const int32_t* expert_count;
    const int32_t* live_tokens;
    const float* grad_loss;
    void* grad_logits;
    int64_t num_tokens;
    int32_t num_experts;
    int32_t num_topk;
    int32_t logits_bytes;
    int32_t idx_bytes;
    uint32_t flags;
    float route_scale;
    float loss_coef;
};

// Gradient of the logits. The row is read again and its scores computed
// again, which is cheaper than storing them. Lane k holds entry k: its
// score's gradient goes through the wavefront's row in LDS to the lane that
// holds the expert.
template <int V, bool kSigmoid>
__global__ void __launch_bounds__(kGateWaves<V> * kWave) gate_backward_kernel(GateBackwardParams p) {
    constexpr int W = kGateWaves<V>;
    extern __shared__ float lds[];  // [W][V * 64] score gradients, zero between tokens
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int E = p.num_experts, K = p.num_topk;
    float* const row = lds + wave * V * kWave;
    float dp[V];  // the loss's gradient of this lane's experts' p: the same for every token
#pragma unroll
    for (int v = 0; v < V; ++v) {
        row[v * kWave + lane] = 0.f;
        dp[v] = 0.f;
    }
    if (p.grad_loss != nullptr) {
        const float n = (float)*p.live_tokens;
        const float unit = n == 0.f ? 0.f : *p.grad_loss * (p.loss_coef * (float)E / ((float)K * n * n));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * kWave + lane;
            if (e < E) dp[v] = unit * (float)p.expert_count[e];
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * W + wave; t < p.num_tokens; t += (int64_t)gridDim.x * W) {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 0.f;
        if (p.mask == nullptr || p.mask[t] != 0) {
            int e = -1;
            float dw = 0.f;
            if (lane < K && p.grad_weights != nullptr) {
                const int64_t at = t * K + lane;
                const int64_t id = p.idx_bytes == 8 ? static_cast<const int64_t*>(p.topk_idx)[at]
                                                    : (int64_t)static_cast<const int32_t*>(p.topk_idx)[at];
                if (id >= 0 && id < E) {
                    e = (int)id;
                    dw = p.grad_weights[at];
                }
            }
            load_row<V>(p.logits, p.logits_bytes, t, E, lane, s);
            const RowSum row_sum = scores<V, kSigmoid>(s);
            // The scores of the taken experts, through the row in LDS.
#pragma unroll
            for (int v = 0; v < V; ++v) row[v * kWave + lane] = s[v];
            __builtin_amdgcn_wave_barrier();
            const float mine = e >= 0 ? row[e] : 0.f;
            __builtin_amdgcn_wave_barrier();
            float ds = p.route_scale * dw;
            if (p.flags & DISPATCH_GATE_NORMALIZE) {
                const float total = wave_sum(mine);
                const float mean = wave_sum(dw * mine);
                ds = total == 0.f ? 0.f : p.route_scale / total * (dw - mean / total);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) row[v * kWave + lane] = 0.f;
            __builtin_amdgcn_wave_barrier();
            if (e >= 0) row[e] = ds;
            __builtin_amdgcn_wave_barrier();
            float d[V];
            float mean = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[v] = row[v * kWave + lane];
                if (kSigmoid) {
                    mean += row_sum.share(s[v]) * dp[v];
                } else {
                    d[v] += dp[v];
                    mean += s[v] * d[v];
                }
            }
            __builtin_amdgcn_wave_barrier();
            mean = wave_sum(mean);
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = kSigmoid ? (d[v] + (dp[v] - mean) * row_sum.inv) * s[v] * (1.f - s[v]) : s[v] * (d[v] - mean);
        }
        if (p.logits_bytes == 2) {
            uint16_t* out = static_cast<uint16_t*>(p.grad_logits) + t * E;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * kWave + lane;
                if (e < E) out[e] = (uint16_t)pack_bf16(s[v], 0.f);
            }
        } else {
            float* out = static_cast<float*>(p.grad_logits) + t * E;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * kWave + lane;
                if (e < E) out[e] = s[v];
            }
        }
    }
}

// f<V> for the fewest V of 1, 2, 4, ..., 64 that hold E experts in 64 lanes.
#define DISPATCH_GATE_BY_V(E, F)                \
    (E) <= 64     ? F(1)                        \
    : (E) <= 128  ? F(2)                        \
    : (E) <= 256  ? F(4)                        \
    : (E) <= 512  ? F(8)                        \
    : (E) <= 1024 ? F(16)                       \
    : (E) <= 2048 ? F(32)                       \
                  : F(64)

}  // namespace

hipError_t launch_gate(const dispatch_gate_problem_t& prob, const void* logits, const float* select_bias,
                       const uint8_t* token_mask, const dispatch_gate_out_t& out, void* workspace,
                       hipStream_t stream) {
    const int E = prob.num_experts;
    GateParams p{};
    p.logits = logits;
    p.bias = select_bias;
    p.mask = token_mask;
    p.topk_idx = out.topk_idx;
    p.topk_weights = out.topk_weights;
    const GateWorkspace ws = gate_workspace(E);
    uint8_t* const base = static_cast<uint8_t*>(workspace);
    p.partial = reinterpret_cast<float*>(base);
    p.ticket = reinterpret_cast<uint32_t*>(base + ws.ticket);
    p.num_tokens = prob.num_tokens;
    p.num_experts = prob.num_experts;
    p.num_topk = prob.num_topk;
    p.logits_bytes = prob.logits_bytes;
    p.idx_bytes = prob.topk_idx_bytes;
    p.flags = prob.flags;
    p.route_scale = prob.route_scale;
    const bool sig = prob.scoring == DISPATCH_GATE_SIGMOID;
    const bool balance = out.loss != nullptr;
    if (prob.num_tokens == 0 && !balance) return hipSuccess;
#define DISPATCH_F(V)                                                                           \
    (sig ? (balance ? (const void*)&gate_kernel<V, true, true> : (const void*)&gate_kernel<V, true, false>)     \
         : (balance ? (const void*)&gate_kernel<V, false, true> : (const void*)&gate_kernel<V, false, false>))
    const void* kernel = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
#define DISPATCH_F(V) kGateWaves<V>
    int waves = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
    // Small workgroups start sooner and spread over more CUs (16 or 1000
    // tokens: 4.7 and 4.5 us, 6.1 and 5.8 with 16 wavefronts); with balance
    // outputs each workgroup leaves a partial row, so there they are large.
    if (!balance) waves = 4;
    // Without balance outputs nothing crosses workgroups and the grid may be
    // as large as the batch.
    const int64_t all = (prob.num_tokens + waves - 1) / waves;
    const int groups = balance ? gate_groups(prob.num_tokens, waves) : (int)(all < 65536 ? all : 65536);
#define DISPATCH_F(V) (V * kWave)
    const int row = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
    const size_t shared = ((size_t)waves * row + (balance ? E + 1 : 0)) * sizeof(float);
    void* args[] = {&p};
    hipError_t err = hipLaunchKernel(kernel, dim3(groups), dim3(waves * kWave), args, shared, stream);
    if (err != hipSuccess || !balance) return err;
    const float* partial = p.partial;
    int n = groups, k = prob.num_topk, e = E;
    float coef = prob.loss_coef;
    int32_t* count = out.expert_count;
    float* prob_sum = out.prob_sum;
    int32_t* live = out.live_tokens;
    float* loss = out.loss;
    double* loss_part = reinterpret_cast<double*>(base + ws.loss_part);
    uint32_t* ticket = p.ticket;
    void* sum_args[] = {&partial, &n, &e, &k, &coef, &count, &prob_sum, &live, &loss, &loss_part, &ticket};
    return hipLaunchKernel((const void*)&gate_sum_kernel, dim3((E + kSumExperts - 1) / kSumExperts),
                           dim3(kSumThreads), sum_args, 0, stream);
}

hipError_t launch_gate_backward(const dispatch_gate_problem_t& prob, const void* logits, const uint8_t* token_mask,
                                const void* topk_idx, const float* grad_weights, const int32_t* expert_count,
                                const int32_t* live_tokens, const float* grad_loss, void* grad_logits,
                                hipStream_t stream) {
    if (prob.num_tokens == 0) return hipSuccess;
    GateBackwardParams p{};
    p.logits = logits;
    p.mask = token_mask;
    p.topk_idx = topk_idx;
    p.grad_weights = grad_weights;
    p.expert_count = expert_count;
    p.live_tokens = live_tokens;
    p.grad_loss = grad_loss;
    p.grad_logits = grad_logits;
    p.num_tokens = prob.num_tokens;
    p.num_experts = prob.num_experts;
    p.num_topk = prob.num_topk;
    p.logits_bytes = prob.logits_bytes;
    p.idx_bytes = prob.topk_idx_bytes;
    p.flags = prob.flags;
    p.route_scale = prob.route_scale;
    p.loss_coef = prob.loss_coef;
    const bool sig = prob.scoring == DISPATCH_GATE_SIGMOID;
    const int E = prob.num_experts;
#define DISPATCH_F(V) (sig ? (const void*)&gate_backward_kernel<V, true> : (const void*)&gate_backward_kernel<V, false>)
    const void* kernel = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
#define DISPATCH_F(V) kGateWaves<V>
    const int waves = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
#define DISPATCH_F(V) (V * kWave)
    const int row = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
    const int64_t all = (prob.num_tokens + waves - 1) / waves;
    // Two workgroups per CU, each wavefront with several tokens: its counts are
    // read once (2048 workgroups: 4 us longer for 65536 tokens).
    const int groups = (int)(all < 512 ? all : 512);
    void* args[] = {&p};
    return hipLaunchKernel(kernel, dim3(groups), dim3(waves * kWave), args, (size_t)waves * row * sizeof(float),
                           stream);
}

}  // namespace moe_dispatch
