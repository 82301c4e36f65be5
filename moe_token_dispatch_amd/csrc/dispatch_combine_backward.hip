// The combine's gradient on gfx950: of the top-k weights, and of the
// expert-major rows.
//
//   grad_weights[t, k] = sum over h of grad_out[t, h] * y[slot, h]
//   grad_y[slot, h] = topk_weights[t, k] * grad_out[t, h],  slot = expert_slot[t, k]
//
// the second in bf16, or quantised to fp8 with a scale per 128 channels. A
// workgroup takes a token: its row of grad_out is read once (once for every
// eight entries) and stays in registers while the rows of its entries pass by,
// eight of them on their way at once. The largest magnitude of a block of
// w * grad_out is |w| times that of grad_out, rounded as the products are: the
// lanes of a block look for it once for all entries.
#include "dispatch_common.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

constexpr int kBatch = 8;      // entries at a time
constexpr int kMaxWaves = 16;  // of a workgroup
constexpr int64_t kMaxGroups = int64_t(1) << 20;  // larger grids loop

struct CombineBackwardParams {
    const int32_t* expert_slot;
    const float* topk_weights;
    const Bf16x8* y;
    const Bf16x8* grad_out;
    float* grad_weights;
    Bf16x8* grad_y;
    uint8_t* grad_q;
    float* grad_sf;
    int64_t num_tokens;
    int64_t expert_rows;
    int32_t vecs;    // vectors of 8 channels in a row
    int32_t blocks;  // blocks of 128 channels
    int32_t num_topk;
};

enum class RowsTo { kNone, kBf16, kFp8 };

template <RowsTo kTo, bool kWeights>
__global__ void __launch_bounds__(kMaxWaves * kWave) combine_backward_kernel(CombineBackwardParams p) {
    __shared__ float part[2][kMaxWaves][kBatch];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int K = p.num_topk;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
        for (int k0 = 0; k0 < K; k0 += kBatch) {
            // Lane b holds entry k0 + b; a slot outside y is dropped, as in the combine.
            int slot = -1;
            float w = 0.f;
            if (lane < kBatch && k0 + lane < K) {
                slot = p.expert_slot[t * K + k0 + lane];
                w = p.topk_weights[t * K + k0 + lane];
            }
            if (slot >= p.expert_rows) slot = -1;
            int s[kBatch];
            float weight[kBatch], dot[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                s[b] = __builtin_amdgcn_readlane(slot, b);
                weight[b] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), b));
                dot[b] = 0.f;
            }
            const bool any = __ballot(slot >= 0) != 0;
            for (int first = wave * kWave; any && first < p.vecs; first += waves * kWave) {
                const int vec = first + lane;
                const bool live = vec < p.vecs;
                Bf16x8 d = {0, 0, 0, 0}, v[kBatch];
                if (live) d = p.grad_out[t * p.vecs + vec];
                if (kWeights) {
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        v[b] = Bf16x8{0, 0, 0, 0};
                        if (s[b] >= 0 && live) v[b] = load_vec<true>(p.y + (int64_t)s[b] * p.vecs + vec);
                    }
                }
                float g[8];
                widen_bf16(d, g);
                float top = 0.f;
                if (kTo == RowsTo::kFp8) {
                    uint32_t most = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t m = __float_as_uint(g[i]) & 0x7fffffffu;
                        most = most > m ? most : m;
                    }
                    top = __uint_as_float(row_max(most));
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (s[b] < 0) continue;
                    const int64_t at = (int64_t)s[b] * p.vecs + vec;
                    if (kTo != RowsTo::kNone) {
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = weight[b] * g[i];
                        if (kTo == RowsTo::kBf16) {
                            if (live) store_vec<true>(p.grad_y + at, narrow_bf16(x));
                        } else {
                            // (By their bits, so that NaN stays.)
                            const uint32_t m = __float_as_uint(weight[b] * top) & 0x7fffffffu;
                            const uint32_t low = __float_as_uint(kAmaxFloor);
                            scale8<true>(x, __uint_as_float(m > low ? m : low), live, live && vec % 16 == 0,
                                         p.grad_q + at * 8, p.grad_sf + (int64_t)s[b] * p.blocks + vec / 16);
                        }
                    }
                    if (kWeights) {
                        float a[8];
                        widen_bf16(v[b], a);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[b] = __builtin_fmaf(g[i], a[i], dot[b]);
                    }
                }
            }
            if (!kWeights) continue;
            // The wavefronts' parts in order. (Two rows of parts in turn: a
            // wavefront may be a batch ahead.)
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const float sum = wave_sum(dot[b]);
                if (lane == 0) part[turn][wave][b] = sum;
            }
            __syncthreads();
            if (threadIdx.x < kBatch && k0 + (int)threadIdx.x < K) {
                float sum = part[turn][0][threadIdx.x];
                for (int i = 1; i < waves; ++i) sum += part[turn][i][threadIdx.x];
                p.grad_weights[t * K + k0 + threadIdx.x] = sum;
            }
            turn ^= 1;
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const dispatch_combine_problem_t& prob, const int32_t* expert_slot,
                                   const float* topk_weights, const void* y, const void* grad_out,
                                   float* grad_weights, void* grad_y, void* grad_q, float* grad_sf,
                                   hipStream_t stream) {
    if (prob.num_tokens == 0) return hipSuccess;
    CombineBackwardParams p{};
    p.expert_slot = expert_slot;
    p.topk_weights = topk_weights;
    p.y = static_cast<const Bf16x8*>(y);
    p.grad_out = static_cast<const Bf16x8*>(grad_out);
    p.grad_weights = grad_weights;
    p.grad_y = static_cast<Bf16x8*>(grad_y);
    p.grad_q = static_cast<uint8_t*>(grad_q);
    p.grad_sf = grad_sf;
    p.num_tokens = prob.num_tokens;
    p.expert_rows = prob.expert_rows;
    p.vecs = (int32_t)(prob.hidden / 8);
    p.blocks = (int32_t)((prob.hidden + DISPATCH_SF_BLOCK - 1) / DISPATCH_SF_BLOCK);
    p.num_topk = prob.num_topk;
    int waves = (p.vecs + kWave - 1) / kWave;
    waves = waves < kMaxWaves ? waves : kMaxWaves;
    const int64_t groups = prob.num_tokens < kMaxGroups ? prob.num_tokens : kMaxGroups;
    using R = RowsTo;
    const bool w = grad_weights != nullptr;
    const void* kernel =
        grad_y ? (w ? (const void*)&combine_backward_kernel<R::kBf16, true> : (const void*)&combine_backward_kernel<R::kBf16, false>)
        : grad_q ? (w ? (const void*)&combine_backward_kernel<R::kFp8, true> : (const void*)&combine_backward_kernel<R::kFp8, false>)
                 : (const void*)&combine_backward_kernel<R::kNone, true>;
    void* args[] = {&p};
    return hipLaunchKernel(kernel, dim3((unsigned)groups), dim3(waves * kWave), args, 0, stream);
}

}  // namespace moe_dispatch
