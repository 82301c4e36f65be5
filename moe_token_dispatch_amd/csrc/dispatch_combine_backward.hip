// The combine's gradient on gfx950: of the top-k weights, and of the
// expert-major rows.
//
//   grad_weights[t, k] = sum over h of grad_out[t, h] * y[slot, h]
//   grad_y[slot, h] = topk_weights[t, k] * grad_out[t, h],  slot = expert_slot[t, k]
//
// the second in bf16, or quantised to fp8 with a scale per 128 channels. A
// workgroup takes up to eight entries of a token: it reads the token's row of
// grad_out once and keeps each vector of it in registers while the entries'
// vectors, all on their way at once, pass by. The largest magnitude of a block
// of w * grad_out is |w| times that of grad_out, rounded as the products are: the
// lanes of a block look for it once for all entries.
//
// It is bound by HBM: 4 bytes a routed channel, 3 with fp8 rows, and 2 a token's.
// 4096 tokens x 8 entries x 7168 channels to fp8 142 us for 770 MB (5.4 TB/s), to
// bf16 189 us for 998 MB; the rows of y and of the result go past the caches
// (through them 163 us to fp8).
#include "dispatch_common.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

constexpr int kMostEntries = 8;  // of a workgroup
constexpr int kMaxWaves = 8;  // of a workgroup: longer rows take several rounds (16: 151 us in place of 142)
constexpr int kCus = 256;
// What moves more goes past the caches: y too, which is otherwise found there
// (256 tokens, 45 MB: 11.5 us, 12.9 past them; 1024, 182 MB: 40.7 and 37.1).
constexpr int64_t kPastBytes = int64_t(128) << 20;
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
    int32_t parts;  // workgroups of a token
    int32_t per;    // entries of one
};

enum class RowsTo { kNone, kBf16, kFp8 };

template <RowsTo kTo, bool kWeights, bool kPast, int kBatch>
__global__ void __launch_bounds__(kMaxWaves * kWave) combine_backward_kernel(CombineBackwardParams p) {
    __shared__ float part[2][kMaxWaves][kBatch];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    int turn = 0;
    for (int64_t item = blockIdx.x; item < p.num_tokens * p.parts; item += gridDim.x) {
        const int64_t t = item / p.parts;
        const int begin = (int)(item - t * p.parts) * p.per;
        const int entries = p.num_topk - begin < p.per ? p.num_topk - begin : p.per;
        const int64_t entry = t * p.num_topk + begin;
        // Lane b holds entry b; a slot outside y is dropped, as in the combine.
        int slot = -1;
        float w = 0.f;
        if (lane < entries) {
            slot = p.expert_slot[entry + lane];
            w = p.topk_weights[entry + lane];
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
                    if (s[b] >= 0 && live) v[b] = load_vec<kPast>(p.y + (int64_t)s[b] * p.vecs + vec);
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
                        // (By their bits, so that NaN stays. An infinite weight's
                        // scale is infinite also beside zeros, whose products are
                        // NaN; the bytes are NaN with either.)
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
        // wavefront may be an item ahead.)
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (b >= entries) break;
            const float sum = wave_sum(dot[b]);
            if (lane == 0) part[turn][wave][b] = sum;
        }
        __syncthreads();
        if ((int)threadIdx.x < entries) {
            float sum = part[turn][0][threadIdx.x];
            for (int i = 1; i < waves; ++i) sum += part[turn][i][threadIdx.x];
            p.grad_weights[entry + threadIdx.x] = sum;
        }
        turn ^= 1;
    }
}

template <RowsTo kTo, int kBatch>
const void* kernel_of(bool weights, bool past) {
    if constexpr (kTo != RowsTo::kNone)
        if (!weights) return (const void*)&combine_backward_kernel<kTo, false, false, kBatch>;  // (loads nothing to keep out)
    return past ? (const void*)&combine_backward_kernel<kTo, true, true, kBatch>
                : (const void*)&combine_backward_kernel<kTo, true, false, kBatch>;
}
// Built for 1, 2, 4 and 8 entries: a small call spends its time on fetching the
// code (16 tokens x 8 x 7168 to fp8, an entry each: 3.7 us in a graph, 4.35 with
// the code for eight; 2000 tokens of one entry of 4096: 8.2 and 11.3 us).
template <RowsTo kTo>
const void* kernel_of(bool weights, bool past, int per) {
    return per <= 1   ? kernel_of<kTo, 1>(weights, past)
           : per <= 2 ? kernel_of<kTo, 2>(weights, past)
           : per <= 4 ? kernel_of<kTo, 4>(weights, past)
                      : kernel_of<kTo, kMostEntries>(weights, past);
}

}  // namespace

hipError_t launch_combine_backward(const dispatch_combine_problem_t& prob, const int32_t* expert_slot,
                                   const float* topk_weights, const void* y, const void* grad_out,
                                   float* grad_weights, void* grad_y, void* grad_q, float* grad_sf,
                                   hipStream_t stream) {
    if (prob.num_tokens == 0 || (!grad_weights && !grad_y && !grad_q)) return hipSuccess;
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
    // Few tokens: their entries on several workgroups, about one per CU (63
    // tokens of 8 entries x 7168 to bf16: 5.8 us with two each, 8.4 with eight;
    // with one each, two workgroups per CU, as with two).
    int parts = (int)(prob.num_tokens < kCus ? kCus / prob.num_tokens : 1);
    parts = parts < p.num_topk ? parts : p.num_topk;
    const int fewest = (p.num_topk + kMostEntries - 1) / kMostEntries;
    parts = parts > fewest ? parts : fewest;
    p.per = (p.num_topk + parts - 1) / parts;
    p.parts = (p.num_topk + p.per - 1) / p.per;
    // As few wavefronts as take the row in the same number of rounds.
    const int segments = (p.vecs + kWave - 1) / kWave, rounds = (segments + kMaxWaves - 1) / kMaxWaves;
    const int waves = (segments + rounds - 1) / rounds;
    const int64_t items = prob.num_tokens * p.parts;
    const int64_t groups = items < kMaxGroups ? items : kMaxGroups;
    const int64_t row = prob.hidden * (2 + (grad_y ? 2 : grad_q ? 1 : 0));
    const bool w = grad_weights != nullptr, past = prob.num_tokens * p.num_topk * row > kPastBytes;
    const void* kernel = grad_y   ? kernel_of<RowsTo::kBf16>(w, past, p.per)
                         : grad_q ? kernel_of<RowsTo::kFp8>(w, past, p.per)
                                  : kernel_of<RowsTo::kNone>(true, past, p.per);
    void* args[] = {&p};
    return hipLaunchKernel(kernel, dim3((unsigned)groups), dim3(waves * kWave), args, 0, stream);
}

}  // namespace moe_dispatch
