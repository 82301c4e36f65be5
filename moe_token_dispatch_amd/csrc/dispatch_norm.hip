// The RMS norm on gfx950, with the residual's addition before it and bf16 or
// fp8 rows behind it, and its gradient.
//
//   h = bf16(x + residual), r = 1 / sqrt(mean(h^2) + eps), y = h r w
//   u = h r, g = grad_y w:  grad_x = r (g - u mean(g u)) + grad_h,
//   grad_w = sum over the rows of grad_y u
//
// A row belongs to as many wavefronts as hold it in registers, V vectors of 8
// channels a lane, so that it is read once; its sums go through LDS. Many rows of
// up to 256 channels share wavefronts, two or four in each. 16 neighbouring lanes
// hold a block of 128 channels, which is quantised from registers as rows of
// their own are. The gradient needs no statistics kept from the forward pass: the
// mean of h^2 is added again beside that of g h.
//
// HBM bounds both: 4096 x 7168 with the residual to bf16 and fp8 rows 46.2 us
// for 265 MB (5.7 TB/s), the gradient 45.6 us for 235 MB (5.2 TB/s), with the
// weight's 45 to 48.6 by the buffers. One row takes 4.2 us, which is the launch.
#include "dispatch_common.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

constexpr int kNormMaxWaves = 16;  // of a workgroup, and so of a row
constexpr int64_t kMaxNormGroups = 1 << 20;  // larger grids loop
constexpr int kCus = 256;
constexpr int kFewNarrow = 1024;  // rows, see lanes_for
// What moves more goes past the caches both ways (the gradient of 4096 x 7168,
// 235 MB: 50.4 us, through the caches 54.4; 20000 x 1024, 164 MB: 31.6 and 36.5;
// the forward pass of 20000 x 1024, 184 MB: 33.3 and 37.8). A smaller result stays
// where its reader finds it.
constexpr int64_t kPastBytes = int64_t(112) << 20;

struct NormParams {
    const Bf16x8* x;
    const Bf16x8* residual;
    const void* weight;
    const int32_t* num_valid_rows;
    Bf16x8* h;
    Bf16x8* y;
    uint8_t* q;
    float* sf;
    int64_t num_rows;
    int32_t vecs;        // vectors of 8 channels in a row
    int32_t blocks;      // blocks of 128 channels, the last one may be short
    int32_t row_waves;   // wavefronts of a row
    int32_t group_rows;  // rows that a workgroup works on at a time
    float per_width;     // 1 / width
    float eps;
    bool weight_half;
};

// 1 / sqrt(x) within 1 ulp for a normal x: the hardware's, and one Newton step
// (0 for an infinite x, which the step has no value for).
__device__ __forceinline__ float inverse_root(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    const float e = __builtin_fmaf(-x * r, r, 1.f);
    return r == 0.f ? 0.f : __builtin_fmaf(0.5f * e, r, r);
}

__device__ __forceinline__ int64_t rows_of(int64_t num_rows, const int32_t* num_valid_rows) {
    if (num_valid_rows == nullptr) return num_rows;
    const int64_t valid = *num_valid_rows;
    return valid < 0 ? 0 : (valid < num_rows ? valid : num_rows);
}

__device__ __forceinline__ void load_weight(const void* weight, bool half, int vec, float (&w)[8]) {
    const Bf16x8* const at = static_cast<const Bf16x8*>(weight);
    if (half) {
        widen_bf16(at[vec], w);
    } else {
        const Bf16x8 a = at[2 * vec], b = at[2 * vec + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __uint_as_float(a[i]), w[4 + i] = __uint_as_float(b[i]);
    }
}

// Sum over a row's lanes in a wavefront, in every one of them.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (kLanes == kWave) return wave_sum(v);
    v = row_sum(v);
    if constexpr (kLanes == 32) v += __shfl_xor(v, 16);
    return v;
}

// kLanes: lanes of a row. Narrow rows share a wavefront.
template <int V, bool kStream, int kLanes>
__global__ void __launch_bounds__(kNormMaxWaves * kWave) norm_kernel(NormParams p) {
    constexpr bool kWhole = kLanes == kWave;
    __shared__ float part[2][kNormMaxWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int mine = kWhole ? wave / p.row_waves : threadIdx.x / kLanes;  // which of the workgroup's rows
    const int step = kWhole ? p.row_waves * kWave : kLanes, first = threadIdx.x - mine * step;
    const int64_t rows = rows_of(p.num_rows, p.num_valid_rows);
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * p.group_rows; base < rows; base += (int64_t)gridDim.x * p.group_rows) {
        const int64_t row = base + mine;
        const bool here = row < rows;
        const int64_t at = row * p.vecs;
        Bf16x8 h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int vec = first + v * step;
            h[v] = Bf16x8{0, 0, 0, 0};
            if (here && vec < p.vecs) h[v] = load_vec<kStream>(p.x + at + vec);
        }
        if (p.residual != nullptr) {
            Bf16x8 r[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int vec = first + v * step;
                r[v] = Bf16x8{0, 0, 0, 0};
                if (here && vec < p.vecs) r[v] = load_vec<kStream>(p.residual + at + vec);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int vec = first + v * step;
                float a[8], b[8];
                widen_bf16(h[v], a);
                widen_bf16(r[v], b);
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] += b[i];
                h[v] = narrow_bf16(a);
                if (here && vec < p.vecs) store_vec<kStream>(p.h + at + vec, h[v]);
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a[8];
            widen_bf16(h[v], a);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(a[i], a[i], sum);
        }
        sum = lanes_sum<kLanes>(sum);
        if (kWhole && p.row_waves > 1) {
            // (Two rows of parts in turn: a wavefront may be a row ahead.)
            if ((threadIdx.x & (kWave - 1)) == 0) part[turn][wave] = sum;
            __syncthreads();
            sum = 0.f;
            for (int w = 0; w < p.row_waves; ++w) sum += part[turn][mine * p.row_waves + w];
            turn ^= 1;
        }
        if (!here) continue;
        const float r = inverse_root(sum * p.per_width + p.eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int vec = first + v * step;
            const bool live = vec < p.vecs;
            if ((vec & ~15) >= p.vecs) break;  // (the lanes of a block stay together)
            float a[8], w[8] = {};
            widen_bf16(h[v], a);
            if (live) load_weight(p.weight, p.weight_half, vec, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = a[i] * r * w[i];
            if (p.y != nullptr && live) store_vec<kStream>(p.y + at + vec, narrow_bf16(a));
            if (p.q != nullptr)
                quantize8<kStream>(a, live, vec % 16 == 0, p.q + (at + vec) * 8, p.sf + row * p.blocks + vec / 16);
        }
    }
}

struct NormBackwardParams {
    const Bf16x8* h;
    const void* weight;
    const Bf16x8* grad_y;
    const Bf16x8* grad_h;
    const int32_t* num_valid_rows;
    Bf16x8* grad_x;
    float* grad_weight;  // a row of sums for each workgroup
    int64_t num_rows;
    int32_t vecs;
    int32_t row_waves;
    int32_t group_rows;
    float per_width;  // 1 / width
    float eps;
    bool weight_half;
};

// With one vector a lane the next row is on its way while this one is worked
// on, and the weight stays in registers: a load of it between the two would be
// waited for behind the next row's. From four vectors on a row is loaded again
// for the second look, there is no room for it beside the weight's sums.
template <int V, bool kStream, bool kWeight, int kLanes>
__global__ void __launch_bounds__(kNormMaxWaves * kWave) norm_backward_kernel(NormBackwardParams p) {
    constexpr bool kWhole = kLanes == kWave;
    constexpr bool kAhead = V == 1, kKeep = V <= 2;
    __shared__ float2 part[2][kNormMaxWaves];
    extern __shared__ float4 sums[];  // with kWeight, and rows beside each other: one row
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int mine = kWhole ? wave / p.row_waves : threadIdx.x / kLanes;
    const int step = kWhole ? p.row_waves * kWave : kLanes, first = threadIdx.x - mine * step;
    const int64_t rows = rows_of(p.num_rows, p.num_valid_rows);
    const int64_t stride = (int64_t)gridDim.x * p.group_rows;
    float dw[kWeight ? V : 1][8] = {};
    float kept_w[8] = {};
    if (kAhead && first < p.vecs) load_weight(p.weight, p.weight_half, first, kept_w);
    const auto weight_of = [&](int vec, float(&w)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = kept_w[i];
        if (!kAhead && vec < p.vecs) load_weight(p.weight, p.weight_half, vec, w);
    };
    const auto load = [&](const Bf16x8* from, int64_t row, int v) {
        const int vec = first + v * step;
        if (from == nullptr || row >= rows || vec >= p.vecs) return Bf16x8{0, 0, 0, 0};
        return load_vec<kStream>(from + row * p.vecs + vec);
    };
    int turn = 0;
    Bf16x8 next_h, next_dy, next_dh;
    const auto load_next = [&](int64_t row) {
        next_h = load(p.h, row, 0);
        next_dy = load(p.grad_y, row, 0);
        next_dh = load(p.grad_h, row, 0);
    };
    Bf16x8 h[V], dy[V], dh;
    int64_t base = (int64_t)blockIdx.x * p.group_rows;
    if (kAhead && base < rows) load_next(base + mine);
    for (; base < rows; base += stride) {
        const int64_t row = base + mine;
        if (kAhead) {
            h[0] = next_h, dy[0] = next_dy, dh = next_dh;
            if (base + stride < rows) load_next(row + stride);
        }
        if (kKeep && !kAhead) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = load(p.h, row, v), dy[v] = load(p.grad_y, row, v);
        }
        float square = 0.f, along = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a[8], d[8], w[8];
            if (!kKeep) h[v] = load(p.h, row, v), dy[v] = load(p.grad_y, row, v);
            weight_of(first + v * step, w);
            widen_bf16(h[v], a);
            widen_bf16(dy[v], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                square = __builtin_fmaf(a[i], a[i], square);
                along = __builtin_fmaf(w[i], d[i] * a[i], along);
            }
        }
        square = lanes_sum<kLanes>(square);
        along = lanes_sum<kLanes>(along);
        if (kWhole && p.row_waves > 1) {
            if ((threadIdx.x & (kWave - 1)) == 0) part[turn][wave] = float2{square, along};
            __syncthreads();
            square = along = 0.f;
            for (int i = 0; i < p.row_waves; ++i) {
                const float2 x = part[turn][mine * p.row_waves + i];
                square += x.x;
                along += x.y;
            }
            turn ^= 1;
        }
        // grad_x = (r w) grad_y - u (r mean(g u)) + grad_h. (Where r is 0 so is u,
        // and the sum of g h may be infinite or have no value.)
        const float r = inverse_root(square * p.per_width + p.eps);
        const float back = r == 0.f ? 0.f : along * p.per_width * r * r;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int vec = first + v * step;
            float a[8], d[8], b[8], w[8];
            if (!kKeep) h[v] = load(p.h, row, v), dy[v] = load(p.grad_y, row, v);
            if (!kAhead) dh = load(p.grad_h, row, v);
            weight_of(vec, w);
            widen_bf16(h[v], a);
            widen_bf16(dy[v], d);
            widen_bf16(dh, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = a[i] * r;
                if (kWeight) dw[kWeight ? v : 0][i] = __builtin_fmaf(d[i], u, dw[kWeight ? v : 0][i]);
                b[i] = __builtin_fmaf(-u, back, __builtin_fmaf(r * w[i], d[i], b[i]));
            }
            if (row < rows && vec < p.vecs) store_vec<kStream>(p.grad_x + row * p.vecs + vec, narrow_bf16(b));
        }
    }
    if constexpr (kWeight) {
        // The workgroup's rows of sums, one after the other, a wavefront's together.
        float4* const to = reinterpret_cast<float4*>(p.grad_weight) + (int64_t)blockIdx.x * p.vecs * 2;
#pragma unroll
        for (int d = kLanes; d < kWave; d *= 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[0][i] += __shfl_xor(dw[0][i], d);
        const int all = p.group_rows / (kWave / kLanes), at = kWhole ? mine : wave;
        for (int n = 0; n < all; ++n) {
            if (n == at && (kWhole || (threadIdx.x & (kWave - 1)) < kLanes)) {
                const bool last = n == all - 1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int vec = first + v * step;
                    if (vec >= p.vecs) continue;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float4 x{dw[v][4 * i], dw[v][4 * i + 1], dw[v][4 * i + 2], dw[v][4 * i + 3]};
                        if (n > 0) {
                            const float4 y = sums[2 * vec + i];
                            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                        }
                        (last ? to : sums)[2 * vec + i] = x;
                    }
                }
            }
            if (all > 1) __syncthreads();
        }
    }
}

// Adds the rows of sums: a workgroup takes 32 channels, 8 threads of four; its
// 128 groups of such threads add every 128th row, four of them on their way at
// once, then the groups of a wavefront and the wavefronts are added in order.
constexpr int kSumThreads = 1024;
constexpr int kSumLanes = 8;
constexpr int kSumGroups = kSumThreads / kSumLanes;

__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float4* partial, int rows, int quads, float4* out) {
    __shared__ float4 part[kSumThreads / kWave][kSumLanes];
    const int g = threadIdx.x / kSumLanes, c = threadIdx.x % kSumLanes;
    const int quad = blockIdx.x * kSumLanes + c;
    float4 s{0.f, 0.f, 0.f, 0.f};
    const auto add = [&](const float4& x) { s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w; };
    if (quad < quads) {
        constexpr int kAtOnce = 4;
        for (int row = g; row < rows; row += kAtOnce * kSumGroups) {
            float4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int at = row + i * kSumGroups;
                x[i] = at < rows ? partial[(int64_t)at * quads + quad] : float4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) add(x[i]);
        }
    }
    for (int step = kSumLanes; step < kWave; step *= 2)
        add(float4{__shfl_xor(s.x, step), __shfl_xor(s.y, step), __shfl_xor(s.z, step), __shfl_xor(s.w, step)});
    if (threadIdx.x % kWave < kSumLanes) part[threadIdx.x / kWave][c] = s;
    __syncthreads();
    if (threadIdx.x >= kSumLanes || quad >= quads) return;
    for (int i = 1; i < kSumThreads / kWave; ++i) add(part[i][c]);
    out[quad] = s;
}

// How a row is cut: V vectors a lane, wavefronts of a row, rows of a workgroup
// at a time, workgroups.
struct NormShape {
    int v, row_waves, group_rows, groups;
    int lanes = kWave;  // of a wavefront for a row: 32 or 16 where narrow rows share one
    int threads() const { return group_rows * row_waves * lanes; }
};

int waves_for(int vecs, int v) { return (vecs + v * kWave - 1) / (v * kWave); }

// Lanes of a row: half or a quarter of a wavefront for narrow rows, from `few`
// rows for each row of a wavefront on. us, with the residual to bf16 and fp8 rows
// / the gradient, and with a wavefront a row (fewer rows: no difference):
//
//   16384 x  64     4.7 /  8.3 ( 7.5 / 10.9)   60000 x  64   8.9 / 11.8 (21.8 / 22.7)
//   16384 x 128     5.6 /  9.5 ( 8.5 / 11.3)   60000 x 128  12.8 / 15.4 (22.4 / 23.2)
//   16384 x 176     6.9 / 10.7 ( 8.7 / 11.7)   60000 x 176  19.7 / 19.1 (28.1 / 24.4)
//   16384 x 256     8.0 / 11.8 ( 9.7 / 12.1)   60000 x 256  25.2 / 25.7 (31.1 / 28.0)
int lanes_for(int64_t rows, int vecs, int64_t few) {
    int lanes = kWave;
    while (lanes > 16 && vecs <= lanes / 2 && rows >= few * (2 * kWave / lanes)) lanes /= 2;
    return lanes;
}

// One vector a lane for few rows, which are bound by latency; two from two
// rows per CU on, wide ones from one (4096 x 7168 channels 46.2 us, 49.1 with one
// and 47.8 with four; 333 x 4096 4.5 us with one, 4.7 with two; 333 x 7168 6.6 and
// 6.2, 64 x 7168 4.25 and 4.4). Narrow rows share a workgroup of four wavefronts.
NormShape norm_shape(int64_t rows, int vecs) {
    NormShape s;
    const bool many = rows >= 2 * kCus ? vecs > kWave : rows > kCus && vecs > 8 * kWave;
    s.v = many ? 2 : 1;
    while (waves_for(vecs, s.v) > kNormMaxWaves) s.v *= 2;
    s.row_waves = waves_for(vecs, s.v);
    s.group_rows = s.row_waves >= 4 ? 1 : 4 / s.row_waves;
    s.lanes = lanes_for(rows, vecs, kFewNarrow);
    s.group_rows *= kWave / s.lanes;
    const int64_t groups = (rows + s.group_rows - 1) / s.group_rows;
    s.groups = (int)(groups < kMaxNormGroups ? groups : kMaxNormGroups);
    return s;
}

// The gradient's workgroups each leave a row of sums, so there are few, one to
// three per CU, with rows beside each other in a workgroup and the next ones on
// their way. Measured, us:
//
//   rows x width     wavefronts of a row, rows of a workgroup: time by workgroups
//    4096 x 7168     14, 1: 256 45.6   512 48   (with 512 the rows of sums cost more)
//    4000 x 4096      8, 2: 256 27.4   512 30.3    8, 1: 512 28.7
//    8191 x 2064      5, 1: 768 25.6   512 31.7    5, 3: 256 27.9
//   14000 x 2048      4, 2: 256 42.1   512 42.9    4, 4: 256 42.9
//    2000 x 2048      4, 2: 256 10.9   512 11.8    4, 4: 256 11.6
//   30000 x  768      2, 4: 512 35.5               2, 8: 256 36.6
//   20000 x  512      1, 8: 512 18.3   256 19.2
//
// A workgroup that takes all rows in a few rounds needs no second kernel: 8 x
// 2048 5.3 us, 7.0 with it; 32 x 512 5.5 and 7.0.
NormShape norm_backward_shape(int64_t rows, int vecs) {
    constexpr int kAlone = 32;  // wavefronts' rows
    NormShape s;
    s.v = 1;
    while (waves_for(vecs, s.v) > kNormMaxWaves) s.v *= 2;
    s.row_waves = waves_for(vecs, s.v);
    const int room = kNormMaxWaves / s.row_waves;
    if (rows * s.row_waves <= kAlone) {
        s.group_rows = rows < 1 ? 1 : (int)(rows < room ? rows : room);
        s.groups = 1;
        return s;
    }
    // (Five wavefronts: three rows would wait for each other.)
    s.group_rows = s.row_waves > 5 ? room : s.row_waves == 5 ? 1 : (room + 1) / 2;
    s.lanes = lanes_for(rows, vecs, 2 * kCus * s.group_rows);  // (so that there is work for as many workgroups)
    s.group_rows *= kWave / s.lanes;
    const int64_t groups = (rows + s.group_rows - 1) / s.group_rows;
    const int most = kCus * (s.row_waves == 5 ? room : s.row_waves > 2 ? 1 : 2);
    s.groups = (int)(groups < most ? groups : most);
    return s;
}

template <int V, int kLanes = kWave>
const void* norm_kernel_of(bool past) {
    return past ? (const void*)&norm_kernel<V, true, kLanes> : (const void*)&norm_kernel<V, false, kLanes>;
}
template <int V, int kLanes = kWave>
const void* norm_backward_of(bool past, bool weight) {
    if (weight)
        return past ? (const void*)&norm_backward_kernel<V, true, true, kLanes>
                    : (const void*)&norm_backward_kernel<V, false, true, kLanes>;
    return past ? (const void*)&norm_backward_kernel<V, true, false, kLanes>
                : (const void*)&norm_backward_kernel<V, false, false, kLanes>;
}

#define DISPATCH_NORM_BY_V(V_, F) ((V_) == 1 ? F(1) : (V_) == 2 ? F(2) : (V_) == 4 ? F(4) : F(8))

}  // namespace

hipError_t launch_rms_norm(const dispatch_rms_norm_problem_t& prob, const void* x, const void* residual,
                           const void* weight, const int32_t* num_valid_rows, void* h, void* y, void* q, float* sf,
                           hipStream_t stream) {
    if (prob.num_rows == 0) return hipSuccess;
    NormParams p{};
    p.x = static_cast<const Bf16x8*>(x);
    p.residual = static_cast<const Bf16x8*>(residual);
    p.weight = weight;
    p.num_valid_rows = num_valid_rows;
    p.h = static_cast<Bf16x8*>(h);
    p.y = static_cast<Bf16x8*>(y);
    p.q = static_cast<uint8_t*>(q);
    p.sf = sf;
    p.num_rows = prob.num_rows;
    p.vecs = (int32_t)(prob.width / 8);
    p.blocks = (int32_t)((prob.width + DISPATCH_SF_BLOCK - 1) / DISPATCH_SF_BLOCK);
    p.per_width = 1.f / (float)prob.width;
    p.eps = prob.eps;
    p.weight_half = prob.weight_bytes == 2;
    const NormShape s = norm_shape(prob.num_rows, p.vecs);
    p.row_waves = s.row_waves;
    p.group_rows = s.group_rows;
    const int64_t channel_bytes = 2 + (residual ? 4 : 0) + (y ? 2 : 0) + (q ? 1 : 0);
    const bool past = prob.num_rows * prob.width * channel_bytes > kPastBytes;
#define DISPATCH_F(V) norm_kernel_of<V>(past)
    const void* kernel = s.lanes == 16   ? norm_kernel_of<1, 16>(past)
                         : s.lanes == 32 ? norm_kernel_of<1, 32>(past)
                                         : DISPATCH_NORM_BY_V(s.v, DISPATCH_F);
#undef DISPATCH_F
    void* args[] = {&p};
    return hipLaunchKernel(kernel, dim3(s.groups), dim3(s.threads()), args, 0, stream);
}

size_t rms_norm_workspace_bytes(const dispatch_rms_norm_problem_t& prob) {
    const NormShape s = norm_backward_shape(prob.num_rows, (int)(prob.width / 8));
    return ((size_t)s.groups * prob.width * sizeof(float) + 255) & ~size_t(255);
}

hipError_t launch_rms_norm_backward(const dispatch_rms_norm_problem_t& prob, const void* h, const void* weight,
                                    const void* grad_y, const void* grad_h, const int32_t* num_valid_rows,
                                    void* grad_x, float* grad_weight, void* workspace, hipStream_t stream) {
    if (prob.num_rows == 0 && grad_weight == nullptr) return hipSuccess;
    NormBackwardParams p{};
    p.h = static_cast<const Bf16x8*>(h);
    p.weight = weight;
    p.grad_y = static_cast<const Bf16x8*>(grad_y);
    p.grad_h = static_cast<const Bf16x8*>(grad_h);
    p.num_valid_rows = num_valid_rows;
    p.grad_x = static_cast<Bf16x8*>(grad_x);
    p.num_rows = prob.num_rows;
    p.vecs = (int32_t)(prob.width / 8);
    p.per_width = 1.f / (float)prob.width;
    p.eps = prob.eps;
    p.weight_half = prob.weight_bytes == 2;
    const NormShape s = norm_backward_shape(prob.num_rows, p.vecs);
    p.row_waves = s.row_waves;
    p.group_rows = s.group_rows;
    int rows = s.groups;
    p.grad_weight = rows == 1 ? grad_weight : static_cast<float*>(workspace);
    const bool past = prob.num_rows * prob.width * (grad_h ? 8 : 6) > kPastBytes;
#define DISPATCH_F(V) norm_backward_of<V>(past, weighs)
    const bool weighs = grad_weight != nullptr;
    const void* kernel = s.lanes == 16   ? norm_backward_of<1, 16>(past, weighs)
                         : s.lanes == 32 ? norm_backward_of<1, 32>(past, weighs)
                                         : DISPATCH_NORM_BY_V(s.v, DISPATCH_F);
#undef DISPATCH_F
    void* args[] = {&p};
    const size_t shared = s.group_rows > 1 && grad_weight != nullptr ? prob.width * sizeof(float) : 0;
    const hipError_t err =
        hipLaunchKernel(kernel, dim3(s.groups), dim3(s.threads()), args, shared, stream);
    if (err != hipSuccess || grad_weight == nullptr || rows == 1) return err;
    const float* partial = p.grad_weight;
    int quads = (int)(prob.width / 4);
    void* sum_args[] = {&partial, &rows, &quads, &grad_weight};
    return hipLaunchKernel((const void*)&norm_sum_kernel, dim3((quads + kSumLanes - 1) / kSumLanes), dim3(kSumThreads),
                           sum_args, 0, stream);
}

}  // namespace moe_dispatch
