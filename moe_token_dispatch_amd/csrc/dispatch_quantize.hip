// Rows to fp8 with one scale per 128 channels on gfx950: of bf16 rows, of
// SwiGLU of bf16 rows, and of SwiGLU's gradient.
//
// A block of 128 channels is 16 lanes of 8 channels: one 16-byte load per
// lane and operand, the block's largest magnitude by four DPP rotations
// within the 16-lane row, one 8-byte store. Nothing is read twice and nothing
// goes through LDS, so the kernel is bound by HBM: 2 bytes read and 1 written
// per channel (4 and 1 for SwiGLU, 6 and 2 for its gradient).
// Measured: 4096 x 7168 rows 16.4 us (5.4 TB/s), SwiGLU's gradient of 32777 rows
// of 2048 89.4 us (6.05 TB/s; a large copy reaches 5.0 to 5.3); 8 rows of 2048
// through SwiGLU 3.9 us, which is the launch.
#include "dispatch_common.hpp"
#include "dispatch_device.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

constexpr int kQuantizeThreads = 256;
constexpr int kLanesPerBlock = 16;
constexpr int kMaxQuantizeGroups = 1 << 20;  // larger grids loop
constexpr int64_t kInfinityCacheBytes = int64_t(256) << 20;

struct QuantizeParams {
    const uint16_t* x;
    const uint16_t* grad;
    const int32_t* num_valid_rows;
    uint8_t* q;
    float* sf;
    int64_t num_rows;
    int64_t width;    // channels of a row of grad / of half a row of h / of x
    uint32_t blocks;  // ceil(width / 128)
};

__device__ __forceinline__ void widen(const u32x4& w, float (&v)[8]) {
    v[0] = bf16_low(w.x), v[1] = bf16_high(w.x), v[2] = bf16_low(w.y), v[3] = bf16_high(w.y);
    v[4] = bf16_low(w.z), v[5] = bf16_high(w.z), v[6] = bf16_low(w.w), v[7] = bf16_high(w.w);
}

template <bool kStream>
__device__ __forceinline__ u32x4 load8(const uint16_t* at) {
    const u32x4* v = reinterpret_cast<const u32x4*>(at);
    return kStream ? __builtin_nontemporal_load(v) : *v;
}

template <QuantizeSource kSource, bool kStream>
__global__ void __launch_bounds__(kQuantizeThreads) quantize_kernel(QuantizeParams p) {
    const int lane = threadIdx.x % kLanesPerBlock;
    int64_t rows = p.num_rows;
    if (p.num_valid_rows != nullptr) {
        const int64_t valid = *p.num_valid_rows;
        rows = valid < 0 ? 0 : (valid < rows ? valid : rows);
    }
    // The host bounds rows * blocks below 2^31.
    const uint32_t total = (uint32_t)rows * p.blocks;
    const uint32_t stride = gridDim.x * (kQuantizeThreads / kLanesPerBlock);
    for (uint32_t b = blockIdx.x * (kQuantizeThreads / kLanesPerBlock) + threadIdx.x / kLanesPerBlock; b < total;
         b += stride) {
        const uint32_t row = b / p.blocks;
        const uint32_t block = b - row * p.blocks;
        const int64_t c = (int64_t)block * 128 + lane * 8;  // this lane's first channel
        const bool live = c < p.width;                      // widths are multiples of 16
        if (kSource == QuantizeSource::kRows) {
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) widen(load8<kStream>(p.x + row * p.width + c), v);
            quantize8<kStream>(v, live, lane == 0, p.q + row * p.width + c, p.sf + b);
        } else {
            float g[8], u[8];
            const uint16_t* h = p.x + row * 2 * p.width + c;
            const u32x4 gw = load8<kStream>(h);
            const u32x4 uw = load8<kStream>(h + p.width);
            widen(gw, g);
            widen(uw, u);
            if (kSource == QuantizeSource::kSwiglu) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = g[i] * near_sigmoid(g[i]) * u[i];
                quantize8<kStream>(g, true, lane == 0, p.q + row * p.width + c, p.sf + b);
            } else {
                float d[8];
                widen(load8<kStream>(p.grad + row * p.width + c), d);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = near_sigmoid(g[i]);
                    const float du = d[i] * g[i] * s;
                    g[i] = d[i] * u[i] * s * (1.f + g[i] * (1.f - s));
                    u[i] = du;
                }
                uint8_t* q = p.q + row * 2 * p.width + c;
                float* sf = p.sf + (int64_t)row * 2 * p.blocks + block;
                quantize8<kStream>(g, true, lane == 0, q, sf);
                quantize8<kStream>(u, true, lane == 0, q + p.width, sf + p.blocks);
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize(QuantizeSource source, const dispatch_quantize_problem_t& prob, const void* x,
                           const void* grad, const int32_t* num_valid_rows, void* q, float* sf,
                           hipStream_t stream) {
    QuantizeParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.grad = static_cast<const uint16_t*>(grad);
    p.num_valid_rows = num_valid_rows;
    p.q = static_cast<uint8_t*>(q);
    p.sf = sf;
    p.num_rows = prob.num_rows;
    p.width = prob.width;
    p.blocks = (uint32_t)((prob.width + 127) / 128);
    const int64_t per = kQuantizeThreads / kLanesPerBlock;
    int64_t groups = (prob.num_rows * p.blocks + per - 1) / per;
    if (groups == 0) return hipSuccess;
    if (groups > kMaxQuantizeGroups) groups = kMaxQuantizeGroups;
    // What does not fit the Infinity Cache goes past the caches both ways
    // (32777 x 4096 channels of SwiGLU's gradient, 541 MB: 86 against 95 us).
    // A smaller result stays where its reader finds it.
    const int64_t channel_bytes = source == QuantizeSource::kRows ? 3 : (source == QuantizeSource::kSwiglu ? 5 : 8);
    const bool stream_past = prob.num_rows * prob.width * channel_bytes > kInfinityCacheBytes;
    const auto pick = [&](const void* past, const void* cached) { return stream_past ? past : cached; };
    using S = QuantizeSource;
    const void* kernel =
        source == S::kRows
            ? pick((const void*)&quantize_kernel<S::kRows, true>, (const void*)&quantize_kernel<S::kRows, false>)
        : source == S::kSwiglu
            ? pick((const void*)&quantize_kernel<S::kSwiglu, true>, (const void*)&quantize_kernel<S::kSwiglu, false>)
            : pick((const void*)&quantize_kernel<S::kSwigluGrad, true>,
                   (const void*)&quantize_kernel<S::kSwigluGrad, false>);
    void* args[] = {&p};
    return hipLaunchKernel(kernel, dim3((unsigned)groups), dim3(kQuantizeThreads), args, 0, stream);
}

}  // namespace moe_dispatch
