// Arithmetic helpers of the gate, quantisation and product kernels (included
// by .hip files only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe_dispatch {

constexpr float kFp8Max = 448.f;  // largest finite e4m3 value
// The floor of a block's largest magnitude: below it 448 / amax would leave
// fp32's range, and a block of zeros would have no scale.
constexpr float kAmaxFloor = 0x1p-100f;

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values rounded to bf16 (to nearest, ties to even), packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Four fp32 values rounded to e4m3 (to nearest, ties to even), packed.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// DPP controls: rotations within a row of 16 lanes, and broadcasts of a
// row's last lane into the following rows.
constexpr int kDppRowShr = 0x110;
constexpr int kDppRowRor = 0x120;
// (also: a lane's neighbour and next but one in its four, its mirror image in
// its eight and in its row.)
constexpr int kDppQuadXor1 = 0xb1;
constexpr int kDppQuadXor2 = 0x4e;
constexpr int kDppRowHalfMirror = 0x141;
constexpr int kDppRowMirror = 0x140;
constexpr int kDppBcast15 = 0x142;
constexpr int kDppBcast31 = 0x143;

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_ror(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kCtrl, 0xf, 0xf, false);
}

// Largest of the 16 lanes of a row, in every lane of the row.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    uint32_t o = dpp_ror<kDppRowRor + 1>(v);
    v = v > o ? v : o;
    o = dpp_ror<kDppRowRor + 2>(v);
    v = v > o ? v : o;
    o = dpp_ror<kDppRowRor + 4>(v);
    v = v > o ? v : o;
    o = dpp_ror<kDppRowRor + 8>(v);
    return v > o ? v : o;
}

// Sum of the 16 lanes of a row, in every lane of the row: the same bits, as
// each step adds a pair of sums that both its lanes have.
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(dpp_ror<kDppRowRor + 8>(__float_as_uint(v)));
    v += __uint_as_float(dpp_ror<kDppRowRor + 4>(__float_as_uint(v)));
    v += __uint_as_float(dpp_ror<kDppRowRor + 2>(__float_as_uint(v)));
    v += __uint_as_float(dpp_ror<kDppRowRor + 1>(__float_as_uint(v)));
    return v;
}

// One block's 8 channels of a lane: quantised to dst, the scale by lane 0.
// kStream: stored past the caches.
template <bool kStream>
__device__ __forceinline__ void quantize8(const float (&v)[8], bool live, bool first, uint8_t* dst, float* sf) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    // The largest magnitude by its bits, which order as the values do, NaN
    // above infinity.
    uint32_t top = __float_as_uint(kAmaxFloor);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
        top = top > m ? top : m;
    }
    const float amax = __uint_as_float(row_max(top));
    const float scale = kFp8Max / amax;
    const u32x2 o = {pack_fp8(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale),
                     pack_fp8(v[4] * scale, v[5] * scale, v[6] * scale, v[7] * scale)};
    if (live) {
        if (kStream)
            __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(dst));
        else
            *reinterpret_cast<u32x2*>(dst) = o;
    }
    if (first) *sf = amax / kFp8Max;
}

// Reductions over the 64 lanes, the result uniform. The order of the sum is
// fixed.
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_float(float old, float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_float<kDppRowShr + 1, 0xf>(0.f, v);
    v += dpp_float<kDppRowShr + 2, 0xf>(0.f, v);
    v += dpp_float<kDppRowShr + 4, 0xf>(0.f, v);
    v += dpp_float<kDppRowShr + 8, 0xf>(0.f, v);
    v += dpp_float<kDppBcast15, 0xa>(0.f, v);
    v += dpp_float<kDppBcast31, 0xc>(0.f, v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Largest of the 64 lanes, uniform.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowShr + 1, 0xf, 0xf, true);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowShr + 2, 0xf, 0xf, true);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowShr + 4, 0xf, 0xf, true);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppRowShr + 8, 0xf, 0xf, true);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppBcast15, 0xa, 0xf, false);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDppBcast31, 0xc, 0xf, false);
    v = v > o ? v : o;
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// 1 / (1 + exp(-z)) from the hardware's exp2 and reciprocal: relative error
// about (|z| + 4) 2^-24, below that of the products it follows.
__device__ __forceinline__ float fast_sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
}

// The same within 3 * 2^-24 for any z (2.2 over the bf16 values), as a row is
// quantised from it and a value further off changes its 8 bits more often: the
// argument's rounding error -z - x ln 2 and the reciprocal's are put right. Far from
// 0 these steps meet infinities, so the ends are settled beside them: a z above
// 2^100 is taken as that (the result is 1 from 17 on, and x would overflow); below
// -88.7 exp(-z) is infinite, the last step has no value, and the maximum makes it 0.
// (A NaN is lost here, not by the z that the result is multiplied with.) SwiGLU's
// gradient of 32777 x 4096 channels takes 89.4 us with it, 85.4 with fast_sigmoid,
// and 113 with expf and a correct division.
__device__ __forceinline__ float near_sigmoid(float z) {
    const float ln2 = 0.693147182f, rest = -1.90465421e-9f;  // ln(2) and what its rounding left
    z = fminf(z, 0x1p100f);
    const float x = -1.44269504f * z;
    const float low = __builtin_fmaf(-rest, x, __builtin_fmaf(-ln2, x, -z));
    const float e = __builtin_amdgcn_exp2f(x);
    const float d = 1.f + __builtin_fmaf(e, low, e);
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaxf(__builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r), 0.f);
}

// 1 / (1 + exp(-z)), the division rounded correctly: what the gate compares.
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

}  // namespace moe_dispatch
