// The experts' product on gfx950: fp8 rows of an expert-major buffer times
// each expert's fp8 weights, with fp32 scales per block of 128 channels.
//
// The weights' rows are the matrix instruction's A operand and the tokens its
// B operand: of a 16 x 16 result a lane then holds four consecutive output
// channels of ONE token, so a block's scale x_sf * w_sf is one number per
// lane and the channels leave as one 8-byte store.
// v_mfma_f32_16x16x128_f8f6f4 takes one 128-channel block whole. Its result
// for the block (C = 0) is scaled and added to the fp32 sums with one fused
// multiply-add per value: four per 32-cycle matrix instruction. (The fp8
// instruction itself adds each run of 16 products in fixed point and drops
// what is below about 2^-14 of the run's largest, on any of its shapes; its
// error, about 5e-5 of a block's typical sum on normal data, is far below the
// operands' own 2^-4. Across blocks all sums are fp32.)
//
// Which channels of the block a lane's 32 bytes stand for does not matter as
// long as both operands agree (the sum runs over all of them): lane group
// g = lane / 16 takes the 16-byte chunks g and g + 4, so that one load
// instruction covers 64 consecutive bytes of 16 rows.
#include "dispatch_common.hpp"
#include "dispatch_device.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kXcds = 8;  // workgroup i runs on XCD i % 8

struct ProductParams {
    const int32_t* psum;
    const int32_t* count;
    const uint8_t* x;
    const float* x_sf;
    const uint8_t* w;
    const float* w_sf;
    void* out;
    float* out_sf;
    int64_t expert_rows;
    int32_t num_experts;
    int32_t K;
    int32_t N;          // weight rows of an expert (2I for the SwiGLU product)
    int32_t k_blocks;   // ceil(K / 128)
    int32_t n_blocks;   // ceil(N / 128)
    int32_t n_tiles;    // tiles of the output's width
};

// A product tile: rows [row, row + rows) of the buffer, tile n of the width.
struct Tile {
    int expert;
    int n;
    int rows;
    int row;
};

// Live rows of expert e: within the buffer, never negative.
__device__ __forceinline__ int live_rows(const ProductParams& p, int e) {
    const int64_t first = p.psum[e];
    int64_t n = p.count[e];
    if (first < 0 || n < 0) n = 0;
    if (first + n > p.expert_rows) n = p.expert_rows - first;
    return n < 0 ? 0 : (int)n;
}

// Inclusive sum over the wavefront's lanes.
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, kDppRowShr + 1, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kDppRowShr + 2, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kDppRowShr + 4, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kDppRowShr + 8, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kDppBcast15, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, kDppBcast31, 0xc, 0xf, false);
    return x;
}

// Row tiles of kRows rows over all experts.
template <int kRows>
__device__ __forceinline__ int count_row_tiles(const ProductParams& p) {
    const int lane = threadIdx.x & (kWave - 1);
    int tiles = 0;
    for (int e = lane; e < p.num_experts; e += kWave) tiles += (live_rows(p, e) + kRows - 1) / kRows;
    return __builtin_amdgcn_readlane(wave_scan(tiles), kWave - 1);
}

// Tile `item` in the order expert, tile of the width, row tile: the row tiles
// that read the same weights follow each other. Every wavefront finds it for
// itself.
template <int kRows>
__device__ __forceinline__ Tile find_tile(const ProductParams& p, int64_t item) {
    const int lane = threadIdx.x & (kWave - 1);
    const int target = (int)item / p.n_tiles;  // its row tile if each were taken whole (the same expert)
    int before = 0;
    Tile t{};
    for (int base = 0; base < p.num_experts; base += kWave) {
        const int e = base + lane;
        const int rows = e < p.num_experts ? live_rows(p, e) : 0;
        const int tiles = (rows + kRows - 1) / kRows;
        const int upto = before + wave_scan(tiles);
        const uint64_t past = __ballot(upto > target);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            const int mine = __builtin_amdgcn_readlane(tiles, l);
            const int first = __builtin_amdgcn_readlane(upto, l) - mine;
            const int live = __builtin_amdgcn_readlane(rows, l);
            const int local = (int)item - first * p.n_tiles;
            // (All uniform; said so, they stay in scalar registers.)
            t.expert = __builtin_amdgcn_readfirstlane(base + l);
            t.n = __builtin_amdgcn_readfirstlane(local / mine);
            const int m = local - t.n * mine;
            t.row = __builtin_amdgcn_readfirstlane(p.psum[t.expert] + m * kRows);
            t.rows = __builtin_amdgcn_readfirstlane(live - m * kRows < kRows ? live - m * kRows : kRows);
            return t;
        }
        before = __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return t;  // not reached for item < row tiles * n_tiles: rows = 0
}

// Workgroup b's i-th item: the items are cut into eight runs, one per XCD, so
// that tiles sharing weights or rows share an L2.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int64_t total) {
    const int64_t run = (total + kXcds - 1) / kXcds;
    return (b % kXcds) * run + b / kXcds;
}

// ------------------------------------------------------ few rows per expert
//
// With few rows per expert the product reads weights and little else. A wave
// holds 64 weight rows x 16 * kTokens tokens of sums and walks every kSplit-th
// block of K, loading the weights straight into the matrix operands: each
// weight byte is used by one wavefront only, so LDS would add a copy and save
// nothing. The kSplit wavefronts of the same 64 rows add their sums through
// LDS at the end, halving their number each time (a fixed order).
template <int kTokens, bool kSwiglu>
struct StreamShape {
    static constexpr int kRowGroups = kSwiglu ? 4 : 1;  // 64 weight rows each
    static constexpr int kSplit = kSwiglu ? 4 : 8;
    static constexpr int kWaves = kRowGroups * kSplit;
    static constexpr int kTileRows = 16 * kTokens;
    static constexpr int kSliceFloats = 64 * kTileRows;  // one wavefront's sums
    static constexpr int kLdsFloats = kRowGroups * (kSplit / 2) * kSliceFloats;
};

__device__ __forceinline__ i32x8 load_block(const uint8_t* row, int k, int K) {
    // Chunks k and k + 64 of the row; beyond K (a multiple of 16) zeros.
    u32x4 lo = {0u, 0u, 0u, 0u}, hi = {0u, 0u, 0u, 0u};
    if (k < K) lo = *reinterpret_cast<const u32x4*>(row + k);
    if (k + 64 < K) hi = *reinterpret_cast<const u32x4*>(row + k + 64);
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__device__ __forceinline__ f32x4 mfma_block(const i32x8& a, const i32x8& b) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

template <int kTokens, bool kSwiglu>
__global__ void __launch_bounds__((StreamShape<kTokens, kSwiglu>::kWaves * kWave))
stream_kernel(ProductParams p) {
    using Shape = StreamShape<kTokens, kSwiglu>;
    extern __shared__ __align__(16) float lds[];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int group = wave % Shape::kRowGroups, split = wave / Shape::kRowGroups;
    const int col = lane & 15, quad = lane >> 4;
    const int64_t total = (int64_t)count_row_tiles<Shape::kTileRows>(p) * p.n_tiles;
    for (int64_t i = blockIdx.x; i < (total + kXcds - 1) / kXcds * kXcds; i += gridDim.x) {
        const int64_t item = xcd_item(i, total);
        if (item >= total) continue;
        const Tile t = find_tile<Shape::kTileRows>(p, item);
        // First weight row of this wavefront: the SwiGLU product's groups 0
        // and 1 take 128 gate rows, 2 and 3 the up rows of the same channels.
        const int n0 = kSwiglu ? t.n * 128 + (group & 1) * 64 + (group >> 1) * (p.N / 2) : t.n * 64;
        const uint8_t* w[4];
        const uint8_t* x[kTokens];
        const float* xs[kTokens];
        const float* ws[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            int n = n0 + f * 16 + col;
            n = n < p.N ? n : p.N - 1;  // (rows past the end are computed and dropped)
            w[f] = p.w + ((int64_t)t.expert * p.N + n) * p.K;
            int nb = (n0 + f * 16) >> 7;
            nb = nb < p.n_blocks ? nb : p.n_blocks - 1;
            ws[f] = p.w_sf + ((int64_t)t.expert * p.n_blocks + nb) * p.k_blocks;
        }
#pragma unroll
        for (int m = 0; m < kTokens; ++m) {
            int r = m * 16 + col;
            r = r < t.rows ? r : t.rows - 1;
            x[m] = p.x + (int64_t)(t.row + r) * p.K;
            xs[m] = p.x_sf + (int64_t)(t.row + r) * p.k_blocks;
        }
        f32x4 acc[4][kTokens];
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int m = 0; m < kTokens; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kb = split; kb < p.k_blocks; kb += Shape::kSplit) {
            const int k = kb * 128 + quad * 16;
            i32x8 a[4], b[kTokens];
            float sx[kTokens];
#pragma unroll
            for (int f = 0; f < 4; ++f) a[f] = load_block(w[f], k, p.K);
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                b[m] = load_block(x[m], k, p.K);
                sx[m] = xs[m][kb];
            }
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float sw = ws[f][kb];
#pragma unroll
                for (int m = 0; m < kTokens; ++m) {
                    const f32x4 y = mfma_block(a[f], b[m]);
                    const float s = sx[m] * sw;
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[f][m][q] = __builtin_fmaf(s, y[q], acc[f][m][q]);
                }
            }
        }
        // Sums of the splits, halving their number.
#pragma unroll
        for (int half = Shape::kSplit / 2; half > 0; half /= 2) {
            f32x4* slice = reinterpret_cast<f32x4*>(lds) +
                           (group * (Shape::kSplit / 2) + (split & (half - 1))) * (Shape::kSliceFloats / 4);
            if (split >= half && split < 2 * half) {
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int m = 0; m < kTokens; ++m) slice[(f * kTokens + m) * kWave + lane] = acc[f][m];
            }
            __syncthreads();
            if (split < half) {
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int m = 0; m < kTokens; ++m) acc[f][m] += slice[(f * kTokens + m) * kWave + lane];
            }
            __syncthreads();
        }
        if (!kSwiglu) {
            if (split == 0) {
                uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int n = n0 + f * 16 + quad * 4;
#pragma unroll
                    for (int m = 0; m < kTokens; ++m) {
                        const int r = m * 16 + col;
                        if (r < t.rows && n < p.N) {  // N is a multiple of 8
                            uint2 o;
                            o.x = pack_bf16(acc[f][m][0], acc[f][m][1]);
                            o.y = pack_bf16(acc[f][m][2], acc[f][m][3]);
                            *reinterpret_cast<uint2*>(out + (int64_t)(t.row + r) * p.N + n) = o;
                        }
                    }
                }
            }
        } else {
            // [token][256] sums: gate channels, then up channels. A row is
            // 4 floats longer than that, so that the 16 tokens of a store
            // fall into different banks.
            constexpr int kRow = 256 + 4;
            static_assert(!kSwiglu || Shape::kTileRows * kRow <= Shape::kLdsFloats, "epilogue rows");
            if (split == 0) {
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int m = 0; m < kTokens; ++m)
                        *reinterpret_cast<f32x4*>(lds + (m * 16 + col) * kRow + group * 64 + f * 16 + quad * 4) =
                            acc[f][m];
            }
            __syncthreads();
            const int I = p.N / 2;
            const int r = threadIdx.x / 16, c = (threadIdx.x & 15) * 8;
            for (int token = r; token < Shape::kTileRows; token += Shape::kWaves * 4) {
                if (token < t.rows) {
                    const float* g = lds + token * kRow + c;
                    float v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = g[q] * sigmoid(g[q]) * g[128 + q];
                    uint8_t* dst = static_cast<uint8_t*>(p.out) + (int64_t)(t.row + token) * I + t.n * 128 + c;
                    quantize8(v, true, c == 0, dst, p.out_sf + (int64_t)(t.row + token) * (I / 128) + t.n);
                }
            }
            __syncthreads();
        }
    }
}

template <int kTokens, bool kSwiglu>
hipError_t launch_stream(ProductParams p, int64_t max_rows, hipStream_t stream) {
    using Shape = StreamShape<kTokens, kSwiglu>;
    p.n_tiles = kSwiglu ? p.N / 256 : (p.N + 63) / 64;
    // Row tiles at most: one of each expert that has a row may be partial.
    const int64_t row_tiles = max_rows / Shape::kTileRows + (max_rows < p.num_experts ? max_rows : p.num_experts);
    int64_t groups = (row_tiles * p.n_tiles + kXcds - 1) / kXcds * kXcds;
    if (groups > 65536) groups = 65536;  // larger batches loop
    if (groups < kXcds) groups = kXcds;
    const size_t shared = Shape::kLdsFloats * sizeof(float);
    void* args[] = {&p};
    return hipLaunchKernel((const void*)&stream_kernel<kTokens, kSwiglu>, dim3((unsigned)groups),
                           dim3(Shape::kWaves * kWave), args, shared, stream);
}

// ----------------------------------------------------- many rows per expert
//
// A workgroup of eight wavefronts computes 256 weight rows x 64 * kMt tokens.
// Both operands go through LDS in stages of one 128-channel block, loaded
// straight into it (no registers), two stages deep: while one is computed the
// next is on its way. Wavefront (h, q) takes weight rows [128 h, 128 h + 128)
// (for the SwiGLU product h = 0 are gate rows and h = 1 the up rows of the same
// channels) and the q-th quarter of the tokens: the weights' scale is then one
// number per wavefront and block. The sums stay in registers: fp32 updates
// need them among the 256 that vector instructions reach, which is what
// bounds a wavefront's tile to 128 x 64.
//
// A stage's row is 128 bytes, eight 16-byte chunks; chunk c of row r lies at
// place c ^ (r % 8), so that the 16 rows a read instruction touches at one
// chunk spread over the banks. Loads into LDS fill it in lane order, so the
// permutation is applied to the addresses they read from.
template <int kMt>
struct TileShape {
    static constexpr int kWaves = 8;
    static constexpr int kTokens = 64 * kMt;
    static constexpr int kWeightBytes = 256 * 128;
    static constexpr int kStageBytes = kWeightBytes + kTokens * 128;
    static constexpr int kScaleBlocks = 8;  // blocks whose x scales are staged at a time
    static constexpr int kScaleFloats = kScaleBlocks * kTokens;
    static constexpr int kLdsBytes = 2 * kStageBytes + 2 * (kScaleFloats + 2 * kScaleBlocks) * 4;
};

typedef __attribute__((address_space(3))) void lds_void;

// Loads eight rows of a stage: 1 KB in lane order at dst. Lane offsets past
// the descriptor's range read as zeros.
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t src, uint8_t* dst, int lane_offset, int k) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)dst, 16, lane_offset, k, 0, 0);
}

__device__ __forceinline__ i32x8 read_fragment(const uint8_t* at, int lo, int hi) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(at + lo);
    const u32x4 b = *reinterpret_cast<const u32x4*>(at + hi);
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

template <int kMt, bool kSwiglu>
__global__ void __launch_bounds__(TileShape<kMt>::kWaves * kWave, 2) tile_kernel(ProductParams p) {
    using Shape = TileShape<kMt>;
    extern __shared__ __align__(16) uint8_t smem[];
    float* const scales = reinterpret_cast<float*>(smem + 2 * Shape::kStageBytes);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int half = wave & 1, quarter = wave >> 1;
    const int col = lane & 15, quad = lane >> 4;
    const int64_t total = (int64_t)count_row_tiles<Shape::kTokens>(p) * p.n_tiles;
    // Reads: this lane's two chunks within the first 16 rows of a fragment.
    const int read_lo = col * 128 + ((quad ^ (col & 7)) << 4);
    const int read_hi = read_lo ^ 64;
    // Loads: this lane's chunk within 8 rows.
    const int load_row = lane >> 3;
    const int load_k = ((lane & 7) ^ load_row) << 4;
    for (int64_t i = blockIdx.x; i < (total + kXcds - 1) / kXcds * kXcds; i += gridDim.x) {
        const int64_t item = xcd_item(i, total);
        if (item >= total) continue;
        const Tile t = find_tile<Shape::kTokens>(p, item);
        // Weight rows of this wavefront's half; the other operand's loads are
        // split over the wavefronts the same way: 32 weight rows and 8 kMt
        // token rows each.
        const int n_half = kSwiglu ? t.n * 128 + half * (p.N / 2) : t.n * 256 + half * 128;
        int n_rows = p.N - n_half;
        n_rows = __builtin_amdgcn_readfirstlane(n_rows < 0 ? 0 : (n_rows > 128 ? 128 : n_rows));
        const int64_t w_row = n_rows > 0 ? (int64_t)t.expert * p.N + n_half : 0;
        const auto w_src = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + w_row * p.K), 0, n_rows * p.K, kBufferWord3);
        const auto x_src =
            __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + (int64_t)t.row * p.K), 0, t.rows * p.K, kBufferWord3);
        const int w_first = quarter * 32, x_first = wave * 8 * kMt;
        // Rows past the last one load that one again; their sums are dropped.
        int w_offset[4], x_offset[kMt];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = w_first + j * 8 + load_row;
            w_offset[j] = (r < n_rows ? r : (n_rows > 0 ? n_rows - 1 : 0)) * p.K + load_k;
        }
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
            const int r = x_first + j * 8 + load_row;
            x_offset[j] = (r < t.rows ? r : t.rows - 1) * p.K + load_k;
        }
        auto load_stage = [&](int kb) {
            uint8_t* const stage = smem + (kb & 1) * Shape::kStageBytes;
            // Chunks past K (a multiple of 16) are sent out of range.
            const int k = kb * 128;
            const int out = k + load_k < p.K ? 0 : INT32_MIN;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_rows(w_src, stage + (half * 128 + w_first + j * 8) * 128, w_offset[j] | out, k);
#pragma unroll
            for (int j = 0; j < kMt; ++j)
                load_rows(x_src, stage + Shape::kWeightBytes + (x_first + j * 8) * 128, x_offset[j] | out, k);
        };
        // Scales, eight blocks at a time: a thread carries kMt blocks of one
        // token's, the first 16 threads one block of a half's weights. (Past
        // the last block the last one is loaded again and not used.)
        constexpr int kS = Shape::kScaleBlocks;
        const int s_token = threadIdx.x / kS * kMt + (threadIdx.x % kS) / (kS / kMt);
        const int s_block = (threadIdx.x % (kS / kMt)) * kMt;
        const int w_half = kSwiglu ? t.n * 128 + ((threadIdx.x / kS) & 1) * (p.N / 2) : t.n * 256 + ((threadIdx.x / kS) & 1) * 128;
        int w_block = w_half >> 7;
        w_block = w_block < p.n_blocks ? w_block : p.n_blocks - 1;
        const float* const s_src =
            p.x_sf + (int64_t)(t.row + (s_token < t.rows ? s_token : t.rows - 1)) * p.k_blocks;
        const float* const ws_src = p.w_sf + ((int64_t)t.expert * p.n_blocks + w_block) * p.k_blocks;
        float s_next[kMt], ws_next;
        auto load_scales = [&](int chunk) {
#pragma unroll
            for (int j = 0; j < kMt; ++j) {
                const int kb = chunk * kS + s_block + j;
                s_next[j] = s_src[kb < p.k_blocks ? kb : p.k_blocks - 1];
            }
            const int kb = chunk * kS + (int)(threadIdx.x % kS);
            ws_next = ws_src[kb < p.k_blocks ? kb : p.k_blocks - 1];
        };
        auto store_scales = [&](int chunk) {
            float* const dst = scales + (chunk & 1) * (Shape::kScaleFloats + 2 * kS);
#pragma unroll
            for (int j = 0; j < kMt; ++j) dst[(s_block + j) * Shape::kTokens + s_token] = s_next[j];
            if (threadIdx.x < 2 * kS) dst[Shape::kScaleFloats + threadIdx.x] = ws_next;
        };

        f32x4 acc[8][kMt];
#pragma unroll
        for (int f = 0; f < 8; ++f)
#pragma unroll
            for (int m = 0; m < kMt; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        load_stage(0);
        load_scales(0);
        store_scales(0);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
            // This wavefront's part of the stage has arrived; past the
            // barrier everybody's has, and the other stage is free.
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            __syncthreads();
            // The next blocks' scales are loaded at the first block of eight
            // and stored at the second, when nobody reads their place.
            const int chunk = kb / kS, in_chunk = kb % kS;
            if (in_chunk == 1) store_scales(chunk + 1);
            if (in_chunk == 0) load_scales(chunk + 1);
            if (kb + 1 < p.k_blocks) load_stage(kb + 1);
            const uint8_t* const stage = smem + (kb & 1) * Shape::kStageBytes;
            const uint8_t* const w_at = stage + half * 128 * 128;
            const uint8_t* const x_at = stage + Shape::kWeightBytes + quarter * 16 * kMt * 128;
            const float* const s_chunk = scales + (chunk & 1) * (Shape::kScaleFloats + 2 * kS);
            const float* const s_at = s_chunk + in_chunk * Shape::kTokens + quarter * 16 * kMt + col;
            const float sw = s_chunk[Shape::kScaleFloats + half * kS + in_chunk];
            i32x8 b[kMt];
            float s[kMt];
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
                b[m] = read_fragment(x_at + m * 16 * 128, read_lo, read_hi);
                s[m] = s_at[m * 16] * sw;
            }
            f32x4 y[kMt];
            i32x8 a = read_fragment(w_at, read_lo, read_hi);
#pragma unroll
            for (int f = 0; f < 9; ++f) {
                // Rows f are multiplied while rows f + 1 are read and the
                // products of rows f - 1 added. (The barriers to scheduling
                // keep the steps apart: moved together, their operands no
                // longer fit the registers.)
                i32x8 next = a;
                if (f < 7) next = read_fragment(w_at + (f + 1) * 16 * 128, read_lo, read_hi);
#pragma unroll
                for (int m = 0; m < kMt; ++m) {
                    const f32x4 last = y[m];
                    if (f < 8) y[m] = mfma_block(a, b[m]);
                    if (f > 0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[f - 1][m][q] = __builtin_fmaf(s[m], last[q], acc[f - 1][m][q]);
                    }
                }
                a = next;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (!kSwiglu) {
            uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
                const int r = (quarter * kMt + m) * 16 + col;
                if (r < t.rows) {
#pragma unroll
                    for (int f = 0; f < 8; ++f) {
                        const int n = f * 16 + quad * 4;
                        if (n < n_rows) {  // N is a multiple of 8
                            uint2 o;
                            o.x = pack_bf16(acc[f][m][0], acc[f][m][1]);
                            o.y = pack_bf16(acc[f][m][2], acc[f][m][3]);
                            *reinterpret_cast<uint2*>(out + (int64_t)(t.row + r) * p.N + n_half + n) = o;
                        }
                    }
                }
            }
        } else {
            // The up wavefronts hand their sums over through LDS, in the
            // order of their registers.
            __syncthreads();
            f32x4* const swap = reinterpret_cast<f32x4*>(smem) + quarter * 8 * kMt * kWave;
            if (half == 1) {
#pragma unroll
                for (int f = 0; f < 8; ++f)
#pragma unroll
                    for (int m = 0; m < kMt; ++m) swap[(f * kMt + m) * kWave + lane] = acc[f][m];
            }
            __syncthreads();
            if (half == 0) {
                const int I = p.N / 2;
#pragma unroll
                for (int m = 0; m < kMt; ++m) {
                    uint32_t top = __float_as_uint(kAmaxFloor);
#pragma unroll
                    for (int f = 0; f < 8; ++f) {
                        const f32x4 u = swap[(f * kMt + m) * kWave + lane];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float g = acc[f][m][q];
                            const float a = g * sigmoid(g) * u[q];
                            acc[f][m][q] = a;
                            const uint32_t mag = __float_as_uint(a) & 0x7fffffffu;
                            top = top > mag ? top : mag;
                        }
                    }
                    // A token's 128 channels are in the four lanes col + 16 i.
                    uint32_t other = __shfl_xor(top, 16);
                    top = top > other ? top : other;
                    other = __shfl_xor(top, 32);
                    top = top > other ? top : other;
                    const float amax = __uint_as_float(top);
                    const float scale = kFp8Max / amax;
                    const int r = (quarter * kMt + m) * 16 + col;
                    if (r < t.rows) {
                        uint8_t* dst = static_cast<uint8_t*>(p.out) + (int64_t)(t.row + r) * I + t.n * 128 + quad * 4;
#pragma unroll
                        for (int f = 0; f < 8; ++f)
                            *reinterpret_cast<uint32_t*>(dst + f * 16) =
                                pack_fp8(acc[f][m][0] * scale, acc[f][m][1] * scale, acc[f][m][2] * scale,
                                         acc[f][m][3] * scale);
                        if (quad == 0) p.out_sf[(int64_t)(t.row + r) * (I / 128) + t.n] = amax / kFp8Max;
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <int kMt, bool kSwiglu>
hipError_t launch_tile(ProductParams p, int64_t max_rows, hipStream_t stream) {
    using Shape = TileShape<kMt>;
    p.n_tiles = kSwiglu ? p.N / 256 : (p.N + 255) / 256;
    const int64_t row_tiles =
        max_rows / Shape::kTokens + (max_rows < p.num_experts ? max_rows : p.num_experts);
    int64_t groups = (row_tiles * p.n_tiles + kXcds - 1) / kXcds * kXcds;
    if (groups > 65536) groups = 65536;
    if (groups < kXcds) groups = kXcds;
    void* args[] = {&p};
    return hipLaunchKernel((const void*)&tile_kernel<kMt, kSwiglu>, dim3((unsigned)groups),
                           dim3(Shape::kWaves * kWave), args, Shape::kLdsBytes, stream);
}

template <bool kSwiglu>
hipError_t launch(const ProductParams& p, int64_t max_rows, hipStream_t stream) {
    const int64_t mean = max_rows / p.num_experts;
    if (mean <= 16) return launch_stream<1, kSwiglu>(p, max_rows, stream);
    if (mean <= 32) return launch_stream<2, kSwiglu>(p, max_rows, stream);
    if (mean <= 64) return launch_tile<1, kSwiglu>(p, max_rows, stream);
    if (mean <= 192) return launch_tile<2, kSwiglu>(p, max_rows, stream);
    return launch_tile<4, kSwiglu>(p, max_rows, stream);
}

}  // namespace

hipError_t launch_expert_product(const dispatch_expert_problem_t& prob, const int32_t* expert_psum,
                                 const int32_t* expert_count, const void* x, const float* x_sf, const void* w,
                                 const float* w_sf, void* out, float* out_sf, hipStream_t stream) {
    if (prob.expert_rows == 0) return hipSuccess;
    ProductParams p{};
    p.psum = expert_psum;
    p.count = expert_count;
    p.x = static_cast<const uint8_t*>(x);
    p.x_sf = x_sf;
    p.w = static_cast<const uint8_t*>(w);
    p.w_sf = w_sf;
    p.out = out;
    p.out_sf = out_sf;
    p.expert_rows = prob.expert_rows;
    p.num_experts = prob.num_experts;
    p.K = (int32_t)prob.in_features;
    p.N = (int32_t)prob.out_features;
    p.k_blocks = (p.K + 127) / 128;
    p.n_blocks = (p.N + 127) / 128;
    const int64_t max_rows = prob.max_routed_rows < prob.expert_rows ? prob.max_routed_rows : prob.expert_rows;
    return out_sf != nullptr ? launch<true>(p, max_rows, stream) : launch<false>(p, max_rows, stream);
}

}  // namespace moe_dispatch
