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
// operands' own 2^-4. Across blocks all sums are fp32. Few rows before an
// activation, see Wide16, go through v_mfma_f32_16x16x32_bf16: fp32 all along.)
//
// Which channels of the block a lane's 32 bytes stand for does not matter as
// long as both operands agree (the sum runs over all of them): lane group
// g = lane / 16 takes the 16-byte chunks g and g + 4, so that one load
// instruction covers 64 consecutive bytes of 16 rows.
//
// Measured, 32 experts: 512 rows, 2048 -> 7168 channels, 90 us, bound by the
// weights' bytes (5.3 TB/s); 32768 rows, 7168 -> 2048, 532 us, bound by the matrix
// instructions and their operands from LDS (1.81 PFLOP/s; the library's 8192^3
// fp8 product, with one scale for all, reaches 2.6 to 2.7).
#include <type_traits>

#include "dispatch_common.hpp"
#include "dispatch_device.hpp"
#include "dispatch_expert_plan.hpp"
#include "dispatch_experts.hpp"
#include "dispatch_math.hpp"

namespace moe_dispatch {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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
    int32_t parts;      // workgroups that share a tile's K
    int32_t slots;      // sums of them that the workspace holds
    f32x4* sums;        // [slots][one workgroup's sums]
    uint32_t* tickets;  // one per tile, zero between calls
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

// Row tiles of kRows rows. Lane l looks at experts l, l + 64, ...; what it
// found of the first 64 stays in registers, so that with at most that many
// experts a workgroup reads their counts once.
template <int kRows>
struct RowTiles {
    int first, rows, tiles, upto;  // lane's expert of the first 64: first row, rows, tiles, tiles up to and with it
    int total;                     // over all experts

    __device__ __forceinline__ explicit RowTiles(const ProductParams& p) {
        const int lane = threadIdx.x & (kWave - 1);
        look(p, lane);
        int more = 0;
        for (int e = lane + kWave; e < p.num_experts; e += kWave) more += (live_rows(p, e) + kRows - 1) / kRows;
        upto = wave_scan(tiles);
        total = __builtin_amdgcn_readlane(upto, kWave - 1);
        if (p.num_experts > kWave) total += __builtin_amdgcn_readlane(wave_scan(more), kWave - 1);
    }
    __device__ __forceinline__ void look(const ProductParams& p, int e) {
        rows = e < p.num_experts ? live_rows(p, e) : 0;
        first = rows > 0 ? p.psum[e] : 0;
        tiles = (rows + kRows - 1) / kRows;
    }
};

// Tile `item` in the order expert, tile of the width, row tile: the row tiles
// that read the same weights follow each other. Every wavefront finds it for
// itself.
template <int kRows>
__device__ __forceinline__ Tile find_tile(const ProductParams& p, RowTiles<kRows> at, int64_t item) {
    const int lane = threadIdx.x & (kWave - 1);
    const int target = (int)item / p.n_tiles;  // its row tile if each were taken whole (the same expert)
    Tile t{};
    for (int base = 0; base < p.num_experts; base += kWave) {
        if (base > 0) {
            const int before = __builtin_amdgcn_readlane(at.upto, kWave - 1);
            at.look(p, base + lane);
            at.upto = before + wave_scan(at.tiles);
        }
        const uint64_t past = __ballot(at.upto > target);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            const int mine = __builtin_amdgcn_readlane(at.tiles, l);
            const int first = __builtin_amdgcn_readlane(at.upto, l) - mine;
            const int live = __builtin_amdgcn_readlane(at.rows, l);
            const int local = (int)item - first * p.n_tiles;
            // (All uniform; said so, they stay in scalar registers.)
            t.expert = __builtin_amdgcn_readfirstlane(base + l);
            t.n = __builtin_amdgcn_readfirstlane(local / mine);
            const int m = local - t.n * mine;
            t.row = __builtin_amdgcn_readlane(at.first, l) + m * kRows;
            t.rows = __builtin_amdgcn_readfirstlane(live - m * kRows < kRows ? live - m * kRows : kRows);
            return t;
        }
    }
    return t;  // not reached for item < row tiles * n_tiles: rows = 0
}

// Workgroup b's i-th item: the items are cut into eight runs, one per XCD, so
// that tiles sharing weights or rows share an L2.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int64_t total) {
    const int64_t run = (total + kXcds - 1) / kXcds;
    return (b % kXcds) * run + b / kXcds;
}

// Eight wavefronts compute 256 weight rows x kTokens tokens. Both operands go
// through LDS in stages of one 128-channel block, loaded straight into it (no
// registers in between), a ring of them deep: while one is computed the next are
// on their way. The wavefronts are kRowWaves x kTokenWaves over the tile.
//
// Many tokens: the fp32 sums fill the registers (vector instructions reach 256
// of them, so a wavefront's tile is at most 128 x 64). Measured with parts of
// the loop taken out (32768 rows, 7168 -> 2048 channels, 531 us): without the
// loads 390 us, with loads that always hit L2 500; a third stage of weights
// (192 tokens) changed nothing. The matrix instructions alone are 250 us.
//
// Few tokens: the product reads weights and little else, and what counts is
// how many bytes are in flight: three stages of four, 96 KB per CU. (A kernel
// that loaded the weights straight into the matrix operands, 16 rows x 64 bytes
// per instruction, took 165 us for 512 rows x 32 experts x 7168 x 2048, this
// one 91.) With fewer tiles than CUs a tile's K is shared by `parts`
// workgroups: each leaves its sums in the workspace and takes a ticket; the
// last one adds them all, in order, and goes on alone.
//
// For the SwiGLU product a tile is 128 gate rows and the 128 up rows of the
// same channels: the first half of the row wavefronts takes the gate rows.
//
// A stage's row is 128 bytes, eight 16-byte chunks; chunk c of row r lies at
// place c ^ (r % 8), so that the 16 rows a read instruction touches at one
// chunk spread over the banks. Loads into LDS fill it in lane order, so the
// permutation is applied to the addresses they read from.
template <int kTokens_, int kRowWaves_, int kStages_, bool kWide_ = false>
struct TileShape {
    static constexpr bool kWide = kWide_;  // operands widened to bf16, the sums of a block in fp32
    static constexpr int kWaves = 8;
    static constexpr int kTokens = kTokens_;
    static constexpr int kStages = kStages_;
    static constexpr int kRowWaves = kRowWaves_;
    static constexpr int kTokenWaves = kWaves / kRowWaves;
    static constexpr int kRows = 256 / kRowWaves;                   // weight rows of a wavefront
    static constexpr int kF = kRows / 16;                           // fragments of them
    static constexpr int kM = kTokens / 16 / kTokenWaves;           // fragments of its tokens
    static constexpr int kWBytes = 256 * 128;      // of a stage
    static constexpr int kXBytes = kTokens * 128;
    // Loads of a wavefront per stage: 32 weight rows, its eighth of the token
    // rows (8 per instruction; fewer use part of the lanes).
    static constexpr int kXLoads = kTokens >= 64 ? kTokens / 64 : 1;
    static constexpr int kXRows = kTokens / kWaves / kXLoads;       // rows of such a load
    static constexpr int kWLoads = 4;
    // Loads of a wavefront that may be outstanding when a block starts: all
    // that were begun after that block's.
    static constexpr int kAhead = (kStages - 2) * (kWLoads + kXLoads);
    static constexpr int kScaleBlocks = 8;                          // blocks whose scales are staged at a time
    static constexpr int kScaleFloats = kScaleBlocks * kTokens;
    static constexpr int kChunkFloats = kScaleFloats + 2 * kScaleBlocks;
    static constexpr int kRingBytes = kStages * (kWBytes + kXBytes);
    static constexpr int kLdsBytes = kRingBytes + 2 * kChunkFloats * 4;
    static constexpr int kSumFloats = 256 * kTokens;                // a tile's sums
    // SwiGLU: a wavefront with all 128 channels of a half hands over through
    // registers, smaller ones through rows of sums in LDS.
    static constexpr int kSumRow = 256 + 4;
    // Rows of the bf16 output in LDS, 16 bytes longer than their 256 channels.
    static constexpr int kOutRow = 512 + 16;
    static_assert(kTokens * kOutRow <= kLdsBytes, "rows of output");
    static constexpr bool kWholeBlock = kRows == 128;
    static_assert(kWholeBlock || kTokens * kSumRow * 4 <= kRingBytes, "rows of sums");
    static_assert(kLdsBytes <= kLdsPerCu, "LDS");
};

// A raw buffer descriptor in scalar registers.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 descriptor(const void* base, int bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    return i32x4{__builtin_amdgcn_readfirstlane((int)at), __builtin_amdgcn_readfirstlane((int)(at >> 32) & 0xffff),
                 __builtin_amdgcn_readfirstlane(bytes), kBufferWord3};
}

__device__ __forceinline__ int lds_address(const void* at) {
    return (int)(uintptr_t)(const __attribute__((address_space(3))) void*)at;
}

// Loads 16 (4) bytes per lane, in lane order, to LDS address dst. Lane offsets past
// the descriptor's range read as zeros. Written out, as the compiler does not
// see that the stage being loaded is not the one being read and puts a wait
// for the load before the reads. It returns nothing (and m0 is the compiler's
// scratch register for such instructions, set before each use); wait_loads()
// stands before the barrier that opens the stage.
__device__ __forceinline__ void load_to_lds(const i32x4& src, int dst, int lane_offset, int k) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(lane_offset), "s"(src), "s"(k), "s"(dst)
                 : "memory");
}

__device__ __forceinline__ void load_dword_to_lds(const i32x4& src, int dst, int lane_offset, int k) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 :
                 : "v"(lane_offset), "s"(src), "s"(k), "s"(dst)
                 : "memory");
}

// Waits until at most kLeft of this wavefront's loads are outstanding (they
// arrive in order; loads other than the stages' only make it wait longer).
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
    static_assert(kLeft < 64, "six bits");
    __builtin_amdgcn_s_waitcnt((kLeft & 15) | (7 << 4) | (15 << 8) | ((kLeft >> 4) << 14));
}

// A barrier that does not wait for loads into LDS.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A lane's 32 channels of a fragment's row as they are, or as bf16, which has
// every e4m3 value.
struct WideFragment {
    bf16x8 part[4];
};

template <bool kWide>
__device__ __forceinline__ auto read_fragment(const uint8_t* at, int lo, int hi) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(at + lo);
    const u32x4 b = *reinterpret_cast<const u32x4*>(at + hi);
    const i32x8 v = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
    if constexpr (kWide) {
        WideFragment wide;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 c0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i], 1.f, false);
            const bf16x2 c1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i], 1.f, true);
            const bf16x2 c2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i + 1], 1.f, false);
            const bf16x2 c3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i + 1], 1.f, true);
            wide.part[i] = bf16x8{c0[0], c0[1], c1[0], c1[1], c2[0], c2[1], c3[0], c3[1]};
        }
        return wide;
    } else {
        return v;
    }
}

__device__ __forceinline__ f32x4 mfma_block(const i32x8& a, const i32x8& b) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_block(const WideFragment& a, const WideFragment& b) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[i], b.part[i], sum, 0, 0, 0);
    return sum;
}

template <class Shape, bool kSwiglu>
__global__ void __launch_bounds__(Shape::kWaves * kWave, 2) product_kernel(ProductParams p) {
    constexpr int kF = Shape::kF, kM = Shape::kM, kS = Shape::kScaleBlocks;
    extern __shared__ __align__(16) uint8_t smem[];
    float* const scales = reinterpret_cast<float*>(smem + Shape::kRingBytes);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row_wave = wave % Shape::kRowWaves, token_wave = wave / Shape::kRowWaves;
    const int col = lane & 15, quad = lane >> 4;
    RowTiles<Shape::kTokens> row_tiles(p);
    const int64_t tiles = (int64_t)row_tiles.total * p.n_tiles;
    const int parts = tiles * p.parts <= p.slots ? p.parts : 1;  // more rows than announced: no room to share
    const int64_t total = tiles * parts;
    // Reads: this lane's two chunks within the first 16 rows of a fragment.
    const int read_lo = col * 128 + ((quad ^ (col & 7)) << 4);
    const int read_hi = read_lo ^ 64;
    // Loads: this lane's row and chunk.
    const int load_row = lane >> 3;
    const int load_k = ((lane & 7) ^ load_row) << 4;
    const int x_first = wave * (Shape::kTokens / Shape::kWaves);
    const int x_load_k = ((lane & 7) ^ ((x_first + load_row) & 7)) << 4;
    // (The row tiles are looked up again for each further item: kept, they
    // would cost the loop over the blocks registers.)
    for (int64_t i = blockIdx.x; i < (total + kXcds - 1) / kXcds * kXcds;
         i += gridDim.x, row_tiles = RowTiles<Shape::kTokens>(p)) {
        const int64_t item = xcd_item(i, total);
        if (item >= total) continue;
        const int tile = (int)item / parts, part = (int)item - tile * parts;
        const Tile t = find_tile(p, row_tiles, tile);
        // The part's blocks of K.
        const int k_first = (int)((int64_t)p.k_blocks * part / parts);
        const int blocks = (int)((int64_t)p.k_blocks * (part + 1) / parts) - k_first;
        // Loads of weights: wavefronts 0 to 3 the first 128 rows of the tile,
        // 4 to 7 the second.
        const int load_half = wave >> 2, w_first = (wave & 3) * 32;
        auto half_row = [&](int half) { return kSwiglu ? t.n * 128 + half * (p.N / 2) : t.n * 256 + half * 128; };
        int n_rows = p.N - half_row(load_half);
        n_rows = __builtin_amdgcn_readfirstlane(n_rows < 0 ? 0 : (n_rows > 128 ? 128 : n_rows));
        const int64_t w_row = n_rows > 0 ? (int64_t)t.expert * p.N + half_row(load_half) : 0;
        const i32x4 w_src = descriptor(p.w + w_row * p.K, n_rows * p.K);
        const i32x4 x_src = descriptor(p.x + (int64_t)t.row * p.K, t.rows * p.K);
        // Rows past the last one are out of the descriptors' range.
        const int w_lane = (w_first + load_row) * p.K + load_k;
        const int x_lane = (x_first + load_row) * p.K + x_load_k;
        // Loads of block b's weights and tokens; past the last block, and for
        // chunks past K (a multiple of 16), out of range.
        auto load_w = [&](int b) {
            const int dst = lds_address(smem) + b % Shape::kStages * Shape::kWBytes + (load_half * 128 + w_first) * 128;
            const int k = (k_first + b) * 128;
            const int out = b < blocks && k + load_k < p.K ? 0 : INT32_MIN;
#pragma unroll
            for (int j = 0; j < Shape::kWLoads; ++j)
                load_to_lds(w_src, dst + j * 8 * 128, (w_lane + j * 8 * p.K) | out, k);
        };
        auto load_x = [&](int b) {
            const int dst = lds_address(smem) + Shape::kStages * Shape::kWBytes + b % Shape::kStages * Shape::kXBytes +
                            x_first * 128;
            const int k = (k_first + b) * 128;
            const int out = b < blocks && k + x_load_k < p.K ? 0 : INT32_MIN;
            if (Shape::kXRows == 8 || load_row < Shape::kXRows) {
#pragma unroll
                for (int j = 0; j < Shape::kXLoads; ++j)
                    load_to_lds(x_src, dst + j * 8 * 128, (x_lane + j * 8 * p.K) | out, k);
            }
        };
        // Scales, eight blocks at a time, one wavefront for each: a lane per
        // token, and the first wavefront's 16 lanes for the weights' halves.
        // (Past the last block the last one is loaded again and not used.)
        constexpr int kSLoads = (Shape::kTokens + kWave - 1) / kWave;
        const i32x4 xs_src = descriptor(p.x_sf + (int64_t)t.row * p.k_blocks, t.rows * p.k_blocks * 4);
        const int64_t ws_first = (int64_t)t.expert * p.n_blocks;
        const i32x4 ws_src = descriptor(p.w_sf + ws_first * p.k_blocks, p.n_blocks * p.k_blocks * 4);
        int w_block = half_row((lane / kS) & 1) >> 7;
        w_block = w_block < p.n_blocks ? w_block : p.n_blocks - 1;
        auto load_scales = [&](int chunk) {
            const int dst = lds_address(scales) + (chunk & 1) * Shape::kChunkFloats * 4;
            int b = chunk * kS + wave;
            b = k_first + (b < blocks ? b : blocks - 1);
#pragma unroll
            for (int j = 0; j < kSLoads; ++j) {
                const int r = j * kWave + lane;
                if (Shape::kTokens >= kWave || lane < Shape::kTokens)
                    load_dword_to_lds(xs_src, dst + (wave * Shape::kTokens + j * kWave) * 4,
                                      (r < t.rows ? r : t.rows - 1) * p.k_blocks * 4, b * 4);
            }
            if (wave == 0 && lane < 2 * kS) {
                int l = chunk * kS + (lane % kS);
                l = k_first + (l < blocks ? l : blocks - 1);
                load_dword_to_lds(ws_src, dst + Shape::kScaleFloats * 4, (w_block * p.k_blocks + l) * 4, 0);
            }
        };

        f32x4 acc[kF][kM];
#pragma unroll
        for (int f = 0; f < kF; ++f)
#pragma unroll
            for (int m = 0; m < kM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        load_scales(0);
#pragma unroll
        for (int b = 0; b < Shape::kStages - 1; ++b) {
            load_x(b);
            load_w(b);
        }
        // The blocks, for a tile whose rows fill kLive of each wavefront's
        // fragments of tokens.
        auto run = [&](auto live_fragments) {
        constexpr int kLive = decltype(live_fragments)::value;
        for (int b = 0; b < blocks; ++b) {
            // This wavefront's part of the block has arrived; past the
            // barrier everybody's has, and the block before is done with.
            wait_loads<Shape::kAhead>();
            lds_barrier();
            const int chunk = b / kS, in_chunk = b % kS;
            if (in_chunk == 0) load_scales(chunk + 1);  // to where nobody reads any more
            // (All at once: one load a step below arrived later and took
            // 602 us where this takes 560, 32768 x 7168 x 2048.)
            load_x(b + Shape::kStages - 1);
            load_w(b + Shape::kStages - 1);
            const uint8_t* const w_at = smem + b % Shape::kStages * Shape::kWBytes + row_wave * Shape::kRows * 128;
            const uint8_t* const x_at = smem + Shape::kStages * Shape::kWBytes + b % Shape::kStages * Shape::kXBytes +
                                        token_wave * 16 * 128;
            const float* const s_chunk = scales + (chunk & 1) * Shape::kChunkFloats;
            const float* const s_at = s_chunk + in_chunk * Shape::kTokens + token_wave * 16 + col;
            const float sw = s_chunk[Shape::kScaleFloats + row_wave / (Shape::kRowWaves / 2) * kS + in_chunk];
            using Fragment = std::conditional_t<Shape::kWide, WideFragment, i32x8>;
            Fragment x[kLive];
            float s[kLive];
#pragma unroll
            for (int m = 0; m < kLive; ++m) {
                x[m] = read_fragment<Shape::kWide>(x_at + m * Shape::kTokenWaves * 16 * 128, read_lo, read_hi);
                // (Below 2^-126 the scales' product is rounded to multiples
                // of 2^-149; a block's sum is under 2^25, so that its part of
                // the result moves by less than 2^-125, an fp32 underflow.)
                s[m] = s_at[m * Shape::kTokenWaves * 16] * sw;
            }
            f32x4 y[kLive];
            Fragment w = read_fragment<Shape::kWide>(w_at, read_lo, read_hi);
#pragma unroll
            for (int f = 0; f <= kF; ++f) {
                // Rows f are multiplied while rows f + 1 are read and the
                // products of rows f - 1 added, four additions behind each
                // matrix instruction, whose 32 cycles they fit into. (Left to
                // the compiler, additions and matrix instructions came in
                // separate runs, 5 % slower; and the steps moved together
                // need more registers than there are.)
                Fragment next = w;
                if (f + 1 < kF) next = read_fragment<Shape::kWide>(w_at + (f + 1) * 16 * 128, read_lo, read_hi);
#pragma unroll
                for (int m = 0; m < kLive; ++m) {
                    const f32x4 last = y[m];
                    if (f < kF) y[m] = mfma_block(w, x[m]);
                    if (f > 0) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[f - 1][m][q] = __builtin_fmaf(s[m], last[q], acc[f - 1][m][q]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                w = next;
            }
        }
        };
        // Fragments of tokens go to the token wavefronts in turn, so that a
        // tile's last rows spread over all of them.
        const int live = (t.rows + 16 * Shape::kTokenWaves - 1) / (16 * Shape::kTokenWaves);
        if (live == 1)
            run(std::integral_constant<int, 1>());
        else if (live == 2)
            run(std::integral_constant<int, (kM < 2 ? kM : 2)>());
        else if (live == 3)
            run(std::integral_constant<int, (kM < 3 ? kM : 3)>());
        else
            run(std::integral_constant<int, kM>());
        wait_loads<0>();  // (those past the last block write zeros to the ring)
        if (parts > 1) {
            // The sums go past the caches that XCDs do not share (sc1 on
            // stores and loads), so that no cache has to be written back or
            // invalidated for them: with release and acquire fences instead,
            // one token's 8 x 4096 x 7168 product took 78 us, unshared 54.
            constexpr int kSums = Shape::kSumFloats / 4;
            const int at = (wave * (kF * kM * kWave) + lane) * 16;
            const auto slot = [&](int q) {
                return __builtin_amdgcn_make_buffer_rsrc((void*)(p.sums + (int64_t)(item - part + q) * kSums), 0,
                                                         kSums * 16, kBufferWord3);
            };
            const auto mine = slot(part);
#pragma unroll
            for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int m = 0; m < kM; ++m)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[f][m]), mine,
                                                           at + (f * kM + m) * kWave * 16, 0, kSc1Policy);
            wait_loads<0>();  // and stores
            uint32_t* const last = reinterpret_cast<uint32_t*>(scales);
            lds_barrier();
            if (threadIdx.x == 0) {
                const uint32_t before =
                    __hip_atomic_fetch_add(p.tickets + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                *last = before == (uint32_t)parts - 1;
                if (before == (uint32_t)parts - 1)
                    __hip_atomic_store(p.tickets + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            lds_barrier();
            const bool go_on = *last != 0;
            lds_barrier();
            if (!go_on) continue;
#pragma unroll
            for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int m = 0; m < kM; ++m) acc[f][m] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < parts; ++q) {
                const auto from = slot(q);
#pragma unroll
                for (int f = 0; f < kF; ++f)
#pragma unroll
                    for (int m = 0; m < kM; ++m)
                        acc[f][m] += __builtin_bit_cast(
                            f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at + (f * kM + m) * kWave * 16, 0,
                                                                         kSc1Policy));
            }
        }
        const int first_token = token_wave * 16 + col;
        if constexpr (!kSwiglu) {
            // Through LDS, so that whole rows of 512 bytes leave (4096 x 8192
            // x 1792 in two rounds of tiles: 68 us; stored straight from the
            // registers, 32 bytes of each of 16 rows at a time, 84).
            lds_barrier();
            const int c0 = (row_wave * Shape::kRows + quad * 4) * 2;
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int f = 0; f < kF; ++f) {
                    uint2 o;
                    o.x = pack_bf16(acc[f][m][0], acc[f][m][1]);
                    o.y = pack_bf16(acc[f][m][2], acc[f][m][3]);
                    *reinterpret_cast<uint2*>(smem + (first_token + m * Shape::kTokenWaves * 16) * Shape::kOutRow + c0 +
                                              f * 32) = o;
                }
            lds_barrier();
            uint16_t* const out = static_cast<uint16_t*>(p.out);
            const int n = t.n * 256 + (lane & 31) * 8;
            if (n < p.N) {  // N is a multiple of 8
                for (int r = wave * 2 + (lane >> 5); r < t.rows; r += 2 * Shape::kWaves)
                    *reinterpret_cast<u32x4*>(out + (int64_t)(t.row + r) * p.N + n) =
                        *reinterpret_cast<const u32x4*>(smem + r * Shape::kOutRow + (lane & 31) * 16);
            }
            lds_barrier();  // the ring is free for the next tile
        } else if constexpr (Shape::kWholeBlock) {
            // The up wavefronts hand their sums over through LDS, in the
            // order of their registers.
            const int I = p.N / 2;
            lds_barrier();
            f32x4* const swap = reinterpret_cast<f32x4*>(smem) + token_wave * kF * kM * kWave;
            if (row_wave == 1) {
#pragma unroll
                for (int f = 0; f < kF; ++f)
#pragma unroll
                    for (int m = 0; m < kM; ++m) swap[(f * kM + m) * kWave + lane] = acc[f][m];
            }
            lds_barrier();
            if (row_wave == 0) {
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    uint32_t top = __float_as_uint(kAmaxFloor);
#pragma unroll
                    for (int f = 0; f < kF; ++f) {
                        const f32x4 u = swap[(f * kM + m) * kWave + lane];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float g = acc[f][m][q];
                            const float a = g * fast_sigmoid(g) * u[q];
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
                    const int r = first_token + m * Shape::kTokenWaves * 16;
                    if (r < t.rows) {
                        uint8_t* dst = static_cast<uint8_t*>(p.out) + (int64_t)(t.row + r) * I + t.n * 128 + quad * 4;
#pragma unroll
                        for (int f = 0; f < kF; ++f)
                            *reinterpret_cast<uint32_t*>(dst + f * 16) =
                                pack_fp8(acc[f][m][0] * scale, acc[f][m][1] * scale, acc[f][m][2] * scale,
                                         acc[f][m][3] * scale);
                        if (quad == 0) p.out_sf[(int64_t)(t.row + r) * (I / 128) + t.n] = amax / kFp8Max;
                    }
                }
            }
            lds_barrier();
        } else {
            // [token][256] sums: gate channels, then up channels. A row is
            // 4 floats longer than that, so that the 16 tokens of a store
            // fall into different banks.
            const int I = p.N / 2;
            float* const sums = reinterpret_cast<float*>(smem);
            lds_barrier();
#pragma unroll
            for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int m = 0; m < kM; ++m)
                    *reinterpret_cast<f32x4*>(sums + (first_token + m * Shape::kTokenWaves * 16) * Shape::kSumRow +
                                              row_wave * Shape::kRows + f * 16 + quad * 4) = acc[f][m];
            lds_barrier();
            const int c = (threadIdx.x & 15) * 8;
            for (int token = threadIdx.x / 16; token < t.rows; token += Shape::kWaves * 4) {
                const float* g = sums + token * Shape::kSumRow + c;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = g[q] * (Shape::kWide ? near_sigmoid(g[q]) : fast_sigmoid(g[q])) * g[128 + q];
                uint8_t* dst = static_cast<uint8_t*>(p.out) + (int64_t)(t.row + token) * I + t.n * 128 + c;
                quantize8<false>(v, true, c == 0, dst, p.out_sf + (int64_t)(t.row + token) * (I / 128) + t.n);
            }
            lds_barrier();
        }
    }
}

using Shape16 = TileShape<16, 8, 4>;
using Shape32 = TileShape<32, 8, 4>;
using Shape64 = TileShape<64, 4, 3>;
using Shape128 = TileShape<128, 2, 3>;
using Shape192 = TileShape<192, 2, 2>;
using Shape256 = TileShape<256, 2, 2>;
// Shape16 for the SwiGLU product of rows that fill no more than one tile of it per
// expert (wide_operands): decoding, bound by the weights' bytes or the launch. Its
// result is rounded to 8 bits, where what the fp8 instruction drops turns single
// roundings: a layer of 1 to 30 rows was off from 64 bits by up to 0.0035 (0.0017 in
// the median, and always with the operands widened). 8 rows on 32 experts, 7168 -> 2 x
// 2048 -> 7168 channels, take 60 to 67 us with either; on 8 experts, 2048 -> 2 x 1024
// -> 2048, 19.2 with these and 18.8; 200 rows there, past the rule, 22.7 and 20.1.
// Widened operands in tiles of 32 and 64 tokens cost up to 35 %, and the other
// product's result is rounded to bf16, 30 times what is dropped.
using Wide16 = TileShape<16, 8, 4, true>;

template <class Shape, bool kSwiglu>
hipError_t launch_product(ProductParams p, const ProductSizes& sizes, void* workspace, hipStream_t stream) {
    static_assert(Shape::kSumFloats == kTileChannels * Shape::kTokens, "a tile's sums");
    p.n_tiles = (p.N + kTileChannels - 1) / kTileChannels;
    const ProductPlan plan = plan_product(Shape::kTokens, sizes);
    p.parts = plan.parts;
    p.slots = plan.parts == 1 ? 0 : (int32_t)(plan.tiles * plan.parts);
    p.tickets = static_cast<uint32_t*>(workspace);
    p.sums = workspace == nullptr ? nullptr
                                  : reinterpret_cast<f32x4*>(static_cast<uint8_t*>(workspace) + kTicketBytes);
    int64_t groups = (plan.tiles * plan.parts + kXcds - 1) / kXcds * kXcds;
    if (groups > 65536) groups = 65536;  // larger batches loop
    if (groups < kXcds) groups = kXcds;
    void* args[] = {&p};
    const void* kernel = (const void*)&product_kernel<Shape, kSwiglu>;
    if constexpr (kSwiglu && Shape::kTokens == Wide16::kTokens)
        if (wide_operands(sizes)) kernel = (const void*)&product_kernel<Wide16, kSwiglu>;
    return hipLaunchKernel(kernel, dim3((unsigned)groups), dim3(Shape::kWaves * kWave), args, Shape::kLdsBytes, stream);
}

template <class Shape>
hipError_t launch_product(const ProductParams& p, const ProductSizes& sizes, void* workspace, hipStream_t stream) {
    return p.out_sf != nullptr ? launch_product<Shape, true>(p, sizes, workspace, stream)
                               : launch_product<Shape, false>(p, sizes, workspace, stream);
}

ProductSizes sizes_of(const dispatch_expert_problem_t& p, bool workspace) {
    return {p.max_routed_rows < p.expert_rows ? p.max_routed_rows : p.expert_rows, p.num_experts,
            (int32_t)p.out_features, (int32_t)((p.in_features + 127) / 128), workspace};
}

}  // namespace

size_t expert_workspace_bytes(const dispatch_expert_problem_t& prob) {
    const ProductSizes sizes = sizes_of(prob, true);
    return plan_product(tile_tokens(sizes), sizes).bytes;
}

hipError_t launch_expert_product(const dispatch_expert_problem_t& prob, const int32_t* expert_psum,
                                 const int32_t* expert_count, const void* x, const float* x_sf, const void* w,
                                 const float* w_sf, void* out, float* out_sf, void* workspace,
                                 hipStream_t stream) {
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
    const ProductSizes sizes = sizes_of(prob, workspace != nullptr);
    switch (tile_tokens(sizes)) {
        case 16: return launch_product<Shape16>(p, sizes, workspace, stream);
        case 32: return launch_product<Shape32>(p, sizes, workspace, stream);
        case 64: return launch_product<Shape64>(p, sizes, workspace, stream);
        case 128: return launch_product<Shape128>(p, sizes, workspace, stream);
        case 192: return launch_product<Shape192>(p, sizes, workspace, stream);
        default: return launch_product<Shape256>(p, sizes, workspace, stream);
    }
}

}  // namespace moe_dispatch
