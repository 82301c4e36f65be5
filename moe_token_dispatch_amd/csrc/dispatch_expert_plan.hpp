// How an experts' product is cut, decided on the host from its sizes alone:
// tokens of a tile, workgroups that share a tile's K, the workspace they need.
// Plain C++, so that tests can ask it without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cmath>

namespace moe_dispatch {

constexpr int kProductCus = 256;
constexpr int kTileChannels = 256;  // weight rows of a tile, of every shape
constexpr int kMaxParts = 16;

// Tokens of a tile, one kernel for each.
constexpr int kTileTokens[] = {16, 32, 64, 128, 192, 256};
constexpr int kTileShapes = sizeof(kTileTokens) / sizeof(kTileTokens[0]);

// Tickets at the start of a workspace, as many as any problem shares tiles
// (then there are at most kProductCus), so that one workspace serves several.
constexpr size_t kTicketBytes = kProductCus * sizeof(uint32_t);

// A product's sizes as the plan sees them.
struct ProductSizes {
    int64_t max_rows;     // rows at most, as announced
    int32_t num_experts;
    int32_t N;            // weight rows of an expert
    int32_t k_blocks;     // ceil(K / 128)
    bool workspace;
};

struct ProductPlan {
    int64_t tiles;  // at most
    int parts;      // workgroups per tile
    size_t bytes;   // of workspace: tickets, then sums (0: nothing shared)
};

inline ProductPlan plan_product(int tokens, const ProductSizes& p) {
    ProductPlan s;
    // Row tiles at most: one of each expert that has a row may be partial.
    const int64_t row_tiles = p.max_rows / tokens + (p.max_rows < p.num_experts ? p.max_rows : p.num_experts);
    s.tiles = row_tiles * ((p.N + kTileChannels - 1) / kTileChannels);
    // As many parts as fill the CUs, each left with four blocks of K or more.
    // (Not of tiles of 128 tokens and more: smaller ones were faster in all of 28
    // problems.)
    const int64_t want = kProductCus / (s.tiles < 1 ? 1 : s.tiles);
    const int64_t most = p.workspace && tokens <= 64 ? p.k_blocks / 4 : 1;
    const int64_t parts = want < most ? want : most;
    s.parts = (int)(parts < 1 ? 1 : (parts > kMaxParts ? kMaxParts : parts));
    const size_t sum_bytes = (size_t)kTileChannels * tokens * sizeof(float);
    s.bytes = s.parts == 1 ? 0 : kTicketBytes + (size_t)(s.tiles * s.parts) * sum_bytes;
    return s;
}

// The shape whose tiles take least time by this estimate: rounds of tiles over
// the CUs, each with its blocks of K and what a tile costs beside them
// (beginning, epilogue, its output), and the sums of tiles that share their K.
// The times are measured ones, us, of the full chip. An expert has about half
// a tile more than its rows fill, fewer where its count (give or take its root)
// fits a few tiles. Weights' bytes cost all shapes alike and are left out.
//
// Measured over 28 problems of 1 to 60 experts, 19 to 18847 rows, 272 to 8192 x 336
// to 8192 channels: the choice is within 8 % of the fastest shape each time (a rule
// by the mean of rows alone took up to 3.6 times that). Some of them, us by
// tokens of a tile:
//                                        16    32    64   128   192   256
//   836 rows on 3, 2656 -> 336           13    12    14    27    31    38
//   2000 rows on 8, 1024 -> 1024         21    17    11    14    15    19
//   6175 rows on 45, 1856 -> 1536       143    89    62    55    65    67
//   4096 rows on 8, 1024 -> 4096        128    77    52    44    39    44
//   2562 rows on 6, 1280 -> 5376        115    73    51    36    42    30
// and where the weights' bytes bound it, 32 experts, 2048 -> 7168, at mean 4, 16, 32
// and 64 rows: 16 tokens 87, 103, 140, 217; 32: 90, 93, 107, 147; 64: 89, 92, 96, 124; 128:
// 93, 97, 100, 111.
struct TileTimes {
    double tile, block;
};
constexpr TileTimes tile_times(int tokens) {
    switch (tokens) {
        case 16: return {3.1, 0.60};
        case 32: return {4.7, 0.65};
        case 64: return {5.7, 0.76};
        case 128: return {7.7, 1.12};
        case 192: return {9.9, 1.46};
        default: return {11.0, 1.70};
    }
}

inline double product_time(int tokens, const ProductSizes& p) {
    const ProductPlan plan = plan_product(tokens, p);
    const double experts = p.max_rows < p.num_experts ? (double)p.max_rows : (double)p.num_experts;
    const double mean = p.max_rows / experts, fill = mean / tokens;
    double per_expert = fill + 0.5;
    if (p.num_experts == 1) {
        per_expert = std::ceil(fill);
    } else if (fill < 3) {
        const double spread = std::sqrt(mean) / tokens;
        const double around = (std::ceil(fill - spread) + std::ceil(fill + spread)) / 2;
        per_expert = around < per_expert ? around : per_expert;
        per_expert = per_expert < 1 ? 1 : per_expert;
    }
    const double tiles = per_expert * experts * ((p.N + kTileChannels - 1) / kTileChannels);
    const TileTimes times = tile_times(tokens);
    double us =
        std::ceil(tiles * plan.parts / kProductCus) * (times.tile + times.block * p.k_blocks / plan.parts);
    if (plan.parts > 1) {
        // The last workgroup's reading, and everybody's writing and reading.
        const double kb = plan.parts * (kTileChannels * tokens) * 4e-3;
        us += 2.5 + 0.012 * kb + tiles * kb * 2 / 5.2e3;
    }
    return us;
}

// Tokens of the tiles that a product takes.
inline int tile_tokens(const ProductSizes& p) {
    if (p.max_rows <= 0) return kTileTokens[0];
    int best = kTileTokens[0];
    double least = product_time(best, p);
    for (int i = 1; i < kTileShapes; ++i) {
        const double us = product_time(kTileTokens[i], p);
        if (us < least) best = kTileTokens[i], least = us;
    }
    return best;
}

// Whether a SwiGLU product in tiles of 16 tokens widens its operands: rows that
// fill no more than one tile of each expert.
inline bool wide_operands(const ProductSizes& p) { return p.max_rows <= (int64_t)kTileTokens[0] * p.num_experts; }

}  // namespace moe_dispatch
