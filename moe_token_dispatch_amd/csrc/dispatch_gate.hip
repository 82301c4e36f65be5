// The gate on gfx950: router logits to the routing table and its weights, the
// per-expert counts and the balance loss, and the gradient of the logits.
//
// One wavefront per token, V = ceil(E / 64) experts per lane (rounded up to a
// power of two) in registers: a row is read once, and its scores, sums and
// choice never leave the wavefront. A lane holds pairs of neighbouring
// experts, which arrive as one load. The next token's row is on its way while
// this one's is worked on; it is widened when its turn comes, so that no load
// is waited for early, but before this one's results are stored, so that it
// does not wait for those either (with single loads, widened as they came,
// 4096 tokens of 256 experts with gradients took 21.1 us, with pairs 17.8).
//
// Choice: K rounds of a wave maximum. Selection compares the fp32 values
// themselves (for softmax the logits, whose order the scores share), so ties
// are exact ties and go to the lowest expert. They are compared as unsigned
// integers that order as the values do: an integer maximum takes one
// instruction where a float maximum also has to quiet NaN. A lane orders each
// pair once; a round then looks at the pairs' first keys alone: the lowest
// pair and lane that hold the maximum are the lowest expert that does.
//
// What bounds it: the rounds, 16 vector and about 24 scalar instructions a
// token, 3.3 us each for 65536 tokens of 256 experts. Many tokens with 65 to
// 256 experts therefore take a form of their own (gate_rows_kernel): 65536
// tokens, top-8, fp32, 28 us for 71 MB on the trace, where this one takes 46. The
// gradient's kernel has no rounds and takes 25.6 us for 140 MB (5.5 TB/s, as a
// large copy). Small batches are bound by the launch, 4.1 us for a call of 333
// tokens.
//
// Balance: a wavefront keeps prob_sum of its lanes' experts in registers over
// all its tokens; a workgroup adds its wavefronts in order and leaves one
// partial row; a second kernel adds the partial rows in order. No float goes
// through an atomic, so the sums do not depend on timing (the counts are
// integers and do go through LDS atomics).
#include <utility>

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
    int32_t* expert_count;  // these by a lone workgroup
    float* prob_sum;
    int32_t* live_tokens;
    float* loss;
    float loss_coef;
    int64_t num_tokens;
    int32_t num_experts;
    int32_t num_topk;
    int32_t idx_bytes;
    uint32_t flags;
    float route_scale;
    int32_t num_groups;  // of a choice by groups, these:
    int32_t topk_groups;
    int32_t group_size;   // experts of a group
    int32_t group_lanes;  // lanes that look at one, as a power of two
    bool group_pairs;     // a group goes by the sum of its two largest choices
};

// Wavefronts per workgroup that leave each enough registers for its V
// experts per lane.
template <int V>
constexpr int kGateWaves = V <= 8 ? 16 : (V == 16 ? 8 : 4);

// A lane's V experts are pairs of neighbours, pair j of lane l from expert
// 2 (64 j + l) (with up to 64 experts a lane has one). With an odd number of
// experts the last pair is moved back to end with them, and its first expert,
// which the pair before has, does not count there; nor does a pair that starts
// past the end.
template <int V>
constexpr int kPair = V < 2 ? V : 2;

template <int V>
struct Pair {
    int start, first;  // where it starts, where it is moved to
    __device__ __forceinline__ Pair(int lane, int v, int32_t E) {
        constexpr int R = kPair<V>;
        start = (v / R * kWave + lane) * R;
        // (E > 32 V if V > 1: the first half of the pairs is whole.)
        first = R * kWave * (v / R + 1) <= 32 * V || start < E - R ? start : E - R;
    }
};

// Expert v of the lane, and whether it counts.
template <int V>
__device__ __forceinline__ int expert_of(int lane, int v, int32_t E) {
    return Pair<V>(lane, v, E).first + v % kPair<V>;
}
template <int V>
__device__ __forceinline__ bool counts(int lane, int v, int32_t E) {
    const Pair<V> pair(lane, v, E);
    return pair.first + v % kPair<V> >= pair.start;
}

// A pair as one access, of rows that start wherever their type may (global
// memory takes accesses of any alignment).
typedef uint32_t Halves2 __attribute__((aligned(2)));
typedef uint32_t Floats2 __attribute__((ext_vector_type(2), aligned(4)));

// Lane's logits of row t as they are in memory, a bf16 pair in one word.
template <int V, bool kHalf>
__device__ __forceinline__ void load_row(const void* logits, int64_t t, int32_t E, int lane, uint32_t (&w)[V]) {
    constexpr int R = kPair<V>;
    const uint16_t* half = static_cast<const uint16_t*>(logits) + t * E;
    const uint32_t* full = static_cast<const uint32_t*>(logits) + t * E;
#pragma unroll
    for (int v = 0; v < V; v += R) {
        const int first = Pair<V>(lane, v, E).first;
        if constexpr (kHalf) {
            if constexpr (R == 2)
                w[v] = *reinterpret_cast<const Halves2*>(half + first);
            else
                w[v] = half[first];
        } else if constexpr (R == 2) {
            const Floats2 x = *reinterpret_cast<const Floats2*>(full + first);
            w[v] = x.x, w[v + 1] = x.y;
        } else {
            w[v] = full[first];
        }
    }
}

// The loaded row as floats, -inf for what does not count.
template <int V, bool kHalf>
__device__ __forceinline__ void widen_row(const uint32_t (&w)[V], int32_t E, int lane, float (&z)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kHalf)
            z[v] = v % 2 == 0 ? bf16_low(w[v]) : bf16_high(w[v - v % 2]);
        else
            z[v] = __uint_as_float(w[v]);
        z[v] = counts<V>(lane, v, E) ? z[v] : kNone;
    }
}

// The gradient of row t's logits.
template <int V, bool kHalf>
__device__ __forceinline__ void store_row(void* grad, int64_t t, int32_t E, int lane, const float (&s)[V]) {
    constexpr int R = kPair<V>;
    uint16_t* const half = static_cast<uint16_t*>(grad) + t * E;
    float* const full = static_cast<float*>(grad) + t * E;
#pragma unroll
    for (int v = 0; v < V; v += R) {
        const Pair<V> pair(lane, v, E);
        const bool whole = pair.first == pair.start;
        const bool second = !whole && counts<V>(lane, v + R - 1, E);  // of a pair that was moved
        if constexpr (kHalf) {
            const uint32_t x = pack_bf16(s[v], s[v + R - 1]);
            uint16_t* const at = half + pair.first;
            if constexpr (R == 2) {
                if (whole) *reinterpret_cast<Halves2*>(at) = x;
                if (second) at[1] = (uint16_t)(x >> 16);
            } else {
                if (whole) *at = (uint16_t)x;
            }
        } else {
            float* const at = full + pair.first;
            if constexpr (R == 2) {
                const Floats2 x = {__float_as_uint(s[v]), __float_as_uint(s[v + 1])};
                if (whole) *reinterpret_cast<Floats2*>(at) = x;
                if (second) at[1] = s[v + 1];
            } else {
                if (whole) *at = s[v];
            }
        }
    }
}

// A row of the lanes' floats in LDS, each pair at the place it would have
// without being moved. slot_of: where expert e's is;
// expert_at: whose a slot is.
template <int V>
__device__ __forceinline__ int lane_slot(int lane, int v) {
    return (v / kPair<V> * kWave + lane) * kPair<V> + v % kPair<V>;
}
template <int V>
__device__ __forceinline__ int slot_of(int e, int32_t E) {
    return kPair<V> == 2 && (E & 1) != 0 && e == E - 1 ? E : e;
}
template <int V>
__device__ __forceinline__ int expert_at(int slot, int32_t E) {
    return kPair<V> == 2 && slot == E ? E - 1 : slot;
}
template <int V>
__device__ __forceinline__ void write_slots(float* row, int lane, const float (&s)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) row[lane_slot<V>(lane, v)] = s[v];
}

// A value as an unsigned integer of the same order, both zeros alike. What is
// never taken, NaN and -inf, gets kNoKey, below every other value's.
constexpr uint32_t kNoKey = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float c) {
    const uint32_t u = __float_as_uint(fmaxf(c + 0.f, kNone));  // (fmaxf drops NaN)
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The value of an order key, -inf of kNoKey.
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((int32_t)key < 0 ? key ^ 0x80000000u : ~key);
}

// exp(x) for x <= 0 from the hardware's exp2: the argument's rounding leaves a
// relative error of |x| 2^-24, far from where exp(x) counts in a sum with 1.
__device__ __forceinline__ float exp_nonpositive(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}

// 1 / x within 1 ulp, exact for 1, for x in [2^-126, 2^126]: the hardware's
// reciprocal and one Newton step, 3 instructions where a division takes 11.
__device__ __forceinline__ float reciprocal(float x) {
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.f), r, r);
}

// A row's sum of scores (before softmax divides by it) and its reciprocal, 0
// for a row whose scores are all 0. (The smallest sigmoid that is not 0, of the
// last fp32 number before exp(-z) is infinite, is 2^-128 (1 + 2^-17): its
// reciprocal is finite, that times another number may not be.)
struct RowSum {
    float sum, inv;
    // s / sum, the product's rounding corrected: a lone score's share is 1, so
    // that its gradient cancels exactly.
    __device__ __forceinline__ float share(float s) const {
        const float p = s * inv;
        return __builtin_fmaf(__builtin_fmaf(-p, sum, s), inv, p);
    }
};

// Scores of a row in place of its logits, whose largest has the key top
// (softmax scores are shares already: their sum is at least 1, or the row has
// nothing).
template <int V, bool kSigmoid>
__device__ __forceinline__ RowSum scores(float (&z)[V], uint32_t top) {
    const float high = top == kNoKey ? 0.f : key_value(top);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kSigmoid)
            z[v] = z[v] == kNone ? 0.f : sigmoid(z[v]);
        else
            z[v] = exp_nonpositive(z[v] - high);
        sum += z[v];
    }
    sum = wave_sum(sum);
    const RowSum r{sum, sum == 0.f ? 0.f : (kSigmoid ? 1.f / sum : reciprocal(sum))};
    if (!kSigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] *= r.inv;
    }
    return r;
}

// A lane's pairs of keys, the larger one of each first, of equal ones the
// lower expert's. A mask bit per lane says whose pairs have changed places:
// a removal then costs two vector instructions a pair, the rest is scalar.
template <int V>
struct Pairs {
    static constexpr int R = kPair<V>, kPairs = V / R;
    uint32_t key[V];
    uint64_t swapped[kPairs];

    __device__ __forceinline__ void sort() {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            swapped[j] = 0;
            if constexpr (R == 2) {
                const uint32_t a = key[2 * j], b = key[2 * j + 1];
                swapped[j] = __ballot(b > a);
                key[2 * j] = a > b ? a : b;
                key[2 * j + 1] = a > b ? b : a;
            }
        }
    }
    // The largest key of the wavefront.
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = key[0];
#pragma unroll
        for (int j = 1; j < kPairs; ++j) m = m > key[j * R] ? m : key[j * R];
        return wave_max(m);
    }
    // Takes the lowest expert whose key is m, the largest, out: its slot.
    __device__ __forceinline__ int take(uint32_t m) {
        uint64_t hit = __ballot(key[0] == m), out[kPairs];
        int pair = 0;
#pragma unroll
        for (int j = 1; j < kPairs; ++j) {
            const uint64_t here = __ballot(key[j * R] == m);
            pair = hit == 0 ? j : pair;
            hit = hit == 0 ? here : hit;
        }
        const int l = __builtin_ctzll(hit);
        const uint64_t bit = uint64_t(1) << l;
        uint64_t order = 0;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const bool here = kPairs == 1 || pair == j;
            out[j] = here ? bit : 0;
            order = here ? swapped[j] : order;
            swapped[j] ^= out[j];
            const bool mine = __builtin_amdgcn_inverse_ballot_w64(out[j]);
            if constexpr (R == 2) key[j * R] = mine ? key[j * R + 1] : key[j * R];
            key[j * R + R - 1] = mine ? kNoKey : key[j * R + R - 1];
        }
        return (pair * kWave + l) * R + (R == 2 ? (int)(order >> l) & 1 : 0);
    }
};

// Two largest keys, and those of two such pairs together.
struct TopTwo {
    uint32_t first = kNoKey, second = kNoKey;
    __device__ __forceinline__ void add(uint32_t key) {
        const uint32_t low = first < key ? first : key;
        second = second > low ? second : low;
        first = first > key ? first : key;
    }
    __device__ __forceinline__ void join(uint32_t other, uint32_t next) {
        second = second > next ? second : next;
        add(other);
    }
    // What a group goes by: its largest choice, or the fp32 sum of its two
    // largest (of a lone one itself; a sum below fp32's range is its lowest
    // number, as the group has something to take).
    __device__ __forceinline__ uint32_t mark(bool pairs) const {
        if (!pairs || second == kNoKey) return first;
        const uint32_t sum = order_key(key_value(first) + key_value(second));
        return sum > kNoKey ? sum : kNoKey + 1;
    }
};

// The lane that stands for an expert's group: (e + 0.5) / size is further from
// a whole number than the product is off, as there are at most 64 groups.
__device__ __forceinline__ int group_lane(int e, float per_size, int log_lanes) {
    return (int)(((float)e + 0.5f) * per_size) << log_lanes;
}

// With the lane that kCtrl pairs this one with.
template <int kCtrl>
__device__ __forceinline__ void join_paired(TopTwo& top) {
    top.join((uint32_t)__builtin_amdgcn_update_dpp(0, (int)top.first, kCtrl, 0xf, 0xf, true),
             (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top.second, kCtrl, 0xf, 0xf, true));
}

// The groups that a token's experts are taken from, a bit for the first lane
// of each: the wavefront's keys go through its row in LDS, the lanes of a group
// look at its experts in turn and join what they found, and the best marks are
// taken, of equal ones the lowest group's. (By their places, a comparison with
// each group's mark, one token of 512 experts in 64 groups took 7.5 us, 5.5 so; 8
// groups the same.)
template <int V>
__device__ __forceinline__ uint64_t open_groups(const uint32_t (&key)[V], float* row, const GateParams& p, int lane) {
#pragma unroll
    for (int v = 0; v < V; ++v) row[lane_slot<V>(lane, v)] = __uint_as_float(key[v]);
    __builtin_amdgcn_wave_barrier();
    const int lanes = 1 << p.group_lanes, part = lane & (lanes - 1), group = lane >> p.group_lanes;
    TopTwo top;
    if (group < p.num_groups) {
        const int first = group * p.group_size;
        for (int i = part; i < p.group_size; i += lanes)
            top.add(__float_as_uint(row[slot_of<V>(first + i, p.num_experts)]));
    }
    __builtin_amdgcn_wave_barrier();
    // (Mirrors pair as steps of 4 and 8 do once fours and eights are alike.)
    if (lanes > 1) join_paired<kDppQuadXor1>(top);
    if (lanes > 2) join_paired<kDppQuadXor2>(top);
    if (lanes > 4) join_paired<kDppRowHalfMirror>(top);
    if (lanes > 8) join_paired<kDppRowMirror>(top);
    for (int step = 16; step < lanes; step *= 2)
        top.join((uint32_t)__shfl_xor((int)top.first, step), (uint32_t)__shfl_xor((int)top.second, step));
    uint32_t mark = part == 0 ? top.mark(p.group_pairs) : kNoKey;
    uint64_t open = 0;
    for (int n = 0; n < p.topk_groups; ++n) {
        const uint32_t m = wave_max(mark);
        if (m == kNoKey) break;
        const int l = __builtin_ctzll(__ballot(mark == m));
        open |= uint64_t(1) << l;
        mark = lane == l ? kNoKey : mark;
    }
    return open;
}

// From the sum of counts times probability sums.
__device__ __forceinline__ float balance_loss(float coef, int E, int K, int live, double sum) {
    return live == 0 ? 0.f : (float)((double)coef * E / ((double)K * live * live) * sum);
}

template <int V, bool kHalf, bool kSigmoid, bool kBalance, bool kGrouped>
__global__ void __launch_bounds__(kGateWaves<V> * kWave) gate_kernel(GateParams p) {
    // A row of scores per wavefront, then with kBalance the workgroup's
    // counts [E] and live tokens [1].
    extern __shared__ float lds[];
    const int W = kBalance ? kGateWaves<V> : (int)blockDim.x / kWave;
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
    uint32_t next[V];
    int next_live = 1;
    const auto load = [&](int64_t row) {
        load_row<V, kHalf>(p.logits, row, E, lane, next);
        if (p.mask != nullptr) next_live = p.mask[row];
    };
    // The loaded row becomes the current one before the last one's results are
    // stored, so that it does not wait for them.
    float s[V];
    bool taken = false;
    const auto arrive = [&] {
        widen_row<V, kHalf>(next, E, lane, s);
        taken = __builtin_amdgcn_readfirstlane(next_live) != 0;
    };
    if (t < p.num_tokens) load(t);
    const auto bias_of = [&](int v) { return p.bias != nullptr ? p.bias[expert_of<V>(lane, v, E)] : 0.f; };
    // Kept in registers where there are enough of them.
    constexpr bool kKeepBias = kSigmoid && V <= 16;
    float bias[kKeepBias ? V : 1];
    if constexpr (kKeepBias) {
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = bias_of(v);
    }
    const float per_size = kGrouped ? 1.f / (float)p.group_size : 0.f;
    // Only experts of the token's groups keep their keys.
    const auto close_groups = [&](uint32_t(&key)[V]) {
        const uint64_t open = open_groups<V>(key, score_row, p, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = group_lane(expert_of<V>(lane, v, E), per_size, p.group_lanes);
            key[v] = (open >> at) & 1 ? key[v] : kNoKey;
        }
    };
    if (t < p.num_tokens) arrive();
    for (; t < p.num_tokens; t += stride) {
        int picked = -1;     // lane k: entry k's slot, then its expert
        float weight = 0.f;  // lane k: its score
        if (t + stride < p.num_tokens) load(t + stride);
        if (taken) {
            Pairs<V> pairs;
            RowSum row_sum;
            uint32_t m;
            if (kSigmoid) {
                bool never[V];
#pragma unroll
                for (int v = 0; v < V; ++v) never[v] = !(s[v] > kNone);
                row_sum = scores<V, true>(s, kNoKey);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float b = kKeepBias ? bias[kKeepBias ? v : 0] : bias_of(v);
                    pairs.key[v] = never[v] ? kNoKey : order_key(s[v] + b);
                }
                if constexpr (kGrouped) close_groups(pairs.key);
                pairs.sort();
                m = pairs.top();
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) pairs.key[v] = order_key(s[v]);
                // (The largest logit's group is among them.)
                if constexpr (kGrouped) close_groups(pairs.key);
                pairs.sort();
                m = pairs.top();
                row_sum = scores<V, false>(s, m);
            }
            write_slots<V>(score_row, lane, s);
            for (int k = 0; m != kNoKey;) {
                const int slot = pairs.take(m);
                picked = lane == k ? slot : picked;
                if (++k == K) break;
                m = pairs.top();
            }
            __builtin_amdgcn_wave_barrier();
            if (picked >= 0) weight = score_row[picked];
            picked = expert_at<V>(picked, E);
            __builtin_amdgcn_wave_barrier();
            if (p.flags & DISPATCH_GATE_NORMALIZE) {
                const float total = wave_sum(weight);
                // (A softmax row's largest share is at least 1 / E. Sigmoid
                // scores may be as small as numbers are: divided first.)
                weight = total == 0.f ? 0.f
                         : kSigmoid   ? p.route_scale * (weight / total)
                                      : p.route_scale * weight * reciprocal(total);
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
        if (t + stride < p.num_tokens) arrive();
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
    write_slots<V>(score_row, lane, prob_sum);
    if (lane == 0) atomicAdd(counts + E, live);
    __syncthreads();
    if (gridDim.x == 1) {
        // A lone workgroup has it all.
        double part = 0.0;
        for (int i = threadIdx.x; i < E; i += W * kWave) {
            const float* at = lds + slot_of<V>(i, E);
            float x = at[0];
#pragma unroll
            for (int w = 1; w < kGateWaves<V>; ++w) x += at[w * V * kWave];
            p.prob_sum[i] = x;
            p.expert_count[i] = counts[i];
            part += (double)counts[i] * (double)x;
        }
        for (int step = kWave / 2; step > 0; step /= 2) part += __shfl_xor(part, step);
        __syncthreads();
        double* const parts = reinterpret_cast<double*>(lds);
        if (lane == 0) parts[wave] = part;
        __syncthreads();
        if (threadIdx.x != 0) return;
        for (int w = 1; w < W; ++w) part += parts[w];
        const int n = counts[E];
        *p.live_tokens = n;
        *p.loss = balance_loss(p.loss_coef, E, K, n, part);
        return;
    }
    float* const out = p.partial + (int64_t)blockIdx.x * (2 * E + 1);
    for (int i = threadIdx.x; i < 2 * E + 1; i += W * kWave) {
        float x = __int_as_float(counts[i - E < 0 ? 0 : i - E]);
        if (i < E) {
            const float* at = lds + slot_of<V>(i, E);
            x = at[0];
#pragma unroll
            for (int w = 1; w < kGateWaves<V>; ++w) x += at[w * V * kWave];
        }
        out[i] = x;
    }
}

// The forward pass of many tokens and up to 256 experts: four tokens per
// wavefront, 16 lanes for each, V = 8 or 16 experts per lane (with groups also 4,
// or 32 for up to 512 experts) in runs of four neighbours (run j of lane c from
// expert 4 (16 j + c); a run that would pass the last expert is moved back, as a
// pair above).
//
// Choice of up to eight: a key and its expert are one number, key * 256 + 255
// - expert (512 and 511 with V = 32), exact in a double (2^52 is added, so that
// its bits are put together by two instructions), and all differ: a maximum and
// a minimum, one full-rate instruction each, order two of them with no tie to
// look at. A lane sorts its numbers, eight at a time, and four times lanes join their best eight with a partner's: the
// larger of each and the partner's opposite are the best eight of both, in a
// bitonic order that three steps sort. What is done once a token above (sums,
// divisions, stores) is done once for four.
//
// Its time does not depend on k; that of the form above does. Measured, us of this
// form and of the one above with k = 3, 4, 6 and 8, without / with balance outputs:
//
//   softmax of fp32         here            k = 3         4            6            8
//   128 experts,  4096   3.8 /  9.7    3.1 /  9.0   3.3 /  9.1   3.7 /  9.4   4.0 /  9.8
//                 8192   3.8 / 10.1    4.0 / 10.0   4.2 / 10.3   4.7 / 11.1   5.2 / 11.7
//                65536  14.4 / 24.1   17.2 / 23.6  18.6 / 25.5  21.8 / 29.4  24.9 / 33.4
//   256 experts,  4096   4.4 / 11.0    3.6 /  9.5   3.9 /  9.8   4.5 / 10.3   5.1 / 10.9
//                 8192   4.6 / 11.5    4.7 / 11.1   5.2 / 11.7   6.2 / 12.8   7.1 / 13.9
//                65536  20.6 / 31.5   22.3 / 30.5  25.1 / 34.1  31.7 / 42.1  38.3 / 49.7
//   sigmoid of bf16
//   128 experts,  8192   5.0 / 11.4    4.3 / 11.0   4.5 / 11.2   5.0 / 12.0   5.5 / 12.7
//                16384   6.9 / 14.4    6.4 / 14.2   6.8 / 14.8   7.7 / 15.8   8.6 / 16.8
//                65536  19.3 / 30.1   19.4 / 29.9  21.1 / 31.7  24.2 / 35.6  27.3 / 39.5
//   256 experts,  8192   6.5 / 13.9    5.5 / 12.5   5.9 / 12.9   6.8 / 14.0   7.8 / 15.1
//                16384   9.5 / 18.9    8.6 / 19.3   9.2 / 20.1  10.9 / 22.4  12.7 / 24.6
//                65536  30.1 / 42.4   27.0 / 46.9  29.6 / 50.8  35.5 / 59.0  42.1 / 67.6
//
// So it is taken for four entries and more from 8192 tokens on, with sigmoid and
// fewer than six from twice as many. (72 experts as 128, 200 as 256.)
constexpr int kBest = 8;
constexpr int kFewestRounds = 4;
constexpr int kFewestSigmoidRounds = 6;  // of less than 2 kManyTokens, or of more than 256 experts
constexpr int64_t kManyTokens = 8192;
constexpr int kRowLanes = 16;
constexpr int kRowTokens = kWave / kRowLanes;
// Wavefronts of a workgroup, and those that share a SIMD's registers.
template <int V>
constexpr int kRowWaves = V > 16 ? 4 : 8;
template <int V>
constexpr int kRowSimdWaves = V > 16 ? 2 : 4;

template <int V>
struct Quad {
    int start, first;  // as of Pair
    __device__ __forceinline__ Quad(int c, int v, int32_t E) {
        start = (v / 4 * kRowLanes + c) * 4;
        // (E > 8 V with V > 4: the first half is whole.)
        first = 4 * kRowLanes * (v / 4 + 1) <= 8 * V || start < E - 4 ? start : E - 4;
    }
};

// (LDS words of these types may be read as others, unlike HIP's uint2 and uint4.)
typedef uint32_t Words2 __attribute__((ext_vector_type(2)));
typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
typedef uint32_t Halves4 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t Floats4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }

// An expert's bits below its key's.
template <int V>
constexpr int kExpertBits = V > 16 ? 9 : 8;
template <int V>
__device__ __forceinline__ double numbered(uint32_t key, int expert) {
    constexpr int kBits = kExpertBits<V>;
    const uint32_t low = key << kBits | (uint32_t)((1 << kBits) - 1 - expert);
    return __builtin_bit_cast(double, (uint64_t)(0x43300000u | key >> (32 - kBits)) << 32 | low);
}

__device__ __forceinline__ void order(double (&x)[kBest], int i, int j) {
    const double a = larger(x[i], x[j]), b = smaller(x[i], x[j]);
    x[i] = a, x[j] = b;
}
// Largest first: Batcher's network of 19 exchanges.
__device__ __forceinline__ void sort(double (&x)[kBest]) {
    order(x, 0, 1), order(x, 2, 3), order(x, 4, 5), order(x, 6, 7);
    order(x, 0, 2), order(x, 1, 3), order(x, 4, 6), order(x, 5, 7);
    order(x, 1, 2), order(x, 5, 6);
    order(x, 0, 4), order(x, 1, 5), order(x, 2, 6), order(x, 3, 7);
    order(x, 2, 4), order(x, 3, 5);
    order(x, 1, 2), order(x, 3, 4), order(x, 5, 6);
}
// The best eight of two sorted lists.
__device__ __forceinline__ void join(double (&x)[kBest], const double (&y)[kBest]) {
#pragma unroll
    for (int i = 0; i < kBest; ++i) x[i] = larger(x[i], y[kBest - 1 - i]);
    order(x, 0, 4), order(x, 1, 5), order(x, 2, 6), order(x, 3, 7);
    order(x, 0, 2), order(x, 1, 3), order(x, 4, 6), order(x, 5, 7);
    order(x, 0, 1), order(x, 2, 3), order(x, 4, 5), order(x, 6, 7);
}
// With the lane that kCtrl pairs this one with.
template <int kCtrl>
__device__ __forceinline__ void join_lanes(double (&x)[kBest]) {
    double y[kBest];
#pragma unroll
    for (int i = 0; i < kBest; ++i) {
        const uint64_t bits = __builtin_bit_cast(uint64_t, x[i]);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)bits, kCtrl, 0xf, 0xf, true);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(bits >> 32), kCtrl, 0xf, 0xf, true);
        y[i] = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    }
    join(x, y);
}

// The best eight of a token's lanes, from each lane's V numbers: the first
// sixteen in best and more, the others from number.
template <int V, typename Number>
__device__ __forceinline__ void best_of(double (&best)[kBest], double (&more)[kBest], const Number& number) {
    sort(best);
    if constexpr (V > kBest) {
        sort(more);
        join(best, more);
    }
#pragma unroll
    for (int v = 2 * kBest; v < V; v += kBest) {
#pragma unroll
        for (int i = 0; i < kBest; ++i) more[i] = number(v + i);
        sort(more);
        join(best, more);
    }
    join_lanes<kDppQuadXor1>(best);
    join_lanes<kDppQuadXor2>(best);
    join_lanes<kDppRowHalfMirror>(best);
    join_lanes<kDppRowMirror>(best);
}

// Where expert e is in a row of runs.
__device__ __forceinline__ int quad_slot(int e, int32_t E) {
    const int past = E % 4;
    return past == 0 || e < E - past ? e : e + 4 - past;
}

// Choice by groups, of up to 32. Where a group is a number of whole runs, a lane
// finds the two largest keys of each of its runs, and these go through LDS; else
// the keys do. The token's 16 lanes, Gp of them side by side for the groups (Gp a
// power of two; with more than 16 groups each lane has two) look for those of
// their group and join what they found by rotations. All of these have its mark
// then, and a group's place is the number of marks above its own, of equal ones
// of lower groups: Gp - 1 rotations. (A maximum and its removal for each group
// taken: 14 instructions for each of them, where a rotation takes 4.) Entries
// past the eighth come from a second pass over the keys below the eighth's.
// Looking for the groups takes longer in the form of one token per wavefront, so
// this one is taken from 8192 tokens on whatever the number of entries. Measured,
// 8 groups, 4 taken, us of this form and of the other with k = 1, 4 and 8, without
// / with balance outputs:
//
//   softmax of fp32         here            k = 1         4            8
//    64 experts,  4096   4.5 / 10.4    4.1 /  9.7   4.3 / 10.4   4.7 / 10.6
//                 8192   5.1 / 10.6    5.7 / 11.5   6.0 / 11.9   6.7 / 12.5
//                65536  17.4 / 24.0   23.1 / 33.8  26.2 / 40.1  31.3 / 47.8
//   128 experts,  4096   5.1 / 11.5    4.5 / 10.5   5.1 / 11.6   5.2 / 11.7
//                 8192   4.9 / 11.8    5.5 / 12.4   6.2 / 13.1   7.1 / 14.1
//                65536  19.1 / 27.5   26.0 / 39.7  30.3 / 47.5  36.5 / 58.1
//   256 experts,  4096   5.9 / 12.7    4.9 / 11.1   5.6 / 11.6   6.8 / 12.6
//                 8192   5.6 / 12.9    6.4 / 13.2   7.7 / 14.4   9.2 / 16.4
//                65536  26.4 / 36.3   32.5 / 47.4  39.6 / 60.2  52.1 / 77.3
//   sigmoid of bf16, pairs
//   256 experts,  4096   7.9 / 15.1    6.0 / 12.3   6.6 / 12.6   7.4 / 13.7
//                 8192   7.8 / 15.7    8.1 / 14.2   9.1 / 15.8  10.8 / 17.9
//                65536  37.8 / 48.3   40.9 / 60.4  48.0 / 72.6  59.7 / 88.7
//
// Groups of other sizes, more than 16 of them or more than eight entries, softmax of
// fp32, 65536 tokens, here / other form: 12 experts in 4 groups, k = 5 17.2 / 25.5;
// 40 in 20, k = 2 22.6 / 24.3; 64 in 8, k = 12 27.1 / 34.6; 128 in 8, k = 12 32.5 /
// 42.0 (8192 tokens 6.8 / 8.1). With 16 experts a lane the registers do not hold it
// (150 in 10, k = 8 61.7 / 50.2; with two wavefronts on a SIMD 49.0 / 46.1 for k = 6),
// so that is left to the other form.
//
// More than 256 experts take 32 a lane and two wavefronts on a SIMD, in groups of
// whole runs only (500 in 20 58.0 / 60.4, sigmoid 79.9 / 67.2, 40000 tokens):
//
//   512 experts in 16, 4 taken  here            k = 3          4              6
//   softmax of fp32,   8192   7.9 / 18.4   10.8 / 17.3   11.0 / 18.4   12.9 / 20.2
//                     16384  14.2 / 25.4   17.6 / 29.4   19.0 / 31.4   22.5 / 35.2
//                     65536  51.5 / 57.4   58.5 / 78.9   64.1 / 86.6   77.4 / 102.5
//   sigmoid of bf16,   8192  12.2 / 25.9   13.1 / 20.6   13.4 / 21.3   15.3 / 23.3
//                     16384  22.5 / 32.7   21.6 / 35.0   22.7 / 36.9   25.7 / 40.7
//                     65536  84.2 / 90.0   73.0 / 101.1  77.6 / 108.7  88.4 / 123.6
//
// So there from four entries on, with sigmoid and no balance outputs from six,
// with balance outputs from twice as many tokens.
constexpr int kMostRowGroups = 2 * kRowLanes;
constexpr int kMostRowEntries = 2 * kBest;
constexpr int kMostAnyExperts = 128;

// Which groups a form is built for.
enum class Groups {
    kNone,
    kRuns,  // up to 16, each a number of whole runs; up to eight entries
    kAny,   // up to 32; up to 16 entries; up to 128 experts
};

// LDS words of a token's runs or keys (8 between the tokens', so that they start
// in other banks), and floats of a wavefront.
__device__ __host__ constexpr int token_words(int v, Groups groups) {
    return groups == Groups::kNone ? 0 : v * kRowLanes / (groups == Groups::kRuns ? 2 : 1) + 8;
}
__device__ __host__ constexpr int row_floats(int v, bool sigmoid, Groups groups) {
    const int scores = (sigmoid ? kRowTokens : 1) * v * kRowLanes, keys = kRowTokens * token_words(v, groups);
    return scores > keys ? scores : keys;
}

// With the lane N places on in a row of 16.
template <int N>
__device__ __forceinline__ void join_rotated(TopTwo& top) {
    const uint32_t first = dpp_ror<kDppRowRor + N>(top.first), second = dpp_ror<kDppRowRor + N>(top.second);
    top.join(first, second);
}

// Adds 1 where the mark of the group N before (modulo Gp) goes before this one.
template <int N>
__device__ __forceinline__ void count_before(uint32_t mark, int group, int& place) {
    place += dpp_ror<kDppRowRor + N>(mark) + (group >= N ? 1u : 0u) > mark ? 1 : 0;
}
template <int kFirst, int... N>
__device__ __forceinline__ void count_from(std::integer_sequence<int, N...>, uint32_t mark, int group, int& place) {
    (count_before<kFirst + N>(mark, group, place), ...);
}
// The same between the first 16 groups and the others: one of the first goes
// before an equal one of the others.
template <int... N>
__device__ __forceinline__ void count_across(std::integer_sequence<int, N...>, uint32_t mark, uint32_t mark2, int& place,
                                             int& place2) {
    place += mark2 > mark ? 1 : 0;
    place2 += mark >= mark2 ? 1 : 0;
    ((place += dpp_ror<kDppRowRor + N + 1>(mark2) > mark ? 1 : 0,
      place2 += dpp_ror<kDppRowRor + N + 1>(mark) >= mark2 ? 1 : 0),
     ...);
}

// A bit for each group of the lane's token that is open.
template <int V, Groups kGroups>
__device__ __forceinline__ uint32_t open_row_groups(const uint32_t (&key)[V], float* mine, const GateParams& p,
                                                    int lane) {
    const int c = lane % kRowLanes;
    const int side = kRowLanes >> p.group_lanes;  // Gp
    const int group = c & (side - 1), part = c / side, parts = 1 << p.group_lanes;
    const bool two = kGroups == Groups::kAny && p.num_groups > kRowLanes;
    float* const row = mine + lane / kRowLanes * token_words(V, kGroups);
    TopTwo top, next;  // of the lane's group, and of the one 16 further on
    if constexpr (kGroups == Groups::kRuns) {
        Words2* const runs = reinterpret_cast<Words2*>(row);
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            TopTwo run;
            const uint32_t a = key[v], b = key[v + 1], d = key[v + 2], e = key[v + 3];
            run.first = a > b ? a : b;
            run.second = a > b ? b : a;
            run.join(d > e ? d : e, d > e ? e : d);
            runs[v / 4 * kRowLanes + c] = Words2{run.first, run.second};
        }
        __builtin_amdgcn_wave_barrier();
        const int size = p.group_size / 4;
        for (int i = part; group < p.num_groups && i < size; i += parts) {
            const Words2 run = runs[group * size + i];
            top.join(run.x, run.y);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v += 4)
            reinterpret_cast<Words4*>(row)[v / 4 * kRowLanes + c] = Words4{key[v], key[v + 1], key[v + 2], key[v + 3]};
        __builtin_amdgcn_wave_barrier();
        const auto at = [&](int e) { return __float_as_uint(row[quad_slot(e, p.num_experts)]); };
        const int first = group * p.group_size, far = first + kRowLanes * p.group_size;
        for (int i = part; i < p.group_size; i += parts) {
            if (first < p.num_experts) top.add(at(first + i));
            if (far < p.num_experts && two) next.add(at(far + i));
        }
    }
    __builtin_amdgcn_wave_barrier();
    // (There are two groups at least: Gp is 2 or more.)
    if (side <= 2) join_rotated<2>(top);
    if (side <= 4) join_rotated<4>(top);
    if (side <= 8) join_rotated<8>(top);
    const uint32_t mark = top.mark(p.group_pairs);
    int place = 0;
    // (Past Gp - 1 rotations the same groups come again.)
    count_before<1>(mark, group, place);
    if (side > 2) count_from<2>(std::make_integer_sequence<int, 2>(), mark, group, place);
    if (side > 4) count_from<4>(std::make_integer_sequence<int, 4>(), mark, group, place);
    if (side > 8) count_from<8>(std::make_integer_sequence<int, 8>(), mark, group, place);
    const auto bits = [&](bool open) {
        const uint64_t all = __ballot(open);
        const uint32_t word = lane < kWave / 2 ? (uint32_t)all : (uint32_t)(all >> 32);
        return (word >> (lane & kRowLanes)) & ((1u << side) - 1);
    };
    if (!two) return bits(place < p.topk_groups && mark != kNoKey);
    const uint32_t mark2 = next.mark(p.group_pairs);
    int place2 = 0;
    const auto others = std::make_integer_sequence<int, kRowLanes - 1>();
    count_from<1>(others, mark2, group, place2);
    count_across(others, mark, mark2, place, place2);
    return bits(place < p.topk_groups && mark != kNoKey) | bits(place2 < p.topk_groups && mark2 != kNoKey) << kRowLanes;
}

template <int V, bool kHalf, bool kSigmoid, bool kBalance, Groups kGroups>
__global__ void __launch_bounds__(kRowWaves<V> * kWave, kRowSimdWaves<V>) gate_rows_kernel(GateParams p) {
    // Sigmoid: the wavefront's rows of scores; groups: its tokens' runs;
    // balance: its sums; then of the workgroup, sigmoid: a row of the selection
    // bias; balance: counts [E] and live tokens [1].
    constexpr bool kGrouped = kGroups != Groups::kNone;
    constexpr int kWaveFloats = row_floats(V, kSigmoid, kGroups);
    extern __shared__ float lds[];
    const int lane = threadIdx.x & (kWave - 1), c = lane % kRowLanes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int E = p.num_experts, K = p.num_topk;
    float* const mine = lds + wave * kWaveFloats;
    float* const bias = lds + kRowWaves<V> * kWaveFloats;
    int* const counts = reinterpret_cast<int*>(bias + (kSigmoid ? V * kRowLanes : 0));
    float prob_sum[V];
    int live = 0;
    if (kBalance) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
        for (int i = threadIdx.x; i < E + 1; i += kRowWaves<V> * kWave) counts[i] = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) prob_sum[v] = 0.f;
    }
    if (kSigmoid)
        for (int e = threadIdx.x; e < E; e += kRowWaves<V> * kWave)
            bias[quad_slot(e, E)] = p.bias != nullptr ? p.bias[e] : 0.f;
    if (kBalance || kSigmoid) __syncthreads();
    const int64_t stride = (int64_t)gridDim.x * kRowWaves<V> * kRowTokens;
    int64_t t0 = ((int64_t)blockIdx.x * kRowWaves<V> + wave) * kRowTokens;  // the wavefront's first token
    constexpr int kWords = kHalf ? V / 2 : V;
    uint32_t next[kWords];
    int next_live = 0;
    const auto load = [&](int64_t first) {
        const int64_t mine_t = first + lane / kRowLanes;
        const int64_t t = mine_t < p.num_tokens ? mine_t : p.num_tokens - 1;
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const int64_t at = t * E + Quad<V>(c, v, E).first;
            if constexpr (kHalf) {
                const Halves4 x = *reinterpret_cast<const Halves4*>(static_cast<const uint16_t*>(p.logits) + at);
                next[v / 2] = x.x, next[v / 2 + 1] = x.y;
            } else {
                const Floats4 x = *reinterpret_cast<const Floats4*>(static_cast<const uint32_t*>(p.logits) + at);
                next[v] = x.x, next[v + 1] = x.y, next[v + 2] = x.z, next[v + 3] = x.w;
            }
        }
        const int on = p.mask != nullptr ? p.mask[t] : 1;
        next_live = mine_t < p.num_tokens ? on : 0;
    };
    float s[V];
    bool taken = false;
    // A token that is masked or past the last has no logit that counts.
    const auto arrive = [&] {
        taken = next_live != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Quad<V> quad(c, v, E);
            const float z = !kHalf        ? __uint_as_float(next[kHalf ? 0 : v])
                            : v % 2 == 0 ? bf16_low(next[v / 2])
                                         : bf16_high(next[v / 2]);
            s[v] = taken && quad.first + v % 4 >= quad.start ? z : kNone;
        }
    };
    // The groups of the lane's runs, where runs are of one (what is past the last
    // group has nothing to take).
    int run_group[V / 4] = {};
    const float per_size = kGroups == Groups::kAny ? 1.f / (float)p.group_size : 0.f;
    if constexpr (kGroups == Groups::kRuns) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) run_group[j] = (j * kRowLanes + c) * 4 / p.group_size & 31;
    }
    if (t0 < p.num_tokens) load(t0);
    if (t0 < p.num_tokens) arrive();
    for (; t0 < p.num_tokens; t0 += stride) {
        if (t0 + stride < p.num_tokens) load(t0 + stride);
        const bool now = taken;
        float sum = 0.f;
        uint32_t keys[V], never = 0;
        // The keys of scores (sigmoid) or logits, without what no choice is.
        const auto key_of_expert = [&](int v) {
            if constexpr (!kSigmoid) return order_key(s[v]);
            return (never >> v) & 1 ? kNoKey : order_key(s[v] + bias[(v / 4 * kRowLanes + c) * 4 + v % 4]);
        };
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (kSigmoid) {
                never |= (!(s[v] > kNone) ? 1u : 0u) << v;
                s[v] = s[v] == kNone ? 0.f : sigmoid(s[v]);
                sum += s[v];
            }
            keys[v] = key_of_expert(v);
        }
        uint32_t open = 0;
        const auto close_groups = [&] {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                int group = run_group[v / 4];
                if (kGroups == Groups::kAny) group = group_lane(Quad<V>(c, v, E).first + v % 4, per_size, 0);
                keys[v] = (open >> group) & 1 ? keys[v] : kNoKey;
            }
        };
        if constexpr (kGrouped) {
            open = open_row_groups<V, kGroups>(keys, mine, p, lane);
            close_groups();
        }
        double best[kBest], more[kBest];
        const auto number = [&](int v) { return numbered<V>(keys[v], Quad<V>(c, v, E).first + v % 4); };
#pragma unroll
        for (int v = 0; v < V && v < 2 * kBest; ++v) (v < kBest ? best : more)[v % kBest] = number(v);
#pragma unroll
        for (int v = V; v < kBest; ++v) best[v] = numbered<V>(kNoKey, 0);
        best_of<V>(best, more, number);
        const auto key_of = [](double x) { return (uint32_t)(__builtin_bit_cast(uint64_t, x) >> kExpertBits<V>); };
        const uint32_t top = key_of(best[0]);
        // Lane c of the token's 16 takes entry c.
        double entry = best[0];
#pragma unroll
        for (int k = 1; k < kBest; ++k) entry = c == k ? best[k] : entry;
        if (kGroups == Groups::kAny && K > kBest) {
            // The entries past the eighth, from what is below that one.
            const double last = best[kBest - 1];
#pragma unroll
            for (int v = 0; v < V; ++v) keys[v] = key_of_expert(v);
            close_groups();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const double x = number(v);
                (v < kBest ? best : more)[v % kBest] = x < last ? x : numbered<V>(kNoKey, 0);
            }
#pragma unroll
            for (int v = V; v < kBest; ++v) best[v] = numbered<V>(kNoKey, 0);
            best_of<V>(best, more, number);
#pragma unroll
            for (int k = 0; k < kBest; ++k) entry = c == kBest + k ? best[k] : entry;
        }
        const float high = top == kNoKey ? 0.f : key_value(top);
        if constexpr (!kSigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = exp_nonpositive(s[v] - high);
                sum += s[v];
            }
        }
        sum = row_sum(sum);
        const RowSum all{sum, sum == 0.f ? 0.f : (kSigmoid ? 1.f / sum : reciprocal(sum))};
        const uint32_t key = key_of(entry);
        constexpr uint32_t kMost = (1u << kExpertBits<V>) - 1;
        const int expert = (int)(kMost - ((uint32_t)__builtin_bit_cast(uint64_t, entry) & kMost));
        const int picked = c < K && key != kNoKey ? expert : -1;
        float weight = 0.f;
        if constexpr (kSigmoid) {
            float* const row = mine + lane / kRowLanes * V * kRowLanes;
#pragma unroll
            for (int v = 0; v < V; ++v) row[(v / 4 * kRowLanes + c) * 4 + v % 4] = s[v];
            __builtin_amdgcn_wave_barrier();
            if (picked >= 0) weight = row[quad_slot(picked, E)];
            __builtin_amdgcn_wave_barrier();
        } else {
            weight = picked >= 0 ? exp_nonpositive(key_value(key) - high) * all.inv : 0.f;
        }
        if (p.flags & DISPATCH_GATE_NORMALIZE) {
            const float total = row_sum(weight);
            weight = total == 0.f ? 0.f
                     : kSigmoid   ? p.route_scale * (weight / total)
                                  : p.route_scale * weight * reciprocal(total);
        } else {
            weight *= p.route_scale;
        }
        if (kBalance) {
#pragma unroll
            for (int v = 0; v < V; ++v) prob_sum[v] += kSigmoid ? all.share(s[v]) : s[v] * all.inv;
            live += now && c == 0 ? 1 : 0;
            if (picked >= 0) atomicAdd(counts + picked, 1);
        }
        if (t0 + stride < p.num_tokens) arrive();
        const int64_t t = t0 + lane / kRowLanes;
        if (c < K && t < p.num_tokens) {
            const int64_t at = t * K + c;
            if (p.idx_bytes == 8)
                static_cast<int64_t*>(p.topk_idx)[at] = picked;
            else
                static_cast<int32_t*>(p.topk_idx)[at] = picked;
            p.topk_weights[at] = weight;
        }
    }
    if (!kBalance) return;
    // The wavefront's four rows, then as above.
#pragma unroll
    for (int v = 0; v < V; ++v) {
        prob_sum[v] += __shfl_xor(prob_sum[v], 16);
        prob_sum[v] += __shfl_xor(prob_sum[v], 32);
        if (lane < kRowLanes) mine[(v / 4 * kRowLanes + c) * 4 + v % 4] = prob_sum[v];
    }
    if (c == 0) atomicAdd(counts + E, live);
    __syncthreads();
    float* const out = p.partial + (int64_t)blockIdx.x * (2 * E + 1);
    for (int i = threadIdx.x; i < 2 * E + 1; i += kRowWaves<V> * kWave) {
        float x = __int_as_float(counts[i - E < 0 ? 0 : i - E]);
        if (i < E) {
            const float* at = lds + quad_slot(i, E);
            x = at[0];
#pragma unroll
            for (int w = 1; w < kRowWaves<V>; ++w) x += at[w * kWaveFloats];
        }
        out[i] = x;
    }
}

// Adds the partial rows. A workgroup takes 16 experts: its 64 groups of 16
// threads add every 64th row, then the groups are added in order. Its part of
// the loss goes to the workspace, and the workgroup that finds itself the last
// adds those, in order too. One workgroup for all experts took 22.8 us for
// 256 rows of 256 experts, this form takes 5.3 (512 rows 5.8; kernel times).
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
        // Eight rows on their way at once (past the last: its own, not added).
        constexpr int kAtOnce = 8;
        for (int g = g0; g < groups; g += kAtOnce * kSumGroups) {
            float a[kAtOnce];
            int b[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int row = g + i * kSumGroups < groups ? g + i * kSumGroups : groups - 1;
                a[i] = partial[row * stride + e];
                b[i] = __float_as_int(partial[row * stride + E + e]);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                s += g + i * kSumGroups < groups ? a[i] : 0.f;
                n += g + i * kSumGroups < groups ? b[i] : 0;
            }
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
#pragma unroll
        for (int i = 0; i < kGateMaxGroups / kWave; ++i) {
            const int g = i * kWave + lane;
            const int here = __float_as_int(partial[(g < groups ? g : groups - 1) * stride + 2 * E]);
            live += g < groups ? here : 0;
        }
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
    // The part goes past the caches that XCDs do not share, and has arrived
    // before the ticket is taken: no cache has to be written back for it.
    uint32_t before = 0;
    if (lane == 0) {
        __hip_atomic_store(loss_part + blockIdx.x, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        before = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if ((uint32_t)__builtin_amdgcn_readfirstlane((int)before) != gridDim.x - 1) return;
    // A lane for each part (one lane for all of them: 16 loads in turn).
    double total = 0.0;
    for (unsigned i = lane; i < gridDim.x; i += kWave)
        total += __hip_atomic_load(loss_part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int step = kWave / 2; step > 0; step /= 2) total += __shfl_xor(total, step);
    if (lane != 0) return;
    *live_tokens = live;
    *loss = balance_loss(loss_coef, E, K, live, total);
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
    int32_t idx_bytes;
    uint32_t flags;
    float route_scale;
    float loss_coef;
};

// Gradient of the logits. The row is read again and its scores computed
// again, which is cheaper than storing them. Lane k holds entry k: its
// score's gradient goes through the wavefront's row in LDS to the lane that
// holds the expert. The row and its entries are loaded before anything is
// waited for.
template <int V, bool kHalf, bool kSigmoid>
__global__ void __launch_bounds__(kGateWaves<V> * kWave) gate_backward_kernel(GateBackwardParams p) {
    constexpr int W = kGateWaves<V>;
    extern __shared__ float lds[];  // [W][V * 64]: a token's scores, then their gradients
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int E = p.num_experts, K = p.num_topk;
    float* const row = lds + wave * V * kWave;
    const int64_t stride = (int64_t)gridDim.x * W;
    int64_t t = (int64_t)blockIdx.x * W + wave;
    uint32_t next[V];
    int next_live = 1;
    uint64_t next_id = 0;
    float next_dw = 0.f;
    const int entry = lane < K ? lane : K - 1;
    const auto load = [&](int64_t token) {
        load_row<V, kHalf>(p.logits, token, E, lane, next);
        if (p.mask != nullptr) next_live = p.mask[token];
        if (p.grad_weights != nullptr) {
            const int64_t at = token * K + entry;
            uint64_t id;
            if (p.idx_bytes == 8)
                id = static_cast<const uint64_t*>(p.topk_idx)[at];
            else
                id = static_cast<const uint32_t*>(p.topk_idx)[at];
            next_id = id;
            next_dw = p.grad_weights[at];
        }
    };
    if (t < p.num_tokens) load(t);
    // As in the forward kernel.
    float z[V];
    bool taken = false;
    int e = -1;  // lane k: entry k's expert
    float dw = 0.f;
    const auto arrive = [&] {
        widen_row<V, kHalf>(next, E, lane, z);
        taken = __builtin_amdgcn_readfirstlane(next_live) != 0;
        const bool any = p.grad_weights != nullptr && lane < K && next_id < (uint64_t)E;
        e = any ? (int)next_id : -1;
        dw = any ? next_dw : 0.f;
    };
    float dp[V];  // the loss's gradient of this lane's experts' p: the same for every token
#pragma unroll
    for (int v = 0; v < V; ++v) dp[v] = 0.f;
    if (p.grad_loss != nullptr) {
        const float n = (float)*p.live_tokens;
        const float unit = n == 0.f ? 0.f : *p.grad_loss * (p.loss_coef * (float)E / ((float)K * n * n));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (counts<V>(lane, v, E)) dp[v] = unit * (float)p.expert_count[expert_of<V>(lane, v, E)];
        }
    }
    if (t < p.num_tokens) arrive();
    for (; t < p.num_tokens; t += stride) {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = z[v];
        if (t + stride < p.num_tokens) load(t + stride);
        if (taken) {
            uint32_t top = kNoKey;
            if (!kSigmoid) {
                float high = s[0];
#pragma unroll
                for (int v = 1; v < V; ++v) high = fmaxf(high, s[v]);
                top = wave_max(order_key(high));
            }
            const RowSum row_sum = scores<V, kSigmoid>(s, top);
            // The scores of the taken experts, through the row in LDS.
            write_slots<V>(row, lane, s);
            __builtin_amdgcn_wave_barrier();
            const float mine = e >= 0 ? row[slot_of<V>(e, E)] : 0.f;
            __builtin_amdgcn_wave_barrier();
            // The entry's score's gradient; with sigmoid, times the score,
            // which may be too small a number to be divided by.
            float ds = p.route_scale * dw;
            if (kSigmoid) ds *= mine;
            if (p.flags & DISPATCH_GATE_NORMALIZE) {
                // (Less the gradient of the entry with the largest score, which
                // changes nothing: a lone entry's weight is constant, and its
                // gradient exactly 0. Another entry's gradient may be far larger
                // than all that comes of it, and its rounding would stay.
                // Softmax entries are in descending order of their scores;
                // sigmoid's may be of something else. Looked for there too,
                // 65536 tokens of 256 experts took 26.8 us, 26.0 without.)
                uint64_t first = __ballot(e >= 0) | uint64_t(1) << (kWave - 1);
                if (kSigmoid) first = __ballot(__float_as_uint(mine) == wave_max(__float_as_uint(mine)));
                const int from = __builtin_ctzll(first);
                dw -= __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dw), from));
                const float total = wave_sum(mine);
                if (kSigmoid) {
                    const float part = total == 0.f ? 0.f : mine / total;
                    ds = p.route_scale * part * (dw - wave_sum(dw * part));
                } else {
                    const float mean = wave_sum(dw * mine);
                    ds = total == 0.f ? 0.f : p.route_scale / total * (dw - mean / total);
                }
            }
            const float zero[V] = {};
            write_slots<V>(row, lane, zero);
            __builtin_amdgcn_wave_barrier();
            if (e >= 0) row[slot_of<V>(e, E)] = ds;
            __builtin_amdgcn_wave_barrier();
            float d[V];
            float mean = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[v] = row[lane_slot<V>(lane, v)];
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
                s[v] = kSigmoid ? (d[v] + (dp[v] - mean) * (s[v] * row_sum.inv)) * (1.f - s[v]) : s[v] * (d[v] - mean);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = 0.f;
        }
        if (t + stride < p.num_tokens) arrive();
        store_row<V, kHalf>(p.grad_logits, t, E, lane, s);
    }
}

template <int V, bool kHalf, bool kGrouped>
const void* gate_kernel_of(bool sigmoid, bool balance) {
    if (sigmoid)
        return balance ? (const void*)&gate_kernel<V, kHalf, true, true, kGrouped>
                       : (const void*)&gate_kernel<V, kHalf, true, false, kGrouped>;
    return balance ? (const void*)&gate_kernel<V, kHalf, false, true, kGrouped>
                   : (const void*)&gate_kernel<V, kHalf, false, false, kGrouped>;
}
template <int V>
const void* gate_kernel_of(bool half, bool sigmoid, bool balance, bool grouped) {
    if (grouped) return half ? gate_kernel_of<V, true, true>(sigmoid, balance) : gate_kernel_of<V, false, true>(sigmoid, balance);
    return half ? gate_kernel_of<V, true, false>(sigmoid, balance) : gate_kernel_of<V, false, false>(sigmoid, balance);
}
template <int V, bool kHalf, Groups kGroups>
const void* gate_rows_half(bool sigmoid, bool balance) {
    if (sigmoid)
        return balance ? (const void*)&gate_rows_kernel<V, kHalf, true, true, kGroups>
                       : (const void*)&gate_rows_kernel<V, kHalf, true, false, kGroups>;
    return balance ? (const void*)&gate_rows_kernel<V, kHalf, false, true, kGroups>
                   : (const void*)&gate_rows_kernel<V, kHalf, false, false, kGroups>;
}
template <int V>
const void* gate_rows_of(bool half, bool sigmoid, bool balance, Groups groups) {
    if (groups == Groups::kRuns)
        return half ? gate_rows_half<V, true, Groups::kRuns>(sigmoid, balance)
                    : gate_rows_half<V, false, Groups::kRuns>(sigmoid, balance);
    if constexpr (V * kRowLanes <= kMostAnyExperts)
        if (groups == Groups::kAny)
            return half ? gate_rows_half<V, true, Groups::kAny>(sigmoid, balance)
                        : gate_rows_half<V, false, Groups::kAny>(sigmoid, balance);
    if constexpr (V > 4 && V <= 16)  // (without groups from 65 experts on)
        return half ? gate_rows_half<V, true, Groups::kNone>(sigmoid, balance)
                    : gate_rows_half<V, false, Groups::kNone>(sigmoid, balance);
    return nullptr;
}

template <int V>
const void* gate_backward_of(bool half, bool sigmoid) {
    if (half)
        return sigmoid ? (const void*)&gate_backward_kernel<V, true, true> : (const void*)&gate_backward_kernel<V, true, false>;
    return sigmoid ? (const void*)&gate_backward_kernel<V, false, true> : (const void*)&gate_backward_kernel<V, false, false>;
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

hipError_t launch_gate(const dispatch_gate_problem_t& prob, const dispatch_gate_groups_t* groups_of,
                       const void* logits, const float* select_bias, const uint8_t* token_mask,
                       const dispatch_gate_out_t& out, void* workspace, hipStream_t stream) {
    const int E = prob.num_experts;
    // (All groups open: the choice is the gate's without them.)
    const bool grouped = groups_of != nullptr && groups_of->topk_groups < groups_of->num_groups;
    GateParams p{};
    p.logits = logits;
    p.bias = select_bias;
    p.mask = token_mask;
    p.topk_idx = out.topk_idx;
    p.topk_weights = out.topk_weights;
    p.expert_count = out.expert_count;
    p.prob_sum = out.prob_sum;
    p.live_tokens = out.live_tokens;
    p.loss = out.loss;
    p.loss_coef = prob.loss_coef;
    const GateWorkspace ws = gate_workspace(E);
    uint8_t* const base = static_cast<uint8_t*>(workspace);
    p.partial = reinterpret_cast<float*>(base);
    p.ticket = reinterpret_cast<uint32_t*>(base + ws.ticket);
    p.num_tokens = prob.num_tokens;
    p.num_experts = prob.num_experts;
    p.num_topk = prob.num_topk;
    p.idx_bytes = prob.topk_idx_bytes;
    p.flags = prob.flags;
    p.route_scale = prob.route_scale;
    if (grouped) {
        p.num_groups = groups_of->num_groups;
        p.topk_groups = groups_of->topk_groups;
        p.group_size = E / p.num_groups;
        p.group_pairs = groups_of->score_experts == 2;
    }
    const bool sig = prob.scoring == DISPATCH_GATE_SIGMOID, half = prob.logits_bytes == 2;
    const bool balance = out.loss != nullptr;
    if (prob.num_tokens == 0 && !balance) return hipSuccess;
    const void* kernel;
    // Wavefronts of a workgroup, their tokens, the floats in LDS of each and of all.
    int waves, per_wave, row, extra = 0;
    const bool wide = E > 256;
    const int64_t many =
        (grouped ? wide && balance : sig && prob.num_topk < kFewestSigmoidRounds) ? 2 * kManyTokens : kManyTokens;
    const int fewest = grouped && !wide ? 1 : wide && sig && !balance ? kFewestSigmoidRounds : kFewestRounds;
    const bool runs = p.group_size % 4 == 0 && p.num_groups <= kRowLanes && prob.num_topk <= kBest;
    const Groups form = !grouped ? Groups::kNone : runs ? Groups::kRuns : Groups::kAny;
    const int most = form == Groups::kAny ? kMostRowEntries : kBest;
    const bool rows_form = E >= (grouped ? 4 : 65) && E <= (form == Groups::kAny ? kMostAnyExperts : form == Groups::kRuns ? 512 : 256) &&
                           prob.num_topk >= fewest && prob.num_topk <= most && prob.num_tokens >= many &&
                           (!grouped || p.num_groups <= kMostRowGroups);
    if (grouped) {
        const int lanes = rows_form ? kRowLanes : kWave;
        while ((2 << p.group_lanes) * p.num_groups <= lanes) ++p.group_lanes;
    }
    if (rows_form) {
        const int v = E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : 32;
        waves = v == 32 ? kRowWaves<32> : kRowWaves<16>, per_wave = kRowTokens;
        kernel = v == 4    ? gate_rows_of<4>(half, sig, balance, form)
                 : v == 8  ? gate_rows_of<8>(half, sig, balance, form)
                 : v == 16 ? gate_rows_of<16>(half, sig, balance, form)
                           : gate_rows_of<32>(half, sig, balance, form);
        row = row_floats(v, sig, form);
        extra = sig ? v * kRowLanes : 0;
    } else {
        per_wave = 1;
#define DISPATCH_F(V) gate_kernel_of<V>(half, sig, balance, grouped)
        kernel = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
#define DISPATCH_F(V) kGateWaves<V>
        waves = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
#define DISPATCH_F(V) (V * kWave)
        row = DISPATCH_GATE_BY_V(E, DISPATCH_F);
#undef DISPATCH_F
        // Small workgroups start sooner and spread over more CUs (16 or 1000
        // tokens: 4.7 and 4.5 us, 6.1 and 5.8 with 16 wavefronts); with balance
        // outputs each workgroup leaves a partial row, so there they are large.
        if (!balance) waves = 4;
    }
    // Without balance outputs nothing crosses workgroups and the grid may be
    // as large as the batch.
    const int64_t all = (prob.num_tokens + waves * per_wave - 1) / (waves * per_wave);
    const int groups = balance ? gate_groups(prob.num_tokens, waves * per_wave) : (int)(all < 65536 ? all : 65536);
    const size_t shared = ((size_t)waves * row + extra + (balance ? E + 1 : 0)) * sizeof(float);
    void* args[] = {&p};
    hipError_t err = hipLaunchKernel(kernel, dim3(groups), dim3(waves * kWave), args, shared, stream);
    if (err != hipSuccess || !balance || groups == 1) return err;
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
    p.idx_bytes = prob.topk_idx_bytes;
    p.flags = prob.flags;
    p.route_scale = prob.route_scale;
    p.loss_coef = prob.loss_coef;
    const bool sig = prob.scoring == DISPATCH_GATE_SIGMOID, half = prob.logits_bytes == 2;
    const int E = prob.num_experts;
#define DISPATCH_F(V) gate_backward_of<V>(half, sig)
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
