// The router: the choice of a token's experts from its logits, the balance loss
// with its counts, and the gradient of both with respect to the logits (formulas:
// include/ep.h). A wave has one token; lane i holds the V consecutive experts
// V i .. V i + V - 1 in registers, V a power of two of at least E / 64, so that
// lower lanes hold lower indices.
//
// Order: a key (a binary32 logit, or a binary64 score + bias) is held as an
// unsigned integer that orders as the number does, 0 for an expert that may not
// be chosen. A round takes the highest key of the wave and clears it. Where binary32 keys
// decide a choice of scores they are taken for it; where 64 bits are needed, a key's halves are
// compared one after the other: the higher one decides unless two experts share it.
//
// Bound by instructions, and for few tokens by the launches. 8192 tokens x 256 experts in
// binary32, settled times of single launches, us: choice (sigmoid, bias, 4 of 8 groups) 9.3, loss
// 5.7 and 5.5 (two launches), gradient of both 7.8; 128 tokens: choice 4.5. Calls on end
// overlap a little, 8.9, 10.8, 7.4 and 4.0, and other times in these comments are of those. The
// logits alone take 1.4 us to read (6.1 TB/s).
#include <type_traits>

#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kRouteWaves = 4;  // tokens of a block

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Over the wave, the same in every lane: neighbours, pairs, quads, eights, then
// the four rows of 16 in order.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<0xB1>(v));
    v = max(v, dpp<0x4E>(v));
    v = max(v, dpp<0x141>(v));
    v = max(v, dpp<0x140>(v));
    return max(max(lane_value(v, 0), lane_value(v, 16)), max(lane_value(v, 32), lane_value(v, 48)));
}

__device__ __forceinline__ float wave_sum(float v) {
    v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u)));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)lane_value((uint32_t)(u >> 32), lane) << 32 | lane_value((uint32_t)u, lane)));
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Integers that order as the numbers do; -0 and +0 are equal.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float((u >> 31) ? u & 0x7FFFFFFFu : ~u); }
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(uint64_t u) {
    return __longlong_as_double((long long)((u >> 63) ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}

constexpr float kLowest = -3.402823466e+38f;
constexpr double kLowest64 = -1.7976931348623157e+308;

// The lane's logits of token t; -infinity past the last expert.
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, int f32, int64_t t, int E, int lane, float l[V]) {
    const int e = lane * V;
    const int64_t at = t * E + e;
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = -__builtin_inff();
    if (E % V == 0) {  // whole vectors
        if (e >= E) return;
        if (f32) {
            typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
            const vec x = *(const vec*)((const float*)logits + at);
#pragma unroll
            for (int v = 0; v < V; ++v) l[v] = x[v];
        } else {
            typedef uint16_t vec __attribute__((ext_vector_type(V), aligned(2)));
            const vec x = *(const vec*)((const uint16_t*)logits + at);
#pragma unroll
            for (int v = 0; v < V; ++v) l[v] = bf16_to_f32(x[v]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e + v < E) l[v] = f32 ? ((const float*)logits)[at + v] : bf16_to_f32(((const uint16_t*)logits)[at + v]);
    }
}

template <int V>
__device__ __forceinline__ float wave_max_logit(const float l[V]) {
    float m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);  // drops a NaN
    return unordered(wave_max(ordered(m == m ? m : -__builtin_inff())));
}

// e^x for x <= 0, within four units 2^-24: 2^t of the rounded product t = x log2(e) (the
// instruction's error is one unit of the last place), times the rest of the product.
// Below 2^-160 it is 0, NaN stays.
__device__ __forceinline__ float exp_negative(float x) {
    const float t = x * 1.44269504f;
    const float rest = __builtin_fmaf(x, 1.44269504f, -t) + x * 1.92596303e-8f;  // log2(e) to 48 bits
    const float y = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(rest, 0.693147181f, 1.0f);
    return t < -160.0f ? 0.0f : y;
}

// 1 / (1 + e^-l), and its slope s (1 - s) without the difference. The reciprocal is
// within one unit of the last place.
__device__ __forceinline__ float sigmoid(float l, float* slope) {
    const float e = exp_negative(-fabsf(l)), y = __builtin_amdgcn_rcpf(1.0f + e);
    *slope = e * y * y;
    return l >= 0.0f ? y : e * y;
}

// exp(l - max l) and their sum over the wave. A row of -infinity alone has none.
template <int V>
__device__ __forceinline__ float softmax_terms(const float l[V], float m, float x[V]) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = l[v] == -__builtin_inff() ? 0.0f : exp_negative(l[v] - m);
        sum += x[v];
    }
    return wave_sum(sum);
}

// A token's scores and their sum: softmax's terms (divided by the sum they are the
// scores), or sigmoids with their slopes.
template <int V>
__device__ __forceinline__ float score_terms(int score, const float l[V], float x[V], float slope[V]) {
    if (score == EP_SCORE_SOFTMAX) return softmax_terms<V>(l, wave_max_logit<V>(l), x);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = sigmoid(l[v], &slope[v]);
        sum += x[v];
    }
    return wave_sum(sum);
}

// Where all of a token's sigmoids are tiny their sum, or a ratio to it, may underflow, and the
// shares would be lost. Below 2^-26 a sigmoid is e^l to less than half a unit, so the shares are
// those of softmax. Such a token is told by its sum, and its shares are taken apart at the end, from
// logits that are read again, so that all others pay for a comparison (balance loss of 8192 x
// 256 10.7 us, with a branch at each token 11.1; gradient 7.3, with the logits kept in registers 7.4).
// Softmax has a sum that small for rows of -infinity alone, whose shares are 0.
constexpr float kFaint = 1.4901161e-8f;  // 2^-26

template <int V>
__device__ __forceinline__ void faint_shares(const void* logits, int f32, int64_t t, int E, int lane, float p[V]) {
    float l[V];
    load_logits<V>(logits, f32, t, E, lane, l);
    const float sum = softmax_terms<V>(l, wave_max_logit<V>(l), p);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= inv;
}

// Orders the LDS accesses of a wave's lanes for the compiler; the hardware keeps them
// in order.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------- choice

// The highest of the wave's keys with its lowest index, which is cleared; false
// when none is left. FULL: keys of 64 bits (hi, lo), otherwise hi alone. Which experts
// have it is known in scalar registers, so most of a round is scalar work beside the
// vector unit: three maxima, four steps over a row of 16, and two operations an expert.
struct Taken {
    uint32_t hi;
    int lane, v;  // where, the same in every lane
};

template <int V, bool FULL>
__device__ __forceinline__ bool take_highest(uint32_t hi[V], const uint32_t lo[V], Taken* t) {
    uint32_t m = hi[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max(m, hi[v]);
    t->hi = wave_max(m);
    if (t->hi == 0) return false;
    uint64_t have[V], any = 0;
    int count = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        have[v] = ballot64(hi[v] == t->hi);
        any |= have[v];
        count += __builtin_popcountll(have[v]);
    }
    if (FULL && count > 1) {  // the lower halves decide
        uint32_t n = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) n = hi[v] == t->hi ? max(n, lo[v]) : n;
        n = wave_max(n);
        any = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            have[v] &= ballot64(lo[v] == n);
            any |= have[v];
        }
    }
    t->lane = __builtin_ctzll(any);
    t->v = 0;
#pragma unroll
    for (int v = V - 1; v > 0; --v) t->v = (have[v] >> t->lane) & 1 ? v : t->v;
    t->v = have[0] >> t->lane & 1 ? 0 : t->v;
    const bool mine = lane_id() == t->lane;
#pragma unroll
    for (int v = 0; v < V; ++v) hi[v] = mine && v == t->v ? 0u : hi[v];
    return true;
}

// A group's key from its highest (first > 0) and second highest; 0: none.
__device__ __forceinline__ uint64_t group_key(uint64_t first, uint64_t second, int best) {
    if (best < 2 || second == 0) return first;
    const double sum = unordered(first) + unordered(second);
    return ordered(sum < kLowest64 ? kLowest64 : sum);
}

// The two highest of two pairs, each in order.
__device__ __forceinline__ void merge_pairs(uint64_t* first, uint64_t* second, uint64_t a, uint64_t b) {
    const bool more = a > *first;
    const uint64_t low = more ? *first : a, high = more ? b : *second;
    *first = more ? a : *first;
    *second = low > high ? low : high;
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
    return (uint64_t)dpp<CTRL>((uint32_t)(v >> 32)) << 32 | dpp<CTRL>((uint32_t)v);
}

// Clears the keys of the experts outside the best groups. Groups that are no power of two of
// whole lanes take one maximum over the wave after another, and no binary32 keys: 8192 tokens, us,
// sigmoids and a bias, 4 of 8 groups by two experts each, top-6: 96 experts 18.9, 192 26.0, 384 42.4,
// where 256, whose groups are, take 8.2; 160 in 8, by one expert each, 19.7, as softmax
// without a bias 12.5.
template <int V, bool FULL>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, int lane, uint32_t hi[V], const uint32_t lo[V]) {
    const int size = a.E / a.G;
    if (a.group_lanes > 0) {
        // A group is a power of two of whole lanes: pairs of its highest keys are merged
        // over them, and every lane ranks its own group.
        const int lanes = a.group_lanes;
        uint64_t first = 0, second = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) merge_pairs(&first, &second, (uint64_t)hi[v] << 32 | (FULL ? lo[v] : 0u), 0);
        if (lanes > 1) merge_pairs(&first, &second, dpp64<0xB1>(first), dpp64<0xB1>(second));
        if (lanes > 2) merge_pairs(&first, &second, dpp64<0x4E>(first), dpp64<0x4E>(second));
        if (lanes > 4) merge_pairs(&first, &second, dpp64<0x141>(first), dpp64<0x141>(second));
        if (lanes > 8) merge_pairs(&first, &second, dpp64<0x140>(first), dpp64<0x140>(second));
        if (lanes > 16) merge_pairs(&first, &second, __shfl_xor(first, 16, kWave), __shfl_xor(second, 16, kWave));
        if (lanes > 32) merge_pairs(&first, &second, __shfl_xor(first, 32, kWave), __shfl_xor(second, 32, kWave));
        const uint64_t key = group_key(first, second, FULL ? a.best : 1);
        // groups that come first: each lane of a group asks about one of them
        int before = 0;
        const int mine = lane & (lanes - 1), base = lane - mine;
        const uint64_t own = lanes < 64 ? (1ull << lanes) - 1 : ~0ull;
        for (int g0 = 0; g0 < a.G; g0 += lanes) {
            const int g = g0 + mine, at = min(g, a.G - 1) * lanes;
            const uint64_t other = __shfl(key, at, kWave);
            const bool ahead = g < a.G && (other > key || (other == key && at < base));
            before += __popcll((ballot64(ahead) >> base) & own);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) hi[v] = before < a.keep ? hi[v] : 0u;
        return;
    }
    uint32_t group_hi[1] = {0u}, group_lo[1] = {0u};  // lane g: group g's
    for (int g = 0; g < a.G; ++g) {
        uint32_t h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            h[v] = e >= g * size && e < (g + 1) * size ? hi[v] : 0u;
        }
        const auto taken = [&]() -> uint64_t {
            Taken t;
            if (!take_highest<V, FULL>(h, lo, &t)) return 0;
            uint32_t low = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) low = FULL && v == t.v ? lane_value(lo[v], t.lane) : low;
            return (uint64_t)t.hi << 32 | low;
        };
        const uint64_t first = taken();
        if (first == 0) continue;
        const uint64_t key = group_key(first, FULL && a.best == 2 ? taken() : 0, FULL ? a.best : 1);
        if (lane == g) {
            group_hi[0] = (uint32_t)(key >> 32);
            group_lo[0] = (uint32_t)key;
        }
    }
    uint64_t kept = 0;
    for (int i = 0; i < a.keep; ++i) {
        Taken t;
        if (!take_highest<1, FULL>(group_hi, group_lo, &t)) break;
        kept |= 1ull << t.lane;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (!((kept >> min((lane * V + v) / size, 63)) & 1)) hi[v] = 0u;
}

// The choice from binary32 keys, where they decide it. Scores: each is off by at most
// `err`, and every comparison that the choice rests on has to be clearer than what its two
// sides can be off by. Where a group's is not: false, and keys of 64 bits choose. Where an
// expert's is not (among them any tie), those that may be chosen are ranked by their keys
// of 64 bits, one a lane; false with a softmax, whose scores take the whole row. Otherwise
// (SCORES false) the keys are the logits. Lane j < k gets the j-th choice and its score (or
// logit); `out`: the wave's LDS. About one token in 1,000 has an unclear choice (sigmoids of 256
// logits, top-8), and a wave that takes both ways ends late. 8192 tokens, us, with this
// first and without it: sigmoids and a bias, 256 experts in 8 groups 8.9, 12.0; 384 experts
// 12.1, 17.3; softmax and a bias, 160 experts 9.1, 10.3; logits, 1024 experts 16.8, 23.7, 256
// of them 8.1, 8.9; but of 128 experts 7.2, 6.9, with softmax and a bias (4096 tokens) 6.2,
// 5.7, with sigmoids 6.8, 7.5, and 64 5.2, 4.9: so from 4 experts a lane on.
constexpr int kNarrowFrom = 4;

struct Choice {
    int e;
    float s;
};

// Descending (Batcher's odd-even merges).
template <int V>
__device__ __forceinline__ void sort_down(uint32_t h[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int d = p; d >= 1; d /= 2)
#pragma unroll
            for (int i = d % p; i + d < V; ++i) {
                if ((i - d % p) % (2 * d) >= d || i / (2 * p) != (i + d) / (2 * p)) continue;
                const uint32_t x = h[i], y = h[i + d];
                h[i] = max(x, y);
                h[i + d] = min(x, y);
            }
}

__device__ __forceinline__ double score64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

template <int V, bool SCORES>
__device__ __forceinline__ bool choose_narrow(const RouteArgs& a, int lane, const float l[V], const float s[V],
                                              const float b[V], const bool open[V], float err, Choice* out,
                                              Choice* mine) {
    constexpr float kUnit = 5.9604645e-8f;    // 2^-24
    constexpr uint32_t kLeast = 0x00400000u;  // half of ordered(kLowest): what lies below is no key
    uint32_t h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float key = SCORES ? s[v] + b[v] : s[v];
        h[v] = open[v] ? ordered(key >= kLowest ? key : kLowest) : 0u;
    }
    if (a.G > 1) {
        const int lanes = a.group_lanes;
        uint32_t first = 0, second = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            second = max(second, min(first, h[v]));
            first = max(first, h[v]);
        }
        const auto merge = [&](uint32_t f, uint32_t n) {
            second = max(max(second, n), min(first, f));
            first = max(first, f);
        };
        if (lanes > 1) merge(dpp<0xB1>(first), dpp<0xB1>(second));
        if (lanes > 2) merge(dpp<0x4E>(first), dpp<0x4E>(second));
        if (lanes > 4) merge(dpp<0x141>(first), dpp<0x141>(second));
        if (lanes > 8) merge(dpp<0x140>(first), dpp<0x140>(second));
        if (lanes > 16) merge(__shfl_xor(first, 16, kWave), __shfl_xor(second, 16, kWave));
        if (lanes > 32) merge(__shfl_xor(first, 32, kWave), __shfl_xor(second, 32, kWave));
        // two keys, each off by its score's error and a unit; a unit of their sum, one of each end
        const bool two = a.best > 1 && second != 0;
        const float f = unordered(first), n = two ? unordered(second) : 0.0f;
        const float off = SCORES ? 2.0f * err + 4.0f * kUnit * (fabsf(f) + fabsf(n)) : 0.0f;
        const float low = first != 0 ? (f + n) - off : -__builtin_inff(), high = first != 0 ? (f + n) + off : -__builtin_inff();
        // groups that come first for sure, and that may; each lane of a group asks about one
        int before = 0, maybe = 0;
        const int at_group = lane & (lanes - 1), base = lane - at_group;
        const uint64_t own = lanes < 64 ? (1ull << lanes) - 1 : ~0ull;
        for (int g0 = 0; g0 < a.G; g0 += lanes) {
            const int g = g0 + at_group, at = min(g, a.G - 1) * lanes;
            const float other_low = __shfl(low, at, kWave), other_high = __shfl(high, at, kWave);
            const bool other = g < a.G && at != base;
            const uint64_t ahead = ballot64(other && (other_low > high || (!SCORES && other_low == high && at < base)));
            before += __popcll((ahead >> base) & own);
            if (SCORES) maybe += __popcll((ballot64(other && !(other_high < low)) >> base) & own);
            else maybe = before;
        }
        if (ballot64(first != 0 && maybe >= a.keep && before < a.keep) != 0) return false;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = maybe < a.keep ? h[v] : 0u;
    }
    // A key's lowest bits make way for the expert's place in its lane, which moves it by less
    // than V units of its last place (two units 2^-24 each, at most); those of a bf16 logit
    // hold nothing, and make way for its whole index, counted down. Each lane's keys are
    // sorted; a round takes the highest of the lanes' first ones.
    const bool exact = !SCORES && !a.f32;
    const float unit = (2 * V + 2) * kUnit;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (exact) {
            const uint32_t key = s[v] == s[v] ? h[v] : h[v] / 2;  // NaN lies below the lowest bf16 number, too
            h[v] = (key & 0xFFFF0000u) | (uint32_t)(0xFFFF - (lane * V + v));
        } else {
            h[v] = (h[v] & ~(uint32_t)(V - 1)) | (uint32_t)(V - 1 - v);
        }
    }
    sort_down<V>(h);
    uint32_t best = 0, chosen = 0;  // lane j: the j-th key, its expert
    const auto take = [&](int n) -> uint32_t {
        const uint32_t m = wave_max(h[0]);
        if (m < kLeast) return 0;
        const int from = __builtin_ctzll(ballot64(h[0] == m));
        const bool now = lane == n, here = lane == from;
        best = now ? m : best;
        const uint32_t e = exact ? 0xFFFF - (m & 0xFFFF) : (uint32_t)from * V + (V - 1 - (m & (V - 1)));
        chosen = now ? e : chosen;
#pragma unroll
        for (int v = 0; v < V - 1; ++v) h[v] = here ? h[v + 1] : h[v];
        h[V - 1] = here ? 0u : h[V - 1];
        return m;
    };
    // whether the higher key of two may be the lower one in truth
    const auto unclear = [&](float x, float y) { return !(x - y > 2.0f * err + unit * (fabsf(x) + fabsf(y))); };
    int n = 0;  // the first one that is not chosen is looked at, too
    while (n < a.k + (exact ? 0 : 1) && take(n) != 0) ++n;
    const uint32_t next = __shfl(best, (lane + 1) & (kWave - 1), kWave);
    const bool close = !exact && lane < a.k && next != 0 && unclear(unordered(best), unordered(next));
    int place = lane;
    if (ballot64(close) != 0) {
        if (SCORES && a.score == EP_SCORE_SOFTMAX) return false;
        // all that may belong to the first k
        const float last = unordered(lane_value(best, a.k - 1));
        while (n > a.k && unclear(last, unordered(lane_value(best, n - 1)))) {
            if (n == kWave) return false;
            if (take(n) == 0) break;
            ++n;
        }
        float x = 0.0f, y = 0.0f;
        const int at = (int)chosen;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float lv = __shfl(l[v], at / V, kWave), bv = SCORES ? __shfl(b[v], at / V, kWave) : 0.0f;
            x = v == at % V ? lv : x;
            y = v == at % V ? bv : y;
        }
        constexpr double kLeastKey = SCORES ? kLowest64 : (double)kLowest;  // of keys of this type: the NaN's
        double key = SCORES ? score64(x) + (double)y : (double)x;
        if (!(key >= kLeastKey)) key = kLeastKey;
        place = 0;
        for (int i = 0; i < n; ++i) {
            const double other = lane_value(key, i);
            const int e = (int)lane_value(chosen, i);
            place += other > key || (other == key && e < at);
        }
    }
    // the scores from the lanes that hold them
    float score = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = __shfl(s[v], (int)chosen / V, kWave);
        score = v == (int)chosen % V ? x : score;
    }
    if (ballot64(close) == 0) {
        if (lane < min(n, a.k)) *mine = Choice{(int)chosen, score};
        return true;
    }
    if (lane < n && place < a.k) out[place] = Choice{(int)chosen, score};
    wave_lds_fence();
    if (lane < min(n, a.k)) *mine = out[lane];
    return true;
}

// FULL: keys are scores + bias, in binary64 where binary32 does not decide; otherwise logits.
template <int V, bool FULL>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(RouteArgs a) {
    __shared__ Choice s_choice[kRouteWaves][kMaxTopk];
    const int lane = lane_id();
    const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kRouteWaves + (threadIdx.x >> 6));
    if (t >= a.T) return;
    int chosen = -1;  // lane j < k: the j-th choice and its weight
    float w = 0.0f;
    if (a.mask == nullptr || a.mask[t] != 0) {
        float l[V], s[V];
        load_logits<V>(a.logits, a.f32, t, a.E, lane, l);
        float max_l = 0.0f, sum = 1.0f;
        Choice mine = {-1, 0.0f};
        const bool narrow = V >= kNarrowFrom && a.narrow;
        if (a.score == EP_SCORE_SOFTMAX) {
            max_l = wave_max_logit<V>(l);
            if (!FULL || narrow) sum = softmax_terms<V>(l, max_l, s);
        }
        float b[V], err = 1e-37f;  // of logits: for those around 0, whose units are no part of them
        bool open[V];
        if (FULL && narrow && a.score == EP_SCORE_SOFTMAX) {
            // The weighted mean of max l - l, which the arguments' roundings count with, is at
            // most log 1024, and x e^-x less than 0.4: in units 2^-24 of the largest score, a
            // term is off by 5, the sum by 7 + 4 + 22, the quotients by 3.
            const float inv = 1.0f / sum;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= inv;
            err = 3.8146973e-6f * inv;  // 64 units
        } else if (FULL && narrow) {
            float slope;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = sigmoid(l[v], &slope);
            err = 3.5762787e-7f;  // 6 units: 10 of a score below a half, 5 of the others
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            b[v] = FULL && a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
            open[v] = l[v] != -__builtin_inff() && b[v] != -__builtin_inff();
            if (!FULL) s[v] = l[v];
        }
        bool decided = false;
        if (narrow)
            decided = choose_narrow<V, FULL>(a, lane, l, s, b, open, err, s_choice[threadIdx.x >> 6], &mine);
        if (!decided) {
            uint32_t hi[V], lo[V];
            if (FULL) {
                double score[V];
                if (a.score == EP_SCORE_SOFTMAX) {
                    double d = 0.0;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        score[v] = l[v] == -__builtin_inff() ? 0.0 : exp((double)l[v] - (double)max_l);
                        d += score[v];
                    }
                    d = wave_sum(d);
#pragma unroll
                    for (int v = 0; v < V; ++v) score[v] /= d;
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) score[v] = score64(l[v]);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    double key = score[v] + (double)b[v];
                    if (!(key >= kLowest64)) key = kLowest64;  // NaN
                    if (!narrow) s[v] = (float)score[v];
                    const uint64_t o = open[v] ? ordered(key) : 0ull;
                    hi[v] = (uint32_t)(o >> 32);
                    lo[v] = (uint32_t)o;
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) hi[v] = open[v] ? ordered(l[v] >= kLowest ? l[v] : kLowest) : 0u;
            }
            if (a.G > 1) keep_groups<V, FULL>(a, lane, hi, lo);
            for (int j = 0; j < a.k; ++j) {
                Taken p;
                if (!take_highest<V, FULL>(hi, lo, &p)) break;
                mine.e = lane == j ? p.lane * V + p.v : mine.e;
            }
            // the chosen experts' scores (or logits) from the lanes that hold them
            const int at = max(mine.e, 0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float x = __shfl(s[v], at / V, kWave);
                mine.s = mine.e >= 0 && v == at % V ? x : mine.s;
            }
        }
        chosen = mine.e;
        w = mine.s;
        if (!FULL && chosen >= 0) {
            float slope;
            w = a.score == EP_SCORE_SOFTMAX ? exp_negative(w - max_l) / sum : sigmoid(w, &slope);
        }
        if (a.renormalize) {
            const float total = wave_sum(w) + 1e-20f;
            w /= total;
        }
        w *= a.scale;
    }
    if (lane >= a.k) return;
    const int64_t at = (int64_t)t * a.k + lane;
    if (a.idx_bits == 64) ((int64_t*)a.idx)[at] = chosen;
    else ((int32_t*)a.idx)[at] = chosen;
    a.w[at] = chosen >= 0 ? w : 0.0f;
}

// ---------------------------------------------------------------- balance loss

// Id j of token t, -1 where it is none of the E experts.
__device__ __forceinline__ int load_id(const void* idx, int idx_bits, int64_t at, int E) {
    if (idx_bits == 64) {
        const int64_t i = ((const int64_t*)idx)[at];
        return i >= 0 && i < E ? (int)i : -1;
    }
    const int32_t i = ((const int32_t*)idx)[at];
    return i >= 0 && i < E ? i : -1;
}

// The first sequence whose end lies past token t (S: none), the same in every lane: the
// wave asks about 64 ends at a time, a 64th of the rest each.
__device__ __forceinline__ int sequence_past(const int32_t* off, int S, int t) {
    int lo = 0, n = S;
    while (n > 0) {
        const int step = (n + 63) / 64, at = lane_id() * step;
        const bool behind = at < n && off[lo + min(at + step, n)] <= t;
        const int c = __builtin_popcountll(ballot64(behind)) * step;
        lo += min(c, n);
        if (step == 1) break;
        n = min(step, n - c);
    }
    return lo;
}

// Tile b (a.tile tokens) by sequence q: a piece of its own at place b + q of the
// partial sums. The pieces of a batch run from (0, 0) up in b or in q, never both,
// so places are distinct. A wave has 2 tokens in flight (4 where 16 waves' sums do not fit
// into LDS); their shares are added in binary32, and those sums in binary64 over the piece. A
// wave's sum is rounded to binary32, which halves its LDS, and so are the waves' sums added: shares
// are positive, so that is off by at most kWaves units 2^-24 of the sum, however long the
// piece. Pieces are added in binary64. 16 waves, 8, 4
// for the 32 tokens of a turn: the batch of 8192 x 256 takes 12.2, 12.8, 15.1 us.
template <int V>
constexpr int kBalanceWaves = V <= 8 ? 16 : 8;

template <int V>
__global__ __launch_bounds__(64 * kBalanceWaves<V>) void k_balance_pieces(BalanceArgs a) {
    constexpr int kWaves = kBalanceWaves<V>, kAhead = kBalanceTurn / kWaves;
    __shared__ float s_sum[kWaves][64 * V];
    __shared__ int s_count[64 * V];
    __shared__ int s_tokens;
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = (int)blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.T);
    if (blockIdx.x == 0 && tid == 0) *a.done = 0;
    int q = a.seq_off != nullptr ? sequence_past(a.seq_off, a.S, t0) : 0;
    for (int at = t0; q < a.S && at < t1; ++q) {
        int from = t0, to = t1;
        if (a.seq_off != nullptr) {
            int end = a.seq_off[q + 1];
            if (end <= at) {  // empty: on to the next one that ends behind this place
                q = max(q, sequence_past(a.seq_off, a.S, at));  // never back, whatever seq_off holds
                if (q >= a.S) break;
                end = a.seq_off[q + 1];
            }
            const int first = a.seq_off[q];
            if (first >= t1) break;
            from = max(t0, first);
            to = min(t1, end);
        }
        at = max(at, to);
        if (from >= to) continue;
        for (int e = tid; e < 64 * V; e += 64 * kWaves) s_count[e] = 0;
        if (tid == 0) s_tokens = 0;
        __syncthreads();
        double sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = 0.0;
        int tokens = 0;
        uint64_t faint = 0;  // whether a token's sigmoids were all tiny
        for (int t = from + wave; t < to; t += kAhead * kWaves) {
            int id[kAhead];
            float l[kAhead][V];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int u = t + i * kWaves;
                id[i] = -1;
                if (u >= to) continue;
                if (lane < a.k) id[i] = load_id(a.idx, a.idx_bits, (int64_t)u * a.k + lane, a.E);
                load_logits<V>(a.logits, a.f32, u, a.E, lane, l[i]);
            }
            float part[V];
#pragma unroll
            for (int v = 0; v < V; ++v) part[v] = 0.0f;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (ballot64(id[i] >= 0) == 0) continue;
                if (id[i] >= 0) atomicAdd(&s_count[id[i]], 1);
                ++tokens;
                float x[V], slope[V];
                const float total = score_terms<V>(a.score, l[i], x, slope);
                const float inv = total < kFaint ? 0.0f : 1.0f / total;
                faint |= ballot64(total < kFaint);
#pragma unroll
                for (int v = 0; v < V; ++v) part[v] += x[v] * inv;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] += (double)part[v];
        }
        if (__builtin_expect(faint != 0, 0)) {  // such tokens again, in order
#pragma unroll 1
            for (int t = from + wave; t < to; t += kWaves) {
                const int id = load_id(a.idx, a.idx_bits, (int64_t)t * a.k + min(lane, a.k - 1), a.E);
                float x[V], slope[V];
                load_logits<V>(a.logits, a.f32, t, a.E, lane, x);
                const float total = score_terms<V>(a.score, x, x, slope);
                if (ballot64(id >= 0) == 0 || ballot64(total < kFaint) == 0) continue;
                faint_shares<V>(a.logits, a.f32, t, a.E, lane, x);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[v] += (double)x[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s_sum[wave][lane * V + v] = (float)sum[v];
        if (lane == 0 && tokens > 0) atomicAdd(&s_tokens, tokens);
        __syncthreads();
        const int64_t place = (int64_t)blockIdx.x + q;
        for (int e = tid; e < a.E; e += 64 * kWaves) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) total += s_sum[i][e];
            a.sums[place * a.E + e] = total;
            a.pairs[place * a.E + e] = s_count[e];
        }
        if (tid == 0) a.tokens[place] = s_tokens;
        __syncthreads();
    }
}

// 64 experts of one sequence a block: their counts, and their part of the sequence's
// term. The block that comes last (a count that the first kernel cleared) adds the
// parts in order, so that nothing depends on which one that is. What passes between blocks
// are atomic stores and loads at agent scope, which go past the caches that blocks do not
// share, so that waiting for the stores orders them before the count; a release would
// write the whole L2 back first (the batch of 8192 x 256: 12.2 us for 10.7). The language does
// not order relaxed accesses: the instructions that they become do, which
// tests/test_balance_order.py reads, so none of them may become a plain one.
__global__ __launch_bounds__(1024) void k_balance_loss(BalanceArgs a) {
    __shared__ double s_sum[16][64];
    __shared__ int s_pairs[16][64];
    __shared__ int s_tokens[16];
    __shared__ int s_last;
    const int tid = threadIdx.x, x = tid & 63, y = tid >> 6;
    const int q = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, e = chunk * 64 + x;
    int from = 0, to = a.T;
    if (a.seq_off != nullptr) {
        from = max(0, a.seq_off[q]);
        to = min(a.T, a.seq_off[q + 1]);
    }
    const int b0 = from / a.tile, b1 = from < to ? (to - 1) / a.tile + 1 : b0;
    double sum = 0.0;
    int pairs = 0, tokens = 0;
    const int column = min(e, a.E - 1);
#pragma unroll 8
    for (int b = b0 + y; b < b1; b += 16) {
        const int64_t at = ((int64_t)b + q) * a.E + column;
        sum += (double)a.sums[at];
        pairs += a.pairs[at];
        tokens += a.tokens[b + q];
    }
    if (e >= a.E) {
        sum = 0.0;
        pairs = 0;
    }
    s_sum[y][x] = sum;
    s_pairs[y][x] = pairs;
    if (x == 0) s_tokens[y] = tokens;
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            sum += s_sum[i][x];
            pairs += s_pairs[i][x];
            tokens += s_tokens[i];
        }
        if (e < a.E) a.counts[(int64_t)q * a.E + e] = pairs;
        sum = wave_sum((double)pairs * sum);
        if (x == 0) {
            __hip_atomic_store(&a.term[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (chunk == 0) __hip_atomic_store(&a.routed[q], tokens, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    // sequences over the lanes of one wave, or of all waves where there are many
    const int threads = a.S <= 64 ? 64 : 1024;
    if (tid >= threads) return;
    const double k = (double)a.k, E = (double)a.E;
    double used = 0.0, loss = 0.0, unit = 0.0;  // unit: of this thread's only sequence, where it has one
    for (int s = tid; s < a.S; s += threads) {
        const int n = __hip_atomic_load(&a.routed[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        double term = 0.0;
#pragma unroll 4
        for (int c = 0; c < a.chunks; ++c)
            term += __hip_atomic_load(&a.term[s * a.chunks + c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        unit = n > 0 ? E / (k * (double)n * (double)n) : 0.0;
        used += n > 0 ? 1.0 : 0.0;
        loss += n > 0 ? unit * term : 0.0;
    }
    used = wave_sum(used);
    loss = wave_sum(loss);
    if (threads > 64) {  // the waves' sums, in order
        if (x == 0) {
            s_sum[0][y] = used;
            s_sum[1][y] = loss;
        }
        __syncthreads();
        used = loss = 0.0;
        for (int i = 0; i < 16; ++i) {
            used += s_sum[0][i];
            loss += s_sum[1][i];
        }
    }
    if (used < 1.0) used = 1.0;
    if (tid == 0) a.loss[0] = (float)(loss / used);
    for (int s = tid; s < a.S; s += threads) {
        if (a.S > threads) {
            const int n = __hip_atomic_load(&a.routed[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            unit = n > 0 ? E / (k * (double)n * (double)n) : 0.0;
        }
        a.coef[s] = (float)(unit / used);
    }
}

// ---------------------------------------------------------------- gradient

template <int V>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_backward(RouteBackwardArgs a) {
    __shared__ int s_pairs[kRouteWaves][64 * V];
    __shared__ float s_grads[kRouteWaves][64 * V];
    const int lane = lane_id();
    const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kRouteWaves + (threadIdx.x >> 6));
    if (t >= a.T) return;
    float grad[V];
#pragma unroll
    for (int v = 0; v < V; ++v) grad[v] = 0.0f;
    // all that depends on nothing is on its way before anything is waited for
    float l[V];
    load_logits<V>(a.logits, a.f32, t, a.E, lane, l);
    const int64_t slot = (int64_t)t * a.k + min(lane, a.k - 1);
    int id = load_id(a.idx, a.idx_bits, slot, a.E);
    float gw = a.grad_w != nullptr ? a.grad_w[slot] : 0.0f;
    int q = 0;
    bool in = a.counts != nullptr;
    if (in && a.seq_off != nullptr) {
        q = sequence_past(a.seq_off, a.S, t);
        in = q < a.S && a.seq_off[q] <= t;
    }
    int32_t pairs_of[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pairs_of[v] = in ? a.counts[(int64_t)q * a.E + min(lane * V + v, a.E - 1)] : 0;
    if (lane >= a.k) {
        id = -1;
        gw = 0.0f;
    }
    if (ballot64(id >= 0) != 0) {
        float s[V], slope[V], u[V], b[V];
        int n[V];
        const bool softmax = a.score == EP_SCORE_SOFTMAX;
        const float total = score_terms<V>(a.score, l, s, slope);
        const bool faint = ballot64(total < kFaint) != 0;
        const float inv = faint ? 0.0f : 1.0f / total;  // the loss's part is 0 here then
        if (softmax) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= inv;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            u[v] = b[v] = 0.0f;
            n[v] = 0;
        }
        if (a.grad_w != nullptr) {
            // scattered through the wave's own LDS, whose accesses stay in order; an expert
            // that a token names twice has its gradients added in order instead
            int* const pairs = s_pairs[threadIdx.x >> 6];
            float* const grads = s_grads[threadIdx.x >> 6];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                pairs[lane * V + v] = 0;
                grads[lane * V + v] = 0.0f;
            }
            wave_lds_fence();
            if (id >= 0) atomicAdd(&pairs[id], 1);
            if (id >= 0) grads[id] = gw;
            wave_lds_fence();
            const uint64_t twice = ballot64(id >= 0 && pairs[id] > 1);
            if (twice != 0) {
                for (int j = 0; j < a.k; ++j) {
                    if (!((twice >> j) & 1)) continue;
                    const int e = (int)lane_value((uint32_t)id, j);
                    float sum = 0.0f;
                    for (int i = 0; i < a.k; ++i) sum += (int)lane_value((uint32_t)id, i) == e ? lane_value(gw, i) : 0.0f;
                    if (lane == j) grads[e] = sum;
                }
                wave_lds_fence();
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                n[v] = pairs[lane * V + v];
                u[v] = grads[lane * V + v];
            }
            if (a.renormalize) {
                float d = 0.0f, q = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d += (float)n[v] * s[v];
                    q += u[v] * s[v];
                }
                const float named = wave_sum(d), sum = named + 1e-20f;
                d = 1.0f / sum;  // one quotient; its products are off by a unit more
                q = wave_sum(q) * d;
                // An expert that is named alone has a share that only 1e-20 keeps from 1. The difference
                // below would be what rounding leaves of it: the share's rest times g instead.
                const int alone = (int)lane_value((uint32_t)id, __builtin_ctzll(ballot64(id >= 0)));
                if (ballot64(id >= 0 && id != alone) == 0) {
                    const float rest = sum == named ? 0.0f : 1e-20f * d;
#pragma unroll
                    for (int v = 0; v < V; ++v) u[v] = n[v] > 0 ? a.scale * (u[v] * rest * d) : 0.0f;
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) u[v] = n[v] > 0 ? a.scale * ((u[v] - (float)n[v] * q) * d) : 0.0f;
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) u[v] *= a.scale;
            }
        }
        if (in) {
            // A constant added to every b changes nothing, and counts of a balanced
            // batch are nearly equal: the first one goes out exactly, as an integer.
            const float f = a.grad_loss[0] * a.coef[q];
            const int first = __builtin_amdgcn_readfirstlane(pairs_of[0]);
            float mean = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane * V + v;
                b[v] = e < a.E ? f * (float)(pairs_of[v] - first) : 0.0f;
                mean += s[v] * b[v];
            }
            mean = wave_sum(mean);
            if (softmax) {
#pragma unroll
                for (int v = 0; v < V; ++v) b[v] -= mean;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) b[v] = (b[v] - mean * inv) * inv;
            }
        }
        if (softmax) {
            float mean = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                u[v] += b[v];
                mean += s[v] * u[v];
            }
            mean = wave_sum(mean);
#pragma unroll
            for (int v = 0; v < V; ++v) grad[v] = s[v] * (u[v] - mean);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) grad[v] = slope[v] * (u[v] + b[v]);
            if (__builtin_expect(in && faint, 0)) {  // p (1 - s) (b - sum p b), and 1 - s is 1
                float p[V], c[V], mean = 0.0f;
                faint_shares<V>(a.logits, a.f32, t, a.E, lane, p);
                const int32_t* const row = a.counts + (int64_t)q * a.E;
                const float f = a.grad_loss[0] * a.coef[q];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    c[v] = f * (float)(row[min(lane * V + v, a.E - 1)] - row[0]);
                    mean += p[v] * c[v];
                }
                mean = wave_sum(mean);
#pragma unroll
                for (int v = 0; v < V; ++v) grad[v] += p[v] * (c[v] - mean);
            }
        }
    }
    const int e = lane * V;
    const int64_t at = (int64_t)t * a.E + e;
    if (a.E % V == 0) {
        if (e >= a.E) return;
        if (a.f32) {
            typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
            vec x;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = grad[v];
            *(vec*)((float*)a.grad + at) = x;
        } else {
            typedef uint16_t vec __attribute__((ext_vector_type(V), aligned(2)));
            vec x;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = (uint16_t)pack_bf16x2(grad[v], 0.0f);
            *(vec*)((uint16_t*)a.grad + at) = x;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (e + v >= a.E) continue;
        if (a.f32) ((float*)a.grad)[at + v] = grad[v];
        else ((uint16_t*)a.grad)[at + v] = (uint16_t)pack_bf16x2(grad[v], 0.0f);
    }
}

// Calls f with V as a template argument: the smallest power of two of at least E / 64.
template <class F>
void for_experts(int E, F f) {
    if (E <= 64) f(std::integral_constant<int, 1>());
    else if (E <= 128) f(std::integral_constant<int, 2>());
    else if (E <= 256) f(std::integral_constant<int, 4>());
    else if (E <= 512) f(std::integral_constant<int, 8>());
    else f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    int V = 1;  // experts of a lane
    while (64 * V < a.E) V *= 2;
    const int size = a.E / a.G, lanes = size / V;
    a.group_lanes = size % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const bool full = a.bias != nullptr || a.best > 1;  // also where all groups stay: equal scores tie
    // scores of bf16 logits alone tie too often
    a.narrow = (!full || a.f32 || a.bias != nullptr) && (a.G == 1 || a.group_lanes > 0);
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (launch_debug()) launch_debug_print("k_route", grid, block, "experts %d keys %d", a.E, full ? 64 : 32);
    for_experts(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (full) hipLaunchKernelGGL((k_route<V, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((k_route<V, false>), grid, block, 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t stream) {
    const int tiles = a.T > 0 ? (a.T + a.tile - 1) / a.tile : 1;  // one clears the count
    const dim3 grid((unsigned)tiles);
    for_experts(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const dim3 block(64 * kBalanceWaves<V>);
        if (launch_debug()) launch_debug_print("k_balance_pieces", grid, block, "experts %d sequences %d", a.E, a.S);
        hipLaunchKernelGGL(k_balance_pieces<V>, grid, block, 0, stream, a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_balance_loss, dim3((unsigned)(a.S * a.chunks)), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (launch_debug()) launch_debug_print("k_route_backward", grid, block, "experts %d", a.E);
    for_experts(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL(k_route_backward<V>, grid, block, 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace ep
