// The router: the choice of a token's experts from its logits, the balance loss
// with its counts, and the gradient of both with respect to the logits (formulas:
// include/ep.h). A wave has one token; lane i holds the V consecutive experts
// V i .. V i + V - 1 in registers, V a power of two of at least E / 64, so that
// lower lanes hold lower indices.
//
// Order: a key (a binary32 logit, or a binary64 score + bias) is held as an
// unsigned integer that orders as the number does, 0 for an expert that may not
// be chosen. A binary64 key's halves are compared one after the other: the
// higher one decides unless two experts share it. A round takes the highest key
// of the wave, its lowest index, and clears it.
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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
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

// exp(l - max l) and their sum over the wave. A row of -infinity alone has none.
template <int V>
__device__ __forceinline__ float softmax_terms(const float l[V], float x[V]) {
    const float m = wave_max_logit<V>(l);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = l[v] == -__builtin_inff() ? 0.0f : expf(l[v] - m);
        sum += x[v];
    }
    return wave_sum(sum);
}

// ---------------------------------------------------------------- choice

// The highest of the wave's keys with its lowest index, which is cleared; false
// when none is left. FULL: keys of 64 bits (hi, lo), otherwise hi alone.
struct Taken {
    uint32_t hi, lo;
    int lane;      // that holds it, the same in every lane
    int v;         // in that lane: which of its experts
};

template <int V, bool FULL>
__device__ __forceinline__ bool take_highest(uint32_t hi[V], const uint32_t lo[V], Taken* t) {
    uint32_t m = hi[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max(m, hi[v]);
    t->hi = wave_max(m);
    if (t->hi == 0) return false;
    t->lo = 0;
    if (FULL) {
        uint32_t n = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) n = hi[v] == t->hi ? max(n, lo[v]) : n;
        t->lo = wave_max(n);
    }
    t->v = V;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
        if (hi[v] == t->hi && (!FULL || lo[v] == t->lo)) t->v = v;
    t->lane = __builtin_ctzll(ballot64(t->v < V));
    const bool mine = lane_id() == t->lane;
#pragma unroll
    for (int v = 0; v < V; ++v) hi[v] = mine && v == t->v ? 0u : hi[v];
    return true;
}

// Clears the keys of the experts outside the best groups.
template <int V, bool FULL>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, int lane, uint32_t hi[V], const uint32_t lo[V]) {
    const int size = a.E / a.G;
    uint32_t group_hi[1] = {0u}, group_lo[1] = {0u};  // lane g: group g's
    for (int g = 0; g < a.G; ++g) {
        uint32_t h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            h[v] = e >= g * size && e < (g + 1) * size ? hi[v] : 0u;
        }
        Taken first, second;
        if (!take_highest<V, FULL>(h, lo, &first)) continue;
        uint64_t key = (uint64_t)first.hi << 32 | first.lo;
        if (FULL && a.best == 2 && take_highest<V, FULL>(h, lo, &second)) {
            const double sum = unordered(key) + unordered((uint64_t)second.hi << 32 | second.lo);
            key = ordered(sum < kLowest64 ? kLowest64 : sum);
        }
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

// FULL: keys are scores + bias in binary64, otherwise logits.
template <int V, bool FULL>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(RouteArgs a) {
    const int lane = lane_id();
    const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kRouteWaves + (threadIdx.x >> 6));
    if (t >= a.T) return;
    int chosen = -1;  // lane j < k: the j-th choice and its weight
    float w = 0.0f;
    if (a.mask == nullptr || a.mask[t] != 0) {
        float l[V], s[V];
        load_logits<V>(a.logits, a.f32, t, a.E, lane, l);
        uint32_t hi[V], lo[V];
        float max_l = 0.0f, sum = 1.0f;
        if (FULL) {
            double score[V];
            if (a.score == EP_SCORE_SOFTMAX) {
                const double m = (double)wave_max_logit<V>(l);
                double d = 0.0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    score[v] = l[v] == -__builtin_inff() ? 0.0 : exp((double)l[v] - m);
                    d += score[v];
                }
                d = wave_sum(d);
#pragma unroll
                for (int v = 0; v < V; ++v) score[v] /= d;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) score[v] = 1.0 / (1.0 + exp(-(double)l[v]));
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = lane * V + v;
                const float b = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
                double key = score[v] + (double)b;
                if (!(key >= kLowest64)) key = kLowest64;  // NaN
                const bool open = l[v] != -__builtin_inff() && b != -__builtin_inff();
                const uint64_t o = open ? ordered(key) : 0ull;
                hi[v] = (uint32_t)(o >> 32);
                lo[v] = (uint32_t)o;
                s[v] = (float)score[v];
            }
        } else {
            if (a.score == EP_SCORE_SOFTMAX) {
                float x[V];
                max_l = wave_max_logit<V>(l);
                sum = softmax_terms<V>(l, x);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                hi[v] = l[v] == -__builtin_inff() ? 0u : ordered(l[v] >= kLowest ? l[v] : kLowest);
                s[v] = l[v];
            }
        }
        if (a.G > 1) keep_groups<V, FULL>(a, lane, hi, lo);
        for (int j = 0; j < a.k; ++j) {
            Taken p;
            if (!take_highest<V, FULL>(hi, lo, &p)) break;
            float x = s[0];
#pragma unroll
            for (int v = 1; v < V; ++v) x = v == p.v ? s[v] : x;
            const int e = (int)lane_value((uint32_t)(lane * V + p.v), p.lane);
            x = lane_value(x, p.lane);
            if (lane == j) {
                chosen = e;
                w = x;
            }
        }
        if (!FULL && chosen >= 0) w = a.score == EP_SCORE_SOFTMAX ? expf(w - max_l) / sum : 1.0f / (1.0f + expf(-w));
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

// The first sequence whose end lies past token t (S: none).
__device__ __forceinline__ int sequence_past(const int32_t* off, int S, int t) {
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Tile b (kBalanceTile tokens) by sequence q: a piece of its own at place b + q of
// the partial sums. The pieces of a batch run from (0, 0) up in b or in q, never
// both, so places are distinct.
template <int V>
__global__ __launch_bounds__(64 * kBalanceWaves) void k_balance_pieces(BalanceArgs a) {
    __shared__ float s_sum[kBalanceWaves][64 * V];
    __shared__ int s_count[64 * V];
    __shared__ int s_tokens;
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = (int)blockIdx.x * kBalanceTile, t1 = min(t0 + kBalanceTile, a.T);
    int q = a.seq_off != nullptr ? sequence_past(a.seq_off, a.S, t0) : 0;
    for (; q < a.S; ++q) {
        int from = t0, to = t1;
        if (a.seq_off != nullptr) {
            const int first = a.seq_off[q];
            if (first >= t1) break;
            from = max(t0, first);
            to = min(t1, a.seq_off[q + 1]);
            if (from >= to) continue;
        }
        for (int e = tid; e < 64 * V; e += 64 * kBalanceWaves) s_count[e] = 0;
        if (tid == 0) s_tokens = 0;
        __syncthreads();
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = 0.0f;
        int tokens = 0;
        for (int t = from + wave; t < to; t += kBalanceWaves) {
            const int id = lane < a.k ? load_id(a.idx, a.idx_bits, (int64_t)t * a.k + lane, a.E) : -1;
            if (ballot64(id >= 0) == 0) continue;
            if (id >= 0) atomicAdd(&s_count[id], 1);
            ++tokens;
            float l[V], x[V];
            load_logits<V>(a.logits, a.f32, t, a.E, lane, l);
            float total;
            if (a.score == EP_SCORE_SOFTMAX) {
                total = softmax_terms<V>(l, x);
            } else {
                total = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = 1.0f / (1.0f + expf(-l[v]));
                    total += x[v];
                }
                total = wave_sum(total);
            }
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] += x[v] * inv;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s_sum[wave][lane * V + v] = sum[v];
        if (lane == 0 && tokens > 0) atomicAdd(&s_tokens, tokens);
        __syncthreads();
        const int64_t place = (int64_t)blockIdx.x + q;
        for (int e = tid; e < a.E; e += 64 * kBalanceWaves) {
            float total = 0.0f;
            for (int i = 0; i < kBalanceWaves; ++i) total += s_sum[i][e];
            a.sums[place * a.E + e] = total;
            a.pairs[place * a.E + e] = s_count[e];
        }
        if (tid == 0) a.tokens[place] = s_tokens;
        __syncthreads();
    }
}

__device__ __forceinline__ double block_sum(double v, double* tmp) {
    v = wave_sum(v);
    __syncthreads();
    if (lane_id() == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += tmp[i];
    return s;
}

// One sequence a block: its counts, its routed tokens and its term of the loss. A
// batch of one sequence has its loss at once.
__global__ __launch_bounds__(1024) void k_balance_sequences(BalanceArgs a) {
    __shared__ double s_tmp[16];
    const int q = blockIdx.x, tid = threadIdx.x;
    int from = 0, to = a.T;
    if (a.seq_off != nullptr) {
        from = max(0, a.seq_off[q]);
        to = min(a.T, a.seq_off[q + 1]);
    }
    const int b0 = from / kBalanceTile, b1 = from < to ? (to - 1) / kBalanceTile + 1 : b0;
    double term = 0.0;
    if (tid < a.E) {
        double sum = 0.0;
        int count = 0;
        for (int b = b0; b < b1; ++b) {
            const int64_t at = ((int64_t)b + q) * a.E + tid;
            sum += (double)a.sums[at];
            count += a.pairs[at];
        }
        a.counts[(int64_t)q * a.E + tid] = count;
        term = (double)count * sum;
    }
    double tokens = 0.0;
    for (int b = b0 + tid; b < b1; b += 1024) tokens += (double)a.tokens[b + q];
    term = block_sum(term, s_tmp);
    tokens = block_sum(tokens, s_tmp);
    if (tid != 0) return;
    const double c = tokens > 0.0 ? (double)a.E / ((double)a.k * tokens * tokens) : 0.0;
    if (a.S == 1) {
        a.coef[0] = (float)c;
        a.loss[0] = (float)(c * term);
    } else {
        a.unit[q] = c;
        a.term[q] = c * term;
    }
}

__global__ __launch_bounds__(1024) void k_balance_loss(BalanceArgs a) {
    __shared__ double s_tmp[16];
    double used = 0.0, loss = 0.0;
    for (int q = threadIdx.x; q < a.S; q += 1024) {
        used += a.unit[q] > 0.0 ? 1.0 : 0.0;
        loss += a.term[q];
    }
    used = block_sum(used, s_tmp);
    loss = block_sum(loss, s_tmp);
    if (used < 1.0) used = 1.0;
    for (int q = threadIdx.x; q < a.S; q += 1024) a.coef[q] = (float)(a.unit[q] / used);
    if (threadIdx.x == 0) a.loss[0] = (float)(loss / used);
}

// ---------------------------------------------------------------- gradient

template <int V>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_backward(RouteBackwardArgs a) {
    const int lane = lane_id();
    const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kRouteWaves + (threadIdx.x >> 6));
    if (t >= a.T) return;
    float grad[V];
#pragma unroll
    for (int v = 0; v < V; ++v) grad[v] = 0.0f;
    const int id = lane < a.k ? load_id(a.idx, a.idx_bits, (int64_t)t * a.k + lane, a.E) : -1;
    if (ballot64(id >= 0) != 0) {
        const float gw = a.grad_w != nullptr && lane < a.k ? a.grad_w[(int64_t)t * a.k + lane] : 0.0f;
        float l[V], s[V], n[V], u[V], b[V];
        load_logits<V>(a.logits, a.f32, t, a.E, lane, l);
        const bool softmax = a.score == EP_SCORE_SOFTMAX;
        float total = 0.0f;
        if (softmax) {
            total = softmax_terms<V>(l, s);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= inv;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = 1.0f / (1.0f + expf(-l[v]));
                total += s[v];
            }
            total = wave_sum(total);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) n[v] = u[v] = b[v] = 0.0f;
        if (a.grad_w != nullptr) {
            for (int j = 0; j < a.k; ++j) {
                const int e = (int)lane_value((uint32_t)id, j) - lane * V;
                const float g = lane_value(gw, j);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    n[v] += e == v ? 1.0f : 0.0f;
                    u[v] += e == v ? g : 0.0f;
                }
            }
            if (a.renormalize) {
                float d = 0.0f, q = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d += n[v] * s[v];
                    q += u[v] * s[v];
                }
                d = wave_sum(d) + 1e-20f;
                q = wave_sum(q) / d;
#pragma unroll
                for (int v = 0; v < V; ++v) u[v] = n[v] > 0.0f ? a.scale * ((u[v] - n[v] * q) / d) : 0.0f;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) u[v] *= a.scale;
            }
        }
        if (a.counts != nullptr) {
            int q = 0;
            bool in = true;
            if (a.seq_off != nullptr) {
                q = __builtin_amdgcn_readfirstlane(sequence_past(a.seq_off, a.S, t));
                in = q < a.S && a.seq_off[q] <= t;
            }
            if (in) {
                // A constant added to every b changes nothing, and counts of a balanced
                // batch are nearly equal: the first one goes out exactly, as an integer.
                const int32_t* c = a.counts + (int64_t)q * a.E;
                const float f = a.grad_loss[0] * a.coef[q];
                const int first = c[0];
                float mean = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e = lane * V + v;
                    b[v] = e < a.E ? f * (float)(c[e] - first) : 0.0f;
                    mean += s[v] * b[v];
                }
                mean = wave_sum(mean);
                if (softmax) {
#pragma unroll
                    for (int v = 0; v < V; ++v) b[v] -= mean;
                } else {
                    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
                    for (int v = 0; v < V; ++v) b[v] = (b[v] - mean * inv) * inv;
                }
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
            for (int v = 0; v < V; ++v) {
                // s (1 - s) without the difference
                const float x = expf(-fabsf(l[v])), y = 1.0f / (1.0f + x);
                grad[v] = x * y * y * (u[v] + b[v]);
            }
        }
    }
    const int e = lane * V;
    const int64_t at = (int64_t)t * a.E + e;
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

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    const bool full = a.bias != nullptr || (a.G > 1 && a.best > 1);
    if (launch_debug()) launch_debug_print("k_route", grid, block, "experts %d keys %d", a.E, full ? 64 : 32);
    for_experts(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (full) hipLaunchKernelGGL((k_route<V, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((k_route<V, false>), grid, block, 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t stream) {
    const int tiles = (a.T + kBalanceTile - 1) / kBalanceTile;
    const dim3 grid((unsigned)tiles), block(64 * kBalanceWaves);
    if (launch_debug()) launch_debug_print("k_balance_pieces", grid, block, "experts %d sequences %d", a.E, a.S);
    if (tiles > 0) {
        for_experts(a.E, [&](auto v) {
            constexpr int V = decltype(v)::value;
            hipLaunchKernelGGL(k_balance_pieces<V>, grid, block, 0, stream, a);
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_balance_sequences, dim3((unsigned)a.S), dim3(1024), 0, stream, a);
    if (a.S > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_balance_loss, dim3(1), dim3(1024), 0, stream, a);
    }
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
