// RMS norm with the residual's addition, and its backward: what stands before
// the router and the dispatch. Forward, for every token t:
//   s    = bf16(x + residual)            (written as `total`; s = x without a residual)
//   rstd = 1 / sqrt(mean_c s^2 + eps)
//   y    = s * rstd * w
// written as bf16, or as E4M3 codes with one scale for each 128 channels, the
// form that a pre-quantised dispatch takes. With u = s * w (exact in binary32:
// two bf16 factors) the FP8 form of a block is
//   q = max|u| / 448, code = E4M3(u / q), scale = q * rstd   (q = 0: code 0, scale 0)
// The row's factor rstd multiplies every channel of a block alike, so it goes
// into the scale alone, and the codes do not depend on how the sum of squares
// was ordered. Backward, with g the gradient of y and gw = g * w:
//   grad_x = bf16( rstd * (gw - s * rstd^2 * mean_c(gw * s)) + grad_total )
//   grad_w = sum_t g * s * rstd          (binary32)
// grad_x is also the gradient of the residual. Sums are binary32 in a fixed
// order: per lane over its channels, butterflies over the waves, the weight
// gradient over the rows of a group and then over the groups in order.
#include "ep_internal.h"

namespace ep {

namespace {

__device__ __forceinline__ void unpack8(uint4 v, float f[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
    }
}

__device__ __forceinline__ uint4 pack8(const float f[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Sum over the threads of a row (the block's x; whole waves), the same in each of
// them: a butterfly over each wave, then the row's waves in order. `tmp` is LDS
// for one float a wave of the block, free again behind the caller's next barrier. Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, float* tmp) {
    const int row_waves = blockDim.x >> 6;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    if (row_waves == 1) return v;
    const int first = threadIdx.y * row_waves;
    if ((threadIdx.x & 63) == 0) tmp[first + (threadIdx.x >> 6)] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < row_waves; ++i) s += tmp[first + i];
    return s;
}

// max|f| over the channels of a block: the 8 of each of 16 consecutive lanes, NaN
// when one of them is (fmaxf would drop it). Magnitudes order like their bit
// patterns, with NaN above infinity.
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float block_max(const float f[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    m = max_with<0xB1>(m);   // quad_perm [1,0,3,2]
    m = max_with<0x4E>(m);   // quad_perm [2,3,0,1]
    m = max_with<0x141>(m);  // row_half_mirror
    m = max_with<0x140>(m);  // row_mirror
    return __uint_as_float(m);
}

// v = f / q, correctly rounded, for |f| <= 448 q (1 + 2^-23). With r the rounded
// reciprocal, the product f r is off by at most two units of the last place; one
// correction by the exact remainder brings it within one, and by Markstein's
// theorem (a quotient within one unit, and a correctly rounded reciprocal) the
// second makes it the rounded quotient. Five operations instead of a division's
// dozen. The remainder keeps f's zeros' sign (y - rem * r), and is exact while
// nothing underflows: |f / q| >= 2^-10, below which every code is a signed zero,
// and q >= 2^-80 leave its last bit at 2^-136. Smaller and huge q divide, and NaN
// and infinite ones, whose NaN quotients stay NaN: only numbers are held to 448.
__device__ __forceinline__ void quotients(const float f[8], float q, float v[8]) {
    if (q >= 0x1p-80f && q <= 0x1p100f) {
        const float r = 1.0f / q;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float y = f[j] * r;
            y = __builtin_fmaf(-__builtin_fmaf(y, q, -f[j]), r, y);
            v[j] = __builtin_fmaf(-__builtin_fmaf(y, q, -f[j]), r, y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = f[j] / q;
            v[j] = y > 448.0f ? 448.0f : y < -448.0f ? -448.0f : y;
        }
    }
}

// A row's threads: whole waves, one vector of 8 channels each (V of them for rows
// of more than 8192 channels), at most 1024. Short rows share a block.
struct RowShape {
    int threads, rows, v;  // of a row; rows of a block; vectors a thread
};

RowShape row_shape(int H) {
    RowShape s;
    const int t = (H / 8 + 63) / 64 * 64;
    s.threads = t < 1024 ? t : 1024;
    s.rows = s.threads <= 256 ? 512 / s.threads : 1;
    s.v = (H / 8 + 1023) / 1024;
    return s;
}

// V vectors of 8 channels a lane: vector i of thread l of a row is i * threads + l.
template <int V, bool FP8>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a) {
    __shared__ float s_sum[16];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int t = V == 1 ? (int)(blockIdx.x * blockDim.y + threadIdx.y) : (int)blockIdx.x;
    const bool live = t < a.T;
    const int64_t row = (int64_t)t * a.H;
    const int nv = live ? a.H / 8 : 0;
    uint4 s[V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * threads + tid;
        s[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c >= nv) continue;
        s[i] = *(const uint4*)(a.x + row + 8 * c);
        float f[8];
        unpack8(s[i], f);
        if (a.residual != nullptr) {
            float r[8];
            unpack8(*(const uint4*)(a.residual + row + 8 * c), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += r[j];
            s[i] = pack8(f);
            *(uint4*)(a.total + row + 8 * c) = s[i];
            unpack8(s[i], f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(f[j], f[j], sum);
    }
    sum = row_sum(sum, s_sum);
    const float rstd = 1.0f / sqrtf(sum / (float)a.H + a.eps);
    if (live && tid == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * threads + tid;
        if (c >= nv) continue;  // whole groups of 16 lanes: H % 128 == 0 for FP8
        float f[8], w[8];
        unpack8(s[i], f);
        unpack8(*(const uint4*)(a.weight + 8 * c), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w[j];
        if (!FP8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= rstd;
            *(uint4*)((uint16_t*)a.y + row + 8 * c) = pack8(f);
        } else {
            const float q = block_max(f) / 448.0f;
            uint32_t code[2] = {0u, 0u};
            if (q != 0.0f) {
                float v[8];
                quotients(f, q, v);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
                    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], p, true);
                    code[j] = (uint32_t)p;
                }
            }
            *(uint2*)((uint8_t*)a.y + row + 8 * c) = make_uint2(code[0], code[1]);
            if ((tid & 15) == 0) a.scales[(int64_t)t * (a.H / 128) + c / 16] = q * rstd;
        }
    }
}

// A row's threads sum the weight gradient of their channels over the rows they
// take, in registers; the rows of a block that share its channels are added
// through LDS at the end, so a block leaves one partial sum of H channels. The
// next row's values are loaded before the present row's sum is waited for.
template <int V, bool BRANCH>
__global__ __launch_bounds__(1024) void k_rms_norm_backward(NormBackwardArgs a) {
    __shared__ float s_sum[2][16];
    __shared__ float s_part[V == 1 ? 8 * 512 : 1];  // several rows a block only with V == 1 and 512 threads
    const int tid = threadIdx.x, threads = blockDim.x;
    const int sub = V == 1 ? threadIdx.y : 0, rows = V == 1 ? blockDim.y : 1;  // long rows have blocks of their own
    const int nv = a.H / 8, step = gridDim.x * rows;
    constexpr bool kAhead = V == 1;  // longer rows have no registers for it, and loads enough in flight
    float gw[V][8];
    uint4 vs[V], vg[V], vt[V];
    float rstd = 0.0f;
    const auto load = [&](int t) {
        const int64_t row = (int64_t)t * a.H;
        if (t < a.T) rstd = a.rstd[t];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * threads + tid;
            vs[i] = vg[i] = vt[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c >= nv || t >= a.T) continue;
            vs[i] = *(const uint4*)(a.total + row + 8 * c);
            vg[i] = *(const uint4*)(a.grad_y + row + 8 * c);
            if (BRANCH && kAhead) vt[i] = *(const uint4*)(a.grad_total + row + 8 * c);
        }
    };
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[i][j] = 0.0f;
    int t = (int)blockIdx.x * rows + sub;
    if (kAhead) load(t);
    int turn = 0;  // two buffers for the rows' sums, so that one barrier a row is enough
    for (int t0 = (int)blockIdx.x * rows; t0 < a.T; t0 += step, t += step, turn ^= 1) {
        if (!kAhead) load(t);
        uint4 s4[V], g4[V], t4[V];
        const float r = rstd;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s4[i] = vs[i];
            g4[i] = vg[i];
            t4[i] = vt[i];
            const int c = i * threads + tid;
            if (c >= nv) continue;
            float s[8], g[8], x[8];
            unpack8(s4[i], s);
            unpack8(g4[i], g);
            unpack8(*(const uint4*)(a.weight + 8 * c), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xhat = s[j] * r;
                dot = __builtin_fmaf(g[j] * x[j], xhat, dot);
                gw[i][j] = __builtin_fmaf(g[j], xhat, gw[i][j]);
            }
        }
        if (kAhead) load(t + step);
        const float mean = row_sum(dot, s_sum[turn]) / (float)a.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * threads + tid;
            if (c >= nv || t >= a.T) continue;
            const int64_t at = (int64_t)t * a.H + 8 * c;
            float s[8], g[8], x[8], o[8];
            unpack8(V < 4 ? s4[i] : *(const uint4*)(a.total + at), s);  // V = 4 has no registers to keep them
            unpack8(V < 4 ? g4[i] : *(const uint4*)(a.grad_y + at), g);
            unpack8(*(const uint4*)(a.weight + 8 * c), x);
            if (BRANCH) unpack8(kAhead ? t4[i] : *(const uint4*)(a.grad_total + at), o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = r * (g[j] * x[j] - s[j] * r * mean);
                o[j] = BRANCH ? v + o[j] : v;
            }
            *(uint4*)(a.grad_x + at) = pack8(o);
        }
    }
    if (V == 1 && rows > 1) {  // rows sub > 0 of the block, in order
        float* p = s_part + (sub * threads + tid) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = gw[0][j];
        __syncthreads();
        if (sub > 0) return;
        for (int k = 1; k < rows; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) gw[0][j] += s_part[(k * threads + tid) * 8 + j];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * threads + tid;
        if (c >= nv) continue;
        float4* p = (float4*)(a.partial + (int64_t)blockIdx.x * a.H + 8 * c);
        p[0] = make_float4(gw[i][0], gw[i][1], gw[i][2], gw[i][3]);
        p[1] = make_float4(gw[i][4], gw[i][5], gw[i][6], gw[i][7]);
    }
}

// grad_weight[c]: the blocks' partial sums in 64 strands (partial p in strand
// p mod 64, in order), then the strands in order.
__global__ __launch_bounds__(1024) void k_rms_norm_grad_weight(const float* partial, float* grad_weight, int parts, int H) {
    __shared__ float s_part[64][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int c = (int)blockIdx.x * 16 + x;
    float v[kNormParts / 64];
#pragma unroll
    for (int i = 0; i < kNormParts / 64; ++i)
        v[i] = c < H && i * 64 + y < parts ? partial[(int64_t)(i * 64 + y) * H + c] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormParts / 64; ++i) sum += v[i];
    s_part[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < H) {
        sum = 0.0f;
        for (int i = 0; i < 64; ++i) sum += s_part[i][x];
        grad_weight[c] = sum;
    }
}

template <int V>
void norm_launch(const NormArgs& a, const RowShape& s, dim3 grid, hipStream_t stream) {
    const dim3 block((unsigned)s.threads, (unsigned)s.rows);
    if (a.scales != nullptr)
        hipLaunchKernelGGL((k_rms_norm<V, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((k_rms_norm<V, false>), grid, block, 0, stream, a);
}

template <int V>
void norm_backward_launch(const NormBackwardArgs& a, const RowShape& s, dim3 grid, hipStream_t stream) {
    const dim3 block((unsigned)s.threads, (unsigned)s.rows);
    if (a.grad_total != nullptr)
        hipLaunchKernelGGL((k_rms_norm_backward<V, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((k_rms_norm_backward<V, false>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const RowShape s = row_shape(a.H);
    const dim3 grid((unsigned)((a.T + s.rows - 1) / s.rows));
    if (launch_debug())
        launch_debug_print("k_rms_norm", grid, dim3((unsigned)(s.threads * s.rows)), "hidden %d", a.H);
    if (s.v <= 1) norm_launch<1>(a, s, grid, stream);
    else if (s.v <= 2) norm_launch<2>(a, s, grid, stream);
    else norm_launch<4>(a, s, grid, stream);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const RowShape s = row_shape(a.H);
    const int need = (a.T + s.rows - 1) / s.rows, parts = need < kNormParts ? need : kNormParts;
    const dim3 grid((unsigned)parts);
    if (launch_debug())
        launch_debug_print("k_rms_norm_backward", grid, dim3((unsigned)(s.threads * s.rows)), "hidden %d", a.H);
    if (parts > 0) {
        if (s.v <= 1) norm_backward_launch<1>(a, s, grid, stream);
        else if (s.v <= 2) norm_backward_launch<2>(a, s, grid, stream);
        else norm_backward_launch<4>(a, s, grid, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_rms_norm_grad_weight, dim3((unsigned)((a.H + 15) / 16)), dim3(1024), 0, stream, a.partial,
                       a.grad_weight, parts, a.H);
    return hipGetLastError();
}

}  // namespace ep
