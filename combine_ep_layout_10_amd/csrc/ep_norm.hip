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

// Sum over the block (at most 16 waves), the same in every thread: a butterfly
// over each wave, then the waves in order. `tmp`: 16 floats of LDS, free again
// after the next barrier of the caller.
__device__ __forceinline__ float block_sum(float v, float* tmp) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    const int nw = blockDim.x >> 6;
    if (nw == 1) return v;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < nw; ++i) s += tmp[i];
    return s;
}

// max over 16 consecutive lanes
__device__ __forceinline__ float max16_dpp(float v) {
    v = max8_dpp(v);
    const int x = __float_as_int(v);
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, false)));  // row_mirror
}

// V vectors of 8 channels a lane: vector i of lane l is i * blockDim + l.
template <int V, bool FP8>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a) {
    __shared__ float s_sum[16];
    const int64_t row = (int64_t)blockIdx.x * a.H;
    const int nv = a.H / 8;
    uint4 s[V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
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
    sum = block_sum(sum, s_sum);
    const float rstd = 1.0f / sqrtf(sum / (float)a.H + a.eps);
    if (threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
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
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
            const float q = max16_dpp(amax) / 448.0f;
            uint32_t code[2] = {0u, 0u};
            if (q > 0.0f) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = fminf(fmaxf(f[j] / q, -448.0f), 448.0f);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
                    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], p, true);
                    code[j] = (uint32_t)p;
                }
            }
            *(uint2*)((uint8_t*)a.y + row + 8 * c) = make_uint2(code[0], code[1]);
            if ((threadIdx.x & 15) == 0) a.scales[(int64_t)blockIdx.x * (a.H / 128) + c / 16] = q * rstd;
        }
    }
}

template <int V>
__global__ __launch_bounds__(1024) void k_rms_norm_backward(NormBackwardArgs a) {
    __shared__ float s_sum[2][16];
    const int nv = a.H / 8;
    float gw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[i][j] = 0.0f;
    int turn = 0;  // two buffers for the block's sums, so that one barrier a row is enough
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = (int64_t)t * a.H;
        const float rstd = a.rstd[t];
        uint4 vs[V], vg[V];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            vs[i] = vg[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c >= nv) continue;
            vs[i] = *(const uint4*)(a.total + row + 8 * c);
            vg[i] = *(const uint4*)(a.grad_y + row + 8 * c);
            float s[8], g[8], w[8];
            unpack8(vs[i], s);
            unpack8(vg[i], g);
            unpack8(*(const uint4*)(a.weight + 8 * c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = s[j] * rstd;
                dot = __builtin_fmaf(g[j] * w[j], x, dot);
                gw[i][j] = __builtin_fmaf(g[j], x, gw[i][j]);
            }
        }
        const float mean = block_sum(dot, s_sum[turn]) / (float)a.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= nv) continue;
            float s[8], g[8], w[8], r[8];
            unpack8(vs[i], s);
            unpack8(vg[i], g);
            unpack8(*(const uint4*)(a.weight + 8 * c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = 0.0f;
            if (a.grad_total != nullptr) unpack8(*(const uint4*)(a.grad_total + row + 8 * c), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] += rstd * (g[j] * w[j] - s[j] * rstd * mean);
            *(uint4*)(a.grad_x + row + 8 * c) = pack8(r);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c >= nv) continue;
        float4* p = (float4*)(a.partial + (int64_t)blockIdx.x * a.H + 8 * c);
        p[0] = make_float4(gw[i][0], gw[i][1], gw[i][2], gw[i][3]);
        p[1] = make_float4(gw[i][4], gw[i][5], gw[i][6], gw[i][7]);
    }
}

// grad_weight[c]: the groups' partial sums, 16 strands in order, then the strands.
__global__ __launch_bounds__(256) void k_rms_norm_grad_weight(const float* partial, float* grad_weight, int parts, int H) {
    __shared__ float s_part[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int c = (int)blockIdx.x * 16 + x;
    float sum = 0.0f;
    if (c < H)
        for (int p = y; p < parts; p += 16) sum += partial[(int64_t)p * H + c];
    s_part[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < H) {
        sum = 0.0f;
        for (int i = 0; i < 16; ++i) sum += s_part[i][x];
        grad_weight[c] = sum;
    }
}

int norm_threads(int H) {
    const int v = (H / 8 + 63) / 64 * 64;
    return v < 1024 ? v : 1024;
}

template <int V>
void norm_launch(const NormArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.T), block((unsigned)norm_threads(a.H));
    if (a.scales != nullptr)
        hipLaunchKernelGGL((k_rms_norm<V, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((k_rms_norm<V, false>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int v = (a.H / 8 + 1023) / 1024;
    if (launch_debug())
        launch_debug_print("k_rms_norm", dim3((unsigned)a.T), dim3((unsigned)norm_threads(a.H)), "hidden %d", a.H);
    if (v <= 1) norm_launch<1>(a, stream);
    else if (v <= 2) norm_launch<2>(a, stream);
    else norm_launch<4>(a, stream);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const int v = (a.H / 8 + 1023) / 1024, parts = norm_backward_parts(a.T);
    const dim3 grid((unsigned)parts), block((unsigned)norm_threads(a.H));
    if (launch_debug()) launch_debug_print("k_rms_norm_backward", grid, block, "hidden %d", a.H);
    if (parts > 0) {
        if (v <= 1) hipLaunchKernelGGL(k_rms_norm_backward<1>, grid, block, 0, stream, a);
        else if (v <= 2) hipLaunchKernelGGL(k_rms_norm_backward<2>, grid, block, 0, stream, a);
        else hipLaunchKernelGGL(k_rms_norm_backward<4>, grid, block, 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_rms_norm_grad_weight, dim3((unsigned)((a.H + 15) / 16)), dim3(256), 0, stream, a.partial,
                       a.grad_weight, parts, a.H);
    return hipGetLastError();
}

}  // namespace ep
