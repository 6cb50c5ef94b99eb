// BF16 products grouped by expert over the receive layout, in the three
// directions of training, for any expert_alignment and any n and k that are
// multiples of 8 (the FP8 product of ep_gemm.hip needs whole 128-row tiles and
// has no backward). With the rows r of expert e that hold a pair:
//   forward      out[r, c]     = bf16( sum_k a[r, k] * b[e, c, k] )
//   grad_input   grad_a[r, k]  = bf16( sum_c g[r, c] * b[e, c, k] )
//   grad_weight  grad_b[e,c,k] = sum_r g[r, c] * a[r, k]   (binary32 or bf16)
// Each is one product C = A B of expert e with a reduction of K values; they
// differ in which operand has the reduction contiguous in memory:
//   forward      A [M rows, K]        B [N, K]   (both contiguous along K)
//   grad_input   A [M rows, K]        B [K, N]
//   grad_weight  A [K rows, M]        B [K rows, N]
// bf16 products are exact in binary32 and the MFMA accumulates in binary32, so
// the only rounding is the output's.
#include "ep_rows_dev.h"

namespace ep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

namespace {

constexpr int kBM = 64, kBN = 64, kBK = 32;
constexpr int kPitch = kBK + 8;  // LDS row pitch (elements): 16-byte reads of 16 rows spread over the banks

// 64 x 32 operand tile into LDS as [64][kPitch], zeros outside `rows` x
// `red`. KMAJOR: element (r, k) at src[k * ld + r], otherwise at src[r * ld + k].
template <bool KMAJOR>
__device__ __forceinline__ void stage(uint16_t* lds, const uint16_t* src, int64_t ld, int r0, int rows, int k0, int red) {
    const int tid = threadIdx.x;  // 256 threads, 8 elements each
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (KMAJOR) {
        const int k = tid >> 3, r = (tid & 7) * 8;
        if (k0 + k < red && r0 + r < rows) v = *(const uint4*)(src + (int64_t)(k0 + k) * ld + r0 + r);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) lds[(r + i) * kPitch + k] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    } else {
        const int r = tid >> 2, k = (tid & 3) * 8;
        if (r0 + r < rows && k0 + k < red) v = *(const uint4*)(src + (int64_t)(r0 + r) * ld + k0 + k);
        *(uint4*)(lds + r * kPitch + k) = v;
    }
}

template <int DIR>
__global__ __launch_bounds__(256) void k_grouped_gemm_bf16(GroupedArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t s_a[kBM * kPitch];
    __shared__ __attribute__((aligned(16))) uint16_t s_b[kBN * kPitch];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int nt_n = (a.N + kBN - 1) / kBN;
    const int n0 = ((int)blockIdx.x % nt_n) * kBN;
    int e, tile;
    if (DIR == kGradWeight) {
        const int nt_m = (a.M + kBM - 1) / kBM;
        tile = (int)(blockIdx.x / nt_n) % nt_m;
        e = (int)(blockIdx.x / nt_n) / nt_m;
    } else if (!find_row_tile(a.rows, kBM, (int)(blockIdx.x / nt_n), &e, &tile)) {
        return;
    }
    const ExpertRows er = expert_rows(a.rows, e);
    const int m0 = tile * kBM;
    const int rows = DIR == kGradWeight ? a.M : er.live;  // valid rows of A
    const int red = DIR == kGradWeight ? er.live : a.K;   // length of the reduction
    const uint16_t* pa = a.a + (int64_t)er.first * (DIR == kGradWeight ? a.M : a.K);
    const uint16_t* pb = DIR == kGradWeight ? a.b + (int64_t)er.first * a.N : a.b + (int64_t)e * a.N * a.K;

    f32x4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < red; k0 += kBK) {
        __syncthreads();
        stage<DIR == kGradWeight>(s_a, pa, DIR == kGradWeight ? a.M : a.K, m0, rows, k0, red);
        stage<DIR != kForward>(s_b, pb, DIR == kForward ? a.K : a.N, n0, a.N, k0, red);
        __syncthreads();
        // wave w: rows 16 w .. 16 w + 15, all 64 columns; operands swapped, so
        // a lane ends up with row lane % 16 and four adjacent columns
        const bf16x8_t fa = *(const bf16x8_t*)(s_a + (16 * w + (lane & 15)) * kPitch + (lane >> 4) * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x8_t fb = *(const bf16x8_t*)(s_b + (16 * i + (lane & 15)) * kPitch + (lane >> 4) * 8);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb, fa, acc[i], 0, 0, 0);
        }
    }
    const int row = m0 + 16 * w + (lane & 15);
    const int64_t crow = DIR == kGradWeight ? (int64_t)e * a.M + row : (int64_t)er.first + row;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = n0 + 16 * i + 4 * (lane >> 4);
        if (row >= rows || col >= a.N) continue;
        if (DIR == kGradWeight && a.out_f32)
            *(float4*)((float*)a.c + crow * a.N + col) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        else
            *(uint2*)((uint16_t*)a.c + crow * a.N + col) =
                make_uint2(pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3]));
    }
    // the expert's last row tile clears its padding rows
    if (DIR != kGradWeight && a.rows.zero_pad && m0 + kBM >= er.live)
        clear_padding((uint16_t*)a.c, a.N, er, n0, kBN);
}

}  // namespace

hipError_t launch_grouped_gemm_bf16(int dir, const GroupedArgs& a, int64_t pairs, hipStream_t stream) {
    const int64_t nt_n = (a.N + kBN - 1) / kBN;
    int64_t mtiles;
    if (dir == kGradWeight)
        mtiles = (int64_t)a.rows.E * ((a.M + kBM - 1) / kBM);
    else
        mtiles = max_row_tiles(a.rows, kBM, pairs);
    const int64_t blocks = mtiles * nt_n;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0xFFFFFF) return hipErrorInvalidValue;  // 2^32 threads a launch
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_bf16", dim3((unsigned)blocks), dim3(256), "direction %d n %d", dir, a.N);
    if (dir == kForward)
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kForward>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    else if (dir == kGradInput)
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kGradInput>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kGradWeight>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ep
