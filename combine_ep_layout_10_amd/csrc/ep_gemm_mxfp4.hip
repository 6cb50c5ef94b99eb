// Products with 4-bit weights over the receive layout: every expert's rows
// (bf16) times its MXFP4 weights (OCP Microscaling: E2M1 codes, two to a byte,
// the lower nibble first, and one E8M0 scale for each 32 consecutive k):
//   out[r, c] = bf16( sum_k a[r, k] * e2m1(code[e, c, k]) * 2^(scale[e, c, k / 32] - 127) )
// A code times its scale is a bf16 value (two significant bits), so the
// conversion is exact, the products are exact in binary32, and the MFMA
// accumulates them in binary32: the only rounding is the output's.
#include "ep_rows_dev.h"

namespace ep {

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x4_v __attribute__((ext_vector_type(4)));

namespace {

// The 8 codes of one word (lowest nibble first) times 2^(e8m0 - 127).
__device__ __forceinline__ bf16x8_v decode_mxfp4(uint32_t word, float scale) {
    const bf16x2_v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0);
    const bf16x2_v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1);
    const bf16x2_v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2);
    const bf16x2_v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3);
    return (bf16x8_v){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

constexpr int kTokens = 16;  // rows of a block's tile
constexpr int kCols = 64;    // output columns of a block: 16 for each of 4 waves

__global__ __launch_bounds__(256) void k_grouped_gemm_mxfp4(Mxfp4Args a) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int nt_n = (a.N + kCols - 1) / kCols;
    int e, local;
    if (!find_expert(a.rows, kTokens, nt_n, &e, &local)) return;
    const ExpertRows er = expert_rows(a.rows, e);
    const int block_n0 = (local % nt_n) * kCols, n0 = block_n0 + 16 * w;
    const int m0 = local / nt_n * kTokens;
    // lane: weight row (output column) and token lane % 16, k piece lane / 16
    const int r16 = lane & 15, g = lane >> 4;
    const int col = min(n0 + r16, a.N - 1);  // columns past N repeat the last and are not stored
    const bool token = m0 + r16 < er.live;
    const uint8_t* pb = a.b + ((int64_t)e * a.N + col) * (a.K / 2);
    const uint8_t* ps = a.b_scales + ((int64_t)e * a.N + col) * (a.K / 32);
    const uint16_t* px = a.x + ((int64_t)er.first + min(m0 + r16, er.live - 1)) * a.K;
    f32x4_v acc = (f32x4_v){0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = 0; kb < a.K / 32; ++kb) {
        const uint32_t word = *(const uint32_t*)(pb + kb * 16 + g * 4);
        const float scale = __uint_as_float((uint32_t)ps[kb] << 23);
        const bf16x8_v x = *(const bf16x8_v*)(px + kb * 32 + g * 8);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_mxfp4(word, scale), x, acc, 0, 0, 0);
    }
    // lane: token r16, columns n0 + 4 g .. + 3
    const int c0 = n0 + 4 * g;
    if (token && c0 < a.N)
        *(uint2*)(a.out + ((int64_t)er.first + m0 + r16) * a.N + c0) =
            make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    if (a.rows.zero_pad && m0 + kTokens >= er.live)
        clear_padding(a.out, a.N, er, block_n0, kCols);
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(const Mxfp4Args& a, int64_t pairs, hipStream_t stream) {
    const int64_t nt_n = (a.N + kCols - 1) / kCols;
    const int64_t blocks = max_row_tiles(a.rows, kTokens, pairs) * nt_n;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0xFFFFFF) return hipErrorInvalidValue;  // 2^32 threads a launch
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_mxfp4", dim3((unsigned)blocks), dim3(256), "n %d k %d", a.N, a.K);
    hipLaunchKernelGGL(k_grouped_gemm_mxfp4, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ep
