// Products with 4-bit weights over the receive layout: every expert's rows
// (bf16) times its MXFP4 weights (OCP Microscaling: E2M1 codes, two to a byte,
// the lower nibble first, and one E8M0 scale for each 32 consecutive k):
//   out[r, c] = bf16( sum_k a[r, k] * e2m1(code[e, c, k]) * 2^(scale[e, c, k / 32] - 127) )
// A code times its scale is a bf16 value (two significant bits), so the
// conversion is exact (v_cvt_scalef32_pk_bf16_fp4, all codes and scales checked
// on MI355X), the products are exact in binary32, and the MFMA accumulates them
// in binary32: the only rounding is the output's.
//
// This is a product for few rows an expert, bound by reading the weights once:
// they go from memory straight into registers, kept kInFlight loads ahead. A
// block of 8 waves takes up to TB rows of one expert by 128 MC / S output
// columns. A wave's piece is 16 MC columns of the weights as the MFMA's first
// operand: in a chunk of 128 k, lane (g, r16) reads the 32 codes of group g of
// column r16 with one 16-byte load, and its scale; word t of the four is the
// operand of MFMA t, whose k are then 32 g + 8 t .. + 7. The rows (the second
// operand, read in the same order of k) are shared by the block through LDS in
// slices of KC values of k, two slices deep; 16-byte chunk c of row r is stored at
// c ^ row_slot(r), which meets each bank once in every read.
// S splits the reduction over the waves of a block, so that a small problem
// still reaches every CU: wave group ks takes the ks-th part of every slice, and
// the S sums are added in order at the end.
#include "ep_mma_dev.h"
#include "ep_rows_dev.h"

namespace ep {

namespace {

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;
constexpr int kInFlight = 8;  // weight loads a wave keeps in flight

__device__ __forceinline__ int row_slot(int r) { return (row_swizzle16(r) << 2) | (r & 3); }

// The 8 codes of one word (lowest nibble first) times 2^(e8m0 - 127).
__device__ __forceinline__ bf16x8_t decode_mxfp4(uint32_t word, float scale) {
    const bf16x2_v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0);
    const bf16x2_v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1);
    const bf16x2_v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2);
    const bf16x2_v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3);
    return (bf16x8_t){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// k values of a slice of rows: 8 chunks for a wave of 16 columns, 4 (so as many
// loads) for one of 32.
template <int MC>
constexpr int slice_k() { return MC == 1 ? 1024 : 512; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, int size) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, size, kBufferFlags);
}

// Rows m0 .. m0 + rows - 1 of the expert (rows <= 16 NT) by the block's columns.
template <int TB, int MC, int S, int NT>
__device__ __forceinline__ void run_tile(const Mxfp4Args& a, const ExpertRows& er, int e, int m0, int rows, int n0,
                                         uint8_t* s_x) {
    constexpr int KC = slice_k<MC>(), NC = KC / 128;   // chunks of a slice
    constexpr int B = NC / S;                          // chunks of a slice that one wave takes
    constexpr int P = kInFlight > B * MC ? kInFlight / (B * MC) : 1;  // slices whose weights are in registers
    constexpr int R = P > 1 ? P : 2;  // slices whose scales are in registers
    constexpr int XL = NT * 16 * KC * 2 / 16 / (64 * kWaves);          // 16-byte loads a thread for a slice of rows
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = w / (kWaves / S), cw = w % (kWaves / S);
    const int slices = (a.K + KC - 1) / KC;
    const int groups = a.K / 32;

    // weights of this wave's columns: columns past N, and k past K, read as zeros
    const int c0 = n0 + 16 * MC * cw;
    const int cols = max(0, min(16 * MC, a.N - c0));
    const int64_t wrow = (int64_t)e * a.N + min(c0, a.N - 1);
    const __amdgpu_buffer_rsrc_t rb = resource(a.b + wrow * (a.K / 2), cols * (a.K / 2));
    const uint8_t* ws = a.b_scales + wrow * groups;
    const __amdgpu_buffer_rsrc_t rx = resource(a.x + ((int64_t)er.first + m0) * a.K, rows * a.K * 2);

    // Codes: chunk b of this wave's B in slice kc. Scales: the 4 B bytes a column
    // that go with them, as words (word b: chunk b, byte g: group g). A byte
    // load for each chunk would cost as many requests as the codes do (313
    // against 220 us at 128 tokens x top-8, 64 experts, 4096 x 7168).
    u32x4_t code[P][B][MC];
    uint32_t scale[R][B][MC];
    auto load = [&](int kc, int p, int b) {
        const int group = (kc * NC + ks * B + b) * 4 + g;
#pragma unroll
        for (int c = 0; c < MC; ++c)
            code[p][b][c] = __builtin_amdgcn_raw_buffer_load_b128(
                rb, group < groups ? (16 * c + r16) * (a.K / 2) + 16 * group : kOutOfRange, 0, 0);
    };
    auto load_scales = [&](int kc, int p) {
        if (kc >= slices) return;
        const int first = (kc * NC + ks * B) * 4;
#pragma unroll
        for (int c = 0; c < MC; ++c) {
            const uint8_t* s = ws + (int64_t)min(16 * c + r16, max(cols - 1, 0)) * groups + first;
            if ((kc + 1) * KC <= a.K) {
                __builtin_memcpy(&scale[p][0][c], s, 4);  // any alignment
#pragma unroll
                for (int b = 1; b < B; ++b) __builtin_memcpy(&scale[p][b][c], s + 4 * b, 4);
            } else {  // the last slice may end inside a word
#pragma unroll
                for (int b = 0; b < B; ++b)
                    scale[p][b][c] = first + 4 * b + g < groups ? (uint32_t)s[4 * b + g] << (8 * g) : 0u;
            }
        }
    };
    u32x4_t xr[XL];
    auto load_rows = [&](int kc) {
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int q = j * 64 * kWaves + tid, row = q / (KC / 8), k = kc * KC + q % (KC / 8) * 8;
            xr[j] = __builtin_amdgcn_raw_buffer_load_b128(rx, k < a.K ? (row * a.K + k) * 2 : kOutOfRange, 0, 0);
        }
    };
    auto store_rows = [&](int stage) {
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int q = j * 64 * kWaves + tid, row = q / (KC / 8), c = q % (KC / 8);
            *(u32x4_t*)(s_x + stage * (TB * KC * 2) + row * (KC * 2) + ((c ^ row_slot(row)) << 4)) = xr[j];
        }
    };

    load_rows(0);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        load_scales(p, p);
#pragma unroll
        for (int b = 0; b < B; ++b) load(p, p, b);
    }
    f32x4_t acc[NT][MC];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < MC; ++c) acc[n][c] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    store_rows(0);
    wait_lgkmcnt0();
    block_barrier();

    for (int kc0 = 0; kc0 < slices; kc0 += R) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int kc = kc0 + r, p = r % P;
            if (kc >= slices) break;
            // the next slice of rows travels while this one is used; its stage
            // was last read a barrier ago
            if (kc + 1 < slices) load_rows(kc + 1);
            if (P == 1) load_scales(kc + 1, (r + 1) % R);
            const uint8_t* x = s_x + (kc & 1) * (TB * KC * 2) + r16 * (KC * 2);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int sub = ks * B + b;
                uint32_t power[MC];
#pragma unroll
                for (int c = 0; c < MC; ++c) power[c] = __builtin_amdgcn_ubfe(scale[r][b][c], 8 * g, 8) << 23;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    bf16x8_t f[MC];
#pragma unroll
                    for (int c = 0; c < MC; ++c)
                        f[c] = decode_mxfp4(code[p][b][c][t], __uint_as_float(power[c]));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const bf16x8_t v =
                            *(const bf16x8_t*)(x + n * (16 * KC * 2) + sub * 256 + (((4 * g + t) ^ row_slot(r16)) << 4));
#pragma unroll
                        for (int c = 0; c < MC; ++c)
                            acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[c], v, acc[n][c], 0, 0, 0);
                    }
                }
                load(kc + P, p, b);
            }
            if (P > 1) load_scales(kc + P, r);
            if (kc + 1 < slices) store_rows((kc + 1) & 1);
            wait_lgkmcnt0();
            block_barrier();
        }
    }

    if (S > 1) {  // the groups' sums, in order
        f32x4_t* sum = (f32x4_t*)s_x;
        if (ks > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < MC; ++c) sum[((w * NT + n) * MC + c) * 64 + lane] = acc[n][c];
        }
        wait_lgkmcnt0();
        block_barrier();
        if (ks > 0) return;
#pragma unroll
        for (int s = 1; s < S; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < MC; ++c)
                    acc[n][c] += sum[(((s * (kWaves / S) + cw) * NT + n) * MC + c) * 64 + lane];
    }
    // lane: row r16 of each piece, columns 4 g .. 4 g + 3
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < MC; ++c) {
            const int row = 16 * n + r16, col = c0 + 16 * c + 4 * g;
            if (row < rows && col < a.N)
                *(uint2*)(a.out + ((int64_t)er.first + m0 + row) * a.N + col) =
                    make_uint2(pack_bf16x2(acc[n][c][0], acc[n][c][1]), pack_bf16x2(acc[n][c][2], acc[n][c][3]));
        }
}

template <int TB, int MC, int S>
__global__ __launch_bounds__(64 * kWaves) void k_grouped_gemm_mxfp4(Mxfp4Args a) {
    constexpr int kCols = 16 * MC * kWaves / S;
    __shared__ __attribute__((aligned(16))) uint8_t s_x[2 * TB * slice_k<MC>() * 2];
    const int nt_n = (a.N + kCols - 1) / kCols;
    int e, local;
    if (!find_expert(a.rows, TB, nt_n, &e, &local)) return;
    const ExpertRows er = expert_rows(a.rows, e);
    // row tiles of one column tile are neighbours: they read the same weights.
    // An expert's rows are cut into tiles of equal size, rounded up to 16.
    const int nt_m = (er.live + TB - 1) / TB, m = local % nt_m;
    const int each = ((er.live + nt_m - 1) / nt_m + 15) & ~15;
    const int m0 = __builtin_amdgcn_readfirstlane(m * each);
    const int rows = __builtin_amdgcn_readfirstlane(min(each, er.live - m0));
    const int n0 = __builtin_amdgcn_readfirstlane(local / nt_m * kCols);
    if (a.rows.zero_pad && m == nt_m - 1) clear_padding(a.out, a.N, er, n0, kCols);
    e = __builtin_amdgcn_readfirstlane(e);
    switch ((rows + 15) / 16) {
        case 1: return run_tile<TB, MC, S, 1>(a, er, e, m0, rows, n0, s_x);
        case 2: if (TB >= 32) return run_tile<TB, MC, S, TB >= 32 ? 2 : 1>(a, er, e, m0, rows, n0, s_x); break;
        case 3: if (TB >= 64) return run_tile<TB, MC, S, TB >= 64 ? 3 : 1>(a, er, e, m0, rows, n0, s_x); break;
        default: if (TB >= 64) return run_tile<TB, MC, S, TB >= 64 ? 4 : 1>(a, er, e, m0, rows, n0, s_x); break;
    }
}

template <int TB, int MC, int S>
hipError_t launch(const Mxfp4Args& a, int64_t pairs, hipStream_t stream) {
    constexpr int kCols = 16 * MC * kWaves / S;
    const int64_t blocks = max_row_tiles(a.rows, TB, pairs) * ((a.N + kCols - 1) / kCols);
    if (blocks > 0x7FFFFF) return hipErrorInvalidValue;  // 2^32 threads a launch
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_mxfp4", dim3((unsigned)blocks), dim3(64 * kWaves), "rows %d split %d n %d k %d",
                           TB, S, a.N, a.K);
    hipLaunchKernelGGL((k_grouped_gemm_mxfp4<TB, MC, S>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(const Mxfp4Args& a, int64_t pairs, hipStream_t stream) {
    if (pairs == 0) return hipSuccess;
    // Rows of a tile: enough for nearly every expert's, so that its weights are
    // read once (an expert's rows scatter around their mean).
    const int64_t experts = pairs < a.rows.E ? pairs : a.rows.E;
    const int64_t mean = (pairs + a.rows.E - 1) / a.rows.E;
    // The reduction is split while that leaves about one block a CU (256 of 8
    // waves), and only where every part keeps 512 of k. One token x 4096 x 7168 on
    // 8, 4, 2, 1 experts: split 1, 2, 4, 8 take 27.5, 16.1, 12.3, 10.5 us, the next
    // smaller split -, 19.2, 14.5, 11.4 us, the next larger 32.3, 18.1, 16.1 us.
    // Never by the device's real CU count: the order of the sums must not depend on it.
    const int64_t waves = experts * ((a.N + 15) / 16);
    int split = waves >= 1536 ? 1 : waves >= 768 ? 2 : waves >= 384 ? 4 : 8;
    while (split > 1 && a.K < 512 * split) split /= 2;
    if (mean > 20) return launch<64, 2, 1>(a, pairs, stream);
    if (mean > 6) {
        switch (split) {
            case 1: return launch<32, 2, 1>(a, pairs, stream);
            case 2: return launch<32, 1, 2>(a, pairs, stream);
            case 4: return launch<32, 1, 4>(a, pairs, stream);
            default: return launch<32, 1, 8>(a, pairs, stream);
        }
    }
    switch (split) {
        case 1: return launch<16, 1, 1>(a, pairs, stream);
        case 2: return launch<16, 1, 2>(a, pairs, stream);
        case 4: return launch<16, 1, 4>(a, pairs, stream);
        default: return launch<16, 1, 8>(a, pairs, stream);
    }
}

}  // namespace ep
