// Products for few rows an expert, bound by reading the weights once: with MXFP4
// weights (always this kernel) and with BF16 weights (the forward product of
// ep_gemm_bf16.hip hands its small batches over). For rows r of expert e:
//   out[r, c] = bf16( sum_k a[r, k] * w[e, c, k] )
// MXFP4 (OCP Microscaling: E2M1 codes, two to a byte, the lower nibble first, one
// E8M0 scale for each 32 consecutive k): w = e2m1(code) * 2^(scale - 127). A code
// times its scale is a bf16 value (two significant bits), so the conversion is
// exact (v_cvt_scalef32_pk_bf16_fp4, all codes and scales checked on MI355X).
// Either way products are exact in binary32, the MFMA accumulates them in
// binary32, and the only rounding is the output's.
//
// The weights go from memory straight into registers, about kInFlight loads
// ahead. A block of 8 waves takes up to TB rows of one expert by 128 MC / S output
// columns. A wave's piece is 16 MC columns of the weights as the MFMA's first
// operand, a chunk of 128 k at a time in four MFMAs: MXFP4 lane (g, r16) reads the
// 32 codes of group g of column r16 with one 16-byte load, and MFMA t takes word t
// (k = 32 g + 8 t .. + 7); BF16 reads the operand of MFMA t (k = 32 t + 8 g .. + 7).
// The rows (the second operand, read in the same order of k) are shared by the
// block through LDS in slices of KC values of k, two slices deep; 16-byte chunk c of
// row r is stored at c ^ W::row_slot(r), which meets each bank once in every read.
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

// The 8 codes of one word (lowest nibble first) times 2^(e8m0 - 127).
__device__ __forceinline__ bf16x8_t decode_mxfp4(uint32_t word, float scale) {
    const bf16x2_v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0);
    const bf16x2_v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1);
    const bf16x2_v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2);
    const bf16x2_v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3);
    return (bf16x8_t){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, int size) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, size, kBufferFlags);
}

// MXFP4 weights of a wave: 16 MC columns from column c0 on, B chunks of a slice
// of NC for each wave group, P slices ahead. Columns past N, and k past K, are zero.
template <int MC, int S>
struct Mxfp4Weights {
    static constexpr int NC = MC == 1 ? 8 : 4, B = NC / S;
    static constexpr int P = kInFlight > B * MC ? kInFlight / (B * MC) : 1;
    static constexpr int R = P > 1 ? P : 2;  // slices whose scales are in registers
    // Scales: the 4 B bytes a column of a wave's chunks, as words (word b: chunk
    // b, byte g: group g). A byte load for each chunk would cost as many requests
    // as the codes do (313 against 220 us at 128 tokens x top-8, 64 experts, 4096 x 7168).
    u32x4_t code[P][B][MC];
    uint32_t scale[R][B][MC];
    __amdgpu_buffer_rsrc_t codes;
    const uint8_t* scales;
    int K, groups, cols, slices, ks, r16, g;

    __device__ __forceinline__ static int row_slot(int r) { return (row_swizzle16(r) << 2) | (r & 3); }
    __device__ __forceinline__ static int row_chunk(int t, int g) { return 4 * g + t; }

    __device__ __forceinline__ void init(const StreamArgs& a, int e, int c0, int wave_part, int n_slices) {
        K = a.K;
        groups = K / 32;
        cols = max(0, min(16 * MC, a.N - c0));
        slices = n_slices;
        ks = wave_part;
        r16 = lane_id() & 15;
        g = lane_id() >> 4;
        const int64_t row = (int64_t)e * a.N + min(c0, a.N - 1);
        codes = resource((const uint8_t*)a.b + row * (K / 2), cols * (K / 2));
        scales = a.b_scales + row * groups;
    }
    __device__ __forceinline__ void load(int kc, int p, int b) {
        const int group = (kc * NC + ks * B + b) * 4 + g;
#pragma unroll
        for (int c = 0; c < MC; ++c)
            code[p][b][c] = __builtin_amdgcn_raw_buffer_load_b128(
                codes, group < groups ? (16 * c + r16) * (K / 2) + 16 * group : kOutOfRange, 0, 0);
    }
    __device__ __forceinline__ void load_scales(int kc, int r) {
        if (kc >= slices) return;
        const int first = (kc * NC + ks * B) * 4;
#pragma unroll
        for (int c = 0; c < MC; ++c) {
            const uint8_t* s = scales + (int64_t)min(16 * c + r16, max(cols - 1, 0)) * groups + first;
            if ((kc + 1) * (128 * NC) <= K) {
#pragma unroll
                for (int b = 0; b < B; ++b) __builtin_memcpy(&scale[r][b][c], s + 4 * b, 4);  // any alignment
            } else {  // the last slice may end inside a word
#pragma unroll
                for (int b = 0; b < B; ++b)
                    scale[r][b][c] = first + 4 * b + g < groups ? (uint32_t)s[4 * b + g] << (8 * g) : 0u;
            }
        }
    }
    __device__ __forceinline__ void first_loads() {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            load_scales(p, p);
#pragma unroll
            for (int b = 0; b < B; ++b) load(p, p, b);
        }
    }
    // around slice kc, which is number r of a round of R
    __device__ __forceinline__ void begin_slice(int kc, int r) {
        if (P == 1) load_scales(kc + 1, (r + 1) % R);
    }
    __device__ __forceinline__ void end_slice(int kc, int r) {
        if (P > 1) load_scales(kc + P, r);
    }
    __device__ __forceinline__ bf16x8_t operand(int r, int b, int t, int c) const {
        const uint32_t power = __builtin_amdgcn_ubfe(scale[r][b][c], 8 * g, 8) << 23;
        return decode_mxfp4(code[r % P][b][c][t], __uint_as_float(power));
    }
};

// BF16 weights, likewise.
template <int MC, int S>
struct Bf16Weights {
    static constexpr int NC = S > 4 ? S : 4, B = NC / S;
    static constexpr int P = B == 1 ? 2 : 1, R = P;
    u32x4_t w[P][B][MC][4];
    __amdgpu_buffer_rsrc_t weights;
    int K, ks, r16, g;

    __device__ __forceinline__ static int row_slot(int r) { return ((r & 3) << 2) | row_swizzle16(r); }
    __device__ __forceinline__ static int row_chunk(int t, int g) { return 4 * t + g; }

    __device__ __forceinline__ void init(const StreamArgs& a, int e, int c0, int wave_part, int) {
        K = a.K;
        ks = wave_part;
        r16 = lane_id() & 15;
        g = lane_id() >> 4;
        const int64_t row = (int64_t)e * a.N + min(c0, a.N - 1);
        weights = resource((const uint16_t*)a.b + row * K, max(0, min(16 * MC, a.N - c0)) * K * 2);
    }
    __device__ __forceinline__ void load(int kc, int p, int b) {
#pragma unroll
        for (int c = 0; c < MC; ++c)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int k = (kc * NC + ks * B + b) * 128 + 32 * t + 8 * g;
                w[p][b][c][t] = __builtin_amdgcn_raw_buffer_load_b128(
                    weights, k < K ? ((16 * c + r16) * K + k) * 2 : kOutOfRange, 0, 0);
            }
    }
    __device__ __forceinline__ void first_loads() {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int b = 0; b < B; ++b) load(p, p, b);
    }
    __device__ __forceinline__ void begin_slice(int, int) {}
    __device__ __forceinline__ void end_slice(int, int) {}
    __device__ __forceinline__ bf16x8_t operand(int r, int b, int t, int c) const {
        return __builtin_bit_cast(bf16x8_t, w[r][b][c][t]);
    }
};

// Rows m0 .. m0 + rows - 1 of the expert (rows <= 16 NT) by the block's columns.
template <class W, int TB, int MC, int S, int NT>
__device__ __forceinline__ void run_tile(const StreamArgs& a, const ExpertRows& er, int e, int m0, int rows, int n0,
                                         uint8_t* s_x) {
    constexpr int KC = 128 * W::NC, B = W::B, P = W::P, R = W::R;
    constexpr int XL = NT * 16 * KC * 2 / 16 / (64 * kWaves);  // 16-byte loads a thread for a slice of rows
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = w / (kWaves / S), cw = w % (kWaves / S);
    const int slices = (a.K + KC - 1) / KC;
    const int c0 = n0 + 16 * MC * cw;
    W weights;
    weights.init(a, e, c0, ks, slices);
    const __amdgpu_buffer_rsrc_t rx = resource(a.x + ((int64_t)er.first + m0) * a.K, rows * a.K * 2);

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
            *(u32x4_t*)(s_x + stage * (TB * KC * 2) + row * (KC * 2) + ((c ^ W::row_slot(row)) << 4)) = xr[j];
        }
    };

    load_rows(0);
    weights.first_loads();
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
            const int kc = kc0 + r;
            if (kc >= slices) break;
            // the next slice of rows travels while this one is used; its place in LDS
            // was last read a barrier ago
            if (kc + 1 < slices) load_rows(kc + 1);
            weights.begin_slice(kc, r);
            const uint8_t* x = s_x + (kc & 1) * (TB * KC * 2) + r16 * (KC * 2);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int sub = ks * B + b;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    bf16x8_t f[MC];
#pragma unroll
                    for (int c = 0; c < MC; ++c) f[c] = weights.operand(r, b, t, c);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const bf16x8_t v =
                            *(const bf16x8_t*)(x + n * (16 * KC * 2) + sub * 256 + ((W::row_chunk(t, g) ^ W::row_slot(r16)) << 4));
#pragma unroll
                        for (int c = 0; c < MC; ++c)
                            acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[c], v, acc[n][c], 0, 0, 0);
                    }
                }
                weights.load(kc + P, r % P, b);
            }
            weights.end_slice(kc, r);
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

template <template <int, int> class WT, int TB, int MC, int S>
__global__ __launch_bounds__(64 * kWaves) void k_grouped_gemm_stream(StreamArgs a) {
    using W = WT<MC, S>;
    constexpr int kCols = 16 * MC * kWaves / S;
    __shared__ __attribute__((aligned(16))) uint8_t s_x[2 * TB * 128 * W::NC * 2];
    const int nt_n = (a.N + kCols - 1) / kCols;
    int e, local;
    if (!find_expert(a.rows, TB, nt_n, &e, &local)) return;
    e = __builtin_amdgcn_readfirstlane(e);
    const ExpertRows er = expert_rows(a.rows, e);
    // row tiles of one column tile are neighbours: they read the same weights.
    // An expert's rows are cut into tiles of equal size, rounded up to 16.
    const int nt_m = (er.live + TB - 1) / TB, m = local % nt_m;
    const int each = ((er.live + nt_m - 1) / nt_m + 15) & ~15;
    const int m0 = __builtin_amdgcn_readfirstlane(m * each);
    const int rows = __builtin_amdgcn_readfirstlane(min(each, er.live - m0));
    const int n0 = __builtin_amdgcn_readfirstlane(local / nt_m * kCols);
    if (a.rows.zero_pad && m == nt_m - 1) clear_padding<kCols>(a.out, a.N, er, n0);
    switch ((rows + 15) / 16) {
        case 1: return run_tile<W, TB, MC, S, 1>(a, er, e, m0, rows, n0, s_x);
        case 2: if (TB >= 32) return run_tile<W, TB, MC, S, TB >= 32 ? 2 : 1>(a, er, e, m0, rows, n0, s_x); break;
        case 3: if (TB >= 64) return run_tile<W, TB, MC, S, TB >= 64 ? 3 : 1>(a, er, e, m0, rows, n0, s_x); break;
        default: if (TB >= 64) return run_tile<W, TB, MC, S, TB >= 64 ? 4 : 1>(a, er, e, m0, rows, n0, s_x); break;
    }
}

template <template <int, int> class WT, int TB, int MC, int S>
hipError_t launch(const StreamArgs& a, int64_t pairs, hipStream_t stream) {
    constexpr int kCols = 16 * MC * kWaves / S;
    const int64_t blocks = max_row_tiles(a.rows, TB, pairs) * ((a.N + kCols - 1) / kCols);
    if (blocks > 0x7FFFFF) return hipErrorInvalidConfiguration;
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_stream", dim3((unsigned)blocks), dim3(64 * kWaves),
                           "rows %d split %d n %d k %d", TB, S, a.N, a.K);
    hipLaunchKernelGGL((k_grouped_gemm_stream<WT, TB, MC, S>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

// Parts of the reduction. It is split while that leaves about one block a CU (256
// of 8 waves), and only where every part keeps 512 of k. MXFP4, one token x 4096 x
// 7168 on 8, 4, 2, 1 experts: split 1, 2, 4, 8 take 27.5, 16.1, 12.3, 10.5 us, the
// next smaller split -, 19.2, 14.5, 11.4 us, the next larger 32.3, 18.1, 16.1 us.
// Never by the device's real CU count: the order of the sums must not depend on it.
int parts(const StreamArgs& a, int64_t pairs) {
    const int64_t waves = (pairs < a.rows.E ? pairs : a.rows.E) * ((a.N + 15) / 16);
    int split = waves >= 1536 ? 1 : waves >= 768 ? 2 : waves >= 384 ? 4 : 8;
    while (split > 1 && a.K < 512 * split) split /= 2;
    return split;
}

// MC1: 16 MC1 columns a wave when the reduction is not split.
template <template <int, int> class WT, int TB, int MC1>
hipError_t launch_split(const StreamArgs& a, int64_t pairs, hipStream_t stream) {
    switch (parts(a, pairs)) {
        case 1: return launch<WT, TB, MC1, 1>(a, pairs, stream);
        case 2: return launch<WT, TB, 1, 2>(a, pairs, stream);
        case 4: return launch<WT, TB, 1, 4>(a, pairs, stream);
        default: return launch<WT, TB, 1, 8>(a, pairs, stream);
    }
}

}  // namespace

// Rows of a tile: enough for nearly every expert's, so that its weights are read
// once (an expert's rows scatter around their mean); smaller tiles hold less LDS
// and fewer registers. Top-8 of 64 experts, us:
//   BF16, 4096 x 4096    mean 4    6    8   10   12   16
//     16 rows               341  347  349  375  372  443
//     32 rows               343  350  353  352  355  355
//   MXFP4, 4096 x 7168   mean 4    6    8   10   12   16   20   24   28   32   48
//     16 rows               190  196  199  217  223
//     32 rows               206  207  207  209  211  216  219  223  262  300  375
//     64 rows                         209       212  216  220  226  236  245  277
// A limit keeps some distance from where it crosses, for counts that scatter more
// than these (uneven routing reads the weights twice for a tile that is too small).
hipError_t launch_grouped_gemm_mxfp4(const StreamArgs& a, int64_t pairs, hipStream_t stream) {
    if (pairs == 0) return hipSuccess;
    const int64_t mean = (pairs + a.rows.E - 1) / a.rows.E;
    if (mean > 20) return launch<Mxfp4Weights, 64, 2, 1>(a, pairs, stream);
    if (mean > 6) return launch_split<Mxfp4Weights, 32, 2>(a, pairs, stream);
    return launch_split<Mxfp4Weights, 16, 1>(a, pairs, stream);
}

hipError_t launch_grouped_gemm_bf16_stream(const StreamArgs& a, int64_t pairs, hipStream_t stream) {
    if (pairs == 0) return hipSuccess;
    const int64_t mean = (pairs + a.rows.E - 1) / a.rows.E;
    if (mean > 6) return launch_split<Bf16Weights, 32, 1>(a, pairs, stream);
    return launch_split<Bf16Weights, 16, 1>(a, pairs, stream);
}

}  // namespace ep
