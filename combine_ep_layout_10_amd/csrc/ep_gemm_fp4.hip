// Products grouped by expert with both operands in MXFP4, on the matrix unit's own
// 4-bit form. For rows r of expert e:
//   out[r, c] = bf16( sum_k a[r, k] * b[e, c, k] ),
// a and b code times power of two; products are exact, sums are the matrix unit's in
// binary32, and the only other rounding is the output's.
//
// The weights go from memory straight into registers; a block of 8 waves takes up to
// TB rows of one expert by 128 / S output columns. A wave's piece is 16 columns
// of the weights as the MFMA's first operand. The reduction runs in units of 512: lane
// (g, r16) reads codes 128 g .. + 127 of its column (four 16-byte loads) with their
// four scales (one word), and MFMA t takes the t-th 32 of each group, so its scale is byte t.
// The rows (second operand) are shared by the block through LDS in slices of NC
// units, two slices deep; 16-byte chunk c of a unit of row r is stored at c ^
// row_slot(r), which meets each bank once in every read. S splits the reduction over
// the waves of a block, so that a small problem still reaches every CU: wave group ks
// takes the ks-th part of every slice, and the S sums are added in order at the end.
// Bound by reading the weights: one token on 8 experts, 4096 x 7168, 25.8 us (4.9 TB/s).
#include <type_traits>

#include "ep_fp4_dev.h"
#include "ep_rows_dev.h"

namespace ep {

namespace {

constexpr int kWaves = 8;
constexpr int kUnit = 512;  // of the reduction: 256 bytes of codes and 16 of scales a row

__device__ __forceinline__ int row_slot(int r) { return ((r & 3) << 2) | row_swizzle16(r); }

// A unit's 16 scales of a row, as the lanes load them (lane group g: scales 4 g .. 4 g +
// 3), to the form the MFMAs take: lane group g has scale 4 t + g in byte t.
__device__ __forceinline__ uint32_t scales_by_mfma(uint32_t w, uint32_t select) {
    // words 0 and 1, 2 and 3, in either half of the wave; then each in every lane group
    const auto halves = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const auto low = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
    const auto high = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
    // byte g of each
    const uint32_t a = __builtin_amdgcn_perm(low[1], low[0], select), b = __builtin_amdgcn_perm(high[1], high[0], select);
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, int size) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, size, kBufferFlags);
}

// Slices: units of a slice, and what a slice of rows takes in LDS (scales padded by
// a word a row, so that 16 rows' words lie in different banks).
template <int TB, int S>
struct Slice {
    static constexpr int B = 2, NC = B * S;       // units of a wave group, and of all
    static constexpr int kCodes = TB * NC * 256;  // bytes
    static constexpr int kPitch = NC * 16 + 4;    // scales of a row
    static constexpr int kBytes = kCodes + TB * kPitch;
};

// Rows m0 .. m0 + rows - 1 of the expert (rows <= 16 NT) by the block's columns.
template <int TB, int S, int NT>
__device__ __forceinline__ void run_tile(const Fp4Args& a, const ExpertRows& er, int e, int m0, int rows, int n0,
                                         uint8_t* s_x) {
    using L = Slice<TB, S>;
    constexpr int NC = L::NC, B = L::B, P = 2;  // P units ahead
    constexpr int kRows = NT * 16, XL = (kRows * NC * 16 + 64 * kWaves - 1) / (64 * kWaves);
    constexpr int SL = (kRows * NC * 4 + 64 * kWaves - 1) / (64 * kWaves);
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = w / (kWaves / S), cw = w % (kWaves / S);
    const int half = a.K / 2, groups = a.K / 32;  // bytes of a row's codes and scales
    const int slices = (a.K + NC * kUnit - 1) / (NC * kUnit);
    const int c0 = n0 + 16 * cw;
    const int cols = max(0, min(16, a.N - c0));
    const int64_t first_col = (int64_t)e * a.N + min(c0, a.N - 1), first_row = (int64_t)er.first + m0;
    const __amdgpu_buffer_rsrc_t rw = resource(a.b + first_col * half, cols * half);
    const __amdgpu_buffer_rsrc_t rx = resource(a.x + first_row * half, rows * half);
    const uint8_t* const w_scales = a.b_scales + first_col * groups;
    const uint8_t* const x_scales = a.x_scales + first_row * groups;

    const uint32_t select = (uint32_t)(0x0400 + 0x0101 * g);  // bytes g of two words, as v_perm_b32 names them
    u32x4_t code[P][4];
    uint32_t scale[P];
    // unit u of the reduction; columns past N, and the reduction past K, are zero
    const auto load = [&](int u, int p) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int byte = u * 256 + t * 64 + g * 16;
            code[p][t] = __builtin_amdgcn_raw_buffer_load_b128(rw, byte < half ? r16 * half + byte : kOutOfRange, 0, 0);
        }
        scale[p] = load_scales4(w_scales + (int64_t)min(r16, max(cols - 1, 0)) * groups, u * 16 + g * 4, groups);
    };
    u32x4_t xr[XL];
    uint32_t xs[SL];
    const auto load_rows = [&](int kc) {
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int q = j * 64 * kWaves + tid, row = q / (NC * 16), byte = (kc * NC * 16 + q % (NC * 16)) * 16;
            xr[j] = __builtin_amdgcn_raw_buffer_load_b128(rx, row < rows && byte < half ? row * half + byte : kOutOfRange,
                                                          0, 0);
        }
#pragma unroll
        for (int j = 0; j < SL; ++j) {
            const int q = j * 64 * kWaves + tid, row = min(q / (NC * 4), rows - 1);
            xs[j] = load_scales4(x_scales + (int64_t)row * groups, (kc * NC * 4 + q % (NC * 4)) * 4, groups);
        }
    };
    const auto store_rows = [&](int kc) {
        uint8_t* const at = s_x + (kc & 1) * L::kBytes;
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int q = j * 64 * kWaves + tid, row = q / (NC * 16), c = q % (NC * 16);
            if (row < kRows) *(u32x4_t*)(at + row * (NC * 256) + ((c ^ row_slot(row & 15)) << 4)) = xr[j];
        }
#pragma unroll
        for (int j = 0; j < SL; ++j) {  // scale 4 t + g of a unit to byte t of word g
            const int q = j * 64 * kWaves + tid, row = q / (NC * 4), c = q % (NC * 4);
            if (row < kRows) {
                uint8_t* const to = at + L::kCodes + row * L::kPitch + c / 4 * 16 + c % 4;
                const uint32_t w = place_scales4(xs[j], (kc * NC * 4 + c) * 4, groups);
#pragma unroll
                for (int i = 0; i < 4; ++i) to[4 * i] = (uint8_t)(w >> (8 * i));
            }
        }
    };

    load_rows(0);
#pragma unroll
    for (int p = 0; p < P; ++p) load(ks * B + p, p);
    f32x4_t acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    store_rows(0);
    wait_lgkmcnt0();
    block_barrier();

    for (int kc = 0; kc < slices; ++kc) {
        // the next slice of rows travels while this one is used; its place in LDS
        // was last read a barrier ago
        if (kc + 1 < slices) load_rows(kc + 1);
        const uint8_t* const x = s_x + (kc & 1) * L::kBytes;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int p = b % P, u = ks * B + b;
            uint32_t row_scale[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                row_scale[n] = *(const uint32_t*)(x + L::kCodes + (16 * n + r16) * L::kPitch + u * 16 + g * 4);
            const uint32_t col_scale = scales_by_mfma(place_scales4(scale[p], (kc * NC + u) * 16 + g * 4, groups), select);
            const auto part = [&](auto tt) {
                constexpr int t = decltype(tt)::value;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const u32x4_t v = *(const u32x4_t*)(x + (16 * n + r16) * (NC * 256) +
                                                        ((16 * u + ((4 * t + g) ^ row_slot(r16))) << 4));
                    acc[n] = mfma_fp4<t, t>(code[p][t], v, acc[n], col_scale, row_scale[n]);
                }
            };
            part(std::integral_constant<int, 0>());
            part(std::integral_constant<int, 1>());
            part(std::integral_constant<int, 2>());
            part(std::integral_constant<int, 3>());
            // the unit P further on in this wave's order: b + P of this slice, or of the next
            load((b + P < B ? kc : kc + 1) * NC + ks * B + (b + P) % B, p);
        }
        if (kc + 1 < slices) store_rows(kc + 1);
        wait_lgkmcnt0();
        block_barrier();
    }

    if (S > 1) {  // the groups' sums, in order
        f32x4_t* sum = (f32x4_t*)s_x;
        if (ks > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) sum[(w * NT + n) * 64 + lane] = acc[n];
        }
        wait_lgkmcnt0();
        block_barrier();
        if (ks > 0) return;
#pragma unroll
        for (int s = 1; s < S; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] += sum[((s * (kWaves / S) + cw) * NT + n) * 64 + lane];
    }
    // lane: row r16 of each piece, columns 4 g .. 4 g + 3
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = 16 * n + r16, col = c0 + 4 * g;
        if (row < rows && col < a.N)
            *(uint2*)(a.out + (first_row + row) * a.N + col) =
                make_uint2(pack_bf16x2(acc[n][0], acc[n][1]), pack_bf16x2(acc[n][2], acc[n][3]));
    }
}

template <int TB, int S>
__global__ __launch_bounds__(64 * kWaves) void k_grouped_gemm_fp4_stream(Fp4Args a) {
    constexpr int kCols = 16 * kWaves / S;
    __shared__ __attribute__((aligned(16))) uint8_t s_x[2 * Slice<TB, S>::kBytes];
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
    if (TB == 16) return run_tile<TB, S, 1>(a, er, e, m0, rows, n0, s_x);
    switch ((rows + 15) / 16) {
        case 1: return run_tile<TB, S, 1>(a, er, e, m0, rows, n0, s_x);
        case 2: return run_tile<TB, S, TB == 64 ? 2 : 1>(a, er, e, m0, rows, n0, s_x);
        case 3: return run_tile<TB, S, TB == 64 ? 3 : 1>(a, er, e, m0, rows, n0, s_x);
        default: return run_tile<TB, S, TB == 64 ? 4 : 1>(a, er, e, m0, rows, n0, s_x);
    }
}

// ---------------------------------------------------------------- whole tiles: 8 waves, 256 x 256

// Wave (wm, wn) computes the 32-row pieces 2 i + wm of the tile by columns 64 wn ..
// + 63, with v_mfma_scale_f32_16x16x128. The reduction runs in steps of 256: both
// operands' slices (rows of 128 bytes, whole cache lines) move from memory to LDS by
// DMA, two steps deep. Lane (g, r16) of the MFMA reads chunks f(g) and f(g) + 1 (16
// bytes, 32 codes) of its row, f = 0, 6, 2, 4, whose scales are two neighbouring bytes.
// Chunk c of row r is stored at c ^ (r / 2 mod 8): with these f a read meets each bank
// once. Scales move in slabs of four steps, 32 bytes a row, two slabs deep; of 16 rows the
// first halves, then the second ones, for the banks again. WORDS: their rows are whole
// words of four bytes, as the DMA needs them. Otherwise a slab's 32 bytes start at
// the word that a row's part starts in, up to 3 bytes before it, and hold three steps; all
// rows of a lane are off by the same number of bytes, since 16 of them are whole words.
// Words that would reach past the tile's last row are left out: the up to 3 scales lost
// there are read apart and put in place in the last steps.
//
// Schedule: the waves form two groups (wm) half a step apart: while one group's MFMAs
// run, the other reads its operands from LDS, then a barrier exchanges the roles.
// Group 0 reads step kb in interval 2 kb, group 1 in the next. The rows' slice is kept
// in two halves, one for each group's pieces, since a half is free one interval after
// its own group has read it. With S steps in LDS,
//   interval 2 kb      sends B of step kb + S - 1 (all waves),
//   interval 2 kb + 1  group 1 sends its own half of A of step kb + S - 1, group 0 its own
//                      half of A of step kb + S; every fourth one the next slab.
// What is sent has 2 S - 2 intervals to land. S is 2, and 3 for tiles of up to 64 rows, which
// wait for the weights (1,024 rows on 64 experts, 4096 x 7168: 177 us, with two steps 193).
//
// 65,536 rows on 32 experts, 4096 x 7168: 0.98 ms settled (0.96 to 1.01 from card to card, 3.9
// PFLOP/s), without WORDS 1.34. MFMAs are
// 55 % busy, at the 1.6 to 1.7 GHz that power leaves; without the DMA it is 0.78 ms, with MFMAs,
// barriers and stores alone 0.73.
constexpr int kTile = 256;
constexpr int kStepBytes = 128;                  // of a row: 256 codes
constexpr int kHalfA = 128 * kStepBytes;         // bytes of a group's half of a slice of A
constexpr int kSliceB = kTile * kStepBytes;
constexpr int kSlabRows = 2 * kTile;             // A's, then B's
constexpr int kSlabRow = 32;                     // bytes of a row in a slab of scales
template <bool WORDS>
constexpr int kSlabSteps = WORDS ? 4 : 3;
// Rows of a tile; 256 of them and the scales of any alignment take more registers than there are.
template <bool WORDS>
constexpr int kTileRows = WORDS ? 256 : 192;
constexpr int kSlab = kSlabRows * kSlabRow;
constexpr int kTileLds = 4 * kHalfA + 2 * kSliceB + 2 * kSlab;  // all of the CU's 160 KiB
constexpr int kStoreLds = 4096;

// LDS of a tile. MI: 32-row pieces of a wave; place: of a step, kb mod kSteps.
template <int MI>
struct TileLds {
    static constexpr int kSteps = MI == 1 ? 3 : 2;
    static constexpr int kHalf = MI == 1 ? kHalfA / 4 : kHalfA;
    static_assert(kSteps * (2 * kHalf + kSliceB) <= 4 * kHalfA + 2 * kSliceB, "the slabs lie behind the steps");
    uint32_t base;
    __device__ __forceinline__ uint32_t a(int place, int half) const { return base + (2 * place + half) * kHalf; }
    __device__ __forceinline__ uint32_t b(int place) const { return base + 2 * kSteps * kHalf + place * kSliceB; }
    __device__ __forceinline__ uint32_t slab(int j) const { return base + 4 * kHalfA + 2 * kSliceB + (j & 1) * kSlab; }
    // the place of the step d <= kSteps further on
    __device__ __forceinline__ static int after(int place, int d) { return place + d >= kSteps ? place + d - kSteps : place + d; }
};

// What a wave sends. MI: 32-row pieces of a wave.
template <int MI, bool WORDS>
struct Sender {
    const uint8_t *a, *b, *s;        // of the tile, reduction step 0; s: this wave's scales
    int half, groups;                // bytes of a row's codes and scales
    int rows, cols, s_bytes;         // that exist
    int steps;
    uint32_t off_a[MI], off_b[4], off_s;
    int w;
    TileLds<MI> lds;

    __device__ __forceinline__ void init(const Fp4Args& g, int64_t first_row, int64_t first_col, int n_rows, int n_cols) {
        const int lane = lane_id(), pos = lane & 7;
        rows = n_rows;
        cols = n_cols;
        a = g.x + first_row * half;
        b = g.b + first_col * half;
        // a group sends its own pieces
#pragma unroll
        for (int j = 0; j < MI; ++j) {
            const int q = (w & 3) * MI + j, in = (q & 3) * 8 + (lane >> 3);  // 8 rows a load
            off_a[j] = __umul24(32 * (2 * (q >> 2) + (w >> 2)) + in, half) + 16 * (pos ^ ((in >> 1) & 7));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = (4 * w + j) * 8 + (lane >> 3);
            off_b[j] = __umul24(r, half) + 16 * (pos ^ ((r >> 1) & 7));
        }
        // scales: waves 0 to 3 those of 64 rows of A each, waves 4 to 7 of B
        const int r0 = 64 * (w & 3), left = (w >= 4 ? cols : rows) - r0;
        s = (w >= 4 ? g.b_scales + first_col * groups : g.x_scales + first_row * groups) + (int64_t)r0 * groups;
        if (WORDS) {
            s_bytes = max(0, left * groups);
            off_s = __umul24((lane >> 5) * 16 + (lane & 15), groups) + (lane & 16);
        } else {
            const int before = (uintptr_t)s & 3;
            s -= before;
            s_bytes = left > 0 ? (before + left * groups) & ~3 : 0;
            off_s = ((before + __umul24(lane >> 1, groups)) & ~3u) + 16 * (lane & 1);
        }
    }
    __device__ __forceinline__ void send_a(int kb, int place, int j) const {
        dma16(a + (int64_t)kb * kStepBytes, kb < steps ? rows * half - kb * kStepBytes : 0, off_a[j],
              lds.a(place, w >> 2) + ((w & 3) * MI + j) * 1024);
    }
    __device__ __forceinline__ void send_b(int kb, int place, int j) const {
        dma16(b + (int64_t)kb * kStepBytes, kb < steps ? cols * half - kb * kStepBytes : 0, off_b[j],
              lds.b(place) + (4 * w + j) * 1024);
    }
    // slab j: steps kSlabSteps j on; a load takes 32 rows
    __device__ __forceinline__ void send_slab(int j) const {
        constexpr int kSteps = kSlabSteps<WORDS>;
        const int size = kSteps * j < steps ? max(0, s_bytes - j * 8 * kSteps) : 0;
#pragma unroll
        for (int d = 0; d < 2; ++d)
            dma16(s + (int64_t)j * 8 * kSteps, size, off_s + 32 * d * groups, lds.slab(j) + (2 * w + d) * 1024);
    }
};

__device__ __forceinline__ u32x4_t read_codes(uint32_t at) { return read_lds_words(at); }
// The pairs of scales of rows 0 and 16 on from `at`, in a word: both rows' words with
// one LDS read, of each the half that `select` names.
typedef uint32_t __attribute__((address_space(3), may_alias)) lds_u32_t;
__device__ __forceinline__ uint32_t read_scales(uint32_t at, uint32_t select) {
    const uint32_t low = *(const lds_u32_t*)at, high = *(const lds_u32_t*)(at + 16 * kSlabRow);
    return __builtin_amdgcn_perm(high, low, select);
}

// The same for scales at any byte: `at` the word that the pairs start in, or lie in the
// next, `shift` bytes on.
__device__ __forceinline__ uint32_t read_scales(uint32_t at, int shift) {
    const lds_u32_t *low = (const lds_u32_t*)at, *high = (const lds_u32_t*)(at + 16 * kSlabRow);
    const uint32_t l = __builtin_amdgcn_alignbyte(low[1], low[0], shift), h = __builtin_amdgcn_alignbyte(high[1], high[0], shift);
    return __builtin_amdgcn_perm(h, l, 0x05040100u);
}

// The pairs of scales of groups g and g + 1 of rows r and r + 16 near a row's end: the `n`
// last scales of row `last`, before `end`, which whole words do not reach, in their place;
// zeros past the last group: 2^-127 by 2^-127.
__device__ __forceinline__ uint32_t finish_scales(uint32_t pairs, int r, int g, int groups, int last, const uint8_t* end) {
    const int first = groups - (int)((uintptr_t)end & 3);
    uint32_t keep = 0xFFFF, mask = 0, bytes = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (g + b >= groups) {
            keep &= ~(0xFFu << (8 * b));
        } else if (g + b >= first) {
            mask |= 0xFFu << (8 * b);
            bytes |= (uint32_t)end[g + b - groups] << (8 * b);
        }
    }
    if (r == last) pairs = (pairs & ~mask) | bytes;
    if (r + 16 == last) pairs = (pairs & ~(mask << 16)) | bytes << 16;
    return pairs & (keep | keep << 16);
}

// The loop of one group of waves over all steps. scales_a, scales_b: the tile's.
template <bool SECOND, int MI, bool WORDS>
__device__ __forceinline__ void multiply(const Sender<MI, WORDS>& send, f32x4_t (&acc)[2 * MI][4], int wn, int groups,
                                         const uint8_t* scales_a, const uint8_t* scales_b) {
    constexpr int kSlab = kSlabSteps<WORDS>;
    const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
    const int first = g == 0 ? 0 : g == 1 ? 6 : g == 2 ? 2 : 4;  // chunk of half 0
    const uint32_t row = r16 * kStepBytes + ((first ^ ((r16 >> 1) & 7)) << 4);
    const uint32_t select = first & 2 ? 0x07060302u : 0x05040100u;
    // where in its slab a lane's first pair of scales starts: A's in the lowest 8 bits, B's in the next
    const int bytes = (((int)(uintptr_t)scales_a + r16 * groups) & 3) + first + ((((int)(uintptr_t)scales_b + r16 * groups) & 3) + first) * 256;
    using Lds = TileLds<MI>;
    constexpr int S = Lds::kSteps, kMore = (S - 2) * (4 + MI);  // loads that may be on their way beside those of two steps
    const Lds lds = send.lds;
    int place = 0;
    for (int kb = 0; kb < send.steps; ++kb, place = Lds::after(place, 1)) {
        const uint32_t at_a = lds.a(place, SECOND ? 1 : 0) + row, at_b = lds.b(place) + wn * 64 * kStepBytes + row;
        const int slab_of = kb / kSlab, in_slab = kb - kSlab * slab_of;
        const uint32_t at_s = lds.slab(slab_of) + (WORDS ? r16 * 16 + (in_slab >> 1) * 256 + (in_slab & 1) * 8 + (first & 4)
                                                         : r16 * kSlabRow + in_slab * 8);
        u32x4_t fa[2][2 * MI], fb[2][4];
        uint32_t sa[MI], sb[2];  // two pieces' pairs of scales a word
        const auto scales = [&](int piece, int byte) {
            const uint32_t at = at_s + piece * kSlabRow;
            return WORDS ? read_scales(at, select) : read_scales(at + (byte & ~3), byte & 3);
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) sb[j] = scales(kTile + 64 * wn + 32 * j, bytes >> 8);
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = scales(64 * i + (SECOND ? 32 : 0), bytes & 255);
        if (!WORDS && 8 * kb + 11 > groups) {  // at most two scales behind this step; ahead of the codes, for their registers
#pragma unroll
            for (int j = 0; j < 2; ++j)
                sb[j] = finish_scales(sb[j], 64 * wn + 32 * j + r16, 8 * kb + first, groups, send.cols - 1,
                                      scales_b + (int64_t)send.cols * groups);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                sa[i] = finish_scales(sa[i], 64 * i + (SECOND ? 32 : 0) + r16, 8 * kb + first, groups, send.rows - 1,
                                      scales_a + (int64_t)send.rows * groups);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[h][j] = read_codes((at_b ^ (h << 4)) + 16 * kStepBytes * j);
#pragma unroll
            for (int i = 0; i < 2 * MI; ++i) fa[h][i] = read_codes((at_a ^ (h << 4)) + 16 * kStepBytes * i);
        }
        const bool slab = in_slab == 0;  // interval 2 kb + 1 sends the next slab
        if (SECOND) {  // interval 2 kb + 1
#pragma unroll
            for (int j = 0; j < MI; ++j) send.send_a(kb + S - 1, Lds::after(place, S - 1), j);
            if (slab) send.send_slab(slab_of + 1);
            // B of step kb + 1 has landed, and all before it
            if (slab) wait_vmcnt<MI + kMore + 2>();
            else wait_vmcnt<MI + kMore>();
        } else {  // interval 2 kb
#pragma unroll
            for (int j = 0; j < 4; ++j) send.send_b(kb + S - 1, Lds::after(place, S - 1), j);
        }
        wait_lgkmcnt0();
        block_barrier();
        if (WORDS && 8 * kb + first >= groups) {  // past the reduction: 2^-127 by 2^-127
#pragma unroll
            for (int j = 0; j < 2; ++j) sb[j] = 0u;
#pragma unroll
            for (int i = 0; i < MI; ++i) sa[i] = 0u;
        }
        __builtin_amdgcn_s_setprio(1);
        // operands swapped: each 16 x 16 piece comes out transposed, lane (g, r16) holding
        // row r16 and columns 4 g .. 4 g + 3
        const auto part = [&](auto hh) {
            constexpr int h = decltype(hh)::value;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if (SECOND) {  // interval 2 kb + 2
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        if (d * 2 * MI / 4 == h * MI + i) send.send_b(kb + S, place, d);
                } else {  // interval 2 kb + 1
#pragma unroll
                    for (int d = 0; d < MI; ++d)
                        if (d * 2 == h * MI + i) send.send_a(kb + S, place, d);
                    if (i == MI - 1 && h == 1 && slab) send.send_slab(slab_of + 1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    acc[2 * i][2 * j] = mfma_fp4<h, h>(fb[h][2 * j], fa[h][2 * i], acc[2 * i][2 * j], sb[j], sa[i]);
                    acc[2 * i][2 * j + 1] = mfma_fp4<2 + h, h>(fb[h][2 * j + 1], fa[h][2 * i], acc[2 * i][2 * j + 1], sb[j], sa[i]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    acc[2 * i + 1][2 * j] = mfma_fp4<h, 2 + h>(fb[h][2 * j], fa[h][2 * i + 1], acc[2 * i + 1][2 * j], sb[j], sa[i]);
                    acc[2 * i + 1][2 * j + 1] = mfma_fp4<2 + h, 2 + h>(fb[h][2 * j + 1], fa[h][2 * i + 1], acc[2 * i + 1][2 * j + 1], sb[j], sa[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        part(std::integral_constant<int, 0>());
        part(std::integral_constant<int, 1>());
        __builtin_amdgcn_s_setprio(0);
        if (SECOND) {  // this group's half of A of step kb + 1 has landed
            wait_vmcnt<4 + kMore>();
        } else {  // B of step kb + 1 has landed, and all before it
            if (slab) wait_vmcnt<MI + kMore + 2>();
            else wait_vmcnt<MI + kMore>();
        }
        block_barrier();
    }
}

// Rows of the tile: MI 32-row pieces for each group.
template <int MI, bool WORDS>
__device__ __forceinline__ void run_whole(const Fp4Args& a, const ExpertRows& er, int e, int m0, int rows, int n0,
                                          bool last, uint32_t lds) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w >> 2, wn = w & 3;
    const int64_t first_row = (int64_t)er.first + m0;
    Sender<MI, WORDS> send;
    send.half = a.K / 2;
    send.groups = a.K / 32;
    send.steps = (a.K + 255) / 256;
    send.w = w;
    send.lds.base = lds;
    send.init(a, first_row, (int64_t)e * a.N + n0, rows, min(kTile, a.N - n0));
    f32x4_t acc[2 * MI][4];
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t *const scales_a = a.x_scales + first_row * send.groups,
                  *const scales_b = a.b_scales + ((int64_t)e * a.N + n0) * send.groups;
    // ahead of interval 0: slab 0, B and A of all steps but one, and group 0's half of A of that
    constexpr int S = TileLds<MI>::kSteps, kMore = (S - 2) * (4 + MI);
    send.send_slab(0);
#pragma unroll
    for (int kb = 0; kb < S - 1; ++kb) {
#pragma unroll
        for (int j = 0; j < 4; ++j) send.send_b(kb, kb, j);
#pragma unroll
        for (int j = 0; j < MI; ++j) send.send_a(kb, kb, j);
    }
    if (wm == 0) {
#pragma unroll
        for (int j = 0; j < MI; ++j) send.send_a(S - 1, S - 1, j);
    }
    wait_vmcnt<MI + kMore>();  // group 1's half of step 0 may still be on its way
    block_barrier();
    const int groups = a.K / 32;
    if (wm == 0) {
        multiply<false, MI, WORDS>(send, acc, wn, groups, scales_a, scales_b);
        block_barrier();
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) send.send_b(S - 1, S - 1, j);
        wait_vmcnt<4 + kMore>();
        block_barrier();  // half a step later
        multiply<true, MI, WORDS>(send, acc, wn, groups, scales_a, scales_b);
    }
    wait_vmcnt<0>();
    block_barrier();  // no wave reads or fills the ring any more

    // stores: each 16 rows are turned through the wave's own LDS, so that neighbouring
    // lanes store neighbouring columns; 16-byte chunks XORed with half the row
    const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
    const uint32_t at = lds + w * kStoreLds;
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u32x2_t v = {pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
            write_lds(at + r16 * 128 + (((2 * j + (g >> 1)) ^ (r16 >> 1)) << 4) + (g & 1) * 8, v);
        }
        const int row = 32 * (i & ~1) + 32 * wm + 16 * (i & 1), col = n0 + 64 * wn + 8 * (lane & 7);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = 8 * s + (lane >> 3);
            const u32x4_t v = read_lds_words(at + r * 128 + (((lane & 7) ^ (r >> 1)) << 4));
            if (row + r < rows && col < a.N) *(u32x4_t*)(a.out + (first_row + row + r) * a.N + col) = v;
        }
    }
    if (a.rows.zero_pad && last) clear_padding<kTile>(a.out, a.N, er, n0);
}

template <bool WORDS>
__global__ __launch_bounds__(512) void k_grouped_gemm_fp4(Fp4Args a) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kTileLds];
    constexpr int kRows = kTileRows<WORDS>;
    const int nt_n = (a.N + kTile - 1) / kTile;
    int e, local, m, n;
    if (!find_expert(a.rows, kRows, nt_n, &e, &local)) return;
    e = __builtin_amdgcn_readfirstlane(e);
    const ExpertRows er = expert_rows(a.rows, e);
    const int nt_m = (er.live + kRows - 1) / kRows;
    order_tiles<2>(local, nt_m, nt_n, &m, &n);
    const int each = ((er.live + nt_m - 1) / nt_m + 63) & ~63;  // rows of a tile; never leaves the last one empty
    const int m0 = __builtin_amdgcn_readfirstlane(m * each), n0 = __builtin_amdgcn_readfirstlane(n * kTile);
    const int rows = __builtin_amdgcn_readfirstlane(min(each, er.live - m0));
    const bool last = m == nt_m - 1;
    const uint32_t lds = lds_offset(s_ring);
    asm volatile("" ::"v"(s_ring) : "memory");  // the ring is written by the DMA alone
    switch ((rows + 63) / 64) {
        case 1: return run_whole<1, WORDS>(a, er, e, m0, rows, n0, last, lds);
        case 2: return run_whole<2, WORDS>(a, er, e, m0, rows, n0, last, lds);
        case 3: return run_whole<3, WORDS>(a, er, e, m0, rows, n0, last, lds);
        default: return run_whole<kRows / 64, WORDS>(a, er, e, m0, rows, n0, last, lds);
    }
}

template <int TB, int S>
hipError_t launch(const Fp4Args& a, int64_t pairs, hipStream_t stream) {
    constexpr int kCols = 16 * kWaves / S;
    const int64_t blocks = max_row_tiles(a.rows, TB, pairs) * ((a.N + kCols - 1) / kCols);
    if (blocks > 0x7FFFFF) return hipErrorInvalidConfiguration;
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_fp4_stream", dim3((unsigned)blocks), dim3(64 * kWaves),
                           "rows %d split %d n %d k %d", TB, S, a.N, a.K);
    hipLaunchKernelGGL((k_grouped_gemm_fp4_stream<TB, S>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_whole(const Fp4Args& a, int64_t pairs, bool words, hipStream_t stream) {
    const int64_t blocks = max_row_tiles(a.rows, words ? kTileRows<true> : kTileRows<false>, pairs) * ((a.N + kTile - 1) / kTile);
    if (blocks > 0x7FFFFF) return hipErrorInvalidConfiguration;
    if (launch_debug())
        launch_debug_print("k_grouped_gemm_fp4", dim3((unsigned)blocks), dim3(512), "n %d k %d words %d", a.N, a.K, (int)words);
    if (words) hipLaunchKernelGGL(k_grouped_gemm_fp4<true>, dim3((unsigned)blocks), dim3(512), 0, stream, a);
    else hipLaunchKernelGGL(k_grouped_gemm_fp4<false>, dim3((unsigned)blocks), dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// Which kernel, by the sizes and the alignment of the scales (never by the device's CU
// count: the order of the sums must not depend on it). us:
//   top-8 of 64 experts, 4096 x 7168, mean rows       1    2    4    6    8   16   32   64  128
//     16 rows a tile                                127  171  187  190  194  253  380  642 1171
//     64 rows                                       127  172  187  190  194  201  210  293  440
//     whole tiles                                   119  160  171  174  176  178  182  216  245
//   top-1 of 32 experts, 4096 x 4096 (512 whole tiles)
//     16 rows                                      40.6 52.3 55.9      57.8 75.8  111  195
//     whole tiles                                  44.4 47.7 52.7      55.8 56.6 59.5 68.7
//   top-1 of 8 experts, 4096 x 7168 (128 whole tiles)
//     16 rows                                      21.7      26.0      26.7 44.6 59.4 92.1  158
//     64 rows                                      21.8      26.2      26.8 27.8 29.7 54.3 71.2
//     whole tiles                                  26.4      30.9      31.3 32.0 33.7 47.4 52.3
//   top-1 of 8 experts, 1536 x 2048 (48 whole tiles)
//     16 rows, split 2                                        6.8       6.9       9.4 16.4 27.1
//     64 rows, split 2                                        7.0       7.0       7.6 12.2 14.4
//     64 rows                                                 8.8       8.8       9.8 11.4 11.6
//     whole tiles                                             9.5       9.5       9.7 12.7 15.0
// and where rows of scales are no whole words:
//   top-8 of 64 experts, 4096 x 7200                       4         8   16   32   64  128
//     64 rows                                            220       226  232  241  333  488
//     whole tiles (192 rows)                             217       222  224  232  261  303
//   top-1 of 32 experts, 4096 x 4064
//     64 rows                                           64.2      67.6      72.2  103
//     whole tiles                                       68.7      72.6      75.4 82.9
//   top-3 of 24 experts, 1000 x 1440 (96 whole tiles)     6   12   38   64  188
//     64 rows                                           7.7  8.0  9.3 13.7 21.7
//     whole tiles                                      12.0 12.0 12.3 14.9 18.7
// Routing that is uneven, the j-th expert's share as j^-1.2, mean rows:
//   top-8 of 64 experts, 4096 x 7168                       2    8        32
//     64 rows                                            121  196       260
//     whole tiles                                        117  164       234
//   top-1 of 8 experts, 4096 x 7168                       16   32   48   64   96  128
//     64 rows                                           33.6 52.6 50.7 51.5 58.6 74.9
//     whole tiles                                       33.5 47.3 51.7 57.0 51.8 55.1
//   top-3 of 24 experts, 1000 x 1440                      12   38   64  100  188
//     64 rows                                            8.9 10.2 13.3 13.8 20.6
//     whole tiles                                       14.3 17.1 17.7 18.0 18.8
// The rule has the mean alone, and loses up to 11 % at its limits there, 30 % at the last one's;
// at that one's 12 and 38 rows it splits the reduction in two, which takes 12.3 and 12.8 (10.9 and 12.9
// where routing is even).
// Whole tiles want the chip full, which a row an expert, met by chance, does not tell; they
// take scales by DMA, so at a word's boundary.
hipError_t launch_grouped_gemm_mxfp4_rows(const Fp4Args& a, int64_t pairs, hipStream_t stream) {
    if (pairs == 0) return hipSuccess;
    const int64_t used = pairs < a.rows.E ? pairs : a.rows.E, mean = (pairs + used - 1) / used;
    // Parts of the reduction of a tile: it is split while that leaves about one block a
    // CU (256 of 8 waves), and only where every part keeps a unit. One token on 8, 4, 2, 1
    // experts, 4096 x 7168: split 1, 2, 4, 8 take 27, 13.8, 9.7, 8.0 us, the next smaller one
    // -, 19.8, 13.0, 9.1 us, the next larger -, 14.8, 14.6 us.
    const auto parts = [&](int64_t row_tiles) {
        const int64_t waves = row_tiles * used * ((a.N + 15) / 16);
        int split = waves >= 1536 ? 1 : waves >= 768 ? 2 : waves >= 384 ? 4 : 8;
        while (split > 1 && a.K < kUnit * split) split /= 2;
        return split;
    };
    const int64_t tiles = (mean + kTile - 1) / kTile * used * ((a.N + kTile - 1) / kTile);
    const bool words = a.K % 128 == 0, aligned = ((uintptr_t)a.x_scales | (uintptr_t)a.b_scales) % 4 == 0;
    const bool full = words ? (mean > 1 && tiles >= 192) || (mean > 48 && tiles >= 96)
                            : (mean > 48 && tiles >= 192) || (mean > 96 && tiles >= 96);
    if (aligned && a.K >= 128 && (full || mean > kTile)) return launch_whole(a, pairs, words, stream);
    if (mean <= 6) {
        switch (parts(1)) {
            case 1: return launch<16, 1>(a, pairs, stream);
            case 2: return launch<16, 2>(a, pairs, stream);
            case 4: return launch<16, 4>(a, pairs, stream);
            default: return launch<16, 8>(a, pairs, stream);
        }
    }
    // an expert's rows scatter around their mean
    return parts((mean + mean / 4 + 63) / 64) > 1 ? launch<64, 2>(a, pairs, stream) : launch<64, 1>(a, pairs, stream);
}

}  // namespace ep
