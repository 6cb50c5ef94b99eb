// Quantisation to MXFP4 (OCP Microscaling Formats): for each 32 consecutive values of
// a row, with m = max|x|,
//   X = max(floor(log2 m) - 2, -127), scale byte X + 127,
//   code = E2M1(x / 2^X), rounded to nearest even and saturated at 6,
// so that the largest magnitude lies in [4, 8) before it is rounded. Powers of two
// divide exactly, so the codes' rounding is the only one; the instruction that makes
// them (v_cvt_scalef32_pk_fp4) was checked on MI355X against this formula for every
// bf16 value and every scale. 32 values with a NaN or an infinity among them have
// scale 255 (NaN) and zero codes; 32 zeros have scale 0.
//
// A lane takes 8 values, four neighbouring lanes share a scale. Bound by memory.
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kQuantWaves = 4;
constexpr int64_t kQuantBlocks = 1 << 22;  // of a launch at most

// Vectors of 8 that a lane has in flight: 65,536 rows of 7168 in bf16 with 1, 2, 3, 4, 8
// take 243, 195, 203, 212, 217 us (1.19 GB: 6.1 TB/s); weights of 8 x 4096 x 4096 in binary32
// with their values, with 1, 2, 4, 151, 153, 158 us (0.88 GB: 5.8 TB/s).
template <bool F32>
constexpr int kQuantAhead = F32 ? 1 : 2;

template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

// A word that the whole wave reads, through the scalar cache.
__device__ __forceinline__ int uniform(const int32_t* p, int64_t i) {
    return *((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p + i);
}

// Whether row `row` of the receive layout holds a pair.
__device__ __forceinline__ bool row_is_live(const QuantArgs& a, int row) {
    if (a.rows.mode == EP_MODE_COMPACT) return row < uniform(a.rows.expert_off, a.rows.E) && uniform(a.row_src, row) >= 0;
    return row % a.rows.C < uniform(a.rows.pad, row / a.rows.C);
}

// F32: x binary32, otherwise bf16. ROWS: only rows that hold a pair, each cut into
// pieces; otherwise the rows follow each other as one. A piece's loads are sent without
// a branch between them, lanes past the end at the last vector: with branches the
// compiler waits for one before it sends the next (250 us for 195).
template <bool F32, bool ROWS>
__global__ __launch_bounds__(kWave * kQuantWaves) void k_quantize_mxfp4(QuantArgs a) {
    constexpr int kAhead = kQuantAhead<F32>, kPiece = kWave * kAhead;  // vectors
    const int lane = lane_id();
    const int64_t step = (int64_t)gridDim.x * kQuantWaves, end = a.vectors;
    int64_t piece = (int64_t)blockIdx.x * kQuantWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (; piece < a.pieces; piece += step) {
        int64_t base = 0, v0 = piece * kPiece;
        if (ROWS) {
            const int64_t row = piece / a.row_pieces;
            if (!row_is_live(a, (int)row)) continue;
            base = row * a.vectors;
            v0 = (piece - row * a.row_pieces) * kPiece;
        }
        uint4 in[kAhead][F32 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t v = v0 + i * kWave + lane;
            const uint4* const from = (const uint4*)a.x + (F32 ? 2 : 1) * (base + (v < end ? v : end - 1));
            in[i][0] = from[0];
            if (F32) in[i][F32 ? 1 : 0] = from[1];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t v = v0 + i * kWave + lane;
            if (v >= end) continue;  // whole groups of four lanes
            const uint32_t* p = (const uint32_t*)&in[i][0];
            // magnitudes order as their bits do, NaN above infinity
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < (F32 ? 8 : 4); ++j) {
                if (F32) m = max(m, p[j] & 0x7FFFFFFFu);
                else m = max(m, max((p[j] << 16) & 0x7FFFFFFFu, p[j] & 0x7FFF0000u));
            }
            m = max_with<0xB1>(m);  // quad_perm [1,0,3,2]
            m = max_with<0x4E>(m);  // quad_perm [2,3,0,1]
            const int power = (int)(m >> 23);  // biased by 127; 0 for subnormal numbers and zeros
            const bool finite = power < 255;
            const uint32_t byte = finite ? (uint32_t)max(power - 2, 0) : 255u;
            const float scale = __uint_as_float(byte << 23);
            uint32_t code = 0;
            if (finite) {
                if (F32) {
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, __uint_as_float(p[0]), __uint_as_float(p[1]), scale, 0);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, __uint_as_float(p[2]), __uint_as_float(p[3]), scale, 1);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, __uint_as_float(p[F32 ? 4 : 0]), __uint_as_float(p[F32 ? 5 : 0]), scale, 2);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, __uint_as_float(p[F32 ? 6 : 0]), __uint_as_float(p[F32 ? 7 : 0]), scale, 3);
                } else {
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2_v, p[0]), scale, 0);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2_v, p[1]), scale, 1);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2_v, p[2]), scale, 2);
                    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2_v, p[3]), scale, 3);
                }
            }
            ((uint32_t*)a.codes)[base + v] = code;
            if ((lane & 3) == 0) a.scales[(base + v) >> 2] = (uint8_t)byte;
            if (a.values != nullptr) {
                uint4 out = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);  // NaN
                if (finite) {
                    out.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 0));
                    out.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 1));
                    out.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 2));
                    out.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 3));
                }
                ((uint4*)a.values)[base + v] = out;
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize_mxfp4(QuantArgs a, int64_t rows, int32_t k, bool live_rows, bool f32, hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    const int64_t piece = kWave * (f32 ? kQuantAhead<true> : kQuantAhead<false>);
    a.vectors = live_rows ? k / 8 : rows * (k / 8);
    a.row_pieces = (a.vectors + piece - 1) / piece;
    a.pieces = live_rows ? rows * a.row_pieces : a.row_pieces;
    const int64_t need = (a.pieces + kQuantWaves - 1) / kQuantWaves;
    const dim3 grid((unsigned)(need < kQuantBlocks ? need : kQuantBlocks)), block(kWave * kQuantWaves);
    if (launch_debug()) launch_debug_print("k_quantize_mxfp4", grid, block, "k %d f32 %d", k, (int)f32);
    if (live_rows) {
        if (f32) hipLaunchKernelGGL((k_quantize_mxfp4<true, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((k_quantize_mxfp4<false, true>), grid, block, 0, stream, a);
    } else {
        if (f32) hipLaunchKernelGGL((k_quantize_mxfp4<true, false>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((k_quantize_mxfp4<false, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace ep
