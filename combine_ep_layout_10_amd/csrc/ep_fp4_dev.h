// MXFP4 operands (OCP Microscaling Formats): E2M1 codes, two to a byte, the lower
// nibble first, and one E8M0 scale for each 32 consecutive values of a row.
#pragma once

#include "ep_mma_dev.h"

namespace ep {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;  // the matrix instructions' number for E2M1

// D = A B + C with both operands' scales applied by the matrix unit: 16 rows of A
// and of B by 128 of the reduction. Lane (g, r) holds 32 consecutive codes of row r,
// and their scale in byte TA (B: TB) of its scale word; which 32 of the reduction group g
// holds is free as long as both operands agree. Checked on MI355X: products of codes and
// scales are exact, and what is more than 23 binary places below a sum's largest
// term is cut off (the tolerance of binary32); scale 255 makes NaN, also of zero codes.
template <int TA, int TB>
__device__ __forceinline__ f32x4_t mfma_fp4(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
    const i32x8_t x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8_t y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, kFp4, kFp4, TA, (int)sa, TB, (int)sb);
}

// Four of a row's `groups` scales from `first` on, as a word; zeros past the last. Loaded
// as they are (any alignment), near a row's end the last four, and put in place where
// they are used: with a branch between, the compiler waits for every load before it (300
// rows on 24 experts, 1000 x 1440: 12.6 us for 11.0).
__device__ __forceinline__ uint32_t load_scales4(const uint8_t* row, int first, int groups) {
    uint32_t w = 0;
    if (groups >= 4) {
        __builtin_memcpy(&w, row + min(first, groups - 4), 4);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < groups) w |= (uint32_t)row[i] << (8 * i);
    }
    return w;
}
__device__ __forceinline__ uint32_t place_scales4(uint32_t w, int first, int groups) {
    const int past = first - max(groups - 4, 0);
    return past < 4 ? w >> (8 * max(past, 0)) : 0u;
}

}  // namespace ep
