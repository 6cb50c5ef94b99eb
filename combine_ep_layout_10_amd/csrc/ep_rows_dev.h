// The row tiles of a receive layout, shared by the products that accept any
// alignment (BF16 and MXFP4).
#pragma once

#include "ep_internal.h"

namespace ep {

// Rows of expert e that hold a pair, its first row, and the rows it owns
// (COMPACT: padding included).
struct ExpertRows {
    int first, live, owned;
};

__device__ __forceinline__ ExpertRows expert_rows(const RowsArgs& a, int e) {
    ExpertRows r;
    if (a.mode == EP_MODE_COMPACT) {
        r.first = a.expert_off[e];
        r.live = a.cnt[e];
        r.owned = a.expert_off[e + 1] - r.first;
    } else {
        r.first = e * a.C;
        r.live = a.pad[e];  // min(cnt, C)
        r.owned = r.live;
    }
    return r;
}

// Row tile m of the whole layout: its expert and its index within the expert,
// experts in order, each with ceil(live / bm) tiles. Every wave finds it by
// itself (64 experts at a time, one a lane, prefix sums over the wave), so no
// barrier and no table in memory is needed. Returns false past the last tile.
__device__ __forceinline__ bool find_row_tile(const RowsArgs& a, int bm, int m, int* expert, int* tile) {
    const int lane = lane_id();
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
        const int e = e0 + lane;
        int n = 0;
        if (e < a.E) n = ((a.mode == EP_MODE_COMPACT ? a.cnt[e] : a.pad[e]) + bm - 1) / bm;
        const int upto = before + wave_inclusive_scan(n);
        const uint64_t past = ballot64(upto > m);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            *expert = e0 + l;
            *tile = m - __builtin_amdgcn_readlane(upto - n, l);
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return false;
}

// Most row tiles of bm rows that `pairs` pairs can need: an expert with c rows
// has ceil(c / bm), so at most one partial tile for each expert that has rows.
inline int64_t max_row_tiles(const RowsArgs& a, int bm, int64_t pairs) {
    return pairs / bm + (pairs < a.E ? pairs : a.E);
}

// Zeros into columns [n0, n0 + width) of the expert's padding rows (bf16
// output of N columns), by the whole block.
__device__ __forceinline__ void clear_padding(uint16_t* out, int N, const ExpertRows& er, int n0, int width) {
    const int per = width / 8;
    for (int i = threadIdx.x; i < (er.owned - er.live) * per; i += blockDim.x) {
        const int col = n0 + (i % per) * 8;
        if (col < N)
            *(uint4*)(out + ((int64_t)er.first + er.live + i / per) * N + col) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace ep
