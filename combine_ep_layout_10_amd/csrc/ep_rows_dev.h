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

// e is the same in every lane, and so is the result (moved to scalar registers).
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
    r.first = __builtin_amdgcn_readfirstlane(r.first);
    r.live = __builtin_amdgcn_readfirstlane(r.live);
    r.owned = __builtin_amdgcn_readfirstlane(r.owned);
    return r;
}

// Pieces of work 0 .. total - 1 are dealt to the 8 XCDs in contiguous ranges
// (block b runs on XCD b mod 8), so that neighbours share operands in one XCD's
// L2: the first piece of this block's XCD.
constexpr int kXcds = 8;

__device__ __forceinline__ int xcd_begin(int total, int xcd) {
    const int q = total / kXcds, r = total % kXcds;
    return xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q;
}

// This block's piece where every piece has a block of its own: the XCD's
// (b / 8)-th.
__device__ __forceinline__ int logical_block(int total) {
    return xcd_begin(total, (int)blockIdx.x % kXcds) + (int)blockIdx.x / kXcds;
}

// Blocks are numbered expert by expert: an expert with c live rows has
// ceil(c / bm) * per of them. Finds this block's expert and its number within
// the expert (both wave-uniform); false when it has no work. The counts are
// known only on the device, so every wave finds its place by itself (64
// experts at a time, one a lane, prefix sums over the wave): no barrier and
// no table in memory.
__device__ __forceinline__ bool find_expert(const RowsArgs& a, int bm, int per, int* expert, int* local) {
    constexpr int kChunks = kMaxExperts / kWave;
    const int lane = lane_id();
    const int32_t* count = a.mode == EP_MODE_COMPACT ? a.cnt : a.pad;  // FIXED: min(cnt, C)
    int upto[kChunks], own[kChunks];  // row tiles up to and with this lane's expert, and its own
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        own[c] = 0;
        if (c * kWave >= a.E) break;
        const int e = c * kWave + lane;
        if (e < a.E) own[c] = (count[e] + bm - 1) / bm;
    }
    int sum = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (c * kWave >= a.E) break;
        upto[c] = sum + wave_inclusive_scan(own[c]);
        sum = __builtin_amdgcn_readlane(upto[c], kWave - 1);
    }
    const int total = sum * per;
    if ((int)blockIdx.x >= total) return false;
    const int L = logical_block(total), m = L / per;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (c * kWave >= a.E) break;
        const uint64_t past = ballot64(upto[c] > m);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            *expert = c * kWave + l;
            *local = L - __builtin_amdgcn_readlane(upto[c] - own[c], l) * per;
            return true;
        }
    }
    return false;
}

// Most row tiles of bm rows that `pairs` pairs can need: an expert with c rows
// has ceil(c / bm), so at most one partial tile for each expert that has rows.
inline int64_t max_row_tiles(const RowsArgs& a, int bm, int64_t pairs) {
    return pairs / bm + (pairs < a.E ? pairs : a.E);
}

// Zeros into columns [n0, n0 + WIDTH) of the expert's padding rows (bf16
// output of N columns), by the whole block: a thread keeps its 8 columns and
// steps over the rows. Rows are counted unsigned: there are less than 2^31 of
// them, so a count one step past the last still fits, where a product of rows
// and columns would not.
template <int WIDTH>
__device__ __forceinline__ void clear_padding(uint16_t* out, int N, const ExpertRows& er, int n0) {
    constexpr int kPer = WIDTH / 8;  // threads of a row; divides the block
    const int col = n0 + (int)threadIdx.x % kPer * 8;
    if (col >= N) return;
    const uint32_t rows = (uint32_t)(er.owned - er.live), step = blockDim.x / kPer;
    uint16_t* at = out + ((int64_t)er.first + er.live) * N + col;
    for (uint32_t r = threadIdx.x / kPer; r < rows; r += step) *(uint4*)(at + (int64_t)r * N) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace ep
