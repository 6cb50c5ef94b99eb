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
//
// One kernel for the three: a block of 8 waves computes a tile of 256 x 256,
// wave (wm, wn) the 16-row pieces 2 i + wm of it by the columns 64 wn .. + 63,
// with v_mfma_f32_16x16x32_bf16. The reduction runs in steps of 64: both
// operands' slices (32 KiB each) move from memory to LDS by DMA, into a ring of
// five. All tails (rows, columns, reduction) are the buffer resource's range
// check, which fills zeros.
//
// Rows: an expert's rows are cut into ceil(rows / 256) tiles of equal size
// (rounded up to 32), and the loop is compiled for every number MI of 32-row
// steps, so an expert with 260 rows costs two tiles of 5/8 and 4/8, and one
// with 6 rows a single piece instead of a whole tile.
//
// Schedule: the waves form two groups (wm), half a step apart: while one
// group's MFMAs run, the other reads its operands from LDS, then a barrier
// exchanges the roles. Each SIMD holds one wave of either group, so its matrix
// unit always has work.
//
// LDS: a slice of an operand that is contiguous along the reduction is
// [256 rows][64 k] (128-byte rows, whole cache lines in memory); its 16-byte
// chunk c of row r is stored at c ^ (r / 2 mod 8). The other operands are
// [64 k][256 columns] (512-byte rows) and are read through the transposing LDS
// read, 4 k by 16 columns; their 32-byte pair of chunks p of row k is stored at
// p ^ f(k), f(k) = k mod 4 + 4 (k / 8 mod 2). Either way a read meets each bank
// once (SQ_LDS_BANK_CONFLICT 0).
#include "ep_mma_dev.h"
#include "ep_rows_dev.h"

namespace ep {

namespace {

constexpr int kTile = 256;
constexpr int kStep = 64;                  // reduction of one step
constexpr int kSlots = 5;                  // slices in LDS: A and B of step 0, of step 1, ... in turn
constexpr int kSlice = kTile * kStep * 2;  // bytes of one operand's slice
constexpr int kLoads = 4;                  // DMA loads of a wave for a slice
constexpr int kGroupRows = 8;                // row tiles that share column tiles in the block order

struct Tile {
    int e;           // expert
    int m0, n0;      // first row (of the expert's) and column
    int rows;        // rows of the tile that exist
    bool last_rows;  // the expert's last row tile
    ExpertRows er;
};

// Tile of logical block `local` among an expert's nt_m x nt_n: groups of
// about kGroupRows row tiles, within a group column by column, so that blocks that
// run together on an XCD share few operand tiles.
__device__ __forceinline__ void order_tiles(int local, int nt_m, int nt_n, int* m, int* n) {
    const int groups = max(1, (nt_m + kGroupRows / 2) / kGroupRows), size = (nt_m + groups - 1) / groups;
    const int g = local / (size * nt_n);
    const int in_group = min(size, nt_m - g * size);
    const int rem = local - g * size * nt_n;
    *n = rem / in_group;
    *m = g * size + rem % in_group;
}

template <int DIR>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, Tile* t) {
    const int nt_n = (a.N + kTile - 1) / kTile;
    int m, n;
    if (DIR == kGradWeight) {
        const int nt_m = (a.M + kTile - 1) / kTile;
        const int L = logical_block((int)gridDim.x);
        t->e = __builtin_amdgcn_readfirstlane(L / (nt_m * nt_n));
        order_tiles(L % (nt_m * nt_n), nt_m, nt_n, &m, &n);
        t->er = expert_rows(a.rows, t->e);
        t->m0 = m * kTile;
        t->rows = min(kTile, a.M - t->m0);
        t->last_rows = false;
    } else {
        int local;
        if (!find_expert(a.rows, kTile, nt_n, &t->e, &local)) return false;
        t->er = expert_rows(a.rows, t->e);
        const int live = t->er.live, nt_m = (live + kTile - 1) / kTile;
        order_tiles(local, nt_m, nt_n, &m, &n);
        const int each = ((live + nt_m - 1) / nt_m + 31) & ~31;  // rows of a tile; never leaves the last one empty
        t->m0 = m * each;
        t->rows = min(each, live - t->m0);
        t->last_rows = m == nt_m - 1;
    }
    t->n0 = n * kTile;
    t->m0 = __builtin_amdgcn_readfirstlane(t->m0);
    t->n0 = __builtin_amdgcn_readfirstlane(t->n0);
    t->rows = __builtin_amdgcn_readfirstlane(t->rows);
    return true;
}

// One operand's way from memory to LDS and to the MFMAs. KMAJOR: the reduction
// runs over the rows in memory (element (r, k) at base[k * ld + r]), otherwise
// along them (base[r * ld + k]). `count`: rows of the tile that exist; `red`:
// length of the reduction.
template <bool KMAJOR>
struct Operand {
    const char* base;  // of the tile, reduction step 0
    int ld;            // bytes between rows
    int count, red;
    uint32_t off[kLoads];  // byte offsets of this lane's loads
    int chunk[2];          // KMAJOR false: chunk (8 values of k) of this lane's even and odd loads

    __device__ __forceinline__ void init(const uint16_t* src, int64_t ld_values, int r0, int rows, int reduction,
                                         int w, int lane) {
        ld = (int)(2 * ld_values);
        count = rows;
        red = reduction;
        base = (const char*)src + (KMAJOR ? 2 * (int64_t)r0 : (int64_t)r0 * ld);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (KMAJOR) {
                const int k = (kLoads * w + j) * 2 + (lane >> 5), pos = lane & 31;
                const int c = (((pos >> 1) ^ swizzle(k)) << 1) | (pos & 1);
                off[j] = 8 * c < rows ? (uint32_t)(k * ld + 16 * c) : kOutOfRange;
            } else {
                const int r = (kLoads * w + j) * 8 + (lane >> 3);
                chunk[j & 1] = (lane & 7) ^ ((r >> 1) & 7);
                off[j] = (uint32_t)(r * ld + 16 * chunk[j & 1]);
            }
        }
    }
    __device__ __forceinline__ static int swizzle(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

    // Step kb's slice to LDS at `to`; steps at or past `steps` load nothing (zeros).
    __device__ __forceinline__ void issue(int kb, int steps, uint32_t to, int w) const {
        const int left = red - kb * kStep;
        to += w * (kLoads * 1024);
        if (KMAJOR) {
            // a lane past the tile's columns is out of range by its offset, a row past the reduction by the size
            const int size = kb < steps ? min(left, kStep) * ld : 0;
            const char* b = base + (int64_t)kb * kStep * ld;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) dma16(b, size, off[j], to + 1024 * j);
        } else {
            const int size = kb < steps ? count * ld - kb * (2 * kStep) : 0;
            const char* b = base + (int64_t)kb * (2 * kStep);
#pragma unroll
            for (int j = 0; j < kLoads; ++j)  // the second case: the reduction's tail
                dma16(b, size, left >= kStep || 8 * chunk[j & 1] < left ? off[j] : kOutOfRange, to + 1024 * j);
        }
    }
};

// The tile's product with MI pieces of 16 rows for each wave, and its stores.
template <int DIR, int MI>
__device__ __forceinline__ void run_tile(const GroupedArgs& a, const Tile& t, uint32_t lds) {
    constexpr bool KA = DIR == kGradWeight, KB = DIR != kForward;  // operands whose reduction runs over rows
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w >> 2, wn = w & 3;
    const int cols = min(kTile, a.N - t.n0);
    const int red = DIR == kGradWeight ? t.er.live : a.K;
    const int steps = (red + kStep - 1) / kStep;

    Operand<KA> A;
    Operand<KB> B;
    if (DIR == kGradWeight) {
        A.init(a.a + (int64_t)t.er.first * a.M, a.M, t.m0, t.rows, red, w, lane);
        B.init(a.b + (int64_t)t.er.first * a.N, a.N, t.n0, cols, red, w, lane);
    } else {
        A.init(a.a + (int64_t)t.er.first * a.K, a.K, t.m0, t.rows, red, w, lane);
        B.init(a.b + (int64_t)t.e * a.N * a.K, DIR == kForward ? a.K : a.N, t.n0, cols, red, w, lane);
    }
    // Addresses of this lane's operands within a slice, first half of the step.
    // Contiguous along k: row 16 p + r16, chunk g (4 further in the second half);
    // piece p is 2048 p bytes on. Otherwise: k = 8 g + r16 / 4 (and 4 further; 32
    // in the second half), values 4 (r16 % 4) of column piece p; pieces that
    // agree in p mod 8 are 256 bytes apart.
    uint32_t ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = 8 * g + (r16 >> 2);
        if (KA) ra[i] = k * 512 + (((2 * i + wm) ^ Operand<true>::swizzle(k)) << 5) + (r16 & 3) * 8;
        else ra[i] = (16 * wm + r16) * 128 + (((4 * (i & 1) + g) ^ ((r16 >> 1) & 7)) << 4);
        if (KB) rb[i] = k * 512 + (((4 * wn + i) ^ Operand<true>::swizzle(k)) << 5) + (r16 & 3) * 8;
        else rb[i] = (64 * wn + r16) * 128 + (((4 * (i & 1) + g) ^ ((r16 >> 1) & 7)) << 4);
    }

    f32x4_t acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

    // Ring: slice q (A of step q / 2 when even, B when odd) lives in slot q mod 5.
    // In interval 2 kb group 0 reads step kb while group 1 computes step kb - 1; in
    // the next one the roles are exchanged. Step kb - 1 has been read by both when
    // interval 2 kb begins, so its two slots take slices 2 kb + 3 and 2 kb + 4 then:
    // all 8 waves send them (group 0 behind its LDS reads, group 1 before its
    // MFMAs). Slice 2 kb + 3 is needed when interval 2 kb + 2 begins: every wave waits
    // for its part of it before the barrier that ends interval 2 kb + 1.
    const auto slot = [&](int q) { return lds + (uint32_t)(q % kSlots) * kSlice; };
    A.issue(0, steps, slot(0), w);
    B.issue(0, steps, slot(1), w);
    A.issue(1, steps, slot(2), w);
    wait_vmcnt<kLoads>();
    block_barrier();
    if (wm == 1) {
        B.issue(1, steps, slot(3), w);
        A.issue(2, steps, slot(4), w);
        block_barrier();
    }
    int qa = 0;  // slot of A of step kb
    for (int kb = 0; kb < steps; ++kb) {
        const auto wrap = [](int q) { return q >= kSlots ? q - kSlots : q; };
        const uint32_t at_a = lds + (uint32_t)qa * kSlice, at_b = lds + (uint32_t)wrap(qa + 1) * kSlice;
        bf16x8_t fa[2][MI], fb[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fb[h][j] = KB ? read_transposed(at_b + rb[j] + 16384 * h, 2048) : read_lds(at_b + rb[h] + 2048 * j);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                fa[h][i] = KA ? read_transposed(at_a + ra[i & 3] + 256 * (i >> 2) + 16384 * h, 2048)
                              : read_lds(at_a + ra[h] + 4096 * i);
        }
        if (wm == 0) {
            B.issue(kb + 1, steps, lds + (uint32_t)wrap(qa + 3) * kSlice, w);
            A.issue(kb + 2, steps, lds + (uint32_t)wrap(qa + 4) * kSlice, w);
        } else {
            wait_vmcnt<kLoads>();
        }
        wait_lgkmcnt0();
        block_barrier();
        qa = wrap(qa + 2);
        if (wm == 1) {
            B.issue(kb + 2, steps, lds + (uint32_t)wrap(qa + 3) * kSlice, w);
            A.issue(kb + 3, steps, lds + (uint32_t)wrap(qa + 4) * kSlice, w);
        }
        __builtin_amdgcn_s_setprio(1);
        // operands swapped: each 16 x 16 piece comes out transposed, lane (g, r16)
        // holding row r16 and columns 4 g .. 4 g + 3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        if (wm == 0) wait_vmcnt<kLoads>();
        block_barrier();
    }
    if (wm == 0) block_barrier();
    wait_vmcnt<0>();

    // Epilogue: the four column pieces of a row are exchanged between the four
    // lane groups, so that a lane holds 16 adjacent columns.
    const int col = t.n0 + 64 * wn + 16 * g;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int row = 16 * (2 * i + wm) + r16;
        const bool live = row < t.rows;
        const int64_t at = ((DIR == kGradWeight ? (int64_t)t.e * a.M : (int64_t)t.er.first) + t.m0 + row) * a.N + col;
        if (DIR == kGradWeight && a.out_f32) {
            uint32_t v[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = __float_as_uint(acc[i][j][q]);
                transpose4(r);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j][q] = r[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live && col + 4 * j < a.N)
                    *(uint4*)((float*)a.c + at + 4 * j) = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
        } else {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = pack_bf16x2(acc[i][j][0], acc[i][j][1]);
                hi[j] = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
            }
            transpose4(lo);
            transpose4(hi);
            if (live && col < a.N) *(uint4*)((uint16_t*)a.c + at) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
            if (live && col + 8 < a.N) *(uint4*)((uint16_t*)a.c + at + 8) = make_uint4(lo[2], hi[2], lo[3], hi[3]);
        }
    }
    if (DIR != kGradWeight && a.rows.zero_pad && t.last_rows) clear_padding((uint16_t*)a.c, a.N, t.er, t.n0, kTile);
}

template <int DIR>
__global__ __launch_bounds__(512) void k_grouped_gemm_bf16(GroupedArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kSlots * kSlice];
    Tile t;
    if (!find_tile<DIR>(a, &t)) return;
    const uint32_t lds = lds_offset(s_ring);
    asm volatile("" ::"v"(s_ring) : "memory");  // the ring is written by the DMA alone
    switch ((t.rows + 31) / 32) {
        case 1: return run_tile<DIR, 1>(a, t, lds);
        case 2: return run_tile<DIR, 2>(a, t, lds);
        case 3: return run_tile<DIR, 3>(a, t, lds);
        case 4: return run_tile<DIR, 4>(a, t, lds);
        case 5: return run_tile<DIR, 5>(a, t, lds);
        case 6: return run_tile<DIR, 6>(a, t, lds);
        case 7: return run_tile<DIR, 7>(a, t, lds);
        default: return run_tile<DIR, 8>(a, t, lds);
    }
}

}  // namespace

hipError_t launch_grouped_gemm_bf16(int dir, const GroupedArgs& a, int64_t pairs, hipStream_t stream) {
    const int64_t nt_n = (a.N + kTile - 1) / kTile;
    const int64_t mtiles = dir == kGradWeight ? (int64_t)a.rows.E * ((a.M + kTile - 1) / kTile)
                                              : max_row_tiles(a.rows, kTile, pairs);
    const int64_t blocks = mtiles * nt_n;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7FFFFF) return hipErrorInvalidValue;  // 2^32 threads a launch
    const dim3 grid((unsigned)blocks), block(512);
    if (launch_debug()) launch_debug_print("k_grouped_gemm_bf16", grid, block, "direction %d n %d", dir, a.N);
    if (dir == kForward)
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kForward>, grid, block, 0, stream, a);
    else if (dir == kGradInput)
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kGradInput>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kGradWeight>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace ep
