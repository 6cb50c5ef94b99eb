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
// Whole tiles (forward, grad_input): a block of 8 waves computes 256 x 256, wave
// (wm, wn) the 16-row pieces 2 i + wm of it by the columns 64 wn .. + 63, with
// v_mfma_f32_16x16x32_bf16. The reduction runs in steps of 64: both operands'
// slices (32 KiB each) move from memory to LDS by DMA, into a ring that fills the
// CU's 160 KiB. All tails (rows, columns, reduction) are the buffer resource's
// range check, which fills zeros.
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
// LDS: a slice of an operand that is contiguous along the reduction has rows of 64
// k (128 bytes, whole cache lines in memory; with steps of 32, half lines, the
// product took 7 % longer); its 16-byte chunk c of row r is stored at
// c ^ (r / 2 mod 8). The other operands have a row of columns for each k and are
// read through the transposing LDS read, 4 k by 16 columns; their 32-byte pair of
// chunks p of row k is stored at p ^ f(k), f(k) = k mod 4 + 4 (k / 8 mod 2). Either
// way a read meets each bank once: the loop has no cycle of SQ_LDS_BANK_CONFLICT
// (what a launch counts, about 1,000 a tile, are the stores' writes).
//
// Half tiles (grad_weight, few tiles): 4 waves, 256 x 128, steps of 32, two blocks
// a CU; described with them. Few rows an expert: ep_gemm_stream.hip.
//
// What bounds it, on MI355X: 65,536 rows x 4096 x 7168 on 32 experts take 2.9 to 3.0
// ms (1.3 PFLOP/s; a library product of 8192^3 reaches 1.46), the matrix units busy
// 73 % of the cycles at the 1.7 GHz that the card holds under this load. The rest is
// the LDS reads and DMA of one group that take longer than the other's MFMAs, tiles
// that are not full, and a tile's first loads and stores. One wave a SIMD with 128 x
// 128 pieces and the accumulators in AGPRs measured 3.6 ms (3.4 then), a ring of five
// steps of 32 as four.
#include "ep_mma_dev.h"
#include "ep_rows_dev.h"

namespace ep {

namespace {

constexpr int kTile = 256;     // rows of a tile
constexpr int kGroupRows = 4;  // row tiles that share column tiles in the block order

struct Tile {
    int e;          // expert
    int m0, n0;     // first row (of the expert's) and column
    int rows;       // rows of the tile that exist
    int last_rows;  // whether it is the expert's last row tile
    ExpertRows er;
};

// This block's tile of kTile rows by COLS columns; false when it has none.
template <int DIR, int COLS>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, Tile* t) {
    const int nt_n = (a.N + COLS - 1) / COLS;
    int m, n;
    if (DIR == kGradWeight) {
        const int nt_m = (a.M + kTile - 1) / kTile;
        const int L = logical_block((int)gridDim.x);
        t->e = __builtin_amdgcn_readfirstlane(L / (nt_m * nt_n));
        order_tiles<kGroupRows>(L % (nt_m * nt_n), nt_m, nt_n, &m, &n);
        t->er = expert_rows(a.rows, t->e);
        t->m0 = m * kTile;
        t->rows = min(kTile, a.M - t->m0);
        t->last_rows = 0;
    } else {
        int local;
        if (!find_expert(a.rows, kTile, nt_n, &t->e, &local)) return false;
        t->er = expert_rows(a.rows, t->e);
        const int live = t->er.live, nt_m = (live + kTile - 1) / kTile;
        order_tiles<kGroupRows>(local, nt_m, nt_n, &m, &n);
        const int each = ((live + nt_m - 1) / nt_m + 31) & ~31;  // rows of a tile; never leaves the last one empty
        t->m0 = m * each;
        t->rows = min(each, live - t->m0);
        t->last_rows = m == nt_m - 1;
    }
    t->n0 = n * COLS;
    t->m0 = __builtin_amdgcn_readfirstlane(t->m0);
    t->n0 = __builtin_amdgcn_readfirstlane(t->n0);
    t->rows = __builtin_amdgcn_readfirstlane(t->rows);
    return true;
}

// One operand's way from memory to LDS and to the MFMAs: slices of WIDTH rows
// (or columns) by STEP of the reduction, moved by WAVES waves. KMAJOR: the
// reduction runs over the rows in memory (element (r, k) at base[k * ld + r]),
// otherwise along them (base[r * ld + k]). `count`: rows of the tile that exist;
// `red`: length of the reduction.
template <bool KMAJOR, int STEP, int WIDTH, int WAVES>
struct Operand {
    static constexpr int kSlice = STEP * WIDTH * 2;            // bytes
    static constexpr int kLoads = kSlice / 1024 / WAVES;       // DMA loads of a wave
    static constexpr int kRow = 2 * (KMAJOR ? WIDTH : STEP);   // bytes of a row in LDS
    static constexpr int kPiece = KMAJOR ? 0 : 16 * kRow;      // from a piece of 16 rows to the next

    const char* base;      // of the tile, reduction step 0
    int ld;                // bytes between rows
    int count, red;
    uint32_t off[kLoads];  // byte offsets of this lane's loads
    int chunk[2];          // KMAJOR false: chunk (8 values of k) of this lane's even and odd loads
    uint32_t at[KMAJOR ? 1 : 2];  // this lane's first operand within a slice (KMAJOR false: of either half)

    // first: the wave's first piece of 16 rows
    __device__ __forceinline__ void init(const uint16_t* src, int64_t ld_values, int r0, int rows, int reduction,
                                         int w, int first) {
        const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
        ld = (int)(2 * ld_values);
        count = rows;
        red = reduction;
        base = (const char*)src + (KMAJOR ? 2 * (int64_t)r0 : (int64_t)r0 * ld);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int byte = (kLoads * w + j) * 1024 + 16 * lane, r = byte / kRow, pos = byte % kRow / 16;
            if (KMAJOR) {
                const int c = (((pos >> 1) ^ pair_swizzle(r)) << 1) | (pos & 1);
                off[j] = 8 * c < rows ? __umul24(r, ld) + 16 * c : kOutOfRange;
            } else {
                chunk[j & 1] = pos ^ chunk_swizzle(r);
                off[j] = __umul24(r, ld) + 16 * chunk[j & 1];
            }
        }
        if (KMAJOR) {
            // k = 8 g + r16 / 4 (and 4 further), values 4 (r16 % 4) of the piece
            const int k = 8 * g + (r16 >> 2);
            at[0] = k * kRow + ((first ^ pair_swizzle(k)) << 5) + (r16 & 3) * 8;
        } else {
            // row r16 of the first piece, chunk g (of the step's second half: 4 further)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at[h] = first * kPiece + r16 * kRow + (((4 * h + g) ^ chunk_swizzle(r16)) << 4);
        }
    }
    __device__ __forceinline__ static int pair_swizzle(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }
    __device__ __forceinline__ static int chunk_swizzle(int r) { return STEP == 64 ? (r >> 1) & 7 : row_swizzle16(r); }

    // Load j of step kb's slice to LDS at `to`; steps at or past `steps` load nothing (zeros).
    __device__ __forceinline__ void issue(int kb, int steps, uint32_t to, int w, int j) const {
        const int left = red - kb * STEP;
        to += (w * kLoads + j) * 1024;
        if (KMAJOR)  // a lane past the tile's columns is out of range by its offset, a row past the reduction by the size
            dma16(base + (int64_t)kb * STEP * ld, kb < steps ? min(left, STEP) * ld : 0, off[j], to);
        else  // the third case: the reduction's tail
            dma16(base + (int64_t)kb * (2 * STEP), kb < steps ? count * ld - kb * (2 * STEP) : 0,
                  left >= STEP || 8 * chunk[j & 1] < left ? off[j] : kOutOfRange, to);
    }
    __device__ __forceinline__ void issue(int kb, int steps, uint32_t to, int w) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) issue(kb, steps, to, w, j);
    }

    // The MFMA operand of the wave's i-th piece, half h (32 of k) of the slice at
    // `slice`. EVERY: the distance of the wave's pieces. KMAJOR: pieces of one
    // cycle of 8 differ from the first in bits that it has clear, so the swizzled
    // place is the first one's XOR the distance; later cycles are 256 bytes on.
    template <int EVERY>
    __device__ __forceinline__ bf16x8_t read(uint32_t slice, int h, int i) const {
        if (KMAJOR) {
            constexpr int kCycle = 8 / EVERY;
            return read_transposed(((slice + at[0]) ^ (EVERY * (i % kCycle) << 5)) + 256 * (i / kCycle) + 32 * kRow * h,
                                   4 * kRow);
        }
        return read_lds(slice + at[h] + EVERY * kPiece * i);
    }
};

// Stores of a wave's MI x 4 pieces: row piece 2 i + wm, columns col .. col + 63.
// The MFMA leaves 16 rows in 16 lanes and 4 columns in each of the four lane
// groups; each 16 rows are turned through the wave's own kStoreLds bytes of LDS at
// `lds`, so that neighbouring lanes store neighbouring columns (a weight gradient of
// 64 x 4096 x 4096 from 24,576 rows: 1.06 ms, binary32 1.43; by exchanges between
// lanes that leave 8 rows side by side, in whole lines as well, 1.09 and 1.49). A
// wave's LDS accesses stay in order. 16-byte chunks are stored XORed with the row
// (binary32), with half the row (bf16, two rows in the 64 banks), so that a read
// meets each bank once. (bf16's writes leave 16 cycles of bank conflicts a wave and
// piece: 512 a half tile, 1,024 a whole one; binary32's none.)
constexpr int kStoreLds = 4096;

template <int DIR, int MI>
__device__ __forceinline__ void store_tile(const GroupedArgs& a, const Tile& t, const f32x4_t (&acc)[MI][4], int wm, int col,
                                           uint32_t lds) {
    int lane = lane_id();
    asm volatile("" : "+v"(lane));  // worked out here: kept over the main loop, its terms would cost registers
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t first = (DIR == kGradWeight ? (int64_t)t.e * a.M : (int64_t)t.er.first) + t.m0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int row = 16 * (2 * i + wm);
        if (DIR == kGradWeight && a.out_f32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                write_lds(lds + r16 * 256 + (((4 * j + g) ^ r16) << 4), __builtin_bit_cast(u32x4_t, acc[i][j]));
            const int c = col + 4 * r16;  // lane (g, r16) stores row 4 s + g, chunk r16
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 4 * s + g;
                const u32x4_t v = read_lds_words(lds + r * 256 + ((r16 ^ r) << 4));
                if (row + r < t.rows && c < a.N) *(u32x4_t*)((float*)a.c + (first + row + r) * a.N + c) = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x2_t v = {pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
                write_lds(lds + r16 * 128 + (((2 * j + (g >> 1)) ^ (r16 >> 1)) << 4) + (g & 1) * 8, v);
            }
            const int c = col + 8 * (lane & 7);  // lane stores row 8 s + lane / 8, chunk lane % 8
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int r = 8 * s + (lane >> 3);
                const u32x4_t v = read_lds_words(lds + r * 128 + (((lane & 7) ^ (r >> 1)) << 4));
                if (row + r < t.rows && c < a.N) *(u32x4_t*)((uint16_t*)a.c + (first + row + r) * a.N + c) = v;
            }
        }
    }
}

template <int DIR, class OpA, class OpB>
__device__ __forceinline__ void init_operands(const GroupedArgs& a, const Tile& t, int cols, int red, int w, int wm,
                                              int wn, OpA& A, OpB& B) {
    if (DIR == kGradWeight) {
        A.init(a.a + (int64_t)t.er.first * a.M, a.M, t.m0, t.rows, red, w, wm);
        B.init(a.b + (int64_t)t.er.first * a.N, a.N, t.n0, cols, red, w, 4 * wn);
    } else {
        A.init(a.a + (int64_t)t.er.first * a.K, a.K, t.m0, t.rows, red, w, wm);
        B.init(a.b + (int64_t)t.e * a.N * a.K, DIR == kForward ? a.K : a.N, t.n0, cols, red, w, 4 * wn);
    }
}

// ---------------------------------------------------------------- whole tiles: 8 waves, 256 columns

// The ring of a tile's slices in 160 KiB of LDS. Steps are read by group 0 in
// interval 2 kb (while group 1 computes step kb - 1) and by group 1 in the next one
// (while group 0 computes step kb); step kb - 1 has been read by both when interval
// 2 kb begins, and its place is filled again from then on.
//   256 rows: five slots of 32 KiB; slice q (A of step q / 2 when even, B when odd)
//   lives in slot q mod 5; interval 2 kb sends slice 2 kb + 3, the next 2 kb + 4.
//   Fewer rows leave room for more steps: 128 rows three, 64 rows four (step kb in
//   place kb mod kSteps); interval 2 kb sends B of step kb + kSteps - 1, the next A.
template <class OpA, class OpB>
struct Ring {
    static constexpr bool kSlots = OpA::kSlice == OpB::kSlice;
    static constexpr int kBytes = 160 * 1024;
    static constexpr int kStepBytes = OpA::kSlice + OpB::kSlice, kSteps = kBytes / kStepBytes;
    static constexpr int kSend = OpA::kLoads + OpB::kLoads;  // loads of a wave for an interval
    // a wave's loads that may be on their way when step kb + 1 has landed, those of interval 2 kb + 1 sent
    static constexpr int kKeep = kSlots ? OpA::kLoads : (kSteps - 2) * kSend;

    const OpA& A;
    const OpB& B;
    int steps;
    uint32_t lds;
    int w;

    __device__ __forceinline__ static int wrap(int q, int n) { return q >= n ? q - n : q; }
    // place: of step kb (slots: that of its slice of A)
    __device__ __forceinline__ uint32_t at_a(int place) const { return lds + place * (kSlots ? OpA::kSlice : kStepBytes); }
    __device__ __forceinline__ uint32_t at_b(int place) const {
        return kSlots ? lds + wrap(place + 1, 5) * OpA::kSlice : at_a(place) + OpA::kSlice;
    }
    __device__ __forceinline__ static int next(int place) { return kSlots ? wrap(place + 2, 5) : wrap(place + 1, kSteps); }
    __device__ __forceinline__ void send_step(int kb) const {
        A.issue(kb, steps, at_a(kb), w);
        B.issue(kb, steps, at_a(kb) + OpA::kSlice, w);
    }
    // ahead of interval 0; step 0 has landed in this wave's part on return
    __device__ __forceinline__ void first() const {
        if (kSlots) {
            A.issue(0, steps, lds, w);
            B.issue(0, steps, lds + OpA::kSlice, w);
            A.issue(1, steps, lds + 2 * OpA::kSlice, w);
        } else {
#pragma unroll
            for (int kb = 0; kb < kSteps - 1; ++kb) send_step(kb);
        }
        wait_vmcnt<kKeep>();
    }
    // load d of what interval 2 kb sends (a slice of B), and the next one (a slice of A)
    __device__ __forceinline__ void send_b(int kb, int place, int d) const {
        if (kSlots) B.issue(kb + 1, steps, lds + wrap(place + 3, 5) * OpA::kSlice, w, d);
        else B.issue(kb + kSteps - 1, steps, at_a(wrap(place + kSteps - 1, kSteps)) + OpA::kSlice, w, d);
    }
    __device__ __forceinline__ void send_a(int kb, int place, int d) const {
        if (kSlots) A.issue(kb + 2, steps, lds + wrap(place + 4, 5) * OpA::kSlice, w, d);
        else A.issue(kb + kSteps - 1, steps, at_a(wrap(place + kSteps - 1, kSteps)), w, d);
    }
};

// The loop of one group of waves over all steps. Every wave sends its part of an
// interval's loads: the group that reads LDS behind its reads, the one that
// computes spread between its MFMAs. A DMA of 1 KiB occupies the CU's address unit
// for 16 cycles, so the loads of a step take 1024 of its 2048 cycles there: sent
// in one interval of the two, they held up the MFMAs (clock reads in the loop:
// 1,400 to 1,800 cycles for 1,024 of MFMA). What step kb + 1 needs is waited for by
// every wave before the barrier that ends interval 2 kb + 1.
template <bool SECOND, int MI, class OpA, class OpB>
__device__ __forceinline__ void multiply(const Ring<OpA, OpB>& ring, f32x4_t (&acc)[MI][4]) {
    using R = Ring<OpA, OpB>;
    constexpr int kSpread = SECOND ? OpB::kLoads : OpA::kLoads;
    int place = 0;
    for (int kb = 0; kb < ring.steps; ++kb) {
        const uint32_t at_a = ring.at_a(place), at_b = ring.at_b(place);
        bf16x8_t fa[2][MI], fb[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[h][j] = ring.B.template read<1>(at_b, h, j);
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[h][i] = ring.A.template read<2>(at_a, h, i);
        }
        if (SECOND) {
#pragma unroll
            for (int d = 0; d < OpA::kLoads; ++d) ring.send_a(kb, place, d);
            wait_vmcnt<R::kKeep>();
        } else {
#pragma unroll
            for (int d = 0; d < OpB::kLoads; ++d) ring.send_b(kb, place, d);
        }
        wait_lgkmcnt0();
        block_barrier();
        const int here = place;
        place = R::next(place);
        __builtin_amdgcn_s_setprio(1);
        // operands swapped: each 16 x 16 piece comes out transposed, lane (g, r16)
        // holding row r16 and columns 4 g .. 4 g + 3
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
                for (int d = 0; d < kSpread; ++d)
                    if (d * 2 * MI / kSpread == h * MI + i) {
                        if (SECOND) ring.send_b(kb + 1, place, d);
                        else ring.send_a(kb, here, d);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        __builtin_amdgcn_s_setprio(0);
        if (!SECOND) wait_vmcnt<R::kKeep>();
        block_barrier();
    }
}

// The tile's product with MI pieces of 16 rows for each wave, and its stores.
template <int DIR, int MI>
__device__ __forceinline__ void run_tile(const GroupedArgs& a, const Tile& t, uint32_t lds) {
    constexpr int kStep = 64, kRows = MI <= 2 ? 64 : MI <= 4 ? 128 : 256;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w >> 2, wn = w & 3;
    using OpA = Operand<false, kStep, kRows, 8>;
    using OpB = Operand<DIR == kGradInput, kStep, kTile, 8>;
    OpA A;
    OpB B;
    init_operands<DIR>(a, t, min(kTile, a.N - t.n0), a.K, w, wm, wn, A, B);
    f32x4_t acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    const Ring<OpA, OpB> ring = {A, B, (a.K + kStep - 1) / kStep, lds, w};
    ring.first();
    block_barrier();
    if (wm == 0) {
        multiply<false, MI>(ring, acc);
        block_barrier();
    } else {
#pragma unroll
        for (int d = 0; d < OpB::kLoads; ++d) ring.send_b(0, 0, d);
        block_barrier();  // half a step later
        multiply<true, MI>(ring, acc);
    }
    wait_vmcnt<0>();
    block_barrier();  // no wave reads or fills the ring any more
    store_tile<DIR, MI>(a, t, acc, wm, t.n0 + 64 * wn, lds + w * kStoreLds);
    if (a.rows.zero_pad && t.last_rows) clear_padding<kTile>((uint16_t*)a.c, a.N, t.er, t.n0);
}

// ---------------------------------------------------------------- half tiles: 4 waves, 128 columns, two blocks a CU

constexpr int kHalf = 128;       // columns
constexpr int kHalfStages = 3;
constexpr int kHalfStage = (kTile + kHalf) * 32 * 2;  // bytes: A's slice, then B's

template <int DIR, int MI>
__device__ __forceinline__ void run_half(const GroupedArgs& a, const Tile& t, uint32_t lds) {
    constexpr int kStep = 32;
    constexpr bool KA = DIR == kGradWeight, KB = DIR != kForward;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w >> 1, wn = w & 1;
    const int red = DIR == kGradWeight ? t.er.live : a.K;
    const int steps = (red + kStep - 1) / kStep;
    Operand<KA, kStep, kTile, 4> A;
    Operand<KB, kStep, kHalf, 4> B;
    constexpr int kLoads = decltype(A)::kLoads + decltype(B)::kLoads;
    init_operands<DIR>(a, t, min(kHalf, a.N - t.n0), red, w, wm, wn, A, B);
    f32x4_t acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};
    const auto issue = [&](int kb, int st) {
        A.issue(kb, steps, lds + st * kHalfStage, w);
        B.issue(kb, steps, lds + st * kHalfStage + decltype(A)::kSlice, w);
    };
    issue(0, 0);
    issue(1, 1);
    int st = 0;
    for (int kb = 0; kb < steps; ++kb) {
        // step kb has landed in every wave's part; every wave has read step kb - 1,
        // whose stage takes step kb + 2. The CU's other block works while this one waits.
        wait_vmcnt<kLoads>();
        block_barrier();
        const uint32_t at = lds + st * kHalfStage;
        bf16x8_t fa[MI], fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[j] = B.template read<1>(at + decltype(A)::kSlice, 0, j);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = A.template read<2>(at, 0, i);
        issue(kb + 2, st == 0 ? kHalfStages - 1 : st - 1);
        wait_lgkmcnt0();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        st = st == kHalfStages - 1 ? 0 : st + 1;
    }
    wait_vmcnt<0>();
    block_barrier();  // no wave reads or fills the ring any more
    store_tile<DIR, MI>(a, t, acc, wm, t.n0 + 64 * wn, lds + w * kStoreLds);
    if (DIR != kGradWeight && a.rows.zero_pad && t.last_rows)
        clear_padding<kHalf>((uint16_t*)a.c, a.N, t.er, t.n0);
}

template <int DIR>
__global__ __launch_bounds__(512) void k_grouped_gemm_bf16(GroupedArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[160 * 1024];
    Tile t;
    if (!find_tile<DIR, kTile>(a, &t)) return;
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

template <int DIR>
__global__ __launch_bounds__(256, 2) void k_grouped_gemm_bf16_half(GroupedArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kHalfStages * kHalfStage];
    Tile t;
    if (!find_tile<DIR, kHalf>(a, &t)) return;
    const uint32_t lds = lds_offset(s_ring);
    asm volatile("" ::"v"(s_ring) : "memory");
    switch ((t.rows + 31) / 32) {
        case 1: return run_half<DIR, 1>(a, t, lds);
        case 2: return run_half<DIR, 2>(a, t, lds);
        case 3: return run_half<DIR, 3>(a, t, lds);
        case 4: return run_half<DIR, 4>(a, t, lds);
        case 5: return run_half<DIR, 5>(a, t, lds);
        case 6: return run_half<DIR, 6>(a, t, lds);
        case 7: return run_half<DIR, 7>(a, t, lds);
        default: return run_half<DIR, 8>(a, t, lds);
    }
}

}  // namespace

hipError_t launch_grouped_gemm_bf16(int dir, const GroupedArgs& a, int64_t pairs, hipStream_t stream) {
    // Few rows an expert: the kernel that streams the weights through registers.
    // 64 tokens x top-6, 64 experts, 4096 x 4096: 346 against 375 us; one token on
    // two experts, 1440 x 3608: 10.6 against 33 us (split reduction); 64 rows x
    // 4096 x 4096 on 8 experts 54 against 63 us, 512 rows on 64 experts 353 against
    // 375 us; at a mean of 15 rows, unevenly spread, 377 us either way.
    if (dir == kForward && pairs <= 16 * (int64_t)a.rows.E) {
        StreamArgs s;
        s.rows = a.rows;
        s.x = a.a;
        s.b = a.b;
        s.b_scales = nullptr;
        s.out = (uint16_t*)a.c;
        s.N = a.N;
        s.K = a.K;
        return launch_grouped_gemm_bf16_stream(s, pairs, stream);
    }
    // Half tiles for the weight gradient: its reductions are a few steps long, and
    // one block's first loads pass behind the other's MFMAs (4096 tokens x top-6, 64
    // experts, 4096 x 4096: 1.06 ms; whole tiles 1.10 ms; blocks that take a run of
    // half tiles and send the next one's first steps ahead of their stores 1.18 ms:
    // the loop alone takes 0.69 ms and the stores alone 0.36 ms, one after the
    // other or side by side). Also where whole tiles would leave
    // half the CUs without one: 16 rows x 4096 x 4096 on 8 experts 63 against 77 us,
    // 480 rows x 2240 x 2832 on 8 experts 36 against 49 us; with 144 whole tiles 29
    // against 27 us. Otherwise whole tiles, which read and move half as much a MFMA:
    // 65,536 rows x 4096 x 7168 on 32 experts 3.0 against 4.7 ms. Never by the
    // device's real CU count: the order of the sums must not depend on it.
    const int64_t row_tiles = pairs / kTile > a.rows.E ? pairs / kTile : pairs < a.rows.E ? pairs : a.rows.E;
    const bool half = dir == kGradWeight || row_tiles * ((a.N + kTile - 1) / kTile) <= 128;
    const int cols = half ? kHalf : kTile, threads = half ? 256 : 512;
    const int64_t nt_n = (a.N + cols - 1) / cols;
    const int64_t mtiles = dir == kGradWeight ? (int64_t)a.rows.E * ((a.M + kTile - 1) / kTile)
                                              : max_row_tiles(a.rows, kTile, pairs);
    const int64_t blocks = mtiles * nt_n;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0xFFFFFFFFll / threads) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(threads);
    if (launch_debug())
        launch_debug_print(half ? "k_grouped_gemm_bf16_half" : "k_grouped_gemm_bf16", grid, block, "direction %d n %d",
                           dir, a.N);
    if (dir == kGradWeight)
        hipLaunchKernelGGL(k_grouped_gemm_bf16_half<kGradWeight>, grid, block, 0, stream, a);
    else if (dir == kForward && half)
        hipLaunchKernelGGL(k_grouped_gemm_bf16_half<kForward>, grid, block, 0, stream, a);
    else if (dir == kGradInput && half)
        hipLaunchKernelGGL(k_grouped_gemm_bf16_half<kGradInput>, grid, block, 0, stream, a);
    else if (dir == kForward)
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kForward>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(k_grouped_gemm_bf16<kGradInput>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace ep
