// Building blocks of the matrix kernels that feed LDS by DMA.
#pragma once

#include "ep_internal.h"

namespace ep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// s_waitcnt with one counter limited (gfx9 encoding: vmcnt bits 3:0 and
// 15:14, expcnt 6:4, lgkmcnt 11:8; the others left at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// Barrier of the block without the compiler's wait for every outstanding
// access: the waits that a stage needs are stated where it is used. Nothing
// is moved across it.
__device__ __forceinline__ void block_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A byte offset that is out of range of every buffer resource made here
// (their sizes stay below 2^30): the DMA then writes zeros (checked on MI355X).
constexpr uint32_t kOutOfRange = 0x7FFFFFF0u;

// 16 bytes a lane from a buffer resource (wave-uniform base and size) at the
// lane's byte offset, to LDS at lds + 16 * lane. Offsets at or past the size
// read as zeros without touching memory, which is how tails and rows past an
// expert's last are cut off. Inline assembly, because for the intrinsic the
// compiler waits for all outstanding DMA before any LDS read; the waits are
// explicit here. m0 goes in as an operand (the asm never writes it). The compiler
// does not see that the asm is a memory instruction, so the asm itself brings the
// wait states that one needs behind a write of its scalar operands: five where a
// vector instruction wrote them (v_readfirstlane, or v_readlane where a scalar
// was spilled), one behind a scalar write of m0. Without them a descriptor
// restored just before the load is read stale, and the load goes astray.
__device__ __forceinline__ void dma16(const void* base, int size, uint32_t off, uint32_t lds) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const i32x4_t r = {__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                       __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)), __builtin_amdgcn_readfirstlane(size),
                       kBufferFlags};
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r), "{m0}"(lds) : "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)(uintptr_t)p; }

// Transposing LDS read (16 lanes share a 4 x 16 block of 16-bit values): lane
// i of a group of 16 passes the address of 4 consecutive values of row i / 4
// and gets column i of the block, rows 0 to 3 (checked on MI355X).
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

__device__ __forceinline__ bf16x8_t read_transposed(uint32_t lds, int second) {
    struct {
        i16x4_t lo, hi;
    } v;
    v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)lds);
    v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(lds + second));
    return __builtin_bit_cast(bf16x8_t, v);
}

// Swizzle of 16-byte LDS reads by the operand lanes of a 16 x 16 MFMA (lane
// (g, r): row r, chunk g). Such a read serves 16 lanes at a time, not in order:
// rows 0-3 and 12-15 of one g together with rows 4-11 of the next (and the
// reverse), so a chunk index XORed with -(r / 4) mod 4 meets each bank once;
// with r / 4 mod 4, half of the LDS cycles were conflicts (SQ_LDS_BANK_CONFLICT).
__device__ __forceinline__ int row_swizzle16(int r) { return -(r >> 2) & 3; }

typedef __attribute__((address_space(3))) bf16x8_t lds_bf16x8_t;
__device__ __forceinline__ bf16x8_t read_lds(uint32_t lds) { return *(const lds_bf16x8_t*)lds; }

// Words to and from LDS at a byte address; any of these may alias.
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t __attribute__((address_space(3), may_alias)) lds_u32x2_t;
typedef u32x4_t __attribute__((address_space(3), may_alias)) lds_u32x4_t;
__device__ __forceinline__ void write_lds(uint32_t lds, u32x2_t v) { *(lds_u32x2_t*)lds = v; }
__device__ __forceinline__ void write_lds(uint32_t lds, u32x4_t v) { *(lds_u32x4_t*)lds = v; }
__device__ __forceinline__ u32x4_t read_lds_words(uint32_t lds) { return *(const lds_u32x4_t*)lds; }

}  // namespace ep
