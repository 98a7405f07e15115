// kda_umma.cuh -- tensor memory and tcgen05 products of the layer operators.
//
// Products here are D [M x N] += A [M x 16] B [16 x N] in fp16 with fp32
// accumulators: D lies in tensor memory, A there too (M = 128: lane = row; two
// halves a column) or in shared memory, B in shared memory; operands in shared
// memory are Core tiles of the unswizzled layout.  With M = 64 rows 16 i .. are
// lanes 32 i .., a warp's own.  One warp
// issues them, all its lanes running the same code and one elected lane the
// MMA: their operands then stay in uniform registers (inside a branch of one
// lane each MMA took 78 cycles to issue).  Measured on B200: an MMA takes 44
// cycles for N = 64 (its issue) and 64 for N = 128, and the commit behind the
// last reaches a waiting warp 230 cycles later.
#pragma once

#include "kda_tiles.cuh"

namespace kdal {

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Consecutive columns of this thread's lane; a warp reaches the 32 lanes of its index modulo 4.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
               : "memory");
}

// Arrives on `mbar` once every product issued by this warp so far is complete.
__device__ __forceinline__ void umma_commit(uint64_t* mbar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_addr(mbar))
      : "memory");
}

// Operand in shared memory: a Core<ROWS> tile of fp16 with its rows as the product's columns (or A's rows; K-major) or
// contracted (MN-major).
template <int ROWS, bool TRANS>
struct Operand {
  static constexpr uint32_t kBlock = Core<ROWS>::kBlock;
  static constexpr uint32_t kStep = TRANS ? 256 : 2 * kBlock;  // bytes from one 16-element step to the next
  uint64_t desc;
  // Leading byte offset: from one 8-element core matrix to the next along the contraction; stride byte offset: along
  // the columns; descriptor version 1 at bit 46.
  __device__ __forceinline__ explicit Operand(uint32_t addr) {
    constexpr uint32_t lbo = TRANS ? 128 : kBlock, sbo = TRANS ? kBlock : 128;
    desc = static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46);
  }
  __device__ __forceinline__ uint64_t at(int step) const { return desc + static_cast<uint64_t>(step * (kStep >> 4)); }
};

// D (+)= A B for one 16-element step; N columns.  Instruction descriptor: fp32 accumulator, fp16 operands, A K-major, B
// MN-major at bit 16, N / 8 at bit 17, M / 16 at bit 24.
template <int N, bool TRANS>
__device__ __forceinline__ void umma(uint32_t d, uint32_t a, uint64_t b, bool accumulate) {
  constexpr uint32_t idesc = (1u << 4) | (TRANS ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
// D = (ah + al) (bh + bl) without al.bl over K elements, the cross terms first (they are 2^-11 of the product, and the
// accumulator's rounding then does not see them behind the large sum).  A: columns hi, lo of K / 2 each; B: planes hi, lo
// `plane` bytes apart.  AEXACT: A is one plane.
template <int N, int K, int ROWS, bool TRANS, bool AEXACT = false>
__device__ __forceinline__ void umma_pairs(uint32_t d, uint32_t a, uint32_t b, uint32_t plane) {
  const Operand<ROWS, TRANS> bh(b), bl(b + plane);
#pragma unroll
  for (int k = 0; k < K / 16; ++k) {
    umma<N, TRANS>(d, a + k * 8, bl.at(k), k > 0);
    if constexpr (!AEXACT) umma<N, TRANS>(d, a + K / 2 + k * 8, bh.at(k), true);
  }
#pragma unroll
  for (int k = 0; k < K / 16; ++k) umma<N, TRANS>(d, a + k * 8, bh.at(k), true);
}

// The same with A [64 rows] in shared memory, both operands pairs (AEXACT: A one plane) of the given tiles.
template <int N, int K, int AROWS, bool ATRANS, int BROWS, bool BTRANS, bool AEXACT>
__device__ __forceinline__ void umma_tiles(uint32_t d, uint32_t a, uint32_t a_plane, uint32_t b, uint32_t b_plane) {
  constexpr uint32_t idesc = (1u << 4) | (ATRANS ? 1u << 15 : 0u) | (BTRANS ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (4u << 24);
  const Operand<AROWS, ATRANS> ah(a), al(a + a_plane);
  const Operand<BROWS, BTRANS> bh(b), bl(b + b_plane);
  auto mma = [&](uint64_t x, uint64_t y, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(x), "l"(y), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  };
#pragma unroll
  for (int k = 0; k < K / 16; ++k) {
    mma(ah.at(k), bl.at(k), k > 0);
    if constexpr (!AEXACT) mma(al.at(k), bh.at(k), true);
  }
#pragma unroll
  for (int k = 0; k < K / 16; ++k) mma(ah.at(k), bh.at(k), true);
}
// 16 lanes x 8 N8 columns in the accumulator layout of mma.sync's m16n8 tiles: acc[n][0, 1] row lane / 4, columns 8 n + 2
// (lane % 4) + {0, 1}, acc[n][2, 3] eight rows on.
__device__ __forceinline__ void tmem_ld_tiles(uint32_t taddr, float (&acc)[4][4]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j >> 2][j & 3] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_ld_tiles(uint32_t taddr, float (&acc)[2][4]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j >> 2][j & 3] = __uint_as_float(r[j]);
}

}  // namespace kdal
