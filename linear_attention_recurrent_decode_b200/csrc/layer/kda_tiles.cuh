// kda_tiles.cuh -- device helpers of the layer operators: fp16 pair tiles, the
// warp-level matrix products on them, and bulk copies with bounded waits.
//
// Accuracy.  The recurrence's fp32 results (states, the gradients of g and
// beta) have to keep fp32's accuracy, which one fp16 or bf16 product does not.
// Every fp32 operand x is therefore held as an fp16 pair x s = hi + lo with a
// power of two s that puts the tile's largest magnitude in [2^13, 2^14): hi has
// 11 significant bits and lo the next 11, so the pair is within 2^-22 of x, or
// within 2^-39 of the tile's largest value where x is far below it (fp16's
// subnormals).  A product takes three MMAs (hi.hi + hi.lo + lo.hi; the dropped
// lo.lo term is 2^-22 relative), two where one side is exact in 11 bits (a bf16
// input), accumulated in fp32.  A bf16 pair would leave 2^-17, a tf32 pair the
// same 2^-22 at half the MMA rate (measured here, mma.sync: 552 TFLOP/s for
// fp16 and bf16, 276 for tf32).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kdal {

constexpr int kC = 64;    // tokens per chunk
constexpr int kB = 16;    // tokens per sub-block
constexpr int kNB = kC / kB;
constexpr int kK = 128;   // key width
constexpr int kV = 128;   // value width

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- launches
// A call's kernels are launched so that one may start while the last blocks of
// the one before it run out (programmatic dependent launch); its blocks find
// their place and set up meanwhile.  A kernel that can be a call's first waits
// before its first access of global memory; the others touch what earlier
// kernels wrote, or write anything, only behind their wait.  Every block waits
// before it ends: a kernel that is complete has everything before it complete.
// Kernels whose grids leave SMs idle may let the next one start earlier; for long
// calls that measured up to 6 % slower, as the next kernel's blocks then take the
// SMs that the running one's last blocks are given.
constexpr uint32_t kSms = 148;
__device__ __forceinline__ void wait_upstream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- scales
// The power of two that puts a tile whose largest magnitude is `m` in
// [2^13, 2^14), kept within 2^+-100: magnitudes from 2^-86 (below, pairs lose
// bits) to 2^115 (above, they overflow), and a scale times a factor that goes
// before it, or the inverse of one times a product's accumulator (up to 2^35),
// stays inside fp32.  Two inverses may be multiplied first: that leaves fp32's
// range only where the product itself does.  1 for a zero, infinite or NaN
// maximum (the values then carry themselves).
__device__ __forceinline__ float pow2_scale(float m) {
  const int e = static_cast<int>(__float_as_uint(m) >> 23) & 0xff;  // m >= 0
  if (e == 0 || e == 255) return 1.f;
  int s = 13 - (e - 127);
  s = s > 100 ? 100 : (s < -100 ? -100 : s);
  return __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
}
// The inverse of a power of two.
__device__ __forceinline__ float pow2_inv(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Largest of non-negative floats over the warp (their bits order like the values).
__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// ---------------------------------------------------------------- fp16 pairs
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// (x, y) as packed hi and lo halves.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = as_u32(h);
  lo = as_u32(__floats2half2_rn(x - f.x, y - f.y));
}
__device__ __forceinline__ float2 join2(uint32_t hi, uint32_t lo) {
  const float2 h = __half22float2(as_half2(hi)), l = __half22float2(as_half2(lo));
  return make_float2(h.x + l.x, h.y + l.y);
}

// ---------------------------------------------------------------- tiles
// Byte offsets of element (r, c) of a 16-bit tile.
//
// Core: 16-byte pieces of eight columns, the pieces of one column block
// contiguous over the ROWS rows.  Eight rows of a piece are one core matrix of
// the tensor cores' unswizzled shared-memory layout, so the same tile serves as
// an operand with its rows as the product's columns (K-major) and, transposed,
// with its rows contracted (MN-major), and as an ldmatrix source without bank
// conflicts; a warp whose lanes own rows writes it in whole lines.  The image in
// global memory is the same: a tile is one bulk copy.
template <int ROWS>
struct Core {
  static constexpr int kBlock = ROWS * 16;  // bytes from one column block to the next
  static __device__ __forceinline__ uint32_t off(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * kBlock + r * 16 + (c & 7) * 2);
  }
};
// Rows of 256 bytes whose 16-byte pieces are permuted by the row: for tiles written a row of 16-byte pieces at a time.
struct Rows128 {
  static __device__ __forceinline__ uint32_t off(int r, int c) {
    return static_cast<uint32_t>(r * 256 + ((((c >> 3) ^ (r & 7)) << 4) | ((c & 7) * 2)));
  }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// A fragment (16 x 16 at (m0, k0)) of a tile stored [m][k] or [k][m].
template <class L>
__device__ __forceinline__ void load_a(uint32_t tile, int m0, int k0, int lane, uint32_t (&a)[4]) {
  ldsm4(tile + L::off(m0 + (lane & 15), k0 + (lane >> 4) * 8), a);
}
template <class L>
__device__ __forceinline__ void load_a_t(uint32_t tile, int m0, int k0, int lane, uint32_t (&a)[4]) {
  ldsm4t(tile + L::off(k0 + (lane & 7) + (lane >> 4) * 8, m0 + ((lane >> 3) & 1) * 8), a);
}
// B fragments of two 8-column tiles (16 x 16 at (k0, n0); b[0..1] columns n0..,
// b[2..3] columns n0 + 8..) of a tile stored [n][k] or [k][n].
template <class L>
__device__ __forceinline__ void load_b(uint32_t tile, int k0, int n0, int lane, uint32_t (&b)[4]) {
  ldsm4(tile + L::off(n0 + (lane & 7) + (lane >> 4) * 8, k0 + ((lane >> 3) & 1) * 8), b);
}
template <class L>
__device__ __forceinline__ void load_b_t(uint32_t tile, int k0, int n0, int lane, uint32_t (&b)[4]) {
  ldsm4t(tile + L::off(k0 + (lane & 15), n0 + (lane >> 4) * 8), b);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The MMA adds to its accumulator with truncation, half an ulp of the running
// sum low on average, so a long chain of them is biased by more than fp32
// rounding.  The cross terms (2^-11 of the product) therefore go ahead of the
// hi.hi terms or into accumulators of their own, and partial sums over a few
// k steps are joined by ordinary additions.
__device__ __forceinline__ void mma_pair(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  mma_f16(c0, a, b[0], b[1]);
  mma_f16(c1, a, b[2], b[3]);
}
// The A fragment pair of 16 accumulator columns (two 8-column tiles) times s.
__device__ __forceinline__ void frag_a(const float (&c0)[4], const float (&c1)[4], float s, uint32_t (&ah)[4],
                                       uint32_t (&al)[4]) {
  split2(c0[0] * s, c0[1] * s, ah[0], al[0]);
  split2(c0[2] * s, c0[3] * s, ah[1], al[1]);
  split2(c1[0] * s, c1[1] * s, ah[2], al[2]);
  split2(c1[2] * s, c1[3] * s, ah[3], al[3]);
}
__device__ __forceinline__ void scale_frag(uint32_t (&a)[4], __half2 f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = as_u32(__hmul2(as_half2(a[i]), f));
}
// 8x8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ---------------------------------------------------------------- tf32 pairs
// For operands whose range is too wide for one fp16 scale (decay factors of up
// to e^+-80 inside a sub-block): x = hi + lo in tf32, three MMAs of k = 8.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// ---------------------------------------------------------------- bulk copies
__device__ __forceinline__ void mbar_init(uint64_t* mbar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(mbar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_expect(uint64_t* mbar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(mbar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(mbar)) : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* mbar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(mbar))
               : "memory");
}
// Polls before a wait gives up: each try_wait suspends for up to some
// microseconds, so this is seconds against the microseconds of any copy here.
constexpr uint32_t kWaitLimit = 1u << 20;
// Waits for the mbarrier's phase of the given parity; false if it gave up.
__device__ __forceinline__ bool mbar_wait(uint64_t* mbar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done) : "r"(smem_addr(mbar)), "r"(parity) : "memory");
    if (done) return true;
  }
  return false;
}
// Orders this thread's ordinary shared-memory accesses before later bulk copies into the same bytes.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- blocks that go on
// A running block takes over a block of the same grid that has not started (cluster launch control): request (one thread;
// the last answer has been read by all) and, once the barrier's phase is done, its index, or -1 if there is none left.
// After a -1 no further request is made.
__device__ __forceinline__ void request_block(uint4* answer, uint64_t* mbar) {
  fence_async();
  mbar_expect(mbar, sizeof(uint4));
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(smem_addr(answer)), "r"(smem_addr(mbar)) : "memory");
}
__device__ __forceinline__ int64_t taken_block(const uint4* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, a;\n\t}\n"
      : "=r"(got), "=r"(x) : "r"(smem_addr(answer)) : "memory");
  fence_async();
  return got ? static_cast<int64_t>(x) : -1;
}

}  // namespace kdal
