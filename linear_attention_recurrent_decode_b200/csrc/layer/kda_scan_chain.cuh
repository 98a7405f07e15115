// kda_scan_chain.cuh -- the scan's sequential kernels: the states from chunk to
// chunk, forwards with the outputs, and their gradients backwards.
//
// Forward, per chunk (see kda_scan_prep.cuh):
//   r = Rt - Wr S0;  U = beta r;  O = scale (Qt S0 + P U);  S1 = Diag(exp(Gamma_C)) S0 + Ke^T U.
// Backward, per chunk in reverse, with the gradient dS1 of its end state:
//   dU = scale P^T dO + Ke dS1
//   dS0 = Diag(exp(Gamma_C)) dS1 + scale Qt^T dO - Wr^T (beta dU).
//
// One CTA a sequence and head.  Everything is transposed so that the 128 value
// columns are the M rows of the tensor cores' products and the lanes of tensor
// memory: four threads a value column keep the state, 32 channels each, in fp32
// registers.  Per chunk they write the state as an fp16 pair into
// tensor memory (the A operand), read S0^T Wr^T back, write U^T there, and add
// the read product U^T Ke to the decayed registers: the fp32 state itself never
// passes through a product's accumulator, and rows never meet, but for the
// scales, one per 32 of them.  The B operands are the record's tiles, straight
// from bulk copies.
//
// Long sequences of few heads would leave most SMs idle.  They are cut into
// segments: a segment's end state is linear in its start state, S -> M S + E.  A
// first call walks every segment from zero (E) and, with no values, from the
// identity (the matrix M, whose columns are 128 more value columns); a small
// kernel joins the segments in order, and a second call walks them all from
// their right starts.  That is three times the work in (1 / segments) of the
// time.  Backwards the transition is M's transpose.
//
// Warps: 0-15 compute, 16 copies, 17 issues the products.  A chunk's critical
// path is two products with a conversion behind each.  The outputs' products run
// behind the state's, under the next chunk's first conversion, and the compute
// warps read them back and store them while that chunk's first product runs
// (four warps of their own for it left 80 registers a thread, too few).
//
// Measured (B200): 4.7 us a chunk forwards, 3.7 without outputs, 6.2 where states
// and residuals are saved, 5.5 backwards, whatever the number of CTAs up to one an
// SM: the latency of that path (conversion, product, read-back, twice), not the
// tensor cores (26 % of their cycles) or memory (36 % of its rate).
#pragma once

#include "kda_scan_common.cuh"
#include "kda_umma.cuh"

namespace kdal {

constexpr int kParts = 4;                    // threads of a value column
constexpr int kComputeWarps = 4 * kParts;
constexpr int kPartK = kK / kParts, kPartT = kC / kParts;  // a thread's channels and tokens
constexpr uint32_t kTmemColumns = 512;

// Shared memory of both chains.  Wr, Ke and the header of two chunks, Qt and P of one.
struct ChainSmem {
  unsigned char wr[2][2 * Record::kPlane], ke[2][2 * Record::kPlane];
  unsigned char qt[2 * Record::kPlane], p[kC * kC * 4];
  unsigned char hdr[2][Record::kHdr];
  alignas(16) float peak[4][kParts][4];      // [exchange][part][quarter of the value columns]
  uint64_t full_wr[2], full_ke[2], full_hdr[2], full_qt, full_p, empty_hdr[2];
  uint64_t state, rows;             // written by the compute warps: the state, U (or dU)
  // Products done, by chunk parity: S0^T Wr^T (or dS1^T Ke^T), the state's with U; with Qt; forward: the outputs' with P.
  // A tile's place is free again once the products that read it are.
  uint64_t first[2], last[2], with_qt, out_done;
  uint64_t d_out;                   // backward: dO is written
  uint64_t end;
  uint32_t tmem;
};
static_assert(sizeof(ChainSmem) <= 232448, "shared memory of an SM");

// A wait that remembers whether any gave up; from then on none waits, and the kernel runs to its end on whatever it has,
// so that every barrier stays matched.  For whole warps `ok` is uniform.
struct Waiter {
  bool ok = true;
  __device__ __forceinline__ void one(uint64_t* bar, int64_t phase) {  // a single thread
    ok = ok && mbar_wait(bar, static_cast<uint32_t>(phase & 1));
  }
  __device__ __forceinline__ void warp(uint64_t* bar, int64_t phase) {
    one(bar, phase);
    ok = __all_sync(0xffffffffu, ok);
  }
};
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void chain_init(ChainSmem& sm) {
  if (threadIdx.x < 32) tmem_alloc(&sm.tmem, kTmemColumns);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.full_wr[i], 1);
      mbar_init(&sm.full_ke[i], 1);
      mbar_init(&sm.full_hdr[i], 1);
      mbar_init(&sm.first[i], 1);
      mbar_init(&sm.last[i], 1);
      mbar_init(&sm.empty_hdr[i], kComputeWarps);
    }
    mbar_init(&sm.full_qt, 1);
    mbar_init(&sm.full_p, 1);
    mbar_init(&sm.with_qt, 1);
    mbar_init(&sm.state, kComputeWarps);
    mbar_init(&sm.rows, kComputeWarps);
    mbar_init(&sm.d_out, kComputeWarps);
    mbar_init(&sm.out_done, 1);
    mbar_init(&sm.end, 1);
    mbar_fence_init();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
}
__device__ __forceinline__ void chain_exit(ChainSmem& sm) {
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x < 32) tmem_dealloc(sm.tmem, kTmemColumns);
}

// The copies of every chunk's tiles, one thread; a tile's copy starts once the products of the tile before it in the
// same place are complete.
template <bool FWD>
__device__ __forceinline__ void chain_copies(ChainSmem& sm, Waiter& w, const unsigned char* rec, int64_t step, int64_t chunks,
                                             bool outputs) {
  int64_t c = 0;
  for (; c < chunks && w.ok; ++c, rec += step) {
    const int b = static_cast<int>(c & 1);
    auto put = [&](void* dst, int off, uint32_t bytes, uint64_t* full) {
      if (!w.ok) return;
      mbar_expect(full, bytes);
      bulk_load(dst, rec + off, bytes, full);
    };
    if (c >= 2) w.one(&sm.empty_hdr[b], (c >> 1) - 1);
    put(sm.hdr[b], 0, Record::kHdr, &sm.full_hdr[b]);
    // Wr is read by the first product forwards, by the last backwards; Ke the other way round
    if (c >= 2) w.one(&sm.first[b], (c >> 1) - 1);
    if constexpr (FWD) put(sm.wr[b], Record::kWr, 2 * Record::kPlane, &sm.full_wr[b]);
    else put(sm.ke[b], Record::kKe, 2 * Record::kPlane, &sm.full_ke[b]);
    if (c >= 2) w.one(&sm.last[b], (c >> 1) - 1);
    if constexpr (FWD) put(sm.ke[b], Record::kKe, 2 * Record::kPlane, &sm.full_ke[b]);
    else put(sm.wr[b], Record::kWr, 2 * Record::kPlane, &sm.full_wr[b]);
    if (!outputs) continue;
    if (c >= 1) w.one(&sm.with_qt, c - 1);
    put(sm.qt, Record::kQt, 2 * Record::kPlane, &sm.full_qt);
    // P: backwards the product with it was issued ahead of the chunk's first
    if (c >= 1) w.one(FWD ? &sm.out_done : &sm.first[b ^ 1], FWD ? c - 1 : (c - 1) >> 1);
    put(sm.p, Record::kP, kC * kC * 4, &sm.full_p);
  }
  // After a wait that gave up: the CTA must not end with copies into it in flight.  The last copy into each place may be.
  if (w.ok || c == 0) return;
  --c;
  for (int64_t d = c > 0 ? c - 1 : 0; d <= c; ++d) {
    mbar_wait(&sm.full_hdr[d & 1], static_cast<uint32_t>((d >> 1) & 1));
    mbar_wait(&sm.full_wr[d & 1], static_cast<uint32_t>((d >> 1) & 1));
    mbar_wait(&sm.full_ke[d & 1], static_cast<uint32_t>((d >> 1) & 1));
    if (outputs) {
      mbar_wait(&sm.full_qt, static_cast<uint32_t>(d & 1));
      mbar_wait(&sm.full_p, static_cast<uint32_t>(d & 1));
    }
  }
}

// A quarter of a value column: the thread's channels of a [K][V] block.
__device__ __forceinline__ void load_state(const float* blk, int v, int part, float (&s)[kPartK]) {
#pragma unroll
  for (int j = 0; j < kPartK; ++j) s[j] = blk == nullptr ? 0.f : blk[(part * kPartK + j) * kV + v];
}
__device__ __forceinline__ void store_state(float* blk, int v, int part, const float (&s)[kPartK]) {
#pragma unroll
  for (int j = 0; j < kPartK; ++j) blk[(part * kPartK + j) * kV + v] = s[j];
}
// The largest of `m` over a quarter's 32 value columns: the four warps that share them.
__device__ __forceinline__ float quarter_max(ChainSmem& sm, int exchange, float m, int part, int quarter) {
  m = warp_max(m);
  sm.peak[exchange][part][quarter] = m;  // every lane the same value
  asm volatile("bar.sync %0, 128;" ::"r"(quarter + 1) : "memory");
  m = fmaxf(fmaxf(sm.peak[exchange][0][quarter], sm.peak[exchange][1][quarter]),
            fmaxf(sm.peak[exchange][2][quarter], sm.peak[exchange][3][quarter]));
  return m;
}

// The largest over all value columns, once every warp is known to have handed its own in.  S0 and r are kept for the
// gradients with one scale each, as the products there contract the value columns; a barrier of all warps for it, twice
// a chunk, made the chains 25 % slower.
__device__ __forceinline__ float all_max(const ChainSmem& sm, int exchange) {
  float m = 0.f;
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    const float4 q = *reinterpret_cast<const float4*>(&sm.peak[exchange][part][0]);
    m = fmaxf(m, fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)));
  }
  return m;
}

// x[n] sc as a pair, this thread's elements `first` .. of K: into tensor memory as the lane's A operand (hi, then lo), or
// into the record's Core<kV> tile [v][element] with planes `plane` apart (apart from each other: the stores to the record
// are issued while the products run).  With `f`, the elements times f[0 .. COUNT - 1] (shared memory).
template <int K, bool TMEM, int COUNT>
__device__ __forceinline__ void write_pair(uint32_t ta, unsigned char* tile, int plane, int v, int first, const float (&x)[COUNT], float sc,
                                           const float* f = nullptr) {
#pragma unroll
  for (int g = 0; g < COUNT / 16; ++g) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 fe = make_float2(sc, sc);
      if (f != nullptr) {
        const float2 y = *reinterpret_cast<const float2*>(f + g * 16 + 2 * e);
        fe = make_float2(y.x * sc, y.y * sc);
      }
      split2(x[g * 16 + 2 * e] * fe.x, x[g * 16 + 2 * e + 1] * fe.y, hi[e], lo[e]);
    }
    if constexpr (TMEM) {
      tmem_st(ta + first / 2 + g * 8, hi);
      tmem_st(ta + K / 2 + first / 2 + g * 8, lo);
    }
    if constexpr (!TMEM) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t off = Core<kV>::off(v, first + g * 16 + e * 8);
        *reinterpret_cast<uint4*>(tile + off) = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
        *reinterpret_cast<uint4*>(tile + plane + off) = make_uint4(lo[4 * e], lo[4 * e + 1], lo[4 * e + 2], lo[4 * e + 3]);
      }
    }
  }
}
// s = s d + f x, x read from tensor memory, d the channels' factors in shared memory.
template <bool DECAY>
__device__ __forceinline__ void add_product(uint32_t ta, const float* d, float f, float (&s)[kPartK]) {
  uint32_t x[kPartK];
  tmem_ld(ta, x);
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < kPartK; j += 4) {
    float4 dj = make_float4(1.f, 1.f, 1.f, 1.f);
    if constexpr (DECAY) dj = *reinterpret_cast<const float4*>(d + j);
    s[j] = fmaf(s[j], dj.x, __uint_as_float(x[j]) * f);
    s[j + 1] = fmaf(s[j + 1], dj.y, __uint_as_float(x[j + 1]) * f);
    s[j + 2] = fmaf(s[j + 2], dj.z, __uint_as_float(x[j + 2]) * f);
    s[j + 3] = fmaf(s[j + 3], dj.w, __uint_as_float(x[j + 3]) * f);
  }
}
template <int N>
__device__ __forceinline__ float abs_max(const float (&x)[N]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(x[j]));
  return m;
}
template <int N>
__device__ __forceinline__ float abs_max(const float (&x)[N], const float* f) {  // of the products with f (shared memory)
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const float4 y = *reinterpret_cast<const float4*>(f + j);
    m = fmaxf(m, fmaxf(fmaxf(fabsf(x[j] * y.x), fabsf(x[j + 1] * y.y)), fmaxf(fabsf(x[j + 2] * y.z), fabsf(x[j + 3] * y.w))));
  }
  return m;
}

// ---------------------------------------------------------------- forward
// Columns of tensor memory.
struct ForwardColumns {
  static constexpr uint32_t kState = 0, kU = 128, kX = 192, kO1 = 256, kO2 = 320, kDelta = 384;
};
constexpr int kChainThreads = (kComputeWarps + 2) * 32;

__global__ void __launch_bounds__(kChainThreads, 1) kda_scan_forward_kernel(const __grid_constant__ ScanParams p) {
  using Col = ForwardColumns;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChainSmem& sm = *reinterpret_cast<ChainSmem*>(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, quarter = warp & 3, v = quarter * 32 + lane;
  // the transitions' call: E and M of a segment in neighbouring blocks
  int64_t slot, h;
  slot_and_head(p, p.transitions ? blockIdx.x >> 1 : blockIdx.x, slot, h);
  const bool map = p.transitions && (blockIdx.x & 1);
  const Segment seg = locate_segment(p, slot);
  const bool last = seg.seg == seg.segs - 1;
  // The last segment's end is nobody's start, and the first's start is known: it has no use for M.
  if (seg.segs == 0 || (p.transitions && (last || (map && seg.seg == 0)))) {
    wait_upstream();
    return;
  }
  const int64_t n = seg.n, start = seg.start + seg.first * kC, len = seg.len - seg.first * kC, chunks = seg.chunks;
  const int64_t blk = state_block(p, n);
  if (blk < 0) {  // inactive: zero outputs
    wait_upstream();
    if (!p.transitions) {
      const int64_t rows = len < chunks * kC ? len : chunks * kC;
      for (int64_t t = threadIdx.x; t < rows * 16; t += kChainThreads)
        *reinterpret_cast<uint4*>(p.out + (start + (t >> 4)) * p.out_ts + h * kV + (t & 15) * 8) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const bool outputs = p.out != nullptr && !p.transitions, save = p.save && !p.transitions;
  chain_init(sm);
  const int64_t sblk = (blk * p.HV + h) * kK * kV, gblk = (slot * p.HV + h) * kK * kV, step = p.HV * p.rec_bytes;
  unsigned char* rec = record(p, first_slot(p, n, seg.start) + seg.first, h);
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0), mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  wait_upstream();
  Waiter w;
  if (warp < kComputeWarps) {
    const int part = warp >> 2;
    float s[kPartK];
    // A segment's start: the first's is the call's, the others' the end of the one before (zero for their E).  The walk for
    // E copies the call's to the first segment's block of seg_map, which has no M, and the walk for the results starts
    // from that copy: s_out may be s_in, and the block of the last segment stores there whenever it is done.
    const float* const call = p.s_in == nullptr ? nullptr : p.s_in + sblk;
    const float* const from = seg.seg > 0 ? (p.transitions ? nullptr : p.seg_state + gblk - p.HV * kK * kV)
                                          : (call == nullptr || p.transitions || seg.segs == 1 ? call : p.seg_map + gblk);
    float* const to = p.transitions ? (map ? p.seg_map : p.seg_state) + gblk : (last && p.s_out != nullptr ? p.s_out + sblk : nullptr);
    load_state(from, v, part, s);
    if (p.transitions && from != nullptr) store_state(p.seg_map + gblk, v, part, s);
    if (map) {
#pragma unroll
      for (int j = 0; j < kPartK; ++j) s[j] = part * kPartK + j == v ? 1.f : 0.f;
    }
    // O = scale (Qt S0 + P U) of a chunk, its factors kept from there: this thread's value column and tokens; neighbours
    // trade a token each, so that a thread stores two values.
    float out_f1 = 0.f, out_f2 = 0.f;
    int64_t left = len - part * kPartT - (lane & 1);
    __nv_bfloat16* out_at = p.out + (start + part * kPartT + (lane & 1)) * p.out_ts + h * kV + (v & ~1);
    auto put_outputs = [&](int64_t c) {  // of each chunk in turn
      w.warp(&sm.out_done, c);
      fence_after_sync();
      const int rows = static_cast<int>(left < kC ? left : kC);
      left -= kC;
      __nv_bfloat16* out = out_at;
      out_at += kC * p.out_ts;
      uint32_t a[kPartT], x[kPartT];
      tmem_ld(mine + Col::kO1 + part * kPartT, a);
      tmem_ld(mine + Col::kO2 + part * kPartT, x);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < kPartT; j += 2, out += 2 * p.out_ts) {
        const float o0 = fmaf(__uint_as_float(a[j]), out_f1, __uint_as_float(x[j]) * out_f2);
        const float o1 = fmaf(__uint_as_float(a[j + 1]), out_f1, __uint_as_float(x[j + 1]) * out_f2);
        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? o0 : o1, 1);
        const __nv_bfloat162 y = lane & 1 ? __floats2bfloat162_rn(got, o1) : __floats2bfloat162_rn(o0, got);
        if (j < rows) *reinterpret_cast<__nv_bfloat162*>(out) = y;
      }
    };
    for (int64_t c = 0; c < chunks; ++c, rec += step) {
      const int b = static_cast<int>(c & 1);
      const float* const hdr = reinterpret_cast<const float*>(sm.hdr[b]);
      // ---- the state as a pair
      const float sc_s = pow2_scale(quarter_max(sm, 2 * b, abs_max(s), part, quarter));
      if (outputs && c > 0) w.warp(&sm.with_qt, c - 1);  // the outputs' product read the last one
      fence_after_sync();
      write_pair<kK, true>(mine + Col::kState, nullptr, 0, v, part * kPartK, s, sc_s);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sm.state, lane);
      float r[kPartT];
      {
        const float4* const rt = reinterpret_cast<const float4*>(rec + Record::kRt) + part * (kPartT / 4) * kV + v;
#pragma unroll
        for (int j = 0; j < kPartT / 4; ++j) {
          const float4 x = map ? make_float4(0.f, 0.f, 0.f, 0.f) : rt[j * kV];
          r[4 * j] = x.x;
          r[4 * j + 1] = x.y;
          r[4 * j + 2] = x.z;
          r[4 * j + 3] = x.w;
        }
      }
      if (outputs && c > 0) put_outputs(c - 1);
      w.warp(&sm.full_hdr[b], c >> 1);
      // ---- r = Rt - S0 Wr, U = beta r
      w.warp(&sm.first[b], c >> 1);
      fence_after_sync();
      {
        const float f = -pow2_inv(sc_s) * pow2_inv(hdr[Record::kScWr]);
        uint32_t x[kPartT];
        tmem_ld(mine + Col::kX + part * kPartT, x);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kPartT; ++j) r[j] = fmaf(__uint_as_float(x[j]), f, r[j]);
      }
      const float* const beta = hdr + Record::kBeta + part * kPartT;
      const float sc_u = pow2_scale(quarter_max(sm, 1, abs_max(r, beta), part, quarter));
      fence_after_sync();
      write_pair<kC, true>(mine + Col::kU, nullptr, 0, v, part * kPartT, r, sc_u, beta);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sm.rows, lane);
      if (save) {
        // Every warp has written its state, and its largest value before that (it is overwritten two chunks on).
        const float peak_s = all_max(sm, 2 * b);
        // r's scale from a bound, |Rt| + 128 |Wr| |S0| (loose by some 2^8 of the 2^17 that a pair has to spare)
        const float sc_saved = pow2_scale(peak_s), sc_r = pow2_scale(fmaf(kK * hdr[Record::kMxWr], peak_s, hdr[Record::kMxRt]));
        write_pair<kK, false>(0, rec + Record::kS, kV * kK * 2, v, part * kPartK, s, sc_saved);
        write_pair<kC, false>(0, rec + Record::kR, Record::kPlane, v, part * kPartT, r, sc_r);
        if (threadIdx.x == 0) {
          float* const sc = reinterpret_cast<float*>(rec + Record::kSc);
          sc[Record::kScS] = sc_saved;
          sc[Record::kScR] = sc_r;
        }
      }
      // ---- S1 = Diag(exp(Gamma_C)) S0 + Ke^T U
      out_f1 = pow2_inv(sc_s) * pow2_inv(hdr[Record::kScQt]) * p.scale;
      out_f2 = pow2_inv(sc_u) * pow2_inv(hdr[Record::kScP]) * p.scale;
      w.warp(&sm.last[b], c >> 1);
      fence_after_sync();
      add_product<true>(mine + Col::kDelta + part * kPartK, hdr + Record::kDecay + part * kPartK, pow2_inv(sc_u) * pow2_inv(hdr[Record::kScKe]), s);
      fence_before_sync();
      warp_arrive(&sm.empty_hdr[b], lane);
    }
    if (outputs && chunks > 0) put_outputs(chunks - 1);
    if (!w.ok) {
      if (lane == 0) set_error(p);
    } else if (to != nullptr) {
      store_state(to, v, part, s);
    }
  } else if (warp == kComputeWarps) {
    if (lane == 0) chain_copies<true>(sm, w, rec, step, chunks, outputs);
    __syncwarp();
  } else {
    for (int64_t c = 0; c < chunks; ++c) {
      const int b = static_cast<int>(c & 1);
      w.warp(&sm.full_wr[b], c >> 1);
      w.warp(&sm.state, c);
      fence_after_sync();
      umma_pairs<kC, kK, kC, false>(tmem + Col::kX, tmem + Col::kState, smem_addr(sm.wr[b]), Record::kPlane);
      umma_commit(&sm.first[b]);
      w.warp(&sm.full_ke[b], c >> 1);
      w.warp(&sm.rows, c);
      fence_after_sync();
      umma_pairs<kK, kC, kC, true>(tmem + Col::kDelta, tmem + Col::kU, smem_addr(sm.ke[b]), Record::kPlane);
      umma_commit(&sm.last[b]);
      if (outputs) {  // over outputs that every warp has read: it wrote its rows after that
        w.warp(&sm.full_qt, c);
        umma_pairs<kC, kK, kC, false>(tmem + Col::kO1, tmem + Col::kState, smem_addr(sm.qt), Record::kPlane);
        umma_commit(&sm.with_qt);
        w.warp(&sm.full_p, c);
        umma_pairs<kC, kC, kC, false>(tmem + Col::kO2, tmem + Col::kU, smem_addr(sm.p), kC * kC * 2);
        umma_commit(&sm.out_done);
      }
    }
    if (chunks > 0) {
      umma_commit(&sm.end);
      mbar_wait(&sm.end, 0);
    }
    __syncwarp();
    if (!w.ok && lane == 0) set_error(p);
  }
  chain_exit(sm);
}

// ---------------------------------------------------------------- backward
// dS1 as a pair and, once its product is done, the product with Wr share columns.
struct BackwardColumns {
  static constexpr uint32_t kState = 0, kDelta = 0, kDO = 128, kU = 160, kX1 = 224, kX2 = 288, kExtra = 352;
};

__global__ void __launch_bounds__(kChainThreads, 1) kda_scan_backward_kernel(const __grid_constant__ ScanParams p) {
  using Col = BackwardColumns;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChainSmem& sm = *reinterpret_cast<ChainSmem*>(smem_raw);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, quarter = warp & 3, v = quarter * 32 + lane;
  int64_t slot, h;
  slot_and_head(p, blockIdx.x, slot, h);
  wait_upstream();  // this may be its call's first kernel
  const Segment seg = locate_segment(p, slot);
  // The first segment's start gradient is the result itself, and nobody's end.
  if (seg.segs == 0 || (p.transitions && seg.seg == 0)) return;
  const int64_t n = seg.n, start = seg.start + seg.first * kC, len = seg.len - seg.first * kC, chunks = seg.chunks;
  chain_init(sm);
  const int64_t sblk = (n * p.HV + h) * kK * kV, gblk = (slot * p.HV + h) * kK * kV, step = p.HV * p.rec_bytes;
  unsigned char* rec = record(p, first_slot(p, n, seg.start) + seg.first + (chunks > 0 ? chunks - 1 : 0), h);
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0), mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  Waiter w;
  // i counts the chunks walked: i = 0 is the last chunk, and barriers' phases go by i
  if (warp < kComputeWarps) {
    const int part = warp >> 2;
    float s[kPartK];
    // a segment's end: the last's is the call's, the others' the start of the one behind (zero for their transition)
    const float* const from = seg.seg == seg.segs - 1 ? (p.d_final == nullptr ? nullptr : p.d_final + sblk)
                                                      : (p.transitions ? nullptr : p.seg_state + gblk + p.HV * kK * kV);
    load_state(from, v, part, s);
    // dO^T: this thread's value column and tokens, exact in fp16 after scaling (bf16 has 8 bits)
    unsigned short raw[kPartT];  // as loaded: packing them would wait for the loads
    int64_t raw_t0 = 0;
    auto fetch = [&](int64_t c) {
      raw_t0 = c * kC + part * kPartT;
#pragma unroll
      for (int j = 0; j < kPartT; ++j)
        raw[j] = *reinterpret_cast<const unsigned short*>(p.d_out + (start + (raw_t0 + j < len ? raw_t0 + j : len - 1)) * p.d_out_ts + h * kV + v);
    };
    float sc_do = 1.f;
    auto put = [&]() {
      float y[kPartT], m = 0.f;
#pragma unroll
      for (int j = 0; j < kPartT; ++j) {
        y[j] = raw_t0 + j < len ? __uint_as_float(static_cast<uint32_t>(raw[j]) << 16) : 0.f;
        m = fmaxf(m, fabsf(y[j]));
      }
      sc_do = pow2_scale(quarter_max(sm, 2, m, part, quarter));
      uint32_t x[kPartT / 2];
#pragma unroll
      for (int j = 0; j < kPartT / 2; ++j)
        x[j] = as_u32(__floats2half2_rn(y[2 * j] * sc_do, y[2 * j + 1] * sc_do));
      fence_after_sync();
      tmem_st(mine + Col::kDO + part * (kPartT / 2), x);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sm.d_out, lane);
    };
    if (chunks > 0) {
      fetch(chunks - 1);
      put();
    }
    for (int64_t i = 0; i < chunks; ++i, rec -= step) {
      const int b = static_cast<int>(i & 1);
      const float* const hdr = reinterpret_cast<const float*>(sm.hdr[b]);
      // ---- dS1 as a pair
      const float sc_s = pow2_scale(quarter_max(sm, 0, abs_max(s), part, quarter));
      fence_after_sync();
      write_pair<kK, true>(mine + Col::kState, nullptr, 0, v, part * kPartK, s, sc_s);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sm.state, lane);
      if (!p.transitions) write_pair<kK, false>(0, rec + Record::kDS, kV * kK * 2, v, part * kPartK, s, sc_s);
      if (i + 1 < chunks) fetch(chunks - 2 - i);
      // ---- decay, and scale Qt^T dO
      w.warp(&sm.full_hdr[b], i >> 1);
      w.warp(&sm.with_qt, i);
      fence_after_sync();
      const float f_do = pow2_inv(sc_do) * p.scale;
      add_product<true>(mine + Col::kExtra + part * kPartK, hdr + Record::kDecay + part * kPartK, f_do * pow2_inv(hdr[Record::kScQt]), s);
      // ---- dU = scale P^T dO + Ke dS1
      w.warp(&sm.first[b], i >> 1);
      fence_after_sync();
      float du[kPartT];
      {
        const float f1 = f_do * pow2_inv(hdr[Record::kScP]), f2 = pow2_inv(sc_s) * pow2_inv(hdr[Record::kScKe]);
        uint32_t x[kPartT], y[kPartT];
        tmem_ld(mine + Col::kX1 + part * kPartT, x);
        tmem_ld(mine + Col::kX2 + part * kPartT, y);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kPartT; ++j) du[j] = fmaf(__uint_as_float(x[j]), f1, __uint_as_float(y[j]) * f2);
      }
      const float* const beta = hdr + Record::kBeta + part * kPartT;
      const float f_wr = -pow2_inv(hdr[Record::kScWr]);
      const float sc_u = pow2_scale(quarter_max(sm, 1, abs_max(du, beta), part, quarter));
      fence_after_sync();
      write_pair<kC, true>(mine + Col::kU, nullptr, 0, v, part * kPartT, du, sc_u, beta);
      warp_arrive(&sm.empty_hdr[b], lane);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sm.rows, lane);
      if (i + 1 < chunks) put();  // the products of this chunk's dO are complete
      if (!p.transitions) {
        const float sc_du = pow2_scale(quarter_max(sm, 3, abs_max(du), part, quarter));
        write_pair<kC, false>(0, rec + Record::kDU, Record::kPlane, v, part * kPartT, du, sc_du);
        if (part == 0 && lane == 0) {
          float* const sc = reinterpret_cast<float*>(rec + Record::kSc);
          sc[Record::kScDS + quarter] = sc_s;
          sc[Record::kScDU + quarter] = sc_du;
        }
      }
      // ---- dS0 = ... - Wr^T (beta dU)
      w.warp(&sm.last[b], i >> 1);
      fence_after_sync();
      add_product<false>(mine + Col::kDelta + part * kPartK, nullptr, pow2_inv(sc_u) * f_wr, s);
      fence_before_sync();
    }
    if (!w.ok) {
      if (lane == 0) set_error(p);
    } else if (p.transitions) {
      store_state(p.seg_state + gblk, v, part, s);
    } else if (seg.seg == 0 && p.d_init != nullptr) {
      store_state(p.d_init + sblk, v, part, s);
    }
  } else if (warp == kComputeWarps) {
    if (lane == 0) chain_copies<false>(sm, w, rec, -step, chunks, true);
    __syncwarp();
  } else {
    auto d_out_products = [&](int64_t i) {
      w.warp(&sm.full_qt, i);
      w.warp(&sm.d_out, i);
      fence_after_sync();
      umma_pairs<kK, kC, kC, true, true>(tmem + Col::kExtra, tmem + Col::kDO, smem_addr(sm.qt), Record::kPlane);
      umma_commit(&sm.with_qt);
      w.warp(&sm.full_p, i);
      umma_pairs<kC, kC, kC, true, true>(tmem + Col::kX1, tmem + Col::kDO, smem_addr(sm.p), kC * kC * 2);
    };
    if (chunks > 0) d_out_products(0);
    for (int64_t i = 0; i < chunks; ++i) {
      const int b = static_cast<int>(i & 1);
      w.warp(&sm.full_ke[b], i >> 1);
      w.warp(&sm.state, i);
      fence_after_sync();
      umma_pairs<kC, kK, kC, false>(tmem + Col::kX2, tmem + Col::kState, smem_addr(sm.ke[b]), Record::kPlane);
      umma_commit(&sm.first[b]);
      w.warp(&sm.full_wr[b], i >> 1);
      w.warp(&sm.rows, i);
      fence_after_sync();
      umma_pairs<kK, kC, kC, true>(tmem + Col::kDelta, tmem + Col::kU, smem_addr(sm.wr[b]), Record::kPlane);
      umma_commit(&sm.last[b]);
      if (i + 1 < chunks) d_out_products(i + 1);
    }
    if (chunks > 0) {
      umma_commit(&sm.end);
      mbar_wait(&sm.end, 0);
    }
    __syncwarp();
    if (!w.ok && lane == 0) set_error(p);
  }
  chain_exit(sm);
}

}  // namespace kdal
