// kda_scan_common.cuh -- parameters, workspace records and the decay factors
// shared by the scan's kernels (see kda_scan_prep.cuh for the mathematics).
#pragma once

#include "kda_tiles.cuh"

namespace kdal {

struct ScanParams {
  const __nv_bfloat16* q; int64_t q_ts;  // [tokens, HV, K], rows q_ts elements apart; likewise below
  const __nv_bfloat16* k; int64_t k_ts;
  const __nv_bfloat16* v; int64_t v_ts;
  const float* g; int64_t g_ts;
  const float* beta; int64_t beta_ts;
  const int32_t* cu;        // [N + 1] packed sequences, or null: N sequences of T tokens
  const float* s_in;        // [N or slots, HV, K, V] or null (zeros)
  float* s_out;             // likewise, or null
  const int32_t* slot_idx;  // [N] or null (sequence n uses block n)
  int64_t num_slots;        // blocks of s_in and s_out when slot_idx is set
  __nv_bfloat16* out; int64_t out_ts;
  unsigned char* ws;
  int64_t rec_bytes;        // bytes of one record
  int64_t tokens, T, HV;
  int32_t N, seq_chunks;    // seq_chunks: ceil(T / C) of the dense form
  float scale;
  int32_t save;             // the forward call keeps what the backward pass reads
  // Segments of a sequence's chunks, walked side by side (see kda_scan_chain.cuh); seg_chunks 0: none.
  int32_t seg_chunks, seq_segs;  // chunks of a segment; segments of a sequence of the dense form
  int32_t transitions;      // the chain call computes the segments' transitions instead of the results
  float* seg_state;         // [segment slots, HV, K, V] states at the segments' ends (or starts, backwards)
  float* seg_map;           // [segment slots, HV, K, K] transition matrices; a first segment's: the state it starts from
  // backward
  const __nv_bfloat16* d_out; int64_t d_out_ts;
  const float* d_final;     // [N, HV, K, V] or null
  __nv_bfloat16* dq; int64_t dq_ts;
  __nv_bfloat16* dk; int64_t dk_ts;
  __nv_bfloat16* dv; int64_t dv_ts;
  float* dg; int64_t dg_ts;
  float* dbeta; int64_t dbeta_ts;
  float* d_init;            // [N, HV, K, V] or null
};

// One record per (chunk slot, head); the chunk slots of sequence n start at
// cu[n] / C + n (n seq_chunks in the dense form), which leaves room for every
// sequence's ceil(length / C) chunks without a scan over the lengths.
struct Record {
  // header: floats
  static constexpr int kDecay = 0;     // [128] exp(Gamma_C)
  static constexpr int kBeta = 128;    // [64]
  static constexpr int kScWr = 192, kScKe = 193, kScQt = 194, kScP = 195, kScY = 196;
  static constexpr int kMxWr = 200, kMxRt = 201;  // the tiles' largest magnitudes
  // byte offsets
  static constexpr int kHdr = 1024;
  static constexpr int kPlane = kC * kK * 2;       // 16 KB: a plane of 64 x 128 elements
  // pairs hi, lo of Core tiles; [rows][columns]
  static constexpr int kP = kHdr;                  // P   [t][s], 8 KB a plane
  static constexpr int kQt = kP + kC * kC * 4;     // Qt  [t][i]
  static constexpr int kWr = kQt + 2 * kPlane;     // Wr  [t][i]
  static constexpr int kKe = kWr + 2 * kPlane;     // Ke  [t][i]
  static constexpr int kRt = kKe + 2 * kPlane;     // Rt^T fp32, [t / 4][v][4]
  static constexpr int64_t kForward = kRt + kV * kC * 4;
  static constexpr int kY = static_cast<int>(kForward);  // beta_t Y [t][s]
  static constexpr int kDn = kY + kC * kC * 4;     // fp32 [4][128]: from k dn to Ke, per sub-block and channel
  static constexpr int kDnBytes = kNB * kK * 4;
  static constexpr int kS = kDn + kDnBytes;        // S0^T [v][i], 32 KB a plane
  static constexpr int kR = kS + kV * kK * 4;      // r^T  [v][t]
  static constexpr int kDS = kR + 2 * kPlane;      // dS1^T [v][i]
  static constexpr int kDU = kDS + kV * kK * 4;    // dU^T [v][t]
  // Scales of the last four; dS1's and dU's one per 32 value columns.
  static constexpr int kSc = kDU + 2 * kPlane;
  static constexpr int kScS = 0, kScR = 1, kScDS = 4, kScDU = 8, kScBytes = 48;
  static constexpr int64_t kTraining = kSc + kScBytes;
};
constexpr int64_t kWsHeader = 256;  // word 0: the error word

__device__ __forceinline__ void set_error(const ScanParams& p) { *reinterpret_cast<volatile int32_t*>(p.ws) = 1; }

__device__ __forceinline__ unsigned char* record(const ScanParams& p, int64_t slot, int64_t h) {
  return p.ws + kWsHeader + (slot * p.HV + h) * p.rec_bytes;
}

// Sequence n's first token and length; offsets are clamped to the tokens
// there are, so that no offset makes an access out of range.
__device__ __forceinline__ void seq_range(const ScanParams& p, int64_t n, int64_t& start, int64_t& len) {
  if (p.cu == nullptr) {
    start = n * p.T;
    len = p.T;
    return;
  }
  int64_t a = __ldg(p.cu + n), b = __ldg(p.cu + n + 1);
  a = a < 0 ? 0 : (a > p.tokens ? p.tokens : a);
  b = b < a ? a : (b > p.tokens ? p.tokens : b);
  start = a;
  len = b - a;
}
__device__ __forceinline__ int64_t first_slot(const ScanParams& p, int64_t n, int64_t start) {
  return p.cu == nullptr ? n * p.seq_chunks : start / kC + n;
}
// The state block of sequence n, or -1 for an inactive one.
__device__ __forceinline__ int64_t state_block(const ScanParams& p, int64_t n) {
  if (p.slot_idx == nullptr) return n;
  const int64_t s = __ldg(p.slot_idx + n);
  return s >= 0 && s < p.num_slots ? s : -1;
}

struct ChunkPos {
  int64_t n, tok;  // sequence, first token of the chunk
  int32_t tc;      // tokens of the chunk; 0: no such chunk
};
// Block index to (slot, head).  32 bits: the launches keep their grids below 2^31, and a 64-bit division takes a
// thousand cycles of every block's life.
__device__ __forceinline__ void slot_and_head(const ScanParams& p, uint32_t block, int64_t& slot, int64_t& h) {
  const uint32_t q = block / static_cast<uint32_t>(p.HV);
  slot = q;
  h = block - q * static_cast<uint32_t>(p.HV);
}
// The last packed sequence with first(n, its first token) <= slot, and its range, or -1; `first` grows with n (decreasing
// offsets end the search somewhere in range).  The lanes of each warp probe 32 sequences at a time: one step to 32
// sequences, two to 1024 (4096 sequences of 64 tokens, one head, us a call: 810, and 2350 looking at all of them).
template <typename F>
__device__ __forceinline__ int64_t find_sequence(const ScanParams& p, int64_t slot, int64_t& start, int64_t& len, F first) {
  uint32_t lo = 0, hi = static_cast<uint32_t>(p.N);
  for (;;) {
    const uint32_t step = (hi - lo + 31) >> 5, n = lo + (threadIdx.x & 31) * step;
    int64_t a = 0, l = 0;
    if (n < hi) seq_range(p, n, a, l);
    const uint32_t found = __ballot_sync(0xffffffffu, n < hi && first(n, a) <= slot);
    if (!found) return -1;
    const int at = 31 - __clz(static_cast<int>(found));
    lo += at * step;
    if (step == 1) {  // a packed call's offsets have 32 bits
      start = __shfl_sync(0xffffffffu, static_cast<int32_t>(a), at);
      len = __shfl_sync(0xffffffffu, static_cast<int32_t>(l), at);
      return lo;
    }
    hi = hi < lo + step ? hi : lo + step;
  }
}
// The chunk of a chunk slot (whole warps call it).
__device__ __forceinline__ ChunkPos locate(const ScanParams& p, int64_t slot) {
  ChunkPos c{0, 0, 0};
  int64_t start, len;
  if (p.cu == nullptr) {
    c.n = slot / p.seq_chunks;
    seq_range(p, c.n, start, len);
  } else {
    c.n = find_sequence(p, slot, start, len, [&](int64_t n, int64_t a) { return first_slot(p, n, a); });
    if (c.n < 0) return c;
  }
  const int64_t t = (slot - first_slot(p, c.n, start)) * kC;
  if (t >= len) return c;
  c.tok = start + t;
  if (state_block(p, c.n) >= 0) c.tc = static_cast<int32_t>(len - t < kC ? len - t : kC);
  return c;
}

// Whether a call whose longest sequence has that many chunks walks its sequences in segments of `len`: two walks of a
// segment (the one for the segments' ends has no outputs, 3.7 us a chunk for 4.7) and joining have to be less than one
// walk of the longest.  Measured, one sequence, us a call whole and in segments, where it is x times a segment: 8192
// tokens x = 2.3 991, 898; 1.8 1108, 1097; 1.5 1219, 1314; 2048 tokens x = 2.3 264, 259; 1.8 299, 308 (782, 764 with
// gradients); 1.5 331, 364.
__host__ __device__ __forceinline__ bool worth_segments(int64_t chunks, int64_t len) { return 4 * chunks >= 7 * len; }

// A CTA's part of a sequence: `chunks` chunks from `first` on, segment `seg` of `segs`.  The segment slots of sequence n
// start at cu[n] / (C seg_chunks) + n, like the chunk slots.
struct Segment {
  int64_t n, start, len;    // the sequence
  int64_t first, chunks;
  int64_t seg, segs;        // segs 0: no such segment
};
// A packed call's sequence of a segment slot, the last one whose first segment slot is not behind it (or -1), its range, and
// whether the call's sequences are cut at all.  A call with segments has at most kMostCut sequences: the lanes of a warp
// load them all at once (whole warps call it; not inlined, it takes registers from the chains).
constexpr int32_t kMostCut = (kSms - 1) / 2;
struct PackedSegment {
  int32_t n, start, len, cut;
};
__device__ __noinline__ PackedSegment find_segment(const int32_t* cu, int32_t N, int64_t tokens, int32_t seg_chunks, int64_t slot) {
  constexpr int32_t kEach = kMostCut / 32 + 1;
  const int32_t rows = static_cast<int32_t>(tokens), lane = threadIdx.x & 31;
  int32_t a[kEach], l[kEach], longest = 0;
#pragma unroll
  for (int32_t j = 0; j < kEach; ++j) {
    a[j] = l[j] = 0;
    if (lane + 32 * j < N) a[j] = __ldg(cu + lane + 32 * j), l[j] = __ldg(cu + lane + 32 * j + 1);
  }
  const int64_t rows_of_segment = static_cast<int64_t>(kC) * seg_chunks;
  PackedSegment s{-1, 0, 0, 0};
#pragma unroll
  for (int32_t j = 0; j < kEach; ++j) {
    if (32 * j >= N) break;
    a[j] = a[j] < 0 ? 0 : (a[j] > rows ? rows : a[j]);  // as in seq_range
    l[j] = (l[j] > rows ? rows : (l[j] < a[j] ? a[j] : l[j])) - a[j];
    longest = l[j] > longest ? l[j] : longest;
    const uint32_t found = __ballot_sync(0xffffffffu, lane + 32 * j < N && a[j] < (slot - (lane + 32 * j) + 1) * rows_of_segment);
    if (found) {
      const int at = 31 - __clz(static_cast<int>(found));
      s.n = 32 * j + at;
      s.start = __shfl_sync(0xffffffffu, a[j], at);
      s.len = __shfl_sync(0xffffffffu, l[j], at);
    }
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  s.cut = worth_segments((static_cast<int64_t>(longest) + kC - 1) / kC, seg_chunks);
  return s;
}
__device__ __forceinline__ int64_t first_segment(const ScanParams& p, int64_t n, int64_t start) {
  return p.cu == nullptr ? n * p.seq_segs : start / (static_cast<int64_t>(kC) * p.seg_chunks) + n;
}
__device__ __forceinline__ int64_t segments_of(const ScanParams& p, int64_t chunks, bool cut) {
  return cut && chunks > 0 ? (chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
}
// The segment of a slot (whole warps call it).
__device__ __forceinline__ Segment locate_segment(const ScanParams& p, int64_t slot) {
  Segment s;
  s.seg = 0, s.segs = 1, s.first = 0;
  if (p.seg_chunks == 0) {
    s.n = slot;
    seq_range(p, s.n, s.start, s.len);
    s.chunks = (s.len + kC - 1) / kC;
    return s;
  }
  bool cut = true;
  if (p.cu == nullptr) {
    s.n = slot / p.seq_segs;
    seq_range(p, s.n, s.start, s.len);
  } else {
    const PackedSegment f = find_segment(p.cu, p.N, p.tokens, p.seg_chunks, slot);
    if (f.n < 0) return Segment{};
    s.n = f.n, s.start = f.start, s.len = f.len;
    cut = f.cut;
  }
  const int64_t chunks = (s.len + kC - 1) / kC;
  s.segs = segments_of(p, chunks, cut);
  s.seg = slot - first_segment(p, s.n, s.start);
  s.first = s.seg * p.seg_chunks;
  s.chunks = s.seg < s.segs - 1 ? p.seg_chunks : chunks - s.first;
  if (s.seg >= s.segs) s.segs = 0;
  return s;
}

// ---------------------------------------------------------------- decays
// A log-decay sum as an unevaluated pair of floats: the low part takes what
// rounding the high part dropped.  A plain fp32 sum over a chunk's tokens is
// off by 1e-6 and more, and so would be the decays (fp64 is exact enough but
// measured 3 us more per chunk here, mostly in its conversions).
struct Sum {
  float hi, lo;
};
__device__ __forceinline__ Sum add(Sum a, float b) {
  const float s = a.hi + b, v = s - a.hi;
  return Sum{s, a.lo + ((a.hi - (s - v)) + (b - v))};
}
__device__ __forceinline__ Sum add(Sum a, Sum b) {
  Sum r = add(a, b.hi);
  r.lo += b.lo;
  return r;
}
__device__ __forceinline__ Sum neg(Sum a) { return Sum{-a.hi, -a.lo}; }
// exp of a pair: the low part enters to first order.
__device__ __forceinline__ float exp_of(Sum x) {
  const float e = expf(x.hi);
  return fmaf(e, x.lo, e);
}
// A log-decay; below -1e4 the decay is zero either way (and -inf would make NaN of differences).
__device__ __forceinline__ float log_decay(float g) { return g < -1e4f ? -1e4f : g; }

// Largest |L - mid| a sub-block may have for its factors exp(+-(L - mid)): they
// and the products of two stay normal fp32 numbers.
constexpr float kSafe = 60.f;

// The decay factors of one sub-block and key channel.  L_t is the cumulative
// log-decay from the sub-block's start.  up[t] = exp(L_t - mu), dn[t] = exp(md
// - L_t).  Within range mu = md = mid, the middle of the L_t, so that
// up[t] dn[s] = exp(L_t - L_s) for every pair; otherwise mu = 0 and md = L_end
// (each factor at most 1 for g <= 0) and pairs inside the sub-block are formed
// one by one from the differences (`exact`).
struct SubFactors {
  Sum mu, md, end;
  bool exact;
};
__device__ __forceinline__ SubFactors sub_factors(const float (&g)[kB], float (&up)[kB], float (&dn)[kB]) {
  SubFactors f;
  Sum L[kB];
  Sum acc{0.f, 0.f};
  float lo = 3e38f, hi = -3e38f;
#pragma unroll
  for (int t = 0; t < kB; ++t) {
    acc = add(acc, g[t]);
    L[t] = acc;
    lo = fminf(lo, acc.hi);
    hi = fmaxf(hi, acc.hi);
  }
  f.end = acc;
  f.exact = !(hi - lo <= 2.f * kSafe);
  const float mid = 0.5f * (hi + lo);
  f.mu = Sum{f.exact ? 0.f : mid, 0.f};
  f.md = f.exact ? acc : f.mu;
#pragma unroll
  for (int t = 0; t < kB; ++t) {
    const Sum x = add(L[t], -f.mu.hi);
    up[t] = exp_of(x);
    dn[t] = exp_of(f.exact ? add(f.md, neg(L[t])) : neg(x));
  }
  return f;
}

// A chunk's log-decays, keys and queries as they lie in memory, in shared memory.
struct RawRows {
  float g[kC][kK];
  __nv_bfloat16 k[kC][kK], q[kC][kK];
};
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Starts the copies of the chunk's rows (rows behind its end: its last one's).  Loaded by the threads that use them, 48
// values of 2 and 4 bytes each, they took 13000 cycles (an SM has only so many requests in flight), against 2500 here.
template <int THREADS>
__device__ __forceinline__ void fetch_rows(const ScanParams& p, int64_t tok, int tc, int64_t h, float (*g)[kK], __nv_bfloat16 (*k)[kK],
                                           __nv_bfloat16 (*q)[kK]) {
  const int tid = threadIdx.x;
  for (int e = tid; e < kC * kK / 8; e += THREADS) {
    const int t = e >> 4, i = (e & 15) * 8;
    const int64_t row = tok + (t < tc ? t : tc - 1);
    cp_async16(&k[t][i], p.k + row * p.k_ts + h * kK + i);
    cp_async16(&q[t][i], p.q + row * p.q_ts + h * kK + i);
  }
  if (((reinterpret_cast<uintptr_t>(p.g) & 15) | (p.g_ts & 3)) == 0) {
    for (int e = tid; e < kC * kK / 4; e += THREADS) {
      const int t = e >> 5, i = (e & 31) * 4;
      cp_async16(&g[t][i], p.g + (tok + (t < tc ? t : tc - 1)) * p.g_ts + h * kK + i);
    }
  } else {  // g may lie on any 4 bytes
    for (int e = tid; e < kC * kK; e += THREADS) {
      const int t = e >> 7, i = e & (kK - 1);
      cp_async4(&g[t][i], p.g + (tok + (t < tc ? t : tc - 1)) * p.g_ts + h * kK + i);
    }
  }
}
// Sub-block b's 16 tokens in channel ch, zeros behind the chunk.
__device__ __forceinline__ void read_sub_block(const float (*gs)[kK], const __nv_bfloat16 (*ks)[kK], const __nv_bfloat16 (*qs)[kK], int tc,
                                               int b, int ch, float (&g)[kB], float (&k)[kB], float (&q)[kB]) {
#pragma unroll
  for (int t = 0; t < kB; ++t) {
    const bool in = b * kB + t < tc;
    g[t] = in ? log_decay(gs[b * kB + t][ch]) : 0.f;
    k[t] = in ? __bfloat162float(ks[b * kB + t][ch]) : 0.f;
    q[t] = in ? __bfloat162float(qs[b * kB + t][ch]) : 0.f;
  }
}

// Split of an fp32 value into a tf32 pair, both rounded to nearest (the MMA
// reads the upper 19 bits of each and would truncate the low part: a bias of
// 2^-23, which the sums of differences behind the decays' gradients show).
__device__ __forceinline__ void tf32_pair(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}

}  // namespace kdal
