// kda_scan_prep.cuh -- the scan's first kernel: everything about a chunk that
// does not depend on the state.
//
// The recurrence, per sequence and head, on the state S [K, V]:
//   S' = Diag(exp(g_t)) S;  r_t = v_t - S'^T k_t;  S = S' + beta_t k_t r_t^T;
//   o_t = scale S^T q_t.
// Over a chunk of C = 64 tokens with the cumulative log-decay Gamma_t from the
// chunk's start and the state S0 there:
//   A_ts = sum_i k_t,i k_s,i exp(Gamma_t,i - Gamma_s,i)  (s < t)
//   P_ts = sum_i q_t,i k_s,i exp(Gamma_t,i - Gamma_s,i)  (s <= t)
//   Kt = k exp(Gamma_t), Qt = q exp(Gamma_t), Ke = k exp(Gamma_C - Gamma_t)
//   r = (I + A diag(beta))^-1 (V - Kt S0) = Rt - Wr S0,
//   O = scale (Qt S0 + P (beta r)),  S1 = Diag(exp(Gamma_C)) S0 + Ke^T (beta r).
// With Y = A (I + diag(beta) A)^-1 (strictly lower triangular) the inverse is
// M = I - Y diag(beta), and its mirror (I + diag(beta) A)^-1 = I - diag(beta) Y
// serves the backward pass: one triangular solve for both, and beta = 0 needs
// no division.  This kernel computes Wr = M Kt, Rt = M V, Ke, Qt, P (and Y).
//
// Decays.  Every factor is kept at most 1 (for g <= 0) by a reference token
// between t and s: pairs across the chunk's middle take their decays to it,
// pairs of neighbouring sub-blocks (16 tokens) inside a half those to the
// border between them, as fp16 pairs.  Inside a sub-block the reference is the
// middle of its cumulative log-decays (see SubFactors), and the products run in
// tf32 pairs, whose range takes the e^+-60 of those factors.
//
// What bounds it: the latency of its phases, each of which leaves half of the
// issue slots empty (the factors 4000 cycles of a chunk's 31000, the products
// inside and across sub-blocks 6000, the tiles' splits 4500, the solve 5700, Rt
// and Wr 5000); 512 threads, one sub-block and channel each (256 left the
// schedulers short of warps), one CTA an SM by its shared memory and registers.
// A block goes on with another chunk, whose rows arrive under the solve (see
// request_block).  Measured (B200): 2112 chunks and heads 274 us, one block a
// chunk 291; a plain copy would move its bytes in 70.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kPrepThreads = 512, kPrepWarps = kPrepThreads / 32;
constexpr int kFP = kK + 4;  // padded rows of the fp32 factors: MMA fragments then touch 32 banks
constexpr int kAP = kC + 4;
constexpr int kHalfPlane = Record::kPlane / 2;  // 32 rows of 128 columns

struct PrepFactors {
  float ku[kC][kFP];  // k up
  float qu[kC][kFP];  // q up
  float kd[kC][kFP];  // k dn
};
struct PrepTiles {    // over the factors once those are in registers; pairs (hi, lo)
  unsigned char kt[2 * Record::kPlane];       // Kt
  unsigned char r32[2][2 * kHalfPlane];       // k, q of tokens 32.. with the decay from token 32's start
  unsigned char c32[2 * kHalfPlane];          // k of tokens ..31 with the decay to there
  unsigned char r16[2][2 * kHalfPlane];       // k, q of sub-blocks 1 and 3 with the decay from their starts
  unsigned char c16[2 * kHalfPlane];          // k of sub-blocks 0 and 2 with the decay to their ends
};
enum PrepMax { kMxV, kMxKt, kMxQt, kMxKe, kMxR32K, kMxR32Q, kMxC32, kMxR16K, kMxR16Q, kMxC16, kMxP, kMxY, kMxWr, kMxRt, kMxBeta, kMxCount };

struct PrepNext {     // the next chunk's rows, over all tiles but Kt once those are read
  unsigned char kt[2 * Record::kPlane];
  RawRows raw;
  uint4 v[kC * kV / 8];
};

struct PrepSmem {
  union {
    PrepFactors f;
    PrepTiles t;
    PrepNext next;
  };
  unsigned char vt[Record::kPlane];     // V tile [t][v]
  float a[kC][kAP];                     // A
  float pm[kC][kAP];                    // P; then the tile M
  float y[kC][kAP];                     // Y
  Sum end[kNB][kK];                     // log-decay of a sub-block
  float up[kNB][kK], dn[kNB][kK];       // to Kt and Qt, to Ke
  float x32[kNB][kK], x16[kNB][kK];     // to the tiles r32 or c32, r16 or c16
  float beta[kC];
  uint32_t mx[kMxCount];                // block maxima (float bits)
  int exact[kNB];
  uint4 taken;                          // the block taken over next
  uint64_t taken_full;
};
static_assert(2 * kC * kC * 2 <= sizeof(float) * kC * kAP, "the M tile fits into pm");
static_assert(sizeof(PrepNext) <= sizeof(PrepTiles), "the raw rows fit over the tiles");
static_assert(sizeof(PrepSmem) <= 232448, "shared memory of an SM");

__device__ __forceinline__ void block_max(uint32_t* slot, float m, int lane) {
  m = warp_max(m);
  if (lane == 0) atomicMax(slot, __float_as_uint(m));
}

// Pairs inside sub-block `b` from the differences themselves: warp w takes row
// w, its lanes four channels each, s running down from t with the
// log-decay between s and t summed on the way.
__device__ __noinline__ void prep_exact_block(const ScanParams& p, PrepSmem& sm, int b, int64_t tok, int tc, int64_t h) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < kB; r += kPrepWarps) {
    const int t = b * kB + r;
    if (t >= tc) continue;
    float kt[4], qt[4], d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = lane + 32 * j;
      kt[j] = __bfloat162float(p.k[(tok + t) * p.k_ts + h * kK + i]);
      qt[j] = __bfloat162float(p.q[(tok + t) * p.q_ts + h * kK + i]);
    }
    for (int s = t; s >= b * kB; --s) {
      float a = 0.f, pv = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = lane + 32 * j;
        const float ke = __bfloat162float(p.k[(tok + s) * p.k_ts + h * kK + i]) * expf(d[j]);
        a = fmaf(kt[j], ke, a);
        pv = fmaf(qt[j], ke, pv);
        d[j] += log_decay(p.g[(tok + s) * p.g_ts + h * kK + i]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        pv += __shfl_xor_sync(0xffffffffu, pv, o);
      }
      if (lane == 0) {
        if (s < t) sm.a[t][s] = a;
        sm.pm[t][s] = pv;
      }
    }
  }
}

// A tile of an fp32 matrix as the A or B operand of the tf32 product, elements f(row, k) and f(k, column).
template <typename F>
__device__ __forceinline__ void tf32_a(F f, int lane, uint32_t (&h)[4], uint32_t (&l)[4]) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) tf32_pair(f(r + (j & 1) * 8, c + (j >> 1) * 4), h[j], l[j]);
}
template <typename F>
__device__ __forceinline__ void tf32_b(F f, int lane, uint32_t (&h)[2], uint32_t (&l)[2]) {
  const int r = lane >> 2, c = lane & 3;
  tf32_pair(f(c, r), h[0], l[0]);
  tf32_pair(f(c + 4, r), h[1], l[1]);
}

// Y's block of ROWS rows from r0 under its diagonal blocks, columns c0 .. c0 + 7 of the ROWS columns from r0 - ROWS:
//   Y21 = (I - Y2 diag(beta2)) A21 (I - diag(beta1) Y1).
// One warp; it reads and writes these columns alone (and finished diagonal blocks).
// Returns the largest magnitude this thread wrote.
template <int ROWS>
__device__ __forceinline__ float solve_below(PrepSmem& sm, int r0, int c0, int lane) {
  constexpr int kM = ROWS / 16;
  const int k0 = r0 - ROWS, r = lane >> 2, c = lane & 3, first = (c0 - k0) / 8;
  float x[kM][4], largest = 0.f;
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    float lo[4] = {}, hi[4] = {};
    for (int kk = first; kk < ROWS / 8; ++kk) {  // Y1[k][n] is zero for k <= n
      uint32_t ah[4], al[4], bh[2], bl[2];
      tf32_a([&](int i, int k) { return sm.a[r0 + m * 16 + i][k0 + kk * 8 + k]; }, lane, ah, al);
      tf32_b([&](int k, int n) { return sm.beta[k0 + kk * 8 + k] * sm.y[k0 + kk * 8 + k][c0 + n]; }, lane, bh, bl);
      mma_tf32(lo, ah, bl);
      mma_tf32(lo, al, bh);
      mma_tf32(hi, ah, bh);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = r0 + m * 16 + r + (e >> 1) * 8, col = c0 + 2 * c + (e & 1);
      x[m][e] = sm.a[row][col] - (hi[e] + lo[e]);
      sm.y[row][col] = x[m][e];
    }
  }
  __syncwarp();
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    float lo[4] = {}, hi[4] = {};
#pragma unroll
    for (int kk = 0; kk < 2 * (m + 1); ++kk) {  // Y2[t][k] is zero for k >= t
      uint32_t ah[4], al[4], bh[2], bl[2];
      tf32_a([&](int i, int k) { return sm.y[r0 + m * 16 + i][r0 + kk * 8 + k]; }, lane, ah, al);
      tf32_b([&](int k, int n) { return sm.beta[r0 + kk * 8 + k] * sm.y[r0 + kk * 8 + k][c0 + n]; }, lane, bh, bl);
      mma_tf32(lo, ah, bl);
      mma_tf32(lo, al, bh);
      mma_tf32(hi, ah, bh);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[m][e] -= hi[e] + lo[e];
  }
  __syncwarp();
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sm.y[r0 + m * 16 + r + (e >> 1) * 8][c0 + 2 * c + (e & 1)] = x[m][e];
      largest = fmaxf(largest, fabsf(x[m][e]));
    }
  return largest;
}

// Elements s0 .. s0 + 7 of row t of a lower triangular matrix stored by blocks of 16 (nothing above the diagonal blocks).
__device__ __forceinline__ void read_row(const float (&m)[kC][kAP], int t, int s0, float (&x)[8]) {
  const bool in = (s0 >> 4) <= (t >> 4);
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const float4 v = *reinterpret_cast<const float4*>(&m[t][s0 + e]);
    x[e] = in ? v.x : 0.f;
    x[e + 1] = in ? v.y : 0.f;
    x[e + 2] = in ? v.z : 0.f;
    x[e + 3] = in ? v.w : 0.f;
  }
}

// 16 x 16 of a product over the 128 channels of two pair tiles [row][i].
__device__ __forceinline__ void pair_product(uint32_t row_tile, int m0, uint32_t col_tile, int n0, int lane, float (&out)[2][4]) {
  float hi[2][2][4] = {}, lo[2][4] = {};
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t ah[4], al[4], bh[4], bl[4];
    load_a<Core<32>>(row_tile, m0, kk * 16, lane, ah);
    load_a<Core<32>>(row_tile + kHalfPlane, m0, kk * 16, lane, al);
    load_b<Core<32>>(col_tile, kk * 16, n0, lane, bh);
    load_b<Core<32>>(col_tile + kHalfPlane, kk * 16, n0, lane, bl);
    mma_pair(lo[0], lo[1], ah, bl);
    mma_pair(lo[0], lo[1], al, bh);
    mma_pair(hi[kk & 1][0], hi[kk & 1][1], ah, bh);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[n][e] = (hi[0][n][e] + hi[1][n][e]) + lo[n][e];
}

__global__ void __launch_bounds__(kPrepThreads, 1) kda_scan_prep_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PrepSmem& sm = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t slot, h;
  slot_and_head(p, blockIdx.x, slot, h);
  if (tid == 0) {
    mbar_init(&sm.taken_full, 1);
    mbar_fence_init();
  }
  wait_upstream();
  ChunkPos pos = locate(p, slot);
  if (pos.tc == 0) return;
  auto fetch = [&]() {
    fetch_rows<kPrepThreads>(p, pos.tok, pos.tc, h, sm.next.raw.g, sm.next.raw.k, sm.next.raw.q);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = tid + j * kPrepThreads, t = c >> 4;
      cp_async16(&sm.next.v[c], p.v + (pos.tok + (t < pos.tc ? t : pos.tc - 1)) * p.v_ts + h * kV + (c & 15) * 8);
    }
  };
  auto scale_of = [&](PrepMax i) { return pow2_scale(__uint_as_float(sm.mx[i])); };
  fetch();
  for (uint32_t phase = 0;; phase ^= 1) {
    const int tc = pos.tc;
    unsigned char* const rec = record(p, slot, h);
    float* const hdr = reinterpret_cast<float*>(rec);
    float be = 0.f;
    if (warp < 2 && tid < tc) be = __ldg(p.beta + (pos.tok + tid) * p.beta_ts + h);
    cp_async_wait_all();
    __syncthreads();
    if (tid == 0) request_block(&sm.taken, &sm.taken_full);
    if (tid < kMxCount) sm.mx[tid] = 0;
    if (tid < kNB) sm.exact[tid] = 0;
    // ---- 1. decay factors: thread = channel and sub-block
    const int ch = tid & (kK - 1), b = tid >> 7;
    SubFactors sf;
    uint4 vraw[2];  // v: kept in registers until the scale is known
    float m_ku = 0.f, m_qu = 0.f, m_kd = 0.f;
    {
      float g[kB], kv[kB], qv[kB], up[kB], dn[kB];
      read_sub_block(sm.next.raw.g, sm.next.raw.k, sm.next.raw.q, tc, b, ch, g, kv, qv);
#pragma unroll
      for (int j = 0; j < 2; ++j) vraw[j] = sm.next.v[tid + j * kPrepThreads];
      __syncthreads();  // the factors go over the rows
      sf = sub_factors(g, up, dn);
#pragma unroll
      for (int t = 0; t < kB; ++t) {
        const float ku = kv[t] * up[t], qu = qv[t] * up[t], kd = kv[t] * dn[t];
        sm.f.ku[b * kB + t][ch] = ku;
        sm.f.qu[b * kB + t][ch] = qu;
        sm.f.kd[b * kB + t][ch] = kd;
        m_ku = fmaxf(m_ku, fabsf(ku));
        m_qu = fmaxf(m_qu, fabsf(qu));
        m_kd = fmaxf(m_kd, fabsf(kd));
      }
      if (sf.exact) sm.exact[b] = 1;
      sm.end[b][ch] = sf.end;
    }
    float m_v = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (((tid + j * kPrepThreads) >> 4) >= tc) vraw[j] = make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {vraw[j].x, vraw[j].y, vraw[j].z, vraw[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m_v = fmaxf(m_v, fabsf(__uint_as_float(w[e] << 16)));
        m_v = fmaxf(m_v, fabsf(__uint_as_float(w[e] & 0xffff0000u)));
      }
    }
    block_max(&sm.mx[kMxV], m_v, lane);
    if (warp < 2) {
      sm.beta[tid] = be;
      hdr[Record::kBeta + tid] = be;
      block_max(&sm.mx[kMxBeta], fabsf(be), lane);
    }
    __syncthreads();

    // ---- 2. channel constants
    {
      Sum before{0.f, 0.f}, after{0.f, 0.f};
      for (int j = 0; j < b; ++j) before = add(before, sm.end[j][ch]);
      for (int j = b + 1; j < kNB; ++j) after = add(after, sm.end[j][ch]);
      const Sum rest = add(sf.end, neg(sf.md));
      const float up = exp_of(add(before, sf.mu)), dn = exp_of(add(after, rest));
      sm.up[b][ch] = up;
      sm.dn[b][ch] = dn;
      if (p.save) reinterpret_cast<float*>(rec + Record::kDn)[b * kK + ch] = dn;
      if (b == 0) hdr[Record::kDecay + ch] = exp_of(add(sf.end, after));
      const float x32 = exp_of(b == 0 ? add(rest, sm.end[1][ch]) : (b == 1 ? rest : (b == 2 ? sf.mu : add(sf.mu, sm.end[2][ch]))));
      const float x16 = exp_of(b & 1 ? sf.mu : rest);
      sm.x32[b][ch] = x32;
      sm.x16[b][ch] = x16;
      block_max(&sm.mx[kMxKt], m_ku * up, lane);
      block_max(&sm.mx[kMxQt], m_qu * up, lane);
      block_max(&sm.mx[kMxKe], m_kd * dn, lane);
      if (b >= 2) {
        block_max(&sm.mx[kMxR32K], m_ku * x32, lane);
        block_max(&sm.mx[kMxR32Q], m_qu * x32, lane);
      } else {
        block_max(&sm.mx[kMxC32], m_kd * x32, lane);
      }
      if (b & 1) {
        block_max(&sm.mx[kMxR16K], m_ku * x16, lane);
        block_max(&sm.mx[kMxR16Q], m_qu * x16, lane);
      } else {
        block_max(&sm.mx[kMxC16], m_kd * x16, lane);
      }
    }
    // ---- 3. A and P inside a sub-block: warp = sub-block, A or P, eight columns
    {
      const int I = warp >> 2, kind = (warp >> 1) & 1, nt = warp & 1;
      const int r = lane >> 2, c = lane & 3;
      float hi[2][4] = {}, lo[4] = {};
      if (!sm.exact[I]) {
        const float (*const X)[kFP] = kind ? sm.f.qu : sm.f.ku;
        const float* const x0 = &X[I * kB + r][c];
        const float* const b0 = &sm.f.kd[I * kB + nt * 8 + r][c];
#pragma unroll
        for (int kk = 0; kk < kK / 8; ++kk) {
          uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
          for (int j = 0; j < 4; ++j) tf32_pair(x0[(j & 1) * 8 * kFP + kk * 8 + (j >> 1) * 4], ah[j], al[j]);
#pragma unroll
          for (int j = 0; j < 2; ++j) tf32_pair(b0[kk * 8 + j * 4], bh[j], bl[j]);
          mma_tf32(lo, ah, bl);
          mma_tf32(lo, al, bh);
          mma_tf32(hi[kk & 1], ah, bh);
        }
      }
      float (*const dst)[kAP] = kind ? sm.pm : sm.a;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = I * kB + r + (e >> 1) * 8, s = I * kB + nt * 8 + 2 * c + (e & 1);
        const float x = (hi[0][e] + hi[1][e]) + lo[e];
        dst[t][s] = s < t + kind ? x : 0.f;
      }
    }
    // ---- 4. tiles of the decayed rows, over the factors; warp = eight channels, lane = token (and the one 32 further on).
    // Qt and Ke stay in registers until the solve leaves most warps idle.
    const int i0 = warp * 8;
    float qu[2][8], kd[2][8];
    // x[8] f[8] sc as a pair of 16-byte pieces
    auto put = [&](unsigned char* hi, unsigned char* lo, uint32_t off, const float (&x)[8], const float (&f)[8], float sc) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[2 * e] * f[2 * e] * sc, x[2 * e + 1] * f[2 * e + 1] * sc, h[e], l[e]);
      *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    };
    auto get = [&](const float* src, float (&f)[8]) {
      *reinterpret_cast<float4*>(&f[0]) = *reinterpret_cast<const float4*>(src);
      *reinterpret_cast<float4*>(&f[4]) = *reinterpret_cast<const float4*>(src + 4);
    };
    {
      float ku[2][8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = j * 32 + lane;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          *reinterpret_cast<float4*>(&ku[j][e]) = *reinterpret_cast<const float4*>(&sm.f.ku[t][i0 + e]);
          *reinterpret_cast<float4*>(&qu[j][e]) = *reinterpret_cast<const float4*>(&sm.f.qu[t][i0 + e]);
          *reinterpret_cast<float4*>(&kd[j][e]) = *reinterpret_cast<const float4*>(&sm.f.kd[t][i0 + e]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = j * 32 + lane, tb = t / kB;  // tb: 0, 1 and then 2, 3
        const uint32_t off = Core<kC>::off(t, i0);
        float f[8];
        get(&sm.up[tb][i0], f);
        put(sm.t.kt, sm.t.kt + Record::kPlane, off, ku[j], f, scale_of(kMxKt));
        get(&sm.x32[tb][i0], f);
        const uint32_t off32 = Core<32>::off(lane, i0), off16 = Core<32>::off(j * kB + (lane & 15), i0);
        if (j == 1) {
          put(sm.t.r32[0], sm.t.r32[0] + kHalfPlane, off32, ku[j], f, scale_of(kMxR32K));
          put(sm.t.r32[1], sm.t.r32[1] + kHalfPlane, off32, qu[j], f, scale_of(kMxR32Q));
        } else {
          put(sm.t.c32, sm.t.c32 + kHalfPlane, off32, kd[j], f, scale_of(kMxC32));
        }
        get(&sm.x16[tb][i0], f);
        if (tb & 1) {
          put(sm.t.r16[0], sm.t.r16[0] + kHalfPlane, off16, ku[j], f, scale_of(kMxR16K));
          put(sm.t.r16[1], sm.t.r16[1] + kHalfPlane, off16, qu[j], f, scale_of(kMxR16Q));
        } else {
          put(sm.t.c16, sm.t.c16 + kHalfPlane, off16, kd[j], f, scale_of(kMxC16));
        }
      }
      const float sc_v = scale_of(kMxV);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = tid + j * kPrepThreads;
        const uint32_t w[4] = {vraw[j].x, vraw[j].y, vraw[j].z, vraw[j].w};
        uint32_t vh[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vh[e] = as_u32(__floats2half2_rn(__uint_as_float(w[e] << 16) * sc_v, __uint_as_float(w[e] & 0xffff0000u) * sc_v));
        *reinterpret_cast<uint4*>(sm.vt + Rows128::off(c >> 4, (c & 15) * 8)) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
      }
    }
    __syncthreads();

    // ---- 5. A and P across sub-blocks: 16 x 16 a warp, eight across the middle, four inside the halves
    if (warp < 12) {
      const bool far = warp < 8;
      const int kind = warp & 1, m0 = far ? ((warp >> 1) & 1) * 16 : ((warp >> 1) & 1) * 16, n0 = far ? (warp >> 2) * 16 : m0;
      float x[2][4];
      pair_product(smem_addr(far ? sm.t.r32[kind] : sm.t.r16[kind]), m0, smem_addr(far ? sm.t.c32 : sm.t.c16), n0, lane, x);
      const float inv = far ? pow2_inv(scale_of(kind ? kMxR32Q : kMxR32K)) * pow2_inv(scale_of(kMxC32))
                            : pow2_inv(scale_of(kind ? kMxR16Q : kMxR16K)) * pow2_inv(scale_of(kMxC16));
      const int t0 = far ? 32 + m0 : 2 * m0 + 16, s0 = far ? n0 : 2 * m0;
      float (*const dst)[kAP] = kind ? sm.pm : sm.a;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          *reinterpret_cast<float2*>(&dst[t0 + (lane >> 2) + hf * 8][s0 + n * 8 + 2 * (lane & 3)]) =
              make_float2(x[n][2 * hf] * inv, x[n][2 * hf + 1] * inv);
    }
    if (sm.exact[0] | sm.exact[1] | sm.exact[2] | sm.exact[3]) {
      for (int j = 0; j < kNB; ++j)
        if (sm.exact[j]) prep_exact_block(p, sm, j, pos.tok, tc, h);
    }
    // the next chunk: its rows arrive over the tiles just read while the rest is computed
    bool more = false, ok = true;
    for (;;) {
      ok = __syncthreads_and(mbar_wait(&sm.taken_full, phase));
      const int64_t block = ok ? taken_block(&sm.taken) : -1;
      if (block < 0) break;
      slot_and_head(p, static_cast<uint32_t>(block), slot, h);
      pos = locate(p, slot);
      more = pos.tc > 0;
      if (more) break;
      __syncthreads();
      if (tid == 0) request_block(&sm.taken, &sm.taken_full);
      phase ^= 1;
    }
    if (more)
      fetch();
    else if (gridDim.x <= kSms)  // one short prompt: 25.7 us a call, 27.1 without; long calls 1 % slower
      launch_dependents();

    auto put_qt_ke = [&]() {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = j * 32 + lane;
        const uint32_t off = Core<kC>::off(t, i0);
        float f[8];
        get(&sm.up[t / kB][i0], f);
        put(rec + Record::kQt, rec + Record::kQt + Record::kPlane, off, qu[j], f, scale_of(kMxQt));
        get(&sm.dn[t / kB][i0], f);
        put(rec + Record::kKe, rec + Record::kKe + Record::kPlane, off, kd[j], f, scale_of(kMxKe));
      }
    };
    // ---- 6. Y = A (I + diag(beta) A)^-1: four warps, the diagonal blocks by substitution, then pairs of blocks
    if (warp < 4) {
      float m = 0.f;
      if (lane < kB) {
        const int r0 = warp * kB;
        float x[kB];
#pragma unroll
        for (int r = 0; r < kB; ++r) x[r] = r > lane ? sm.a[r0 + r][r0 + lane] : 0.f;
#pragma unroll
        for (int s = 0; s < kB - 1; ++s) {
          const float w = -sm.beta[r0 + s] * x[s];
#pragma unroll
          for (int r = s + 1; r < kB; ++r) x[r] = fmaf(sm.a[r0 + r][r0 + s], w, x[r]);
        }
#pragma unroll
        for (int r = 0; r < kB; ++r) {
          sm.y[r0 + r][r0 + lane] = x[r];
          m = fmaxf(m, fabsf(x[r]));
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      m = fmaxf(m, solve_below<16>(sm, 16 + (warp >> 1) * 32, (warp >> 1) * 32 + (warp & 1) * 8, lane));
      asm volatile("bar.sync 1, 128;" ::: "memory");
      m = fmaxf(m, solve_below<32>(sm, 32, warp * 8, lane));
      block_max(&sm.mx[kMxY], m, lane);
      put_qt_ke();
    } else {  // the other warps: Qt, Ke and P to the record
      put_qt_ke();
      const int w = tid - 128;
      float m = 0.f;
      for (int e = w; e < kC * kC; e += kPrepThreads - 128)
        if (((e >> 4) & 3) <= (e >> 10)) m = fmaxf(m, fabsf(sm.pm[e >> 6][e & 63]));
      block_max(&sm.mx[kMxP], m, lane);
      asm volatile("bar.sync 2, 384;" ::: "memory");
      const float sc_p = scale_of(kMxP);
      if (w == 0) hdr[Record::kScP] = sc_p;
      for (int c = w; c < kC * kC / 8; c += kPrepThreads - 128) {
        const int t = c & 63, s0 = (c >> 6) * 8;
        float x[8];
        read_row(sm.pm, t, s0, x);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[2 * e] * sc_p, x[2 * e + 1] * sc_p, hi[e], lo[e]);
        *reinterpret_cast<uint4*>(rec + Record::kP + Core<kC>::off(t, s0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(rec + Record::kP + kC * kC * 2 + Core<kC>::off(t, s0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    __syncthreads();
    // ---- 7. the tile M = I - Y diag(beta) (over P), and diag(beta) Y to the record
    const float y_beta = __uint_as_float(sm.mx[kMxY]) * __uint_as_float(sm.mx[kMxBeta]);
    const float sc_m = pow2_scale(fmaxf(1.f, y_beta)), sc_y = pow2_scale(y_beta), sc_v = scale_of(kMxV), sc_kt = scale_of(kMxKt);
    unsigned char* const mt = reinterpret_cast<unsigned char*>(&sm.pm[0][0]);
    {
      const int t = tid & 63, s0 = (tid >> 6) * 8;
      const float bt = sm.beta[t];
      float x[8];
      read_row(sm.y, t, s0, x);
      uint32_t hi[4], lo[4], yh[4], yl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = s0 + 2 * e;
        split2(((t == s ? 1.f : 0.f) - x[2 * e] * sm.beta[s]) * sc_m, ((t == s + 1 ? 1.f : 0.f) - x[2 * e + 1] * sm.beta[s + 1]) * sc_m,
               hi[e], lo[e]);
        split2(x[2 * e] * bt * sc_y, x[2 * e + 1] * bt * sc_y, yh[e], yl[e]);
      }
      const uint32_t off = Core<kC>::off(t, s0);
      *reinterpret_cast<uint4*>(mt + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(mt + kC * kC * 2 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (p.save) {
        *reinterpret_cast<uint4*>(rec + Record::kY + off) = make_uint4(yh[0], yh[1], yh[2], yh[3]);
        *reinterpret_cast<uint4*>(rec + Record::kY + kC * kC * 2 + off) = make_uint4(yl[0], yl[1], yl[2], yl[3]);
      }
    }
    __syncthreads();

    // ---- 8. Rt^T = V^T M^T: warp = 16 value columns, token sub-blocks 0 and 3 or 1 and 2 (five products each)
    const uint32_t mt_a = smem_addr(mt), kt_a = smem_addr(sm.t.kt), vt_a = smem_addr(sm.vt);
    const int g16 = (warp & 7) * 16, first = warp >> 3;  // sub-blocks `first` and 3 - first
    float* const rt = reinterpret_cast<float*>(rec + Record::kRt);
    float m_rt = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int nb = u ? 3 - first : first;
      float hi[2][4] = {}, lo[2][4] = {};
      for (int kk = 0; kk <= nb; ++kk) {  // s sub-blocks up to it
        uint32_t av[4], bh[4], bl[4];
        load_a_t<Rows128>(vt_a, g16, kk * 16, lane, av);
        load_b<Core<kC>>(mt_a, kk * 16, nb * 16, lane, bh);
        load_b<Core<kC>>(mt_a + kC * kC * 2, kk * 16, nb * 16, lane, bl);
        mma_pair(lo[0], lo[1], av, bl);
        mma_pair(hi[0], hi[1], av, bh);
      }
      const float inv = pow2_inv(sc_m) * pow2_inv(sc_v);
      const int v0 = g16 + (lane >> 2), t0 = nb * 16 + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float2 x = make_float2((hi[n][2 * hf] + lo[n][2 * hf]) * inv, (hi[n][2 * hf + 1] + lo[n][2 * hf + 1]) * inv);
          *reinterpret_cast<float2*>(rt + ((t0 + n * 8) >> 2) * (kV * 4) + (v0 + hf * 8) * 4 + (t0 & 3)) = x;
          m_rt = fmaxf(m_rt, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
    }
    block_max(&sm.mx[kMxRt], m_rt, lane);
    // ---- 9. Wr = M Kt: warp = 16 key channels, the same token sub-blocks
    float acc[2][2][4];
    float m_wr = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int mb = u ? 3 - first : first;
      float hi[2][4] = {}, lo[2][4] = {};
      for (int kk = 0; kk <= mb; ++kk) {
        uint32_t ah[4], al[4], bh[4], bl[4];
        load_b_t<Core<kC>>(kt_a, kk * 16, g16, lane, bh);
        load_b_t<Core<kC>>(kt_a + Record::kPlane, kk * 16, g16, lane, bl);
        load_a<Core<kC>>(mt_a, mb * 16, kk * 16, lane, ah);
        load_a<Core<kC>>(mt_a + kC * kC * 2, mb * 16, kk * 16, lane, al);
        mma_pair(lo[0], lo[1], ah, bl);
        mma_pair(lo[0], lo[1], al, bh);
        mma_pair(hi[0], hi[1], ah, bh);
      }
      const float inv = pow2_inv(sc_m) * pow2_inv(sc_kt);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[u][n][e] = (hi[n][e] + lo[n][e]) * inv;
          m_wr = fmaxf(m_wr, fabsf(acc[u][n][e]));
        }
    }
    block_max(&sm.mx[kMxWr], m_wr, lane);
    __syncthreads();
    const float sc_wr = scale_of(kMxWr);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t hi, lo;
          split2(acc[u][n][2 * hf] * sc_wr, acc[u][n][2 * hf + 1] * sc_wr, hi, lo);
          const uint32_t off = Core<kC>::off((u ? 3 - first : first) * 16 + hf * 8 + (lane >> 2), g16 + n * 8 + 2 * (lane & 3));
          *reinterpret_cast<uint32_t*>(rec + Record::kWr + off) = hi;  // a warp's are a whole line of the Core tile
          *reinterpret_cast<uint32_t*>(rec + Record::kWr + Record::kPlane + off) = lo;
        }
    if (tid == 0) {
      hdr[Record::kScWr] = sc_wr;
      hdr[Record::kScKe] = scale_of(kMxKe);
      hdr[Record::kScQt] = scale_of(kMxQt);
      hdr[Record::kScY] = sc_y;
      hdr[Record::kMxWr] = __uint_as_float(sm.mx[kMxWr]);
      hdr[Record::kMxRt] = __uint_as_float(sm.mx[kMxRt]);
    }
    if (!more) {
      if (!ok && tid == 0) set_error(p);
      return;
    }
  }
}

}  // namespace kdal
