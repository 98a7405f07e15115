// kda_scan_grad.cuh -- the scan's gradients of a chunk, once the states and
// their gradients are known at its ends (kda_scan_chain.cuh).
//
// With dU (the gradient of U = beta r), S0 and dS1 of the chunk:
//   y = dU - Y^T (beta dU),  dR = beta y,  dV = dR,  dbeta = sum_v r y
//   dQt = scale dO S0^T, dKt = -dR S0^T, dKe = (beta r) dS1^T
//   dP = scale dO (beta r)^T (s <= t),  dA = -dR (beta r)^T (s < t)
// and, over the pairs of the chunk with E_ts = exp(Gamma_t - Gamma_s),
//   dq_t  = dQt_t exp(Gamma_t) + sum_s dP_ts k_s E_ts
//   dk_t  = [dKt_t exp(Gamma_t) + sum_s dA_ts k_s E_ts]                      "row"
//         + [dKe_t exp(Gamma_C - Gamma_t) + sum_s (dP_st q_s + dA_st k_s) E_st] "column"
// dg_t is what crosses token t: the products q dq + k dk of every pair (t', s) with s < t <= t', with S0 as the earliest s
// and dS1 as the latest t'.  For t in sub-block b that is
//   sum_{t' >= t in b} (in-block pairs' row minus column, and rows' from before b)
//   + sum_{s < t in b} (columns' from behind b, and Ke dKe) + sum_{s before b} Ke dKe + exp(Gamma_C) sum_v S0 dS1
//   + sum_{blocks behind b} rows' from before them - sum_{b and blocks behind} columns' from behind them.
// A sum of rows minus columns over the whole rest of the chunk is the same, but every pair behind t comes in twice there
// and cancels, a token with itself (P_tt) and dKe with sum_v S1 dS1 too: under strong decays that left dg ten times less
// exact.
//
// The decays are applied sub-block by sub-block (16 tokens) on the
// accumulators: a row block I starts from its dQt and, for J = 0 .. I - 1,
// multiplies by the decay up to J's reference, adds dP_IJ (k dn)_J on the
// tensor cores and multiplies by the rest of J's decay; column blocks run
// through the later blocks in reverse the same way.  All factors stay at most
// 1 (see SubFactors), and no product is formed twice.
//
// What bounds it, like the chunk preparation: the latency of its phases on one
// block of 512 threads an SM (its operands fill the shared memory).  Of a chunk's
// 47000 cycles the first loads take 8000, y and the factors 10000, the products
// with the states and exp(Gamma_C) sum_v S0 dS1 7000, the pairs 19000 (tf32
// splits and MMAs, half of either's rate).  Measured (B200): 2112 chunks and
// heads 399 us; a plain copy would move its bytes in 120.  Blocks that go on with
// the next chunk and fetch its first operands under the decays' gradients, as the
// preparation's do, were 20 us slower.
#pragma once

#include "kda_scan_common.cuh"
#include "kda_umma.cuh"

namespace kdal {

constexpr int kGradThreads = 512;  // 256 left the schedulers short of warps: each phase waits on its own loads
static_assert(kGradThreads == 512, "the count of the barrier ahead of dKe");
constexpr int kGP = kK + 8;  // padded rows of the fp32 factors, read as [k][n] fragments
constexpr int kDP = kC + 4;

struct GradSmem {
  // The operand tiles; later dP and dA over the first, and the factors after them.
  unsigned char s0[kV * kK * 4];             // S0^T [v][i] hi, lo; before: the chunk's raw rows
  unsigned char ds[kV * kK * 4];             // dS1^T; before: dU^T and beta Y
  unsigned char dr[2 * Record::kPlane];      // dR^T [v][t]
  unsigned char r[2 * Record::kPlane];       // r^T [v][t]
  unsigned char dO[Record::kPlane];          // dO [t][v], one plane
  // exp(mu), exp(md), exp(end - mu), exp(end - md) per sub-block and channel
  float emu[kNB][kK], emd[kNB][kK], eru[kNB][kK], erd[kNB][kK];
  float hdr[Record::kHdr / 4];
  float dn[kNB][kK];                         // from k dn to Ke
  float sc[Record::kScBytes / 4];
  float ended[kNB][kK];                      // Ke dKe summed per sub-block
  float dbeta[8][kC];
  float dp_own[kC];                          // dP_tt
  uint32_t mx_do, mx_dr;
  uint32_t exact[kNB][kK / 32];              // channels out of the factors' range, a bit each
  uint64_t bar[5];                           // dU, Y and r; S0; dS1; dP and dA; the other products
  uint32_t tmem;
};
// Columns of tensor memory: products of 64 tokens (M) with 128 channels or 64 tokens.
struct GradColumns {
  static constexpr uint32_t kDQ = 0, kDKRow = 128, kDKCol = 256, kDP = 384, kDA = 448, kAll = 512;
};
struct GradPairs {  // over s0 .. dO once those are dead
  float dp[kC][kDP], da[kC][kDP];
  float up[kC][kGP], dn[kC][kGP];            // exp(L - mu), exp(md - L)
  float ku[kC][kGP], qu[kC][kGP], kd[kC][kGP];  // k up, q up, k dn
  float rows[kNB][kK], columns[kNB][kK];     // parts of the decays' gradients, summed per sub-block
};
static_assert(sizeof(GradPairs) <= offsetof(GradSmem, emu), "the factors fit over the operand tiles");
static_assert(2 * sizeof(float) * kC * kDP <= kV * kK * 4, "dP and dA fit over S0");
static_assert(sizeof(GradSmem) <= 232448, "shared memory of an SM");

// A 16 x 16 A-fragment pair to rows v0.. of a tile, columns c0..
template <class L>
__device__ __forceinline__ void store_frag(unsigned char* tile, int plane, int v0, int c0, int lane, const uint32_t (&ah)[4],
                                           const uint32_t (&al)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t off = L::off(v0 + (lane >> 2) + (j & 1) * 8, c0 + (j >> 1) * 8 + 2 * (lane & 3));
    *reinterpret_cast<uint32_t*>(tile + off) = ah[j];
    *reinterpret_cast<uint32_t*>(tile + plane + off) = al[j];
  }
}
// [16 value columns x 16 tokens] of an accumulator pair, rounded to bf16, to rows (token, 16 values).
__device__ __forceinline__ void store_out16(__nv_bfloat16* out, int64_t ts, int t0, int tc, int lane, const float (&c0)[4],
                                            const float (&c1)[4], float f) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float(&c)[4] = j ? c1 : c0;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(c[0] * f, c[1] * f), hi = __floats2bfloat162_rn(c[2] * f, c[3] * f);
    const uint32_t a = transpose8(*reinterpret_cast<const uint32_t*>(&lo)), b = transpose8(*reinterpret_cast<const uint32_t*>(&hi));
    const int t = t0 + j * 8 + (lane >> 2);
    if (t < tc) {
      *reinterpret_cast<uint32_t*>(out + t * ts + 2 * (lane & 3)) = a;
      *reinterpret_cast<uint32_t*>(out + t * ts + 8 + 2 * (lane & 3)) = b;
    }
  }
}

// Direct sums inside sub-block b for a channel i whose decays are out of the
// factors' range: one accumulator element (t, i), pairs from the log-decays
// between them.  Only such channels' elements: for all of a sub-block with one,
// the gradients took three times as long.
__device__ __noinline__ float3 grad_exact_element(const ScanParams& p, const GradPairs& f, int b, int64_t tok, int tc, int64_t h,
                                                  int t, int i) {
  if (t >= tc) return make_float3(0.f, 0.f, 0.f);
  float d = 0.f, dq = 0.f, dkr = 0.f, dkc = 0.f;
  for (int s = t; s >= b * kB; --s) {
    const float ke = __bfloat162float(p.k[(tok + s) * p.k_ts + h * kK + i]) * expf(d);
    dq = fmaf(f.dp[t][s], ke, dq);
    dkr = fmaf(f.da[t][s], ke, dkr);
    d += log_decay(p.g[(tok + s) * p.g_ts + h * kK + i]);
  }
  d = 0.f;
  for (int s = t; s < (b + 1) * kB && s < tc; ++s) {
    if (s > t) d += log_decay(p.g[(tok + s) * p.g_ts + h * kK + i]);
    const float e = expf(d);
    dkc = fmaf(f.dp[s][t] * e, __bfloat162float(p.q[(tok + s) * p.q_ts + h * kK + i]), dkc);
    dkc = fmaf(f.da[s][t] * e, __bfloat162float(p.k[(tok + s) * p.k_ts + h * kK + i]), dkc);
  }
  return make_float3(dq, dkr, dkc);
}

// A operand a (rows r0.., k0.. k), stored [row][k] (or [k][row] if TRANS); B operand b rows k0.., channels i0...
template <bool TRANS>
__device__ __forceinline__ void pair_a(const float (*a)[kDP], int r0, int k0, int lane, uint32_t (&ah)[4], uint32_t (&al)[4]) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = r0 + r + (j & 1) * 8, k = k0 + c + (j >> 1) * 4;
    tf32_pair(TRANS ? a[k][row] : a[row][k], ah[j], al[j]);
  }
}
__device__ __forceinline__ void pair_b(const float (*b)[kGP], int k0, int i0, int lane, uint32_t (&bh)[2], uint32_t (&bl)[2]) {
  const int r = lane >> 2, c = lane & 3;
  tf32_pair(b[k0 + c][i0 + r], bh[0], bl[0]);
  tf32_pair(b[k0 + c + 4][i0 + r], bh[1], bl[1]);
}
// c += (ah + al) (bh + bl) without al.bl, the cross terms first.  The MMA adds to its accumulator with truncation: c is a
// few products' alone, and joins a longer sum by an ordinary addition.
__device__ __forceinline__ void mma3_tf32(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[2],
                                          const uint32_t (&bl)[2]) {
  mma_tf32(c, ah, bl);
  mma_tf32(c, al, bh);
  mma_tf32(c, ah, bh);
}
__device__ __forceinline__ void scale_cols(float (&acc)[4][4], const float* f) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 d = *reinterpret_cast<const float2*>(f + n * 8);
    acc[n][0] *= d.x;
    acc[n][1] *= d.y;
    acc[n][2] *= d.x;
    acc[n][3] *= d.y;
  }
}
__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&x)[4], float f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[e], f, acc[e]);
}

__global__ void __launch_bounds__(kGradThreads, 1) kda_scan_grad_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  GradSmem& sm = *reinterpret_cast<GradSmem*>(smem_raw);
  GradPairs& pr = *reinterpret_cast<GradPairs*>(smem_raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  int64_t slot, h;
  slot_and_head(p, blockIdx.x, slot, h);
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(&sm.bar[i], 1);
    mbar_fence_init();
    sm.mx_do = sm.mx_dr = 0;
  }
  const ChunkPos pos = locate(p, slot);
  const int tc = pos.tc;
  wait_upstream();
  if (tc == 0) return;
  if (warp == 0) tmem_alloc(&sm.tmem, GradColumns::kAll);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const unsigned char* const rec = record(p, slot, h);
  RawRows& raw = *reinterpret_cast<RawRows*>(sm.s0);
  static_assert(sizeof(RawRows) <= sizeof(sm.s0), "the raw rows fit");
  // ---- dO as an fp16 tile (exact after scaling); its loads go ahead of the copies, which keep the SM's port busy
  const int ch = tid & (kK - 1), sub = tid >> 7;
  {
    uint4 raw_do[2];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = tid & 63, pc = (tid >> 6) + 8 * j;
      raw_do[j] = *reinterpret_cast<const uint4*>(p.d_out + (pos.tok + (t < tc ? t : tc - 1)) * p.d_out_ts + h * kV + pc * 8);
    }
    if (tid == 0) {
      mbar_expect(&sm.bar[0], Record::kHdr + Record::kScBytes + Record::kDnBytes + 2 * Record::kPlane + kC * kC * 4 + 2 * Record::kPlane);
      bulk_load(sm.hdr, rec, Record::kHdr, &sm.bar[0]);
      bulk_load(sm.sc, rec + Record::kSc, Record::kScBytes, &sm.bar[0]);
      bulk_load(sm.dn, rec + Record::kDn, Record::kDnBytes, &sm.bar[0]);
      bulk_load(sm.ds, rec + Record::kDU, 2 * Record::kPlane, &sm.bar[0]);
      bulk_load(sm.ds + 2 * Record::kPlane, rec + Record::kY, kC * kC * 4, &sm.bar[0]);
      bulk_load(sm.r, rec + Record::kR, 2 * Record::kPlane, &sm.bar[0]);
    }
    fetch_rows<kGradThreads>(p, pos.tok, tc, h, raw.g, raw.k, raw.q);  // for step 3
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if ((tid & 63) >= tc) raw_do[j] = make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {raw_do[j].x, raw_do[j].y, raw_do[j].z, raw_do[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    }
    m = warp_max(m);
    if (lane == 0) atomicMax(&sm.mx_do, __float_as_uint(m));
    __syncthreads();
    const float sc = pow2_scale(__uint_as_float(sm.mx_do));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = tid & 63, pc = (tid >> 6) + 8 * j;
      uint32_t w[4] = {raw_do[j].x, raw_do[j].y, raw_do[j].z, raw_do[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = as_u32(__floats2half2_rn(__uint_as_float(w[e] << 16) * sc, __uint_as_float(w[e] & 0xffff0000u) * sc));
      *reinterpret_cast<uint4*>(sm.dO + Core<kC>::off(t, pc * 8)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  const float sc_do = pow2_scale(__uint_as_float(sm.mx_do));
  bool ok = __syncthreads_and(mbar_wait(&sm.bar[0], 0));  // if a wait gives up, the block goes on to its end on what it has
  const uint32_t a_s0 = smem_addr(sm.s0), a_ds = smem_addr(sm.ds), a_dr = smem_addr(sm.dr), a_r = smem_addr(sm.r), a_do = smem_addr(sm.dO);
  const float* const beta = sm.hdr + Record::kBeta;

  // ---- 1. y^T = dU^T - dU^T (beta Y); dR, dV, dbeta: warp = 16 value columns, token sub-blocks 0 and 3 or 1 and 2
  // (five products each)
  {
    const int grp = warp & 7, v0 = grp * 16, first = warp >> 3;
    const uint32_t a_y = a_ds + 2 * Record::kPlane;
    __nv_bfloat16* const dv = p.dv + pos.tok * p.dv_ts + h * kV + v0;
    float dr[2][2][4] = {}, m_dr = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int nb = u ? 3 - first : first;  // the sub-block of tokens
      auto& acc = dr[u];
      uint32_t dh[4], dl[4];
      for (int kk = 3; kk >= nb; --kk) {     // s sub-block; Y[s][t] is zero for t >= s
        uint32_t bh[4], bl[4];
        load_a<Core<kV>>(a_ds, v0, kk * 16, lane, dh);
        load_a<Core<kV>>(a_ds + Record::kPlane, v0, kk * 16, lane, dl);
        load_b_t<Core<kC>>(a_y, kk * 16, nb * 16, lane, bh);
        load_b_t<Core<kC>>(a_y + kC * kC * 2, kk * 16, nb * 16, lane, bl);
        float x[2][4] = {};
        mma_pair(x[0], x[1], dh, bl);
        mma_pair(x[0], x[1], dl, bh);
        mma_pair(x[0], x[1], dh, bh);
        const float f = pow2_inv(sm.sc[Record::kScDU + (grp >> 1)]) * pow2_inv(sm.hdr[Record::kScY]);
        add_scaled(acc[0], x[0], f);
        add_scaled(acc[1], x[1], f);
      }
      // dh, dl now hold the sub-block's own dU
      const float inv = pow2_inv(sm.sc[Record::kScDU + (grp >> 1)]), inv_r = pow2_inv(sm.sc[Record::kScR]);
      uint32_t rh[4], rl[4];
      load_a<Core<kV>>(a_r, v0, nb * 16, lane, rh);
      load_a<Core<kV>>(a_r + Record::kPlane, v0, nb * 16, lane, rl);
      float db[4] = {0.f, 0.f, 0.f, 0.f};  // tokens nb 16 + 2 (lane & 3) + {0, 1, 8, 9}
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // fragment register j: rows + (j & 1) 8, columns + (j >> 1) 8
        const float2 du = join2(dh[j], dl[j]), r = join2(rh[j], rl[j]);
        float(&c)[4] = acc[j >> 1];
        const int e = (j & 1) * 2, t = nb * 16 + (j >> 1) * 8 + 2 * (lane & 3);
        const float y0 = fmaf(du.x, inv, -c[e]), y1 = fmaf(du.y, inv, -c[e + 1]);
        db[(j >> 1) * 2] = fmaf(y0, r.x * inv_r, db[(j >> 1) * 2]);
        db[(j >> 1) * 2 + 1] = fmaf(y1, r.y * inv_r, db[(j >> 1) * 2 + 1]);
        c[e] = y0 * beta[t];
        c[e + 1] = y1 * beta[t + 1];
        m_dr = fmaxf(m_dr, fmaxf(fabsf(c[e]), fabsf(c[e + 1])));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
        if (lane < 4) sm.dbeta[grp][nb * 16 + (j >> 1) * 8 + 2 * lane + (j & 1)] = db[j];
      }
      store_out16(dv, p.dv_ts, nb * 16, tc, lane, acc[0], acc[1], 1.f);
    }
    m_dr = warp_max(m_dr);
    if (lane == 0) atomicMax(&sm.mx_dr, __float_as_uint(m_dr));
    __syncthreads();
    const float sc = pow2_scale(__uint_as_float(sm.mx_dr));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t dh[4], dl[4];
      frag_a(dr[u][0], dr[u][1], sc, dh, dl);
      store_frag<Core<kV>>(sm.dr, Record::kPlane, v0, (u ? 3 - first : first) * 16, lane, dh, dl);
    }
  }
  cp_async_wait_all();
  fence_async();  // dO and dR come before the products' reads, the reads of dU and Y before dS1 is copied over them
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  // ---- 2. The products on the tensor cores, issued by two warps among the others' work on the decay factors: dP = dO r,
  // dA = -dR r and, once S0 and dS1 are there, dQt = dO S0^T, dKt = -dR S0^T, dKe = r dS1^T (scales and signs come later).
  const float sc_do_inv = pow2_inv(sc_do), sc_dr_inv = pow2_inv(pow2_scale(__uint_as_float(sm.mx_dr)));
  if (tid < tc) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sm.dbeta[w][tid];
    p.dbeta[(pos.tok + tid) * p.dbeta_ts + h] = s;
  }
  // ---- 3. decay factors: thread = channel and sub-block
  float up[kB], dn[kB], kv[kB], qv[kB];
  {
    float g[kB];
    read_sub_block(raw.g, raw.k, raw.q, tc, sub, ch, g, kv, qv);
    fence_async();
    __syncthreads();  // the rows are read: S0 goes over them
    if (tid == 0) {
      mbar_expect(&sm.bar[1], kV * kK * 4);
      bulk_load(sm.s0, rec + Record::kS, kV * kK * 4, &sm.bar[1]);
      mbar_expect(&sm.bar[2], kV * kK * 4);
      bulk_load(sm.ds, rec + Record::kDS, kV * kK * 4, &sm.bar[2]);
    }
    if (warp == 0) {
      umma_tiles<kC, kV, kC, false, kV, true, true>(tmem + GradColumns::kDP, a_do, 0, a_r, Record::kPlane);
      umma_tiles<kC, kV, kV, true, kV, true, false>(tmem + GradColumns::kDA, a_dr, Record::kPlane, a_r, Record::kPlane);
      umma_commit(&sm.bar[3]);
    }
    const SubFactors f = sub_factors(g, up, dn);
    const uint32_t out_of_range = __ballot_sync(0xffffffffu, f.exact);
    if (lane == 0) sm.exact[sub][warp & 3] = out_of_range;
    sm.emu[sub][ch] = exp_of(f.mu);
    sm.emd[sub][ch] = exp_of(f.md);
    sm.eru[sub][ch] = exp_of(add(f.end, neg(f.mu)));
    sm.erd[sub][ch] = exp_of(add(f.end, neg(f.md)));
  }
  // ---- 4. exp(Gamma_C) sum_v S0 dS1: warp = eight channels, lanes over the value columns; lane e < 8 keeps channel e's
  // dS1 has a scale per 32 value columns, which dKe contracts: r (done with otherwise) takes up the differences
  ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar[3], 0)) && ok;
  const float sc_ds = fminf(fminf(sm.sc[Record::kScDS], sm.sc[Record::kScDS + 1]), fminf(sm.sc[Record::kScDS + 2], sm.sc[Record::kScDS + 3]));
  fence_after_sync();
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // a plane's half of the column blocks; lanes over the value columns
    const int piece = tid + j * kGradThreads;
    const __half2 f = __float2half2_rn(sc_ds * pow2_inv(sm.sc[Record::kScDS + ((piece & (kV - 1)) >> 5)]));
    uint4& x = *reinterpret_cast<uint4*>(sm.r + piece * 16);
    uint32_t y[4] = {x.x, x.y, x.z, x.w};
    scale_frag(y, f);
    x = make_uint4(y[0], y[1], y[2], y[3]);
  }
  fence_async();
  ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar[1], 0)) && ok;
  if (warp == 1) {
    umma_tiles<kK, kV, kC, false, kV, true, true>(tmem + GradColumns::kDQ, a_do, 0, a_s0, kV * kK * 2);
    umma_tiles<kK, kV, kV, true, kV, true, false>(tmem + GradColumns::kDKRow, a_dr, Record::kPlane, a_s0, kV * kK * 2);
  }
  ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar[2], 0)) && ok;
  if (warp == 1) {  // r is complete when every warp is here; the others need not wait
    asm volatile("bar.sync 1, 512;" ::: "memory");
    umma_tiles<kK, kV, kV, true, kV, true, false>(tmem + GradColumns::kDKCol, a_r, Record::kPlane, a_ds, kV * kK * 2);
    umma_commit(&sm.bar[4]);
  } else {
    asm volatile("bar.arrive 1, 512;" ::: "memory");
  }
  float e_sum = 0.f;
  {
    float x[8] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t off = Core<kV>::off(q * 32 + lane, warp * 8);
      const uint4 sh = *reinterpret_cast<const uint4*>(sm.s0 + off), sl = *reinterpret_cast<const uint4*>(sm.s0 + kV * kK * 2 + off);
      const uint4 dh = *reinterpret_cast<const uint4*>(sm.ds + off), dl = *reinterpret_cast<const uint4*>(sm.ds + kV * kK * 2 + off);
      const uint32_t a[4] = {sh.x, sh.y, sh.z, sh.w}, al[4] = {sl.x, sl.y, sl.z, sl.w};
      const uint32_t d[4] = {dh.x, dh.y, dh.z, dh.w}, ld[4] = {dl.x, dl.y, dl.z, dl.w};
      const float inv_ds = pow2_inv(sm.sc[Record::kScDS + q]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 s = join2(a[e], al[e]), ds = join2(d[e], ld[e]);
        x[2 * e] = fmaf(s.x * ds.x, inv_ds, x[2 * e]);
        x[2 * e + 1] = fmaf(s.y * ds.y, inv_ds, x[2 * e + 1]);
      }
    }
    const float inv = pow2_inv(sm.sc[Record::kScS]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = 16; o; o >>= 1) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
      if (lane == e) e_sum = x[e] * inv * sm.hdr[Record::kDecay + warp * 8 + e];
    }
  }
  // ---- 5. the factors, dP and dA over the operand tiles
  ok = __syncthreads_and(mbar_wait(&sm.bar[4], 0) && ok);  // every product is done, and every warp with S0 and dS1
  fence_after_sync();
#pragma unroll
  for (int t = 0; t < kB; ++t) {
    pr.up[sub * kB + t][ch] = up[t];
    pr.dn[sub * kB + t][ch] = dn[t];
    pr.ku[sub * kB + t][ch] = kv[t] * up[t];
    pr.qu[sub * kB + t][ch] = qv[t] * up[t];
    pr.kd[sub * kB + t][ch] = kv[t] * dn[t];
  }
  const int I = warp & 3, i0 = (warp >> 2) * 32;  // the warp's tokens (its lanes of tensor memory) and channels
  const uint32_t mine = tmem + (static_cast<uint32_t>(I * 32) << 16);
  if (const int si = warp >> 2; si <= I) {        // none above the diagonal
    float cp[2][4], ca[2][4];
    tmem_ld_tiles(mine + GradColumns::kDP + si * 16, cp);
    tmem_ld_tiles(mine + GradColumns::kDA + si * 16, ca);
    const float inv_r = pow2_inv(sm.sc[Record::kScR]), fp = inv_r * sc_do_inv * p.scale, fa = -inv_r * sc_dr_inv;
    const int t = I * 16 + (lane >> 2), s = si * 16 + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tt = t + (e >> 1) * 8, ss = s + n * 8 + (e & 1);
        const float b = beta[ss];
        const float x = cp[n][e] * fp * b;
        if (ss == tt) sm.dp_own[tt] = x;
        pr.dp[tt][ss] = ss < tt ? x : 0.f;
        pr.da[tt][ss] = ss < tt ? ca[n][e] * fa * b : 0.f;
      }
  }
  // ---- 6. the products with the states into registers: tokens I 16 .., channels i0 ..
  const int row = I * 16 + (lane >> 2), col = i0 + 2 * (lane & 3);  // this thread's rows: row, row + 8; channels col + 8 n, + 1
  float dq[4][4], dkr[4][4], dkc[4][4] = {};
  tmem_ld_tiles(mine + GradColumns::kDQ + i0, dq);
  tmem_ld_tiles(mine + GradColumns::kDKRow + i0, dkr);
  {
    const float inv_s = pow2_inv(sm.sc[Record::kScS]), fq = inv_s * sc_do_inv * p.scale, fk = -inv_s * sc_dr_inv;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dq[n][e] *= fq;
        dkr[n][e] *= fk;
      }
  }
  __syncthreads();

  // ---- 7. the pairs
  // q or k again, at this thread's elements (rows behind the chunk: the last one's); read where they are used, not kept
  auto fetch = [&](const __nv_bfloat16* x, int64_t ts, __nv_bfloat162 (&to)[4][2]) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const __nv_bfloat16* const at = x + (pos.tok + (row + hf * 8 < tc ? row + hf * 8 : tc - 1)) * ts + h * kK + col;
#pragma unroll
      for (int n = 0; n < 4; ++n) to[n][hf] = *reinterpret_cast<const __nv_bfloat162*>(at + n * 8);
    }
  };
  auto put_out = [&](__nv_bfloat16* to, int64_t ts, int n, int hf, float x, float y) {
    const int t = row + hf * 8;
    if (t < tc) *reinterpret_cast<__nv_bfloat162*>(to + (pos.tok + t) * ts + h * kK + col + n * 8) = __floats2bfloat162_rn(x, y);
  };
  // the products with block J's keys; with its queries and keys
  auto row_block = [&](int J, float (&xq)[4][4], float (&xk)[4][4]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t ph[4], pl[4], ah[4], al[4];
      pair_a<false>(pr.dp, I * 16, J * 16 + kk * 8, lane, ph, pl);
      pair_a<false>(pr.da, I * 16, J * 16 + kk * 8, lane, ah, al);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t bh[2], bl[2];
        pair_b(pr.kd, J * 16 + kk * 8, i0 + n * 8, lane, bh, bl);
        mma3_tf32(xq[n], ph, pl, bh, bl);
        mma3_tf32(xk[n], ah, al, bh, bl);
      }
    }
  };
  auto column_block = [&](int J, float (&x)[4][4]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t ph[4], pl[4], ah[4], al[4];
      pair_a<true>(pr.dp, I * 16, J * 16 + kk * 8, lane, ph, pl);
      pair_a<true>(pr.da, I * 16, J * 16 + kk * 8, lane, ah, al);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t bh[2], bl[2];
        pair_b(pr.qu, J * 16 + kk * 8, i0 + n * 8, lane, bh, bl);
        mma3_tf32(x[n], ph, pl, bh, bl);
        pair_b(pr.ku, J * 16 + kk * 8, i0 + n * 8, lane, bh, bl);
        mma3_tf32(x[n], ah, al, bh, bl);
      }
    }
  };
  // sums of a block's rows per channel, to the block's lanes 0 .. 3
  auto block_sum = [&](float (&x)[4][2], float (*to)[kK]) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x[n][e] += __shfl_xor_sync(0xffffffffu, x[n][e], o);
        if (lane < 4) to[I][col + n * 8 + e] = x[n][e];
      }
  };
  // This thread's channels whose pairs inside the block have to be summed directly: bit 8 n + e; nearly always none.
  const uint32_t exact_word = sm.exact[I][warp >> 2], exact = exact_word >> (2 * (lane & 3));
  {  // rows: earlier tokens
    for (int J = 0; J < I; ++J) {
      scale_cols(dq, &sm.emd[J][col]);
      scale_cols(dkr, &sm.emd[J][col]);
      float xq[4][4] = {}, xk[4][4] = {};  // this block's alone: see mma3_tf32
      row_block(J, xq, xk);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        add_scaled(dq[n], xq[n], 1.f);
        add_scaled(dkr[n], xk[n], 1.f);
      }
      scale_cols(dq, &sm.erd[J][col]);
      scale_cols(dkr, &sm.erd[J][col]);
    }
    scale_cols(dq, &sm.emu[I][col]);
    scale_cols(dkr, &sm.emu[I][col]);
    float xq[4][4] = {}, xk[4][4] = {}, sum[4][2] = {};
    __nv_bfloat162 qe[4][2], ke[4][2];
    fetch(p.q, p.q_ts, qe);
    fetch(p.k, p.k_ts, ke);
    row_block(I, xq, xk);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = pr.up[row + (e >> 1) * 8][col + n * 8 + (e & 1)];
        dq[n][e] *= u;
        dkr[n][e] *= u;
        xq[n][e] *= u;
        xk[n][e] *= u;
      }
    if (exact_word) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((exact >> (8 * n + (e & 1))) & 1) {
            const float3 d = grad_exact_element(p, pr, I, pos.tok, tc, h, row + (e >> 1) * 8, col + n * 8 + (e & 1));
            xq[n][e] = d.x;
            xk[n][e] = d.y;
          }
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float own = sm.dp_own[row + hf * 8];
        const float2 q2 = __bfloat1622float2(qe[n][hf]), k2 = __bfloat1622float2(ke[n][hf]);
        float2 y;
        auto element = [&](int e, float q, float k) {
          const float before = fmaf(q, dq[n][e], k * dkr[n][e]), inside = fmaf(q, xq[n][e], k * xk[n][e]);
          sum[n][e & 1] += before;
          dq[n][e] = fmaf(own, k, dq[n][e] + xq[n][e]);
          dkr[n][e] = fmaf(own, q, dkr[n][e] + xk[n][e]);
          return before + inside;
        };
        y.x = element(2 * hf, q2.x, k2.x);
        y.y = element(2 * hf + 1, q2.y, k2.y);
        *reinterpret_cast<float2*>(&pr.up[row + hf * 8][col + n * 8]) = y;  // this thread's own elements
        put_out(p.dq, p.dq_ts, n, hf, dq[n][2 * hf], dq[n][2 * hf + 1]);
      }
    block_sum(sum, pr.rows);
  }
  {  // columns: later tokens
    for (int J = kNB - 1; J > I; --J) {
      scale_cols(dkc, &sm.eru[J][col]);
      float x[4][4] = {};
      column_block(J, x);
#pragma unroll
      for (int n = 0; n < 4; ++n) add_scaled(dkc[n], x[n], 1.f);
      scale_cols(dkc, &sm.emu[J][col]);
    }
    scale_cols(dkc, &sm.erd[I][col]);
    float x[4][4] = {}, ended[4][4], sum[4][2] = {};
    __nv_bfloat162 ke[4][2];
    fetch(p.k, p.k_ts, ke);
    column_block(I, x);
    tmem_ld_tiles(mine + GradColumns::kDKCol + i0, ended);  // dKe
    const float inv_r = pow2_inv(sm.sc[Record::kScR]) * pow2_inv(sc_ds), b0 = beta[row] * inv_r, b1 = beta[row + 8] * inv_r;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float d = pr.dn[row + (e >> 1) * 8][col + n * 8 + (e & 1)], f = sm.dn[I][col + n * 8 + (e & 1)];
        dkc[n][e] *= d;
        x[n][e] *= d;
        ended[n][e] *= (e >> 1 ? b1 : b0) * (f * d);
      }
    if (exact_word) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((exact >> (8 * n + (e & 1))) & 1)
            x[n][e] = grad_exact_element(p, pr, I, pos.tok, tc, h, row + (e >> 1) * 8, col + n * 8 + (e & 1)).z;
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float2& at = *reinterpret_cast<float2*>(&pr.up[row + hf * 8][col + n * 8]);
        const float2 k2 = __bfloat1622float2(ke[n][hf]);
        float2 y = at, z;
        auto element = [&](int e, float k, float& inside) {
          const float behind = k * dkc[n][e];
          sum[n][e & 1] += behind;
          inside = fmaf(-k, x[n][e], inside);
          dkr[n][e] += (dkc[n][e] + x[n][e]) + ended[n][e];  // dk
          return fmaf(k, ended[n][e], behind);
        };
        z.x = element(2 * hf, k2.x, y.x);
        z.y = element(2 * hf + 1, k2.y, y.y);
        at = y;
        *reinterpret_cast<float2*>(&pr.dn[row + hf * 8][col + n * 8]) = z;
        put_out(p.dk, p.dk_ts, n, hf, dkr[n][2 * hf], dkr[n][2 * hf + 1]);
      }
    }
    block_sum(sum, pr.columns);
  }
  fence_before_sync();
  __syncthreads();  // the factors are dead: the decays' gradients go over them
  // ---- 8. dg: thread = channel and sub-block
  float* const ev = &pr.qu[0][0];  // [128]
  if (lane < 8) ev[warp * 8 + lane] = e_sum;
  float lead[kB], ahead = 0.f;  // of the sub-block: the columns' from behind it and Ke dKe, ahead of each token
#pragma unroll
  for (int t = 0; t < kB; ++t) {
    lead[t] = ahead;
    ahead += pr.dn[sub * kB + t][ch];
  }
  sm.ended[sub][ch] = ahead - pr.columns[sub][ch];
  __syncthreads();
  {
    float acc = ev[ch];
    for (int j = 0; j < sub; ++j) acc += sm.ended[j][ch];
    float cross = -pr.columns[sub][ch];
    for (int j = sub + 1; j < kNB; ++j) cross += pr.rows[j][ch] - pr.columns[j][ch];
    acc += cross;
#pragma unroll
    for (int t = kB - 1; t >= 0; --t) {
      const int tt = sub * kB + t;
      acc += pr.up[tt][ch];
      if (tt < tc) p.dg[(pos.tok + tt) * p.dg_ts + h * kK + ch] = acc + lead[t];
    }
  }
  if (!ok && tid == 0) set_error(p);
  if (warp == 0) tmem_dealloc(tmem, GradColumns::kAll);
}

}  // namespace kdal
