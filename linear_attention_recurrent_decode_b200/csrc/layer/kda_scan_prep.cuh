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
// Decays.  Every factor is kept at most 1 (for g <= 0) by splitting the chunk
// into sub-blocks of 16 tokens: for t in sub-block I and s in an earlier J,
// exp(Gamma_t - Gamma_s) = up_t exp(mu_I + L_J+1 + .. + L_I-1 + L_J - md_J) dn_s
// (see SubFactors), the middle factor per channel from fp64 sums; inside a
// sub-block up_t dn_s alone.  These products run in tf32 pairs, whose range
// takes the e^+-60 of a sub-block's factors; the triangular products that
// follow in fp16 pairs.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kPrepThreads = 256;
constexpr int kFP = kK + 4;  // padded rows of the fp32 factors: MMA fragments then touch 32 banks
constexpr int kAP = kC + 4;

struct PrepSmem {
  float ku[kC][kFP];            // k up
  float qu[kC][kFP];            // q up
  float kd[kC][kFP];            // k dn
  float a[kC][kAP];             // A; the first part holds the fp64 sums before
  float pm[kC][kAP];            // P; then the tile M
  float y[kC][kAP];             // Y
  unsigned char kt[2 * Record::kPlane];  // Kt tile hi, lo; then Wr
  unsigned char vt[Record::kPlane];      // V tile [t][v]
  float up[kNB][kK];            // exp(Gamma at the sub-block's start + mu)
  float dn[kNB][kK];            // exp(Gamma_C - (Gamma at its start + md))
  float cross[6][kK];           // the middle factor of the six (I, J < I)
  float beta[kC];
  uint32_t mx[8];               // block maxima (float bits): v, kt, qt, ke, p, y, wr, beta
  int exact[kNB];
  ChunkPos pos;
};
static_assert(sizeof(double) * 3 * kNB * kK <= sizeof(float) * kC * kAP, "the fp64 sums fit into a");
static_assert(2 * kC * kC * 2 <= sizeof(float) * kC * kAP, "the M tile fits into pm");

__device__ __forceinline__ void block_max(uint32_t* slot, float m, int lane) {
  m = warp_max(m);
  if (lane == 0) atomicMax(slot, __float_as_uint(m));
}

// Pairs inside sub-block `b` from the differences themselves: warp w takes two
// rows, its lanes four channels each, s running down from t with the
// log-decay between s and t summed on the way.
__device__ __noinline__ void prep_exact_block(const ScanParams& p, PrepSmem& sm, int b, int64_t tok, int tc, int64_t h) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < kB; r += kPrepThreads / 32) {
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

__global__ void __launch_bounds__(kPrepThreads, 1) kda_scan_prep_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PrepSmem& sm = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t slot = blockIdx.x / p.HV, h = blockIdx.x - slot * p.HV;
  if (tid < 8) sm.mx[tid] = 0;
  if (tid < kNB) sm.exact[tid] = 0;
  const ChunkPos pos = locate(p, slot, &sm.pos);
  const int tc = pos.tc;
  if (tc == 0) return;
  __syncthreads();
  unsigned char* const rec = record(p, slot, h);
  float* const hdr = reinterpret_cast<float*>(rec);

  // ---- 1. decay factors: thread = channel, two sub-blocks
  const int ch = tid & (kK - 1), half = tid >> 7;
  double* const dsum = reinterpret_cast<double*>(&sm.a[0][0]);  // [3][kNB][kK]: mu, md, end
  float m_ku[2], m_qu[2], m_kd[2];
#pragma unroll
  for (int b2 = 0; b2 < 2; ++b2) {
    const int b = half * 2 + b2;
    float g[kB], kv[kB], qv[kB], up[kB], dn[kB];
#pragma unroll
    for (int t = 0; t < kB; ++t) {
      const int64_t tk = pos.tok + b * kB + t;
      const bool in = b * kB + t < tc;
      g[t] = in ? log_decay(__ldg(p.g + tk * p.g_ts + h * kK + ch)) : 0.f;
      kv[t] = in ? __bfloat162float(p.k[tk * p.k_ts + h * kK + ch]) : 0.f;
      qv[t] = in ? __bfloat162float(p.q[tk * p.q_ts + h * kK + ch]) : 0.f;
    }
    const SubFactors f = sub_factors(g, up, dn);
    m_ku[b2] = m_qu[b2] = m_kd[b2] = 0.f;
#pragma unroll
    for (int t = 0; t < kB; ++t) {
      const float a = kv[t] * up[t], c = qv[t] * up[t], d = kv[t] * dn[t];
      sm.ku[b * kB + t][ch] = a;
      sm.qu[b * kB + t][ch] = c;
      sm.kd[b * kB + t][ch] = d;
      m_ku[b2] = fmaxf(m_ku[b2], fabsf(a));
      m_qu[b2] = fmaxf(m_qu[b2], fabsf(c));
      m_kd[b2] = fmaxf(m_kd[b2], fabsf(d));
    }
    if (f.exact) sm.exact[b] = 1;
    dsum[b * kK + ch] = f.mu;
    dsum[(kNB + b) * kK + ch] = f.md;
    dsum[(2 * kNB + b) * kK + ch] = f.end;
  }
  // v: 16-byte pieces, kept in registers until the scale is known
  uint4 vraw[4];
  float m_v = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = tid + j * kPrepThreads, t = c >> 4, pc = c & 15;
    vraw[j] = t < tc ? *reinterpret_cast<const uint4*>(p.v + (pos.tok + t) * p.v_ts + h * kV + pc * 8) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {vraw[j].x, vraw[j].y, vraw[j].z, vraw[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m_v = fmaxf(m_v, fabsf(__uint_as_float(w[e] << 16)));
      m_v = fmaxf(m_v, fabsf(__uint_as_float(w[e] & 0xffff0000u)));
    }
  }
  block_max(&sm.mx[0], m_v, lane);
  if (warp < 2) {
    const float b = tid < tc ? __ldg(p.beta + (pos.tok + tid) * p.beta_ts + h) : 0.f;
    sm.beta[tid] = b;
    hdr[Record::kBeta + tid] = b;
    block_max(&sm.mx[7], fabsf(b), lane);
  }
  __syncthreads();

  // ---- 2. channel constants
#pragma unroll
  for (int b2 = 0; b2 < 2; ++b2) {
    const int b = half * 2 + b2;
    double before = 0.0, after = 0.0;
    for (int j = 0; j < b; ++j) before += dsum[(2 * kNB + j) * kK + ch];
    for (int j = b + 1; j < kNB; ++j) after += dsum[(2 * kNB + j) * kK + ch];
    const double mu = dsum[b * kK + ch], md = dsum[(kNB + b) * kK + ch], end = dsum[(2 * kNB + b) * kK + ch];
    const float up = exp_of(before + mu), dn = exp_of(after + (end - md));
    sm.up[b][ch] = up;
    sm.dn[b][ch] = dn;
    if (b == 0) hdr[Record::kDecay + ch] = exp_of(end + after);
    m_ku[b2] *= up;
    m_qu[b2] *= up;
    m_kd[b2] *= dn;
  }
  for (int e = half; e < 6; e += 2) {  // (I, J): (1,0) (2,0) (2,1) (3,0) (3,1) (3,2)
    const int I = e < 1 ? 1 : (e < 3 ? 2 : 3), J = e - I * (I - 1) / 2;
    double s = dsum[I * kK + ch] + (dsum[(2 * kNB + J) * kK + ch] - dsum[(kNB + J) * kK + ch]);
    for (int j = J + 1; j < I; ++j) s += dsum[(2 * kNB + j) * kK + ch];
    sm.cross[e][ch] = exp_of(s);
  }
  block_max(&sm.mx[1], fmaxf(m_ku[0], m_ku[1]), lane);
  block_max(&sm.mx[2], fmaxf(m_qu[0], m_qu[1]), lane);
  block_max(&sm.mx[3], fmaxf(m_kd[0], m_kd[1]), lane);
  __syncthreads();
  for (int e = tid; e < kC * kAP; e += kPrepThreads) {
    (&sm.a[0][0])[e] = 0.f;
    (&sm.pm[0][0])[e] = 0.f;
    (&sm.y[0][0])[e] = 0.f;
  }
  const float sc_v = pow2_scale(__uint_as_float(sm.mx[0])), sc_kt = pow2_scale(__uint_as_float(sm.mx[1]));
  const float sc_qt = pow2_scale(__uint_as_float(sm.mx[2])), sc_ke = pow2_scale(__uint_as_float(sm.mx[3]));

  // ---- 3. tiles of the decayed rows: Kt and V to shared memory, Qt and Ke to the record
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = tid + j * kPrepThreads, t = c >> 4, i0 = (c & 15) * 8, b = t / kB;
    const uint32_t off = off128(t, i0);
    uint32_t hi[4], lo[4], qh[4], ql[4], eh[4], el[4], vh[4];
    const uint32_t w[4] = {vraw[j].x, vraw[j].y, vraw[j].z, vraw[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 2 * e;
      const float2 up = *reinterpret_cast<const float2*>(&sm.up[b][i]), dn = *reinterpret_cast<const float2*>(&sm.dn[b][i]);
      const float2 ku = *reinterpret_cast<const float2*>(&sm.ku[t][i]), qu = *reinterpret_cast<const float2*>(&sm.qu[t][i]);
      const float2 kd = *reinterpret_cast<const float2*>(&sm.kd[t][i]);
      split2(ku.x * up.x * sc_kt, ku.y * up.y * sc_kt, hi[e], lo[e]);
      split2(qu.x * up.x * sc_qt, qu.y * up.y * sc_qt, qh[e], ql[e]);
      split2(kd.x * dn.x * sc_ke, kd.y * dn.y * sc_ke, eh[e], el[e]);
      vh[e] = as_u32(__floats2half2_rn(__uint_as_float(w[e] << 16) * sc_v, __uint_as_float(w[e] & 0xffff0000u) * sc_v));
    }
    *reinterpret_cast<uint4*>(sm.kt + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sm.kt + Record::kPlane + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(sm.vt + off) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
    *reinterpret_cast<uint4*>(rec + Record::kQt + off) = make_uint4(qh[0], qh[1], qh[2], qh[3]);
    if (p.save) *reinterpret_cast<uint4*>(rec + Record::kQt + Record::kPlane + off) = make_uint4(ql[0], ql[1], ql[2], ql[3]);
    *reinterpret_cast<uint4*>(rec + Record::kKe + off) = make_uint4(eh[0], eh[1], eh[2], eh[3]);
    *reinterpret_cast<uint4*>(rec + Record::kKe + Record::kPlane + off) = make_uint4(el[0], el[1], el[2], el[3]);
  }
  __syncthreads();

  // ---- 4. A and P: 40 units of 16 x 8 (ten sub-block pairs, A or P, two column tiles), five a warp
  for (int u = warp; u < 40; u += kPrepThreads / 32) {
    const int nt = u & 1, kind = (u >> 1) & 1, pr = u >> 2;  // pr: 0..5 below the diagonal, 6..9 on it
    const int I = pr < 6 ? (pr < 1 ? 1 : (pr < 3 ? 2 : 3)) : pr - 6, J = pr < 6 ? pr - I * (I - 1) / 2 : I;
    if (I == J && sm.exact[I]) continue;
    const float (*const X)[kFP] = kind ? sm.qu : sm.ku;
    const int r = lane >> 2, c = lane & 3;
    const float* const x0 = &X[I * kB + r][c];
    const float* const b0 = &sm.kd[J * kB + nt * 8 + r][c];
    const float* const f = pr < 6 ? &sm.cross[pr][c] : nullptr;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int kk = 0; kk < kK; kk += 8) {
      const float f0 = f ? f[kk] : 1.f, f1 = f ? f[kk + 4] : 1.f;
      uint32_t ah[4], al[4], bh[2], bl[2];
      tf32_split(x0[kk] * f0, ah[0], al[0]);
      tf32_split(x0[8 * kFP + kk] * f0, ah[1], al[1]);
      tf32_split(x0[kk + 4] * f1, ah[2], al[2]);
      tf32_split(x0[8 * kFP + kk + 4] * f1, ah[3], al[3]);
      tf32_split(b0[kk], bh[0], bl[0]);
      tf32_split(b0[kk + 4], bh[1], bl[1]);
      mma3_tf32(acc, ah, al, bh, bl);
    }
    float (*const dst)[kAP] = kind ? sm.pm : sm.a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = I * kB + r + (e >> 1) * 8, s = J * kB + nt * 8 + 2 * c + (e & 1);
      dst[t][s] = kind ? (s <= t ? acc[e] : 0.f) : (s < t ? acc[e] : 0.f);
    }
  }
  __syncthreads();
  if (sm.exact[0] | sm.exact[1] | sm.exact[2] | sm.exact[3]) {
    for (int b = 0; b < kNB; ++b)
      if (sm.exact[b]) prep_exact_block(p, sm, b, pos.tok, tc, h);
    __syncthreads();
  }

  // ---- 5. Y = A (I + diag(beta) A)^-1 by sub-blocks: the diagonal ones by substitution ...
  if (tid < kC) {
    const int b = tid / kB, j = tid % kB;
    float yv[kB];
#pragma unroll
    for (int r = 0; r < kB; ++r) {
      float x = sm.a[b * kB + r][tid];
#pragma unroll
      for (int s = 0; s < r; ++s) x = fmaf(-sm.a[b * kB + r][b * kB + s] * sm.beta[b * kB + s], yv[s], x);
      yv[r] = r > j ? x : 0.f;
      sm.y[b * kB + r][tid] = yv[r];
    }
  } else {
    float m = 0.f;  // the other warps: P's maximum
    for (int e = tid - kC; e < kC * kC; e += kPrepThreads - kC) m = fmaxf(m, fabsf(sm.pm[e >> 6][e & 63]));
    block_max(&sm.mx[4], m, lane);
  }
  __syncthreads();
  {
    const float sc_p = pow2_scale(__uint_as_float(sm.mx[4]));
    if (tid == 0) hdr[Record::kScP] = sc_p;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = tid + j * kPrepThreads, t = c >> 3, s0 = (c & 7) * 8;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(sm.pm[t][s0 + 2 * e] * sc_p, sm.pm[t][s0 + 2 * e + 1] * sc_p, hi[e], lo[e]);
      *reinterpret_cast<uint4*>(rec + Record::kP + off64(t, s0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (p.save)
        *reinterpret_cast<uint4*>(rec + Record::kP + kC * kC * 2 + off64(t, s0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  // ... the rows of sub-blocks below from Y_I = (I - Y_II beta) (A_I - A_I,<I beta Y_<I)
  for (int I = 1; I < kNB; ++I) {
    const int cols = I * kB;
    float x[3];
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int e = tid + u * kPrepThreads, r = I * kB + (e & 15), j = e >> 4;
      if (j < cols) {
        float acc = sm.a[r][j];
        for (int s = j & ~(kB - 1); s < cols; ++s) acc = fmaf(-sm.a[r][s] * sm.beta[s], sm.y[s][j], acc);
        sm.y[r][j] = acc;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int e = tid + u * kPrepThreads, r = I * kB + (e & 15), j = e >> 4;
      if (j < cols) {
        x[u] = sm.y[r][j];
        for (int s = I * kB; s < r; ++s) x[u] = fmaf(-sm.y[r][s] * sm.beta[s], sm.y[s][j], x[u]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int e = tid + u * kPrepThreads, r = I * kB + (e & 15), j = e >> 4;
      if (j < cols) sm.y[r][j] = x[u];
    }
    __syncthreads();
  }
  {
    float m = 0.f;
    for (int e = tid; e < kC * kC; e += kPrepThreads) m = fmaxf(m, fabsf(sm.y[e >> 6][e & 63]));
    block_max(&sm.mx[5], m, lane);
  }
  __syncthreads();
  // ---- 6. the tile M = I - Y diag(beta) (over P), and diag(beta) Y to the record
  const float y_beta = __uint_as_float(sm.mx[5]) * __uint_as_float(sm.mx[7]);
  const float sc_m = pow2_scale(fmaxf(1.f, y_beta)), sc_y = pow2_scale(y_beta);
  unsigned char* const mt = reinterpret_cast<unsigned char*>(&sm.pm[0][0]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = tid + j * kPrepThreads, t = c >> 3, s0 = (c & 7) * 8;
    uint32_t hi[4], lo[4], yh[4], yl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s = s0 + 2 * e;
      const float y0 = sm.y[t][s], y1 = sm.y[t][s + 1];
      split2(((t == s ? 1.f : 0.f) - y0 * sm.beta[s]) * sc_m, ((t == s + 1 ? 1.f : 0.f) - y1 * sm.beta[s + 1]) * sc_m, hi[e], lo[e]);
      split2(y0 * sm.beta[t] * sc_y, y1 * sm.beta[t] * sc_y, yh[e], yl[e]);
    }
    *reinterpret_cast<uint4*>(mt + off64(t, s0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(mt + kC * kC * 2 + off64(t, s0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (p.save) {
      *reinterpret_cast<uint4*>(rec + Record::kY + off64(t, s0)) = make_uint4(yh[0], yh[1], yh[2], yh[3]);
      *reinterpret_cast<uint4*>(rec + Record::kY + kC * kC * 2 + off64(t, s0)) = make_uint4(yl[0], yl[1], yl[2], yl[3]);
    }
  }
  __syncthreads();

  // ---- 7. Rt^T = V^T M^T: warp = 16 value columns
  const uint32_t mt_a = smem_addr(mt), kt_a = smem_addr(sm.kt), vt_a = smem_addr(sm.vt);
  {
    float acc[8][4] = {};
#pragma unroll
    for (int kk = 0; kk < kNB; ++kk) {  // s sub-block
      uint32_t av[4];
      load_a_t<128>(vt_a, warp * 16, kk * 16, lane, av);
#pragma unroll
      for (int nb = kk; nb < kNB; ++nb) {  // t sub-blocks from it on
        uint32_t bh[4], bl[4];
        load_b<64>(mt_a, kk * 16, nb * 16, lane, bh);
        load_b<64>(mt_a + kC * kC * 2, kk * 16, nb * 16, lane, bl);
        mma2(acc[2 * nb], acc[2 * nb + 1], av, bh, bl);
      }
    }
    const float inv = pow2_inv(sc_m) * pow2_inv(sc_v);
    float* const rt = reinterpret_cast<float*>(rec + Record::kRt);
    const int v0 = warp * 16 + (lane >> 2), t0 = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      *reinterpret_cast<float2*>(rt + v0 * kC + n * 8 + t0) = make_float2(acc[n][0] * inv, acc[n][1] * inv);
      *reinterpret_cast<float2*>(rt + (v0 + 8) * kC + n * 8 + t0) = make_float2(acc[n][2] * inv, acc[n][3] * inv);
    }
  }
  // ---- 8. Wr = M Kt: warp = 16 key channels, all rows
  float acc[4][2][4] = {};
#pragma unroll
  for (int kk = 0; kk < kNB; ++kk) {
    uint32_t bh[4], bl[4];
    load_b_t<128>(kt_a, kk * 16, warp * 16, lane, bh);
    load_b_t<128>(kt_a + Record::kPlane, kk * 16, warp * 16, lane, bl);
#pragma unroll
    for (int mb = kk; mb < kNB; ++mb) {
      uint32_t ah[4], al[4];
      load_a<64>(mt_a, mb * 16, kk * 16, lane, ah);
      load_a<64>(mt_a + kC * kC * 2, mb * 16, kk * 16, lane, al);
      mma3(acc[mb][0], acc[mb][1], ah, al, bh, bl);
    }
  }
  {
    const float inv = pow2_inv(sc_m) * pow2_inv(sc_kt);
    float m = 0.f;
#pragma unroll
    for (int mb = 0; mb < 4; ++mb)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[mb][n][e] *= inv;
          m = fmaxf(m, fabsf(acc[mb][n][e]));
        }
    block_max(&sm.mx[6], m, lane);
  }
  __syncthreads();  // every warp is done with Kt
  const float sc_wr = pow2_scale(__uint_as_float(sm.mx[6]));
#pragma unroll
  for (int mb = 0; mb < 4; ++mb)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t hi, lo;
        split2(acc[mb][n][2 * hf] * sc_wr, acc[mb][n][2 * hf + 1] * sc_wr, hi, lo);
        const uint32_t off = off128(mb * 16 + hf * 8 + (lane >> 2), warp * 16 + n * 8 + 2 * (lane & 3));
        *reinterpret_cast<uint32_t*>(sm.kt + off) = hi;
        *reinterpret_cast<uint32_t*>(sm.kt + Record::kPlane + off) = lo;
      }
  if (tid == 0) {
    hdr[Record::kScWr] = sc_wr;
    hdr[Record::kScKe] = sc_ke;
    hdr[Record::kScQt] = sc_qt;
    hdr[Record::kScY] = sc_y;
  }
  __syncthreads();
  for (int c = tid; c < 2 * Record::kPlane / 16; c += kPrepThreads)
    *reinterpret_cast<uint4*>(rec + Record::kWr + 16 * c) = *reinterpret_cast<const uint4*>(sm.kt + 16 * c);
}

}  // namespace kdal
