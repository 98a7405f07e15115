// kda_scan_chain.cuh -- the scan's sequential kernels: the states from chunk to
// chunk, forwards with the outputs, and their gradients backwards.
//
// Forward, per chunk (see kda_scan_prep.cuh):
//   r = Rt - Wr S0;  O = scale (Qt S0 + P (beta r));  S1 = Diag(exp(Gamma_C)) S0 + Ke^T (beta r).
// Backward, per chunk in reverse, with the gradient dS1 of its end state:
//   dU = scale P^T dO + Ke dS1                          (the gradient of U = beta r)
//   dS0 = Diag(exp(Gamma_C)) dS1 + scale Qt^T dO - Wr^T (beta dU).
//
// The value columns are independent, so a warp owns 16 of them and keeps its
// whole slice of the (transposed) state, S^T [16 x 128], in 64 accumulator
// registers a thread; the chunk's r^T [16 x 64] is a second accumulator.  As
// the accumulator layout of one product is the A-operand layout of the next,
// the state never leaves the registers and warps never exchange anything: per
// chunk a warp only reads the chunk's tiles, which come through a ring of bulk
// copies that all warps of the CTA share.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kRing = 6;                                  // stages of the ring
constexpr int kStageBytes = 2 * Record::kPlane + Record::kHdr;  // 33 KB: two planes and a header

struct ChainSmem {
  unsigned char stage[kRing][kStageBytes];
  uint64_t full[kRing], empty[kRing];
};

// What a stage holds: up to two pieces of a record.
struct Piece {
  int off0, bytes0, off1, bytes1;
};
// Forward: header and Wr; P (hi) and Qt (hi); header and Ke.
__device__ __forceinline__ Piece forward_piece(int s) {
  if (s == 0) return Piece{0, Record::kHdr, Record::kWr, 2 * Record::kPlane};
  if (s == 1) return Piece{Record::kP, kC * kC * 2, Record::kQt, Record::kPlane};
  return Piece{0, Record::kHdr, Record::kKe, 2 * Record::kPlane};
}
// Backward: header and P; Ke; header and Qt; Wr.
__device__ __forceinline__ Piece backward_piece(int s) {
  if (s == 0) return Piece{0, Record::kHdr + kC * kC * 4, 0, 0};
  if (s == 1) return Piece{Record::kKe, 2 * Record::kPlane, 0, 0};
  if (s == 2) return Piece{0, Record::kHdr, Record::kQt, 2 * Record::kPlane};
  return Piece{Record::kWr, 2 * Record::kPlane, 0, 0};
}

// A warp's place in the ring.  One thread of the CTA (warp 0's lane 0) also
// refills it: as it comes to an item it starts the copy of the item kAhead
// further on, into the stage that every warp released kRing - kAhead items ago
// (a ninth warp for this would cost each thread a quarter of its registers).
constexpr int kAhead = 4;
template <bool FWD>
struct Ring {
  static constexpr int kPer = FWD ? 3 : 4;
  const ScanParams& p;
  ChainSmem& sm;
  int64_t slot0, h, nch;
  int lane;
  bool producer;
  int64_t it = 0;      // items released
  int64_t filled = 0;  // items whose copies were started (producer)
  bool ok = true;

  __device__ __forceinline__ void fill(int64_t item) {
    if (item >= nch * kPer) return;
    const int st = static_cast<int>(item % kRing);
    if (item >= kRing) ok = ok && mbar_wait(&sm.empty[st], static_cast<uint32_t>((item / kRing - 1) & 1));
    if (!ok) return;
    const int64_t c = item / kPer;
    const Piece pc = FWD ? forward_piece(static_cast<int>(item % kPer)) : backward_piece(static_cast<int>(item % kPer));
    const unsigned char* const rec = record(p, slot0 + (FWD ? c : nch - 1 - c), h);
    mbar_expect(&sm.full[st], static_cast<uint32_t>(pc.bytes0 + pc.bytes1));
    bulk_load(sm.stage[st], rec + pc.off0, static_cast<uint32_t>(pc.bytes0), &sm.full[st]);
    if (pc.bytes1) bulk_load(sm.stage[st] + pc.bytes0, rec + pc.off1, static_cast<uint32_t>(pc.bytes1), &sm.full[st]);
    ++filled;
  }
  __device__ __forceinline__ void start() {
    if (producer)
      for (int j = 0; j < kAhead; ++j) fill(j);
  }
  // Item it + ahead (0 or 1): its address once it is there.
  __device__ __forceinline__ uint32_t wait(int ahead = 0) {
    const int64_t i = it + ahead;
    const int st = static_cast<int>(i % kRing);
    if (producer) fill(i + kAhead);
    ok = ok && mbar_wait(&sm.full[st], static_cast<uint32_t>((i / kRing) & 1));
    return smem_addr(sm.stage[st]);
  }
  __device__ __forceinline__ const float* floats() const { return reinterpret_cast<const float*>(sm.stage[it % kRing]); }
  __device__ __forceinline__ void release() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[it % kRing]);
    ++it;
  }
  // After a wait that gave up: the CTA must not end with copies into it in flight.
  __device__ __forceinline__ void abandon() {
    if (lane == 0) set_error(p);
    if (producer)
      for (int64_t j = filled > kRing ? filled - kRing : 0; j < filled; ++j)
        mbar_wait(&sm.full[j % kRing], static_cast<uint32_t>((j / kRing) & 1));
  }
};

__device__ __forceinline__ void chain_init(ChainSmem& sm, int warps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], warps);
    }
    mbar_fence_init();
  }
  __syncthreads();
}

__device__ __forceinline__ float max4(const float (&a)[4], float m) {
  return fmaxf(fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])), fmaxf(fabsf(a[2]), fabsf(a[3]))), m);
}

// A 16 x 16 A-fragment pair to rows v0.. of a tile, columns c0..
template <int COLS>
__device__ __forceinline__ void store_frag(unsigned char* tile, int plane, int v0, int c0, int lane, const uint32_t (&ah)[4],
                                           const uint32_t (&al)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t off = tile_off<COLS>(v0 + (lane >> 2) + (j & 1) * 8, c0 + (j >> 1) * 8 + 2 * (lane & 3));
    *reinterpret_cast<uint32_t*>(tile + off) = ah[j];
    *reinterpret_cast<uint32_t*>(tile + plane + off) = al[j];
  }
}

// The state slice of 16 value columns: element (v, i) in the accumulator layout
// from or to a [K][V] block.
__device__ __forceinline__ void load_state(const float* blk, int v0, int lane, float (&s)[16][4]) {
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[n][e] = blk == nullptr ? 0.f : blk[(n * 8 + 2 * (lane & 3) + (e & 1)) * kV + v0 + (lane >> 2) + (e >> 1) * 8];
}
__device__ __forceinline__ void store_state(float* blk, int v0, int lane, const float (&s)[16][4], float f) {
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      blk[(n * 8 + 2 * (lane & 3) + (e & 1)) * kV + v0 + (lane >> 2) + (e >> 1) * 8] = s[n][e] * f;
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

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) kda_scan_forward_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChainSmem& sm = *reinterpret_cast<ChainSmem*>(smem_raw);
  constexpr int kTiles = 8 / WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x / kTiles;
  const int group = static_cast<int>(blockIdx.x - unit * kTiles) * WARPS + warp;  // 16 value columns
  const int64_t n = unit / p.HV, h = unit - n * p.HV;
  int64_t start, len;
  seq_range(p, n, start, len);
  const int64_t nch = (len + kC - 1) / kC, slot0 = first_slot(p, n, start), blk = state_block(p, n);
  const int v0 = group * 16;
  if (blk < 0) {  // inactive: zero outputs
    for (int64_t t = lane; t < len * 2; t += 32)
      *reinterpret_cast<uint4*>(p.out + (start + (t >> 1)) * p.out_ts + h * kV + v0 + (t & 1) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  chain_init(sm, WARPS);
  const int64_t sblk = (blk * p.HV + h) * kK * kV;
  float s[16][4];
  load_state(p.s_in == nullptr ? nullptr : p.s_in + sblk, v0, lane, s);
  float f = 1.f;  // the state is s f
  Ring<true> ring{p, sm, slot0, h, nch, lane, threadIdx.x == 0};
  ring.start();
  bool alive = true;  // no wait gave up, for any lane
  for (int64_t c = 0; c < nch; ++c) {
    unsigned char* const rec = record(p, slot0 + c, h);
    const int tc = static_cast<int>(len - c * kC < kC ? len - c * kC : kC);
    // Rt^T, needed after the first product
    float2 rt[8][2];
    {
      const float* const src = reinterpret_cast<const float*>(rec + Record::kRt) + (v0 + (lane >> 2)) * kC + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rt[j][0] = *reinterpret_cast<const float2*>(src + j * 8);
        rt[j][1] = *reinterpret_cast<const float2*>(src + 8 * kC + j * 8);
      }
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= f;
      m = max4(s[j], m);
    }
    const float sc_s = pow2_scale(warp_max(m));
    // ---- r^T = Rt^T - S0^T Wr^T, and S0^T Qt^T (one fp16 product: it is rounded to bf16 with the output)
    const uint32_t a_wr = ring.wait() + Record::kHdr;
    const float sc_wr = ring.floats()[Record::kScWr], sc_qt = ring.floats()[Record::kScQt], sc_p = ring.floats()[Record::kScP];
    const float sc_ke = ring.floats()[Record::kScKe];
    float r[8][4] = {}, o[8][4] = {};
    const uint32_t a_p = ring.wait(1), a_qt = a_p + kC * kC * 2;  // read along with the first
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      uint32_t ah[4], al[4];
      frag_a(s[2 * kk], s[2 * kk + 1], sc_s, ah, al);
      if (p.save) store_frag<128>(rec + Record::kS, kV * kK * 2, v0, kk * 16, lane, ah, al);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        uint32_t bh[4], bl[4];
        load_b<128>(a_wr, kk * 16, nb * 16, lane, bh);
        load_b<128>(a_wr + Record::kPlane, kk * 16, nb * 16, lane, bl);
        mma3(r[2 * nb], r[2 * nb + 1], ah, al, bh, bl);
        load_b<128>(a_qt, kk * 16, nb * 16, lane, bh);
        mma_f16(o[2 * nb], ah, bh[0], bh[1]);
        mma_f16(o[2 * nb + 1], ah, bh[2], bh[3]);
      }
    }
    // beta, before the header's stage is released
    float2 beta[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) beta[j] = *reinterpret_cast<const float2*>(ring.floats() + Record::kBeta + j * 8 + 2 * (lane & 3));
    ring.release();
    {
      const float inv = pow2_inv(sc_s) * pow2_inv(sc_wr);
      float mr = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j][0] = fmaf(-inv, r[j][0], rt[j][0].x);
        r[j][1] = fmaf(-inv, r[j][1], rt[j][0].y);
        r[j][2] = fmaf(-inv, r[j][2], rt[j][1].x);
        r[j][3] = fmaf(-inv, r[j][3], rt[j][1].y);
        mr = max4(r[j], mr);
      }
      if (p.save) {
        const float sc_r = pow2_scale(warp_max(mr));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t ah[4], al[4];
          frag_a(r[2 * kk], r[2 * kk + 1], sc_r, ah, al);
          store_frag<64>(rec + Record::kR, Record::kPlane, v0, kk * 16, lane, ah, al);
        }
        if (lane == 0) {
          reinterpret_cast<float*>(rec)[Record::kScS + group] = sc_s;
          reinterpret_cast<float*>(rec)[Record::kScR + group] = sc_r;
        }
      }
    }
    // ---- U^T = r^T diag(beta)
    float mu = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j][0] *= beta[j].x;
      r[j][1] *= beta[j].y;
      r[j][2] *= beta[j].x;
      r[j][3] *= beta[j].y;
      mu = max4(r[j], mu);
    }
    const float sc_u = pow2_scale(warp_max(mu));
    uint32_t uh[4][4], ul[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a(r[2 * kk], r[2 * kk + 1], sc_u, uh[kk], ul[kk]);
    // ---- O^T = scale (S0^T Qt^T + U^T P^T)
    {
      const float inv_s = pow2_inv(sc_s) * pow2_inv(sc_qt), inv_u = pow2_inv(sc_u) * pow2_inv(sc_p);
      float o2[8][4] = {};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int nb = kk; nb < 4; ++nb) {
          uint32_t bh[4];
          load_b<64>(a_p, kk * 16, nb * 16, lane, bh);
          mma_f16(o2[2 * nb], uh[kk], bh[0], bh[1]);
          mma_f16(o2[2 * nb + 1], uh[kk], bh[2], bh[3]);
        }
      ring.release();
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = fmaf(o[j][e], inv_s, o2[j][e] * inv_u);
      if (p.out != nullptr) {
        __nv_bfloat16* const out = p.out + (start + c * kC) * p.out_ts + h * kV + v0;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) store_out16(out, p.out_ts, nb * 16, tc, lane, o[2 * nb], o[2 * nb + 1], p.scale);
      }
    }
    // ---- S1^T = S0^T Diag(exp(Gamma_C)) + U^T Ke, in the products' scale
    const uint32_t a_ke = ring.wait() + Record::kHdr;
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
    {
      const float up = sc_u * sc_ke;
      f = pow2_inv(sc_u) * pow2_inv(sc_ke);
      const float* const dc = ring.floats() + Record::kDecay + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 d = *reinterpret_cast<const float2*>(dc + j * 8);
        s[j][0] *= d.x * up;
        s[j][1] *= d.y * up;
        s[j][2] *= d.x * up;
        s[j][3] *= d.y * up;
      }
#pragma unroll
      for (int nb = 0; nb < 8; ++nb)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t bh[4], bl[4];
          load_b_t<128>(a_ke, kk * 16, nb * 16, lane, bh);
          load_b_t<128>(a_ke + Record::kPlane, kk * 16, nb * 16, lane, bl);
          mma3(s[2 * nb], s[2 * nb + 1], uh[kk], ul[kk], bh, bl);
        }
    }
    ring.release();
  }
  if (!alive) {  // a copy never came: the state is not written
    ring.abandon();
    return;
  }
  if (p.s_out != nullptr) store_state(p.s_out + sblk, v0, lane, s, f);
}

// ---------------------------------------------------------------- backward
constexpr int kDoPitch = 48;                       // bytes per token row of a warp's 16 columns of dO (32 used)
constexpr int kDoBytes = kC * kDoPitch;

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) kda_scan_backward_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChainSmem& sm = *reinterpret_cast<ChainSmem*>(smem_raw);
  constexpr int kTiles = 8 / WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x / kTiles;
  const int group = static_cast<int>(blockIdx.x - unit * kTiles) * WARPS + warp;
  const int64_t n = unit / p.HV, h = unit - n * p.HV;
  int64_t start, len;
  seq_range(p, n, start, len);
  const int64_t nch = (len + kC - 1) / kC, slot0 = first_slot(p, n, start);
  const int v0 = group * 16;
  chain_init(sm, WARPS);
  unsigned char* const dob = smem_raw + sizeof(ChainSmem) + warp * kDoBytes;
  const uint32_t dob_a = smem_addr(dob);
  const int64_t sblk = (n * p.HV + h) * kK * kV;
  float s[16][4];
  load_state(p.d_final == nullptr ? nullptr : p.d_final + sblk, v0, lane, s);
  float f = 1.f;
  Ring<false> ring{p, sm, slot0, h, nch, lane, threadIdx.x == 0};
  ring.start();
  bool alive = true;
  uint4 dor[4];  // the next chunk's rows of dO: 16-byte piece (lane + 32 j): token / half of the columns
  auto fetch = [&](int64_t c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 32 * j, t = e >> 1;
      dor[j] = c >= 0 && c * kC + t < len
                   ? *reinterpret_cast<const uint4*>(p.d_out + (start + c * kC + t) * p.d_out_ts + h * kV + v0 + (e & 1) * 8)
                   : make_uint4(0, 0, 0, 0);
    }
  };
  fetch(nch - 1);
  for (int64_t c = nch - 1; c >= 0; --c) {
    unsigned char* const rec = record(p, slot0 + c, h);
    // ---- dO^T as the A operand (exact in fp16 after scaling: bf16 has 8 bits)
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {dor[j].x, dor[j].y, dor[j].z, dor[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    }
    const float sc_do = pow2_scale(warp_max(m));
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 32 * j;
      uint32_t w[4] = {dor[j].x, dor[j].y, dor[j].z, dor[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = as_u32(__floats2half2_rn(__uint_as_float(w[q] << 16) * sc_do, __uint_as_float(w[q] & 0xffff0000u) * sc_do));
      *reinterpret_cast<uint4*>(dob + (e >> 1) * kDoPitch + (e & 1) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    uint32_t da[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      ldsm4t(dob_a + (kk * 16 + (lane & 7) + (lane >> 4) * 8) * kDoPitch + ((lane >> 3) & 1) * 16, da[kk]);
    fetch(c - 1);

    // ---- dU^T = scale dO^T P + dS1^T Ke^T
    const uint32_t a_p = ring.wait() + Record::kHdr;
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
    const float sc_p = ring.floats()[Record::kScP], sc_ke = ring.floats()[Record::kScKe];
    const float sc_qt = ring.floats()[Record::kScQt], sc_wr = ring.floats()[Record::kScWr];
    float du[8][4] = {};
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)  // t sub-block; P[t][s] is zero for s > t
#pragma unroll
      for (int nb = 0; nb <= kk; ++nb) {
        uint32_t bh[4], bl[4];
        load_b_t<64>(a_p, kk * 16, nb * 16, lane, bh);
        load_b_t<64>(a_p + kC * kC * 2, kk * 16, nb * 16, lane, bl);
        mma2(du[2 * nb], du[2 * nb + 1], da[kk], bh, bl);
      }
    float2 beta[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) beta[j] = *reinterpret_cast<const float2*>(ring.floats() + Record::kBeta + j * 8 + 2 * (lane & 3));
    ring.release();
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= f;
      m = max4(s[j], m);
    }
    const float sc_s = pow2_scale(warp_max(m));
    const uint32_t a_ke = ring.wait();
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
    {
      float acc[8][4] = {};
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t ah[4], al[4];
        frag_a(s[2 * kk], s[2 * kk + 1], sc_s, ah, al);
        store_frag<128>(rec + Record::kDS, kV * kK * 2, v0, kk * 16, lane, ah, al);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t bh[4], bl[4];
          load_b<128>(a_ke, kk * 16, nb * 16, lane, bh);
          load_b<128>(a_ke + Record::kPlane, kk * 16, nb * 16, lane, bl);
          mma3(acc[2 * nb], acc[2 * nb + 1], ah, al, bh, bl);
        }
      }
      ring.release();
      const float inv_p = pow2_inv(sc_do) * pow2_inv(sc_p) * p.scale, inv_s = pow2_inv(sc_s) * pow2_inv(sc_ke);
      m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) du[j][e] = fmaf(du[j][e], inv_p, acc[j][e] * inv_s);
        m = max4(du[j], m);
      }
    }
    {
      const float sc_du = pow2_scale(warp_max(m));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t ah[4], al[4];
        frag_a(du[2 * kk], du[2 * kk + 1], sc_du, ah, al);
        store_frag<64>(rec + Record::kDU, Record::kPlane, v0, kk * 16, lane, ah, al);
      }
      if (lane == 0) {
        reinterpret_cast<float*>(rec)[Record::kScDS + group] = sc_s;
        reinterpret_cast<float*>(rec)[Record::kScDU + group] = sc_du;
      }
    }
    // ---- dS0^T = dS1^T Diag(exp(Gamma_C)) + scale dO^T Qt - (beta dU)^T Wr
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      du[j][0] *= -beta[j].x;
      du[j][1] *= -beta[j].y;
      du[j][2] *= -beta[j].x;
      du[j][3] *= -beta[j].y;
      m = max4(du[j], m);
    }
    const float sc_b = pow2_scale(warp_max(m));
    const uint32_t a_qt = ring.wait() + Record::kHdr;
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
    const float* const dc = ring.floats() + Record::kDecay + 2 * (lane & 3);
    const float scale_inv = pow2_inv(sc_do) * pow2_inv(sc_qt) * p.scale;
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      float x0[4] = {}, x1[4] = {};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t bh[4], bl[4];
        load_b_t<128>(a_qt, kk * 16, nb * 16, lane, bh);
        load_b_t<128>(a_qt + Record::kPlane, kk * 16, nb * 16, lane, bl);
        mma2(x0, x1, da[kk], bh, bl);
      }
      const float2 d0 = *reinterpret_cast<const float2*>(dc + nb * 16), d1 = *reinterpret_cast<const float2*>(dc + nb * 16 + 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * nb][e] = fmaf(s[2 * nb][e], e & 1 ? d0.y : d0.x, x0[e] * scale_inv);
        s[2 * nb + 1][e] = fmaf(s[2 * nb + 1][e], e & 1 ? d1.y : d1.x, x1[e] * scale_inv);
      }
    }
    ring.release();
    uint32_t uh[4][4], ul[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a(du[2 * kk], du[2 * kk + 1], sc_b, uh[kk], ul[kk]);
    const uint32_t a_wr = ring.wait();
    if (!(alive = __all_sync(0xffffffffu, ring.ok))) break;
    {
      const float upw = sc_b * sc_wr;
      f = pow2_inv(sc_b) * pow2_inv(sc_wr);
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] *= upw;
#pragma unroll
      for (int nb = 0; nb < 8; ++nb)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t bh[4], bl[4];
          load_b_t<128>(a_wr, kk * 16, nb * 16, lane, bh);
          load_b_t<128>(a_wr + Record::kPlane, kk * 16, nb * 16, lane, bl);
          mma3(s[2 * nb], s[2 * nb + 1], uh[kk], ul[kk], bh, bl);
        }
    }
    ring.release();
  }
  if (!alive) {
    ring.abandon();
    return;
  }
  if (p.d_init != nullptr) store_state(p.d_init + sblk, v0, lane, s, f);
}

}  // namespace kdal
