// kda_scan_chain.cuh -- the scan's sequential kernels: the states from chunk to
// chunk, forwards with the outputs, and their gradients backwards.
//
// Forward, per chunk (see kda_scan_prep.cuh):
//   r = Rt - Wr S0;  U = beta r;  O = scale (Qt S0 + P U);  S1 = Diag(exp(Gamma_C)) S0 + Ke^T U.
// Backward, per chunk in reverse, with the gradient dS1 of its end state:
//   dU = scale P^T dO + Ke dS1
//   dS0 = Diag(exp(Gamma_C)) dS1 + scale Qt^T dO - Wr^T (beta dU).
//
// The value columns are independent: a strip is 16 of them, and a CTA walks the
// chunks with one, two or four strips that share the chunk's tiles (a ring of
// bulk copies).  A strip is four warps, one on each of the SM's schedulers,
// because the chain's latency is what bounds it: one warp a strip, with no
// exchange at all, measured 5.4 us a chunk forward and 7.3 us backward, against
// 1.8 and 2.4 us here (one sequence, 8 heads).  Each warp keeps a quarter of the transposed
// state, S^T [16 x 32 channels], in 16 accumulator registers a thread.  Per
// chunk the warps of a strip exchange twice through shared memory: the sums
// over their channels of S0^T Wr^T (each warp joins those of its 16 tokens),
// then the resulting U^T as MMA fragments.  The accumulator layout of one
// product is the A-operand layout of the next, so nothing is rearranged.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kStageBytes = 2 * Record::kPlane + Record::kHdr;  // 33 KB: two planes and a header
constexpr int kDoPitch = 48;  // bytes per token row of a strip's 16 columns of dO (32 used)

// Exchange buffers of a strip.
struct Strip {
  float4 part[4][3][2][32];  // [from][to, without from][column tile of to's 16 tokens][lane]
  uint4 u[4][2][32];         // U^T fragments per 16 tokens: hi, lo
  uint4 s[4][2][32];         // forward: S^T fragments (hi) per 32 channels
};
struct StripBack {
  float4 part[4][3][2][32];
  uint4 u[4][2][32];
  unsigned char dO[2][kC * kDoPitch];  // this chunk's and the next one's, [t][v] in fp16
  float sc_u[4], sc_do[2][4];
};
struct StripScales {
  float u[4], s[4];
};

template <int STRIPS>
struct ChainCfg {
  static constexpr int kRing = STRIPS == 4 ? 4 : 5;
  static constexpr int kAhead = kRing - 2;  // items copied ahead of the one in use
  struct Common {
    unsigned char stage[kRing][kStageBytes];
    uint64_t full[kRing], empty[kRing];
  };
  struct Forward : Common {
    Strip strip[STRIPS];
    StripScales sc[STRIPS];
  };
  struct Backward : Common {
    StripBack strip[STRIPS];
  };
};

// What a stage holds: up to two pieces of a record.
struct Piece {
  int off0, bytes0, off1, bytes1;
};
// Forward: header and Wr; P (hi) and Qt (hi); header and Ke.
// Backward: header and Ke; P; header and Qt; Wr.
template <bool FWD>
__device__ __forceinline__ Piece piece(int s) {
  if constexpr (FWD) {
    if (s == 0) return Piece{0, Record::kHdr, Record::kWr, 2 * Record::kPlane};
    if (s == 1) return Piece{Record::kP, kC * kC * 2, Record::kQt, Record::kPlane};
    return Piece{0, Record::kHdr, Record::kKe, 2 * Record::kPlane};
  } else {
    if (s == 0) return Piece{0, Record::kHdr, Record::kKe, 2 * Record::kPlane};
    if (s == 1) return Piece{Record::kP, kC * kC * 4, 0, 0};
    if (s == 2) return Piece{0, Record::kHdr, Record::kQt, 2 * Record::kPlane};
    return Piece{Record::kWr, 2 * Record::kPlane, 0, 0};
  }
}

// A warp's place in the ring.  One thread of the CTA also refills it: as it
// comes to an item it starts the copy of the item kAhead further on, into the
// stage that every warp released kRing - kAhead items ago.
template <bool FWD, int STRIPS>
struct Ring {
  using Cfg = ChainCfg<STRIPS>;
  static constexpr int kPer = FWD ? 3 : 4, kRing = Cfg::kRing;
  const ScanParams& p;
  typename Cfg::Common& sm;
  const unsigned char* rec;  // of the next item to copy
  int64_t step;              // to the next chunk's record
  int32_t items, lane;
  bool producer;
  int32_t it = 0, stage = 0, phase = 0;  // the next item to release
  int32_t put = 0, put_stage = 0, put_phase = 0, put_piece = 0;
  bool ok = true;

  __device__ __forceinline__ void fill() {
    if (put >= items) return;
    if (put >= kRing) ok = ok && mbar_wait(&sm.empty[put_stage], static_cast<uint32_t>(put_phase ^ 1));
    if (!ok) return;
    const Piece pc = piece<FWD>(put_piece);
    mbar_expect(&sm.full[put_stage], static_cast<uint32_t>(pc.bytes0 + pc.bytes1));
    bulk_load(sm.stage[put_stage], rec + pc.off0, static_cast<uint32_t>(pc.bytes0), &sm.full[put_stage]);
    if (pc.bytes1)
      bulk_load(sm.stage[put_stage] + pc.bytes0, rec + pc.off1, static_cast<uint32_t>(pc.bytes1), &sm.full[put_stage]);
    ++put;
    if (++put_stage == kRing) {
      put_stage = 0;
      put_phase ^= 1;
    }
    if (++put_piece == kPer) {
      put_piece = 0;
      rec += step;
    }
  }
  __device__ __forceinline__ void start() {
    if (producer)
      for (int j = 0; j < Cfg::kAhead; ++j) fill();
  }
  // The current item, once it is there.  A warp whose wait gave up goes on without waiting, so that the strip's barriers
  // stay matched; `ok` is uniform over the warp.
  __device__ __forceinline__ const unsigned char* wait() {
    if (producer) fill();
    ok = ok && mbar_wait(&sm.full[stage], static_cast<uint32_t>(phase));
    ok = __all_sync(0xffffffffu, ok);
    return sm.stage[stage];
  }
  __device__ __forceinline__ void release() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[stage]);
    ++it;
    if (++stage == kRing) {
      stage = 0;
      phase ^= 1;
    }
  }
  // After a wait that gave up: the CTA must not end with copies into it in flight.
  __device__ __forceinline__ void abandon() {
    if (lane == 0) set_error(p);
    if (producer)
      for (int32_t j = put > kRing ? put - kRing : 0; j < put; ++j)
        mbar_wait(&sm.full[j % kRing], static_cast<uint32_t>((j / kRing) & 1));
  }
};

template <typename Common>
__device__ __forceinline__ void chain_init(Common& sm, int ring, int warps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], warps);
    }
    mbar_fence_init();
  }
  __syncthreads();
}
// Barrier of a strip's four warps.
__device__ __forceinline__ void strip_sync(int strip) { asm volatile("bar.sync %0, 128;" ::"r"(strip + 1) : "memory"); }

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
__device__ __forceinline__ uint4 vec(const uint32_t (&a)[4]) { return make_uint4(a[0], a[1], a[2], a[3]); }
__device__ __forceinline__ void unvec(uint4 v, uint32_t (&a)[4]) {
  a[0] = v.x;
  a[1] = v.y;
  a[2] = v.z;
  a[3] = v.w;
}

// 16 value columns x 32 channels of a [K][V] block in the accumulator layout: element (v, i).
__device__ __forceinline__ void load_state(const float* blk, int v0, int i0, int lane, float (&s)[4][4]) {
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[n][e] = blk == nullptr ? 0.f : blk[(i0 + n * 8 + 2 * (lane & 3) + (e & 1)) * kV + v0 + (lane >> 2) + (e >> 1) * 8];
}
__device__ __forceinline__ void store_state(float* blk, int v0, int i0, int lane, const float (&s)[4][4]) {
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      blk[(i0 + n * 8 + 2 * (lane & 3) + (e & 1)) * kV + v0 + (lane >> 2) + (e >> 1) * 8] = s[n][e];
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

// The sums over a warp's 32 channels, S^T [16 x 32] B^T [32 x 64 tokens] with B a pair tile [t][i], in true units.
__device__ __forceinline__ void channel_sums(uint32_t tile, int i0, int lane, const uint32_t (&ah)[2][4], const uint32_t (&al)[2][4],
                                             float inv, float (&x)[8][4]) {
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    uint32_t bh[2][4], bl[2][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      load_b<128>(tile, i0 + kk * 16, nb * 16, lane, bh[kk]);
      load_b<128>(tile + Record::kPlane, i0 + kk * 16, nb * 16, lane, bl[kk]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * nb][e] = x[2 * nb + 1][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      mma_pair(x[2 * nb], x[2 * nb + 1], ah[kk], bl[kk]);
      mma_pair(x[2 * nb], x[2 * nb + 1], al[kk], bh[kk]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) mma_pair(x[2 * nb], x[2 * nb + 1], ah[kk], bh[kk]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * nb][e] *= inv;
      x[2 * nb + 1][e] *= inv;
    }
  }
}
// Hands each warp of the strip the sums of its 16 tokens.
__device__ __forceinline__ void put_sums(float4 (&part)[4][3][2][32], int quarter, int lane, const float (&x)[8][4]) {
#pragma unroll
  for (int to = 0; to < 4; ++to)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (to != quarter) {
        const float(&c)[4] = x[2 * to + j];
        part[quarter][to > quarter ? to - 1 : to][j][lane] = make_float4(c[0], c[1], c[2], c[3]);
      }
}
// This warp's tokens: its own sums and the other three warps', in a fixed order.
__device__ __forceinline__ void take_sums(const float4 (&part)[4][3][2][32], int quarter, int lane, const float (&x)[8][4],
                                          float (&own)[2][4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float4 c[4];
#pragma unroll
    for (int from = 0; from < 4; ++from) {
      c[from] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from != quarter) c[from] = part[from][quarter > from ? quarter - 1 : quarter][j][lane];
    }
#pragma unroll
    for (int to = 0; to < 4; ++to)
      if (to == quarter) {
        const float(&m)[4] = x[2 * to + j];
        c[to] = make_float4(m[0], m[1], m[2], m[3]);
      }
    own[j][0] = (c[0].x + c[1].x) + (c[2].x + c[3].x);
    own[j][1] = (c[0].y + c[1].y) + (c[2].y + c[3].y);
    own[j][2] = (c[0].z + c[1].z) + (c[2].z + c[3].z);
    own[j][3] = (c[0].w + c[1].w) + (c[2].w + c[3].w);
  }
}
// s += f U^T [16 x 16 tokens] B [16 tokens x 32 channels] with B a pair tile [t][i].
template <bool PAIR>
__device__ __forceinline__ void add_outer(uint32_t tile, int t0, int i0, int lane, const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          float f, float (&s)[4][4]) {
#pragma unroll
  for (int nb = 0; nb < 2; ++nb) {
    uint32_t bh[4], bl[4];
    load_b_t<128>(tile, t0, i0 + nb * 16, lane, bh);
    load_b_t<128>(tile + Record::kPlane, t0, i0 + nb * 16, lane, bl);
    float x0[4] = {}, x1[4] = {};
    mma_pair(x0, x1, ah, bl);
    if constexpr (PAIR) mma_pair(x0, x1, al, bh);
    mma_pair(x0, x1, ah, bh);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[2 * nb][e] = fmaf(x0[e], f, s[2 * nb][e]);
      s[2 * nb + 1][e] = fmaf(x1[e], f, s[2 * nb + 1][e]);
    }
  }
}
// s = s Diag(exp(Gamma_C)) for the warp's channels.
__device__ __forceinline__ void decay_state(const float* decay, int lane, float (&s)[4][4]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 d = *reinterpret_cast<const float2*>(decay + n * 8 + 2 * (lane & 3));
    s[n][0] *= d.x;
    s[n][1] *= d.y;
    s[n][2] *= d.x;
    s[n][3] *= d.y;
  }
}

template <int STRIPS>
__global__ void __launch_bounds__(STRIPS * 128, 1) kda_scan_forward_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<typename ChainCfg<STRIPS>::Forward*>(smem_raw);
  constexpr int kTiles = 8 / STRIPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, strip = warp >> 2, quarter = warp & 3;
  const int64_t unit = blockIdx.x / kTiles;
  const int group = static_cast<int>(blockIdx.x - unit * kTiles) * STRIPS + strip;  // 16 value columns
  const int64_t n = unit / p.HV, h = unit - n * p.HV;
  int64_t start, len;
  seq_range(p, n, start, len);
  const int32_t nch = static_cast<int32_t>((len + kC - 1) / kC);
  const int64_t slot0 = first_slot(p, n, start), blk = state_block(p, n);
  const int v0 = group * 16, i0 = quarter * 32, t0 = quarter * 16;
  if (blk < 0) {  // inactive: zero outputs
    for (int64_t t = quarter * 32 + lane; t < len * 2; t += 128)
      *reinterpret_cast<uint4*>(p.out + (start + (t >> 1)) * p.out_ts + h * kV + v0 + (t & 1) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  chain_init(sm, ChainCfg<STRIPS>::kRing, STRIPS * 4);
  Strip& st = sm.strip[strip];
  StripScales& sc = sm.sc[strip];
  const int64_t sblk = (blk * p.HV + h) * kK * kV, step = p.HV * p.rec_bytes;
  unsigned char* rec = record(p, slot0, h);
  Ring<true, STRIPS> ring{p, sm, rec, step, nch * 3, lane, threadIdx.x == 0};
  ring.start();
  float s[4][4];
  load_state(p.s_in == nullptr ? nullptr : p.s_in + sblk, v0, i0, lane, s);
  for (int32_t c = 0; c < nch; ++c, rec += step) {
    const int tc = static_cast<int>(len - static_cast<int64_t>(c) * kC < kC ? len - static_cast<int64_t>(c) * kC : kC);
    float2 rt[2][2];  // Rt^T of this warp's tokens, needed after the first product
    {
      const float* const src = reinterpret_cast<const float*>(rec + Record::kRt) + (v0 + (lane >> 2)) * kC + t0 + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rt[j][0] = *reinterpret_cast<const float2*>(src + j * 8);
        rt[j][1] = *reinterpret_cast<const float2*>(src + 8 * kC + j * 8);
      }
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max4(s[j], m);
    const float sc_s = pow2_scale(warp_max(m));
    uint32_t ah[2][4], al[2][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      frag_a(s[2 * kk], s[2 * kk + 1], sc_s, ah[kk], al[kk]);
      st.s[quarter][kk][lane] = vec(ah[kk]);
    }
    // ---- the sums of S0^T Wr^T over this warp's channels, to the warps of their tokens
    float x[8][4];
    const unsigned char* const wr = ring.wait();
    const float* const hdr = reinterpret_cast<const float*>(wr);
    const float sc_qt = hdr[Record::kScQt], sc_p = hdr[Record::kScP], sc_ke = hdr[Record::kScKe];
    channel_sums(smem_addr(wr) + Record::kHdr, i0, lane, ah, al, pow2_inv(sc_s) * pow2_inv(hdr[Record::kScWr]), x);
    put_sums(st.part, quarter, lane, x);
    if (lane == 0) sc.s[quarter] = sc_s;
    if (p.save) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        store_frag<128>(rec + Record::kS, kV * kK * 2, v0, i0 + kk * 16, lane, ah[kk], al[kk]);
    }
    float2 beta[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) beta[j] = *reinterpret_cast<const float2*>(hdr + Record::kBeta + t0 + j * 8 + 2 * (lane & 3));
    ring.release();
    strip_sync(strip);
    // ---- r^T and U^T of this warp's tokens
    float r[2][4];
    take_sums(st.part, quarter, lane, x, r);
    float mr = 0.f, mu = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r[j][0] = rt[j][0].x - r[j][0];
      r[j][1] = rt[j][0].y - r[j][1];
      r[j][2] = rt[j][1].x - r[j][2];
      r[j][3] = rt[j][1].y - r[j][3];
      mr = max4(r[j], mr);
    }
    float u[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[j][e] = r[j][e] * (e & 1 ? beta[j].y : beta[j].x);
      mu = max4(u[j], mu);
    }
    {
      const float sc_u = pow2_scale(warp_max(mu));
      uint32_t uh[4], ul[4];
      frag_a(u[0], u[1], sc_u, uh, ul);
      st.u[quarter][0][lane] = vec(uh);
      st.u[quarter][1][lane] = vec(ul);
      if (lane == 0) sc.u[quarter] = sc_u;
    }
    // ---- O^T = scale (S0^T Qt^T + U^T P^T), this warp's tokens (one fp16 product: it is rounded to bf16)
    const uint32_t a_p = smem_addr(ring.wait()), a_qt = a_p + kC * kC * 2;
    float o[2][4] = {};
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
      float y[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t a[4], b[4];
        unvec(st.s[qd][kk][lane], a);
        load_b<128>(a_qt, qd * 32 + kk * 16, t0, lane, b);
        mma_pair(y[0], y[1], a, b);
      }
      const float f = pow2_inv(sc.s[qd]) * pow2_inv(sc_qt);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = fmaf(y[j][e], f, o[j][e]);
    }
    strip_sync(strip);
    // ---- S1^T = S0^T Diag(exp(Gamma_C)) + U^T Ke
    const bool out = p.out != nullptr;
    uint32_t uh[4][4], ul[4][4];
    float fu[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      unvec(st.u[kk][0][lane], uh[kk]);
      unvec(st.u[kk][1][lane], ul[kk]);
      fu[kk] = pow2_inv(sc.u[kk]);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      if (kk <= quarter) {
        float y[2][4] = {};
        uint32_t b[4];
        load_b<64>(a_p, kk * 16, t0, lane, b);
        mma_pair(y[0], y[1], uh[kk], b);
        const float f = fu[kk] * pow2_inv(sc_p);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = fmaf(y[j][e], f, o[j][e]);
      }
    ring.release();
    const unsigned char* const ke = ring.wait();
    decay_state(reinterpret_cast<const float*>(ke) + Record::kDecay + i0, lane, s);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      add_outer<true>(smem_addr(ke) + Record::kHdr, kk * 16, i0, lane, uh[kk], ul[kk], fu[kk] * pow2_inv(sc_ke), s);
    ring.release();
    if (out) store_out16(p.out + (start + static_cast<int64_t>(c) * kC) * p.out_ts + h * kV + v0, p.out_ts, t0, tc, lane, o[0], o[1], p.scale);
    if (p.save) {
      const float sc_r = pow2_scale(warp_max(mr));
      uint32_t rh[4], rl[4];
      frag_a(r[0], r[1], sc_r, rh, rl);
      store_frag<64>(rec + Record::kR, Record::kPlane, v0, t0, lane, rh, rl);
      if (lane == 0) {
        float* const scales = reinterpret_cast<float*>(rec + Record::kSc);
        scales[Record::kScS + group * 4 + quarter] = sc_s;
        scales[Record::kScR + group * 4 + quarter] = sc_r;
      }
    }
  }
  if (!ring.ok) {  // a copy never came: the state is not written
    ring.abandon();
    return;
  }
  if (p.s_out != nullptr) store_state(p.s_out + sblk, v0, i0, lane, s);
}

// ---------------------------------------------------------------- backward
template <int STRIPS>
__global__ void __launch_bounds__(STRIPS * 128, 1) kda_scan_backward_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<typename ChainCfg<STRIPS>::Backward*>(smem_raw);
  constexpr int kTiles = 8 / STRIPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, strip = warp >> 2, quarter = warp & 3;
  const int64_t unit = blockIdx.x / kTiles;
  const int group = static_cast<int>(blockIdx.x - unit * kTiles) * STRIPS + strip;
  const int64_t n = unit / p.HV, h = unit - n * p.HV;
  int64_t start, len;
  seq_range(p, n, start, len);
  const int32_t nch = static_cast<int32_t>((len + kC - 1) / kC);
  const int64_t slot0 = first_slot(p, n, start);
  const int v0 = group * 16, i0 = quarter * 32, t0 = quarter * 16;
  chain_init(sm, ChainCfg<STRIPS>::kRing, STRIPS * 4);
  StripBack& st = sm.strip[strip];
  const int64_t sblk = (n * p.HV + h) * kK * kV, step = p.HV * p.rec_bytes;
  unsigned char* rec = record(p, slot0 + (nch > 0 ? nch - 1 : 0), h);
  Ring<false, STRIPS> ring{p, sm, rec, -step, nch * 4, lane, threadIdx.x == 0};
  ring.start();
  float s[4][4];
  load_state(p.d_final == nullptr ? nullptr : p.d_final + sblk, v0, i0, lane, s);

  // dO, one 16-byte piece a thread (this warp: its 16 tokens), exact in fp16 after scaling: bf16 has 8 bits
  const int dt = t0 + (lane >> 1), dh = lane & 1;
  auto fetch = [&](int32_t c) {
    const int64_t t = static_cast<int64_t>(c) * kC + dt;
    return c >= 0 && t < len ? *reinterpret_cast<const uint4*>(p.d_out + (start + t) * p.d_out_ts + h * kV + v0 + dh * 8)
                             : make_uint4(0, 0, 0, 0);
  };
  auto put_do = [&](uint4 raw, int buf) {
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    const float sc = pow2_scale(warp_max(m));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = as_u32(__floats2half2_rn(__uint_as_float(w[e] << 16) * sc, __uint_as_float(w[e] & 0xffff0000u) * sc));
    *reinterpret_cast<uint4*>(st.dO[buf] + dt * kDoPitch + dh * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane == 0) st.sc_do[buf][quarter] = sc;
  };
  put_do(fetch(nch - 1), (nch - 1) & 1);
  strip_sync(strip);

  for (int32_t c = nch - 1; c >= 0; --c, rec -= step) {
    const uint4 next_do = fetch(c - 1);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max4(s[j], m);
    const float sc_s = pow2_scale(warp_max(m));
    uint32_t ah[2][4], al[2][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      frag_a(s[2 * kk], s[2 * kk + 1], sc_s, ah[kk], al[kk]);
      store_frag<128>(rec + Record::kDS, kV * kK * 2, v0, i0 + kk * 16, lane, ah[kk], al[kk]);
    }
    // ---- the sums of dS1^T Ke^T over this warp's channels, to the warps of their tokens
    float x[8][4];
    const unsigned char* const ke = ring.wait();
    const float* const hdr = reinterpret_cast<const float*>(ke);
    const float sc_p = hdr[Record::kScP], sc_qt = hdr[Record::kScQt], sc_wr = hdr[Record::kScWr];
    channel_sums(smem_addr(ke) + Record::kHdr, i0, lane, ah, al, pow2_inv(sc_s) * pow2_inv(hdr[Record::kScKe]), x);
    put_sums(st.part, quarter, lane, x);
    float2 beta[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) beta[j] = *reinterpret_cast<const float2*>(hdr + Record::kBeta + t0 + j * 8 + 2 * (lane & 3));
    ring.release();
    // ---- scale dO^T P of this warp's tokens
    uint32_t da[4][4];
    float fd[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      ldsm4t(smem_addr(st.dO[c & 1]) + (kk * 16 + (lane & 7) + (lane >> 4) * 8) * kDoPitch + ((lane >> 3) & 1) * 16, da[kk]);
      fd[kk] = pow2_inv(st.sc_do[c & 1][kk]) * p.scale;
    }
    const uint32_t a_p = smem_addr(ring.wait());
    float du[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)  // t sub-block; P[t][s] is zero for s > t
      if (kk >= quarter) {
        uint32_t bh[4], bl[4];
        load_b_t<64>(a_p, kk * 16, t0, lane, bh);
        load_b_t<64>(a_p + kC * kC * 2, kk * 16, t0, lane, bl);
        float y[2][4] = {};
        mma_pair(y[0], y[1], da[kk], bl);
        mma_pair(y[0], y[1], da[kk], bh);
        const float f = fd[kk] * pow2_inv(sc_p);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) du[j][e] = fmaf(y[j][e], f, du[j][e]);
      }
    ring.release();
    strip_sync(strip);
    // ---- dU^T of this warp's tokens; -beta dU^T to the strip
    float own[2][4], m2 = 0.f;
    take_sums(st.part, quarter, lane, x, own);
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        du[j][e] += own[j][e];
        own[j][e] = -du[j][e] * (e & 1 ? beta[j].y : beta[j].x);
      }
      m = max4(du[j], m);
      m2 = max4(own[j], m2);
    }
    {
      const float sc_u = pow2_scale(warp_max(m2));
      uint32_t uh[4], ul[4];
      frag_a(own[0], own[1], sc_u, uh, ul);
      st.u[quarter][0][lane] = vec(uh);
      st.u[quarter][1][lane] = vec(ul);
      if (lane == 0) st.sc_u[quarter] = sc_u;
    }
    put_do(next_do, (c & 1) ^ 1);
    // ---- dS0^T = dS1^T Diag(exp(Gamma_C)) + scale dO^T Qt - (beta dU)^T Wr
    const unsigned char* const qt = ring.wait();
    decay_state(reinterpret_cast<const float*>(qt) + Record::kDecay + i0, lane, s);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      add_outer<false>(smem_addr(qt) + Record::kHdr, kk * 16, i0, lane, da[kk], da[kk], fd[kk] * pow2_inv(sc_qt), s);
    ring.release();
    strip_sync(strip);
    const uint32_t a_wr = smem_addr(ring.wait());
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t uh[4], ul[4];
      unvec(st.u[kk][0][lane], uh);
      unvec(st.u[kk][1][lane], ul);
      add_outer<true>(a_wr, kk * 16, i0, lane, uh, ul, pow2_inv(st.sc_u[kk]) * pow2_inv(sc_wr), s);
    }
    ring.release();
    {
      const float sc_du = pow2_scale(warp_max(m));
      uint32_t uh[4], ul[4];
      frag_a(du[0], du[1], sc_du, uh, ul);
      store_frag<64>(rec + Record::kDU, Record::kPlane, v0, t0, lane, uh, ul);
      if (lane == 0) {
        float* const scales = reinterpret_cast<float*>(rec + Record::kSc);
        scales[Record::kScDS + group * 4 + quarter] = sc_s;
        scales[Record::kScDU + group * 4 + quarter] = sc_du;
      }
    }
  }
  if (!ring.ok) {
    ring.abandon();
    return;
  }
  if (p.d_init != nullptr) store_state(p.d_init + sblk, v0, i0, lane, s);
}

}  // namespace kdal
