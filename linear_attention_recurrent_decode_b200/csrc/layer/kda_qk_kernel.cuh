// kda_qk_kernel.cuh -- per-head norm of queries and keys with the position
// rotation, and its gradients.
//
// Forward per row and head: n = x i w with i = rsqrt(sum x^2 (/ D) + eps), then
// each pair (a, b) of the first rot components to (a c - b s, a s + b c).
// Backward from dy: the rotation's transpose turns back, g; then with x^ = x i
//   dw = sum over rows and heads of g x^,   dx = i (g w - x^ sum(g w x^) (/ D)).
//
// What bounds it: device memory, one read and one write of every element; next
// the instructions, and of those the angles'.  A thread holds 8 components (16
// bytes) of a head, the head's threads are a power of two of neighbouring lanes
// (unused ones idle for D = 96), sums go by shuffles.  A tile is 256 threads'
// heads, VPT each, of one tensor; its rows' cos and sin are computed once, in
// shared memory, and shared by all heads, while the loads are in flight.
//
// Measured (B200, 16384 rows, D = 128): forward, 32 + 32 heads rotated in
// interleaved pairs, 98 us, 5.5 TB/s (0.83 of the measured copy rate); 32 + 8
// heads with weights in halves 75 us (0.68; 0.86 of the issue slots), without
// rotation 52 us (0.97).  Four heads a thread and five blocks an SM against 81,
// 80 and 74 us (32 + 8 heads) for three, five and six heads.  Backward with
// weights, 32 + 8 heads, 131 us, 3.8 TB/s, 0.72 of the issue slots; without
// rotation 96.  Two heads a thread and four blocks an SM against 138 and 157 us
// for three and five blocks; three heads are alike; loading the next tile ahead
// of computing one, or its angles, was slower.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kdal {

constexpr int kQkThreads = 256;
constexpr int kQkMaxCtas = 1024;  // of the backward pass: rows of its partial sums
constexpr int kQkBackwardCtas = 4;  // an SM

struct QkTensor {
  const __nv_bfloat16* x; int64_t x_ts;
  __nv_bfloat16* y; int64_t y_ts;          // forward output, or dx
  const __nv_bfloat16* dy; int64_t dy_ts;
  const __nv_bfloat16* w;
  float* dw;
  int64_t items;                           // rows * heads
  int64_t tiles;
  uint64_t div64;                          // ceil(2^64 / heads) and ceil(2^32 / heads), 0 for one head: an item's row by
  uint32_t div32;                          // a multiplication (exact: see kMaxHeads); a division cost 50 instructions a head
  int32_t heads, ctas;                     // ctas: blocks that share the tiles
};
// The quotient by multiplication is exact while n heads < 2^32 (or 2^64): n is below heads + 1024 in 32 bits, below 2^51
// in 64.
constexpr int kMaxHeads = 4096;
struct QkParams {
  QkTensor t[2];
  const void* pos;
  const double* freq;
  float* partial;          // [ctas][D]: sums for dw
  int64_t rows;
  int32_t D, rot, lanes;   // lanes: log2 of a head's threads
  int32_t norm, pos64;
  float eps, scale, inv_d; // inv_d: 1 / D for the mean, 1 for the sum
};
enum QkRotate { kQkNone, kQkHalves, kQkInterleaved };

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Sum over the 2^LANES neighbouring lanes of a head.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = 1; o < (1 << LANES); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of rows row0 .. row0 + span - 1, [span][rot / 2], a row's pairs in the order [pair of pairs of a thread]
// [thread][2], so that neighbouring lanes read neighbouring 16 bytes (in pair order they met in two of the banks).  The angle is
// position * inv_freq in fp64, taken in half turns and reduced to one turn
// there; cos and sin then see an argument exact to fp32.
__device__ __forceinline__ void qk_table(const QkParams& p, int64_t row0, int span, float2* tab) {
  const int half = p.rot >> 1;
  for (int e = threadIdx.x; e < span * half; e += kQkThreads) {
    const int r = e / half, i = e - r * half;
    const int64_t row = row0 + r;
    if (row >= p.rows) break;
    const double pos = p.pos64 ? static_cast<double>(static_cast<const int64_t*>(p.pos)[row])
                               : static_cast<double>(static_cast<const int32_t*>(p.pos)[row]);
    double u = pos * p.freq[i] * 0.318309886183790671538;  // 1 / pi
    u -= 2.0 * rint(0.5 * u);
    float s, c;
    sincospif(static_cast<float>(u), &s, &c);
    const int at = ((((i & 3) >> 1) * (half >> 2) + (i >> 2)) << 1) + (i & 1);  // four pairs of a thread
    tab[r * half + at] = make_float2(c * p.scale, s * p.scale);
  }
}

// Where a thread's 8 components lie in a head, four and four.  Neighbours but for the halves' layout, where both
// partners of a pair are the same thread's: with 8 neighbours each, trading them by shuffles was 10 % of the time.
template <QkRotate ROT>
struct QkPlace {
  int32_t o0, o1;
  __device__ __forceinline__ QkPlace(const QkParams& p, int l) {
    const bool apart = ROT == kQkHalves && l * 8 < p.rot;
    o0 = apart ? l * 4 : l * 8;
    o1 = apart ? (p.rot >> 1) + l * 4 : l * 8 + 4;
  }
  __device__ __forceinline__ uint4 load(const __nv_bfloat16* head) const {
    if constexpr (ROT != kQkHalves) return *reinterpret_cast<const uint4*>(head + o0);
    const uint2 a = *reinterpret_cast<const uint2*>(head + o0), b = *reinterpret_cast<const uint2*>(head + o1);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* head, uint4 x) const {
    if constexpr (ROT != kQkHalves) {
      *reinterpret_cast<uint4*>(head + o0) = x;
    } else {
      *reinterpret_cast<uint2*>(head + o0) = make_uint2(x.x, x.y);
      *reinterpret_cast<uint2*>(head + o1) = make_uint2(x.z, x.w);
    }
  }
};

// This thread's 8 components turned by the row's angles (cs: its row of the table), backwards if BACK.
template <QkRotate ROT, bool BACK>
__device__ __forceinline__ void qk_rotate(const QkParams& p, const float2* cs, int l, float (&f)[8]) {
  if (ROT == kQkNone || l * 8 >= p.rot) return;
  const float4* const t4 = reinterpret_cast<const float4*>(cs) + l;
  constexpr int kA = ROT == kQkHalves ? 1 : 2, kB = ROT == kQkHalves ? 4 : 1;  // pair i: components kA i and kA i + kB
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 t = t4[e * (p.rot >> 3)];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float c = i ? t.z : t.x, s = BACK ? -(i ? t.w : t.y) : (i ? t.w : t.y);
      float &x = f[kA * (2 * e + i)], &y = f[kA * (2 * e + i) + kB];
      const float a = x, b = y;
      x = a * c - b * s;
      y = a * s + b * c;
    }
  }
}

// A thread's heads of a tile: the tile starts `rem` heads into row row0.
template <int LANES, int VPT>
struct QkTile {
  static constexpr int kGroups = kQkThreads >> LANES;
  int64_t row0;
  int32_t rem, r[VPT], head[VPT];  // row within the tile, head
  bool in[VPT];
  __device__ __forceinline__ QkTile(const QkTensor& t, int64_t tile, int grp, bool used) {
    const int64_t item0 = tile * (kGroups * VPT);
    row0 = t.div64 ? static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(item0), t.div64)) : item0;
    rem = static_cast<int32_t>(item0 - row0 * t.heads);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = grp + j * kGroups;
      in[j] = used && item0 + i < t.items;
      const uint32_t at = in[j] ? static_cast<uint32_t>(rem + i) : 0u;  // the table has no rows behind the last one
      r[j] = static_cast<int32_t>(t.div32 ? __umulhi(at, t.div32) : at);
      head[j] = static_cast<int32_t>(at) - r[j] * t.heads;
    }
  }
  __device__ __forceinline__ int span(const QkTensor& t) const {
    const uint32_t last = static_cast<uint32_t>(rem + kGroups * VPT - 1);
    return static_cast<int>(t.div32 ? __umulhi(last, t.div32) : last) + 1;
  }
};

template <QkRotate ROT, int LANES, int VPT>
__global__ void __launch_bounds__(kQkThreads, 5) kda_qk_forward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) float2 tab[];
  const int which = blockIdx.x >= p.t[0].tiles;
  const QkTensor& t = p.t[which];
  const int grp = threadIdx.x >> LANES, l = threadIdx.x & ((1 << LANES) - 1);
  const bool used = l * 8 < p.D;
  const QkTile<LANES, VPT> it(t, static_cast<int64_t>(blockIdx.x) - (which ? p.t[0].tiles : 0), grp, used);
  const QkPlace<ROT> at(p, l);
  const __nv_bfloat16* const xb = t.x + it.row0 * t.x_ts;
  __nv_bfloat16* const yb = t.y + it.row0 * t.y_ts;
  uint4 x[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    x[j] = it.in[j] ? at.load(xb + it.r[j] * t.x_ts + it.head[j] * p.D) : make_uint4(0, 0, 0, 0);
  float w[8];
  const bool weighted = t.w != nullptr;
  if (weighted && used) unpack8(at.load(t.w), w);
  if constexpr (ROT != kQkNone) {
    qk_table(p, it.row0, it.span(t), tab);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float f[8];
    unpack8(x[j], f);
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
      const float inv = rsqrtf(fmaf(head_sum<LANES>(ss), p.inv_d, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
      if (weighted) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w[e];
      }
    }
    qk_rotate<ROT, false>(p, tab + it.r[j] * (p.rot >> 1), l, f);
    if (it.in[j]) at.store(yb + it.r[j] * t.y_ts + it.head[j] * p.D, pack8(f));
  }
}

// Blocks [0, t[0].ctas) walk q's tiles, the rest k's, so that a thread sums dw's contributions of its 8 components in
// registers; a block then leaves one row of partial sums.
template <QkRotate ROT, int LANES, int VPT>
__global__ void __launch_bounds__(kQkThreads, kQkBackwardCtas) kda_qk_backward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) float2 tab[];
  constexpr int kGroups = kQkThreads >> LANES;
  const int which = blockIdx.x >= p.t[0].ctas;
  const QkTensor& t = p.t[which];
  const int grp = threadIdx.x >> LANES, l = threadIdx.x & ((1 << LANES) - 1);
  const bool used = l * 8 < p.D, weighted = t.w != nullptr;
  const QkPlace<ROT> at(p, l);
  float w[8], dw[8] = {};
  if (weighted && used) unpack8(at.load(t.w), w);
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) - (which ? p.t[0].ctas : 0); tile < t.tiles; tile += t.ctas) {
    const QkTile<LANES, VPT> it(t, tile, grp, used);
    const __nv_bfloat16* const xb = t.x + it.row0 * t.x_ts;
    const __nv_bfloat16* const db = t.dy + it.row0 * t.dy_ts;
    __nv_bfloat16* const yb = t.y + it.row0 * t.y_ts;
    uint4 x[VPT], dy[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      x[j] = dy[j] = make_uint4(0, 0, 0, 0);
      if (it.in[j]) {
        if (p.norm) x[j] = at.load(xb + it.r[j] * t.x_ts + it.head[j] * p.D);
        dy[j] = at.load(db + it.r[j] * t.dy_ts + it.head[j] * p.D);
      }
    }
    if constexpr (ROT != kQkNone) {
      qk_table(p, it.row0, it.span(t), tab);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[8], g[8];
      unpack8(dy[j], g);
      qk_rotate<ROT, true>(p, tab + it.r[j] * (p.rot >> 1), l, g);
      if (p.norm) {
        unpack8(x[j], f);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        const float inv = rsqrtf(fmaf(head_sum<LANES>(ss), p.inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;  // x^
        if (weighted) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (it.in[j]) dw[e] = fmaf(g[e], f[e], dw[e]);
            g[e] *= w[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sg = fmaf(g[e], f[e], sg);
        sg = head_sum<LANES>(used ? sg : 0.f) * p.inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = inv * fmaf(-f[e], sg, g[e]);
      }
      if (it.in[j]) at.store(yb + it.r[j] * t.y_ts + it.head[j] * p.D, pack8(g));
    }
    if constexpr (ROT != kQkNone) __syncthreads();  // the table is rewritten
  }
  if (t.dw == nullptr) return;
  float* const red = reinterpret_cast<float*>(tab);  // [groups][D]
  if (used) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[grp * p.D + (e < 4 ? at.o0 + e : at.o1 + e - 4)] = dw[e];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kQkThreads) {
    float s = 0.f;
    for (int i = 0; i < kGroups; ++i) s += red[i * p.D + d];
    p.partial[static_cast<int64_t>(blockIdx.x) * p.D + d] = s;
  }
}

// dw from the blocks' partial sums: one block a tensor and 32 components, thread (component, part of the blocks).
__global__ void __launch_bounds__(1024) kda_qk_weight_kernel(const __grid_constant__ QkParams p) {
  __shared__ double part[32][33];
  const QkTensor& t = p.t[blockIdx.y];
  if (t.dw == nullptr) return;
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, d = blockIdx.x * 32 + c;
  const int first = blockIdx.y ? p.t[0].ctas : 0;
  double s = 0.0;
  if (d < p.D)
    for (int i = w; i < t.ctas; i += 32) s += static_cast<double>(p.partial[static_cast<int64_t>(first + i) * p.D + d]);
  part[w][c] = s;
  __syncthreads();
  if (w == 0 && d < p.D) {
    for (int i = 1; i < 32; ++i) s += part[i][c];
    t.dw[d] = static_cast<float>(s);
  }
}

}  // namespace kdal
