// kda_qk_kernel.cuh -- per-head norm of queries and keys with the position
// rotation, and its gradients.
//
// Forward per row and head: n = x i w with i = rsqrt(sum x^2 (/ D) + eps), then
// each pair (a, b) of the first rot components to (a c - b s, a s + b c).
// Backward from dy: the rotation's transpose turns back, g; then with x^ = x i
//   dw = sum over rows and heads of g x^,   dx = i (g w - x^ sum(g w x^) (/ D)).
//
// What bounds it: device memory, one read and one write of every element.  A
// thread holds 8 components (16 bytes) of a head, the head's threads are a
// power of two of neighbouring lanes (unused ones idle for D = 96), sums and
// the halves' partners go by shuffles.  A tile is 256 threads' heads, VPT each,
// of one tensor; its rows' cos and sin are computed once, in shared memory, and
// shared by all heads, while the loads are in flight.  VPT = 4 keeps four loads
// in flight a thread; with few heads (fewer tiles than twice the SMs) VPT = 1
// spreads them over more of the SMs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kdal {

constexpr int kQkThreads = 256;
constexpr int kQkMaxCtas = 1024;  // of the backward pass: rows of its partial sums

struct QkTensor {
  const __nv_bfloat16* x; int64_t x_ts;
  __nv_bfloat16* y; int64_t y_ts;          // forward output, or dx
  const __nv_bfloat16* dy; int64_t dy_ts;
  const __nv_bfloat16* w;
  float* dw;
  int64_t items;                           // rows * heads
  int64_t tiles;
  int32_t heads, ctas;                     // ctas: blocks that share the tiles
};
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
// Sum over the 2^lanes neighbouring lanes of a head.
__device__ __forceinline__ float head_sum(float x, int lanes) {
  for (int o = 1; o < (1 << lanes); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of rows row0 .. row0 + span - 1, [span][rot / 2].  The angle is
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
    tab[e] = make_float2(c * p.scale, s * p.scale);
  }
}

// This thread's 8 components turned by the row's angles (cs: its row of the table); sign -1 turns back.
template <QkRotate ROT>
__device__ __forceinline__ void qk_rotate(const QkParams& p, const float2* cs, int l, float sign, float (&f)[8]) {
  if constexpr (ROT == kQkInterleaved) {
    if (l * 8 >= p.rot) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = cs[l * 4 + e];
      const float s = sign * t.y, a = f[2 * e], b = f[2 * e + 1];
      f[2 * e] = a * t.x - b * s;
      f[2 * e + 1] = a * s + b * t.x;
    }
  } else if constexpr (ROT == kQkHalves) {
    const int hv = p.rot >> 4;  // threads of a half
    const bool first = l < hv, in = l < 2 * hv;
    const int lane = threadIdx.x & 31, from = in ? (first ? lane + hv : lane - hv) : lane;
    float other[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = __shfl_sync(0xffffffffu, f[e], from);
    if (!in) return;
    const float sg = first ? -sign : sign;
    const float2* const t = cs + (first ? l : l - hv) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * t[e].x + sg * t[e].y * other[e];
  }
}

// The items of a tile that this thread takes part in.
struct QkItem {
  int64_t row;
  int32_t r, head;  // row within the tile, head
  bool in;
};
__device__ __forceinline__ QkItem qk_item(const QkTensor& t, int64_t item0, int64_t row0, int rem, int i, bool used) {
  QkItem it;
  it.r = (rem + i) / t.heads;
  it.head = rem + i - it.r * t.heads;
  it.row = row0 + it.r;
  it.in = used && item0 + i < t.items;
  if (!it.in) it.r = 0;  // the table has no rows behind the last one
  return it;
}

template <QkRotate ROT, int VPT>
__global__ void __launch_bounds__(kQkThreads) kda_qk_forward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) float2 tab[];
  const int which = blockIdx.x >= p.t[0].tiles;
  const QkTensor& t = p.t[which];
  const int64_t tile = static_cast<int64_t>(blockIdx.x) - (which ? p.t[0].tiles : 0);
  const int grp = threadIdx.x >> p.lanes, l = threadIdx.x & ((1 << p.lanes) - 1), groups = kQkThreads >> p.lanes;
  const int64_t item0 = tile * (groups * VPT), row0 = item0 / t.heads;
  const int rem = static_cast<int>(item0 - row0 * t.heads);
  const bool used = l * 8 < p.D;
  uint4 x[VPT];
  QkItem it[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    it[j] = qk_item(t, item0, row0, rem, grp + j * groups, used);
    x[j] = it[j].in ? *reinterpret_cast<const uint4*>(t.x + it[j].row * t.x_ts + it[j].head * p.D + l * 8) : make_uint4(0, 0, 0, 0);
  }
  float w[8];
  if (t.w != nullptr && used) unpack8(__ldg(reinterpret_cast<const uint4*>(t.w) + l), w);
  if constexpr (ROT != kQkNone) {
    qk_table(p, row0, (rem + groups * VPT - 1) / t.heads + 1, tab);
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
      const float inv = rsqrtf(fmaf(head_sum(ss, p.lanes), p.inv_d, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
      if (t.w != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w[e];
      }
    }
    qk_rotate<ROT>(p, tab + it[j].r * (p.rot >> 1), l, 1.f, f);
    if (it[j].in) *reinterpret_cast<uint4*>(t.y + it[j].row * t.y_ts + it[j].head * p.D + l * 8) = pack8(f);
  }
}

// Blocks [0, t[0].ctas) walk q's tiles, the rest k's, so that a thread sums dw's contributions of its 8 components in
// registers; a block then leaves one row of partial sums.
template <QkRotate ROT, int VPT>
__global__ void __launch_bounds__(kQkThreads) kda_qk_backward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) float2 tab[];
  const int which = blockIdx.x >= p.t[0].ctas;
  const QkTensor& t = p.t[which];
  const int grp = threadIdx.x >> p.lanes, l = threadIdx.x & ((1 << p.lanes) - 1), groups = kQkThreads >> p.lanes;
  const bool used = l * 8 < p.D;
  float w[8], dw[8] = {};
  if (t.w != nullptr && used) unpack8(__ldg(reinterpret_cast<const uint4*>(t.w) + l), w);
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) - (which ? p.t[0].ctas : 0); tile < t.tiles; tile += t.ctas) {
    const int64_t item0 = tile * (groups * VPT), row0 = item0 / t.heads;
    const int rem = static_cast<int>(item0 - row0 * t.heads);
    uint4 x[VPT], dy[VPT];
    QkItem it[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      it[j] = qk_item(t, item0, row0, rem, grp + j * groups, used);
      x[j] = dy[j] = make_uint4(0, 0, 0, 0);
      if (it[j].in) {
        if (p.norm) x[j] = *reinterpret_cast<const uint4*>(t.x + it[j].row * t.x_ts + it[j].head * p.D + l * 8);
        dy[j] = *reinterpret_cast<const uint4*>(t.dy + it[j].row * t.dy_ts + it[j].head * p.D + l * 8);
      }
    }
    if constexpr (ROT != kQkNone) {
      qk_table(p, row0, (rem + groups * VPT - 1) / t.heads + 1, tab);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[8], g[8];
      unpack8(dy[j], g);
      qk_rotate<ROT>(p, tab + it[j].r * (p.rot >> 1), l, -1.f, g);
      if (p.norm) {
        unpack8(x[j], f);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        const float inv = rsqrtf(fmaf(head_sum(ss, p.lanes), p.inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;  // x^
        if (t.w != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (it[j].in) dw[e] = fmaf(g[e], f[e], dw[e]);
            g[e] *= w[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sg = fmaf(g[e], f[e], sg);
        sg = head_sum(used ? sg : 0.f, p.lanes) * p.inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = inv * fmaf(-f[e], sg, g[e]);
      }
      if (it[j].in) *reinterpret_cast<uint4*>(t.y + it[j].row * t.y_ts + it[j].head * p.D + l * 8) = pack8(g);
    }
    if constexpr (ROT != kQkNone) __syncthreads();  // the table is rewritten
  }
  if (t.dw == nullptr) return;
  float* const red = reinterpret_cast<float*>(tab);  // [groups][D]
  if (used) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[grp * p.D + l * 8 + e] = dw[e];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kQkThreads) {
    float s = 0.f;
    for (int i = 0; i < groups; ++i) s += red[i * p.D + d];
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
