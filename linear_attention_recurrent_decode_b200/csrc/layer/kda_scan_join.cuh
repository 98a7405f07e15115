// kda_scan_join.cuh -- joins the segments of a sequence (see kda_scan_chain.cuh).
//
// Forwards, with E the end state of a segment walked from zero (the first from
// its real start) and M its transition matrix, the real ends are, in order,
//   E_g <- E_g + M_g E_{g-1},   g = 1 .. segments - 2,
// backwards, with F the gradient at a segment's start,
//   F_g <- F_g + M_g^T F_{g+1},  g = segments - 2 .. 1.
// One CTA a sequence, head and 16 of the 128 columns, which are independent; the
// columns stay in shared memory from step to step, and the next matrix is copied
// while this one is used.  fp32 throughout: 128 x 128 x 16 products a step are
// too few for the tensor cores to matter, and the step's latency is the copy's.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kJoinThreads = 256, kJoinCols = 16;
constexpr int kJoinPitch = kK + 4;  // rows read across rows of a warp: no two in the same banks

struct JoinSmem {
  float map[2][kK][kJoinPitch];
  float s[kK][kJoinCols];
};

template <bool BACK>
__global__ void __launch_bounds__(kJoinThreads) kda_scan_join_kernel(const __grid_constant__ ScanParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  JoinSmem& sm = *reinterpret_cast<JoinSmem*>(smem_raw);
  constexpr int kGroups = kV / kJoinCols;
  const int64_t unit = blockIdx.x / kGroups, n = unit / p.HV, h = unit - n * p.HV;
  const int v0 = static_cast<int>(blockIdx.x - unit * kGroups) * kJoinCols, tid = threadIdx.x;
  int64_t start, len;
  seq_range(p, n, start, len);
  const int64_t chunks = (len + kC - 1) / kC, segs = (chunks + p.seg_chunks - 1) / p.seg_chunks;
  if (segs < 3 || state_block(p, n) < 0) return;
  const int64_t slot0 = first_segment(p, n, start), steps = segs - 2;
  auto block = [&](int64_t g) { return ((slot0 + g) * p.HV + h) * kK * kV; };
  auto copy = [&](int64_t g, int buf) {
    const float* const src = p.seg_map + block(g);
    for (int e = tid; e < kK * kK / 4; e += kJoinThreads) cp_async16(&sm.map[buf][e >> 5][(e & 31) * 4], src + e * 4);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t first = BACK ? segs - 2 : 1;
  copy(first, 0);
  {
    const float* const src = p.seg_state + block(BACK ? segs - 1 : 0) + v0;
    for (int e = tid; e < kK * kJoinCols; e += kJoinThreads) sm.s[e / kJoinCols][e % kJoinCols] = src[(e / kJoinCols) * kV + e % kJoinCols];
  }
  const int k = tid >> 1, c = (tid & 1) * 8;  // this thread's row and columns
  for (int64_t i = 0; i < steps; ++i) {
    const int64_t g = BACK ? first - i : first + i;
    if (i + 1 < steps) copy(BACK ? g - 1 : g + 1, static_cast<int>((i + 1) & 1));
    float* const dst = p.seg_state + block(g) + k * kV + v0 + c;
    float acc[8];
    *reinterpret_cast<float4*>(&acc[0]) = *reinterpret_cast<const float4*>(dst);
    *reinterpret_cast<float4*>(&acc[4]) = *reinterpret_cast<const float4*>(dst + 4);
    if (i + 1 < steps) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const auto& m = sm.map[i & 1];
#pragma unroll 4
    for (int j = 0; j < kK; j += 4) {
      float f[4];
      if constexpr (BACK) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = m[j + e][k];
      } else {
        *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(&m[k][j]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 a = *reinterpret_cast<const float4*>(&sm.s[j + e][c]), b = *reinterpret_cast<const float4*>(&sm.s[j + e][c + 4]);
        acc[0] = fmaf(f[e], a.x, acc[0]);
        acc[1] = fmaf(f[e], a.y, acc[1]);
        acc[2] = fmaf(f[e], a.z, acc[2]);
        acc[3] = fmaf(f[e], a.w, acc[3]);
        acc[4] = fmaf(f[e], b.x, acc[4]);
        acc[5] = fmaf(f[e], b.y, acc[5]);
        acc[6] = fmaf(f[e], b.z, acc[6]);
        acc[7] = fmaf(f[e], b.w, acc[7]);
      }
    }
    __syncthreads();  // the columns and this matrix are read
    *reinterpret_cast<float4*>(&sm.s[k][c]) = *reinterpret_cast<const float4*>(&acc[0]);
    *reinterpret_cast<float4*>(&sm.s[k][c + 4]) = *reinterpret_cast<const float4*>(&acc[4]);
    *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(&acc[0]);
    *reinterpret_cast<float4*>(dst + 4) = *reinterpret_cast<const float4*>(&acc[4]);
  }
}

}  // namespace kdal
