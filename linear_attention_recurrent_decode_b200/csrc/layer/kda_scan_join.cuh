// kda_scan_join.cuh -- joins the segments of a sequence (see kda_scan_chain.cuh).
//
// Forwards, with E the end state of a segment walked from zero (the first from
// its real start) and M its transition matrix, the real ends are, in order,
//   E_g <- E_g + M_g E_{g-1},   g = 1 .. segments - 2,
// backwards, with F the gradient at a segment's start,
//   F_g <- F_g + M_g^T F_{g+1},  g = segments - 2 .. 1.
// One CTA a sequence, head and 16 of the 128 columns, which are independent.  The
// steps' latency bounds it: each element of a matrix is used once per CTA, so the
// fragments of the tf32 products (pairs, three products: fp32 accuracy) go from
// global memory straight to registers, a step ahead, and only the columns pass
// through shared memory.  Measured: 3 us a step (its
// loads' latency), against 5 us for fp32 products with the matrix staged in
// shared memory.
#pragma once

#include "kda_scan_common.cuh"

namespace kdal {

constexpr int kJoinThreads = 256, kJoinCols = 16;
constexpr int kJoinPitch = 18;  // floats of a row of the columns: fragments then touch 32 banks

template <bool BACK>
__global__ void __launch_bounds__(kJoinThreads, 1) kda_scan_join_kernel(const __grid_constant__ ScanParams p) {
  __shared__ float col[kK][kJoinPitch];
  constexpr int kGroups = kV / kJoinCols;
  int64_t n, h;
  slot_and_head(p, blockIdx.x / kGroups, n, h);
  const int v0 = static_cast<int>(blockIdx.x % kGroups) * kJoinCols, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  int64_t start, len;
  seq_range(p, n, start, len);
  const bool cut = p.cu == nullptr || find_segment(p.cu, p.N, p.tokens, p.seg_chunks, 0).cut;
  const int64_t segs = segments_of(p, (len + kC - 1) / kC, cut);
  wait_upstream();
  if (gridDim.x <= kSms) launch_dependents();  // 1 us of 268 for one sequence of 8192 tokens, 8 heads
  if (segs < 3 || state_block(p, n) < 0) return;
  const int64_t slot0 = first_segment(p, n, start), steps = segs - 2, first = BACK ? segs - 2 : 1;
  auto block = [&](int64_t g) { return ((slot0 + g) * p.HV + h) * kK * kV; };
  // The warp's 16 rows of the result.  Forwards the matrix is the left operand, [16 rows][128]; backwards (transposed) the
  // right one, 128 x 16, and the result comes out transposed.  A thread's contracted indices are 16 g + 4 c .. + 3.
  float m[64];
  auto fetch = [&](int64_t g) {
    const float* const src = p.seg_map + block(g);
#pragma unroll
    for (int kg = 0; kg < 8; ++kg) {
      if constexpr (BACK) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2*>(&m[kg * 8 + 2 * j]) = *reinterpret_cast<const float2*>(src + (kg * 16 + 4 * c + j) * kK + warp * 16 + 2 * r);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(&m[kg * 8 + 4 * j]) = *reinterpret_cast<const float4*>(src + (warp * 16 + r + 8 * j) * kK + kg * 16 + 4 * c);
      }
    }
  };
  // Row and column of this thread's result element e of tile t.
  auto row = [&](int t, int e) { return warp * 16 + (BACK ? 2 * (2 * c + (e & 1)) + t : r + (e >> 1) * 8); };
  auto column = [&](int t, int e) { return BACK ? r + (e >> 1) * 8 : t * 8 + 2 * c + (e & 1); };
  fetch(first);
  {
    const float* const src = p.seg_state + block(BACK ? segs - 1 : 0) + v0;
    for (int e = tid; e < kK * kJoinCols; e += kJoinThreads) col[e / kJoinCols][e % kJoinCols] = src[(e / kJoinCols) * kV + e % kJoinCols];
  }
  for (int64_t i = 0; i < steps; ++i) {
    const int64_t g = BACK ? first - i : first + i;
    float* const dst = p.seg_state + block(g) + v0;
    float base[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) base[t][e] = dst[row(t, e) * kV + column(t, e)];
    uint32_t mh[64], ml[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) tf32_pair(m[j], mh[j], ml[j]);
    if (i + 1 < steps) fetch(BACK ? g - 1 : g + 1);
    __syncthreads();  // the columns are there
    float sum[2][4] = {};
#pragma unroll
    for (int kg = 0; kg < 8; ++kg) {
      float part[2][4] = {}, lo[2][4] = {};  // of these 16 alone: one long chain of products waits 30 cycles for each
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float* const at = &col[kg * 16 + 4 * c + 2 * s][r];
        if constexpr (BACK) {
          uint32_t ah[4], al[4];  // (column r or r + 8, index 2 s or 2 s + 1)
          tf32_pair(at[0], ah[0], al[0]);
          tf32_pair(at[8], ah[1], al[1]);
          tf32_pair(at[kJoinPitch], ah[2], al[2]);
          tf32_pair(at[kJoinPitch + 8], ah[3], al[3]);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int j = kg * 8 + 4 * s + t;
            const uint32_t bh[2] = {mh[j], mh[j + 2]}, bl[2] = {ml[j], ml[j + 2]};
            mma_tf32(lo[t], ah, bl);
            mma_tf32(lo[t], al, bh);
            mma_tf32(part[t], ah, bh);
          }
        } else {
          const int j = kg * 8 + 2 * s;
          const uint32_t ah[4] = {mh[j], mh[j + 4], mh[j + 1], mh[j + 5]}, al[4] = {ml[j], ml[j + 4], ml[j + 1], ml[j + 5]};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t bh[2], bl[2];
            tf32_pair(at[t * 8], bh[0], bl[0]);
            tf32_pair(at[kJoinPitch + t * 8], bh[1], bl[1]);
            mma_tf32(lo[t], ah, bl);
            mma_tf32(lo[t], al, bh);
            mma_tf32(part[t], ah, bh);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] += part[t][e] + lo[t][e];
    }
    __syncthreads();  // the columns are read
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = base[t][e] + sum[t][e];
        col[row(t, e)][column(t, e)] = x;
        dst[row(t, e) * kV + column(t, e)] = x;
      }
  }
}

}  // namespace kdal
