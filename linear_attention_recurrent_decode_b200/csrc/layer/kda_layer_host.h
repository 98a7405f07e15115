// kda_layer_host.h -- host-side argument checks of the layer operators.
#pragma once

#include "kda_host_util.h"

namespace kda_layer {

using namespace kda_host;

// A strided row buffer an entry point reads or writes.
struct Rows {
  const void* p;
  int64_t rows, stride, width;  // elements
  int elem;                     // bytes per element
};
inline Rows dense(const void* p, int64_t elems, int elem) { return Rows{p, 1, elems, elems, elem}; }

inline bool span(const Rows& r, Range* out) {
  int64_t bytes = 0;
  if (r.p == nullptr || r.rows <= 0) {
    *out = Range{0, 0};
    return true;
  }
  if (!span_bytes(r.rows, r.stride, r.width, r.elem, &bytes) || bytes > INT64_MAX / 2) return false;
  *out = range_of(r.p, bytes);
  return true;
}

// Whether two row buffers share no byte: apart, or interleaved rows of one
// buffer (equal strides) with disjoint columns.  False also for sizes whose
// extent overflows.
inline bool disjoint(const Rows& a, const Rows& b) {
  Range ra, rb;
  if (!span(a, &ra) || !span(b, &rb)) return false;
  if (!overlaps(ra, rb)) return true;
  const int64_t sa = a.stride * a.elem, sb = b.stride * b.elem;
  if (sa != sb) return false;
  const int64_t wa = a.width * a.elem, wb = b.width * b.elem;
  int64_t d = static_cast<int64_t>(rb.lo - ra.lo) % sa;  // two's complement difference
  if (d < 0) d += sa;
  return wa <= d && d + wb <= sa;
}

// SMs of the current device.
inline int sm_count() {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  int v = dev < kMaxDevices ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
    if (dev < kMaxDevices) cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace kda_layer
