// kda_scan_api.cu -- C ABI of the scan (include/layer/kda_scan.h): validation,
// workspace sizes and launches.  Nothing here allocates or synchronises.
#include <atomic>
#include <cstdint>

#include "kda_layer_host.h"
#include "kda_scan_chain.cuh"
#include "kda_scan_grad.cuh"
#include "kda_scan_join.cuh"
#include "kda_scan_prep.cuh"
#include "layer/kda_scan.h"

namespace {

using namespace kda_layer;
namespace ks = kdal;

constexpr int kChainSmem = static_cast<int>(sizeof(ks::ChainSmem));

// Dynamic shared memory allowances, once per device.
cudaError_t prepare_kernels() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit && (ready.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  cudaError_t e = cudaSuccess;
  auto allow = [&](auto kernel, int smem) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  allow(ks::kda_scan_prep_kernel, static_cast<int>(sizeof(ks::PrepSmem)));
  allow(ks::kda_scan_forward_kernel, kChainSmem);
  allow(ks::kda_scan_backward_kernel, kChainSmem);
  allow(ks::kda_scan_grad_kernel, static_cast<int>(sizeof(ks::GradSmem)));
  if (e == cudaSuccess && bit) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Chunk slots of the whole call (see Record); false on overflow.
bool chunk_slots(int64_t N, int64_t T, bool packed, int64_t* slots) {
  if (packed) return !__builtin_add_overflow(T / ks::kC, N, slots);
  return mul_ok(N, T / ks::kC + (T % ks::kC != 0), slots);
}

// Chunks of a segment, 0 for none, and the segment slots of the call.  Segments are for calls whose sequences and heads
// leave half the SMs idle or more, with room for a sequence of 24 chunks (below, walking it twice and joining cost what
// the segments save); as long as the first of the two walks, two blocks a segment, then fills the SMs once, and at least
// 8 chunks.  Where the longest sequence is not much longer than one, all are walked whole (worth_segments): a packed
// call's lengths are on the device, so it may launch the walk for the segments' ends and the join for none, 8 us.
// Measured, us a call: 8192 tokens of 8 heads 635 without and 269 with segments, with gradients 1753 and 674.
constexpr int64_t kSms = ks::kSms;
bool segments(int64_t N, int64_t T, bool packed, int64_t HV, int32_t* seg_chunks, int64_t* slots) {
  const int64_t total = packed ? T / ks::kC : (T + ks::kC - 1) / ks::kC;  // the longest sequence's chunks at most
  *seg_chunks = 0;
  *slots = N;
  int64_t units;
  if (!mul_ok(N, HV, &units)) return false;
  if (units > ks::kMostCut || total < 24) return true;
  const int64_t all = (packed ? total : total * N) * HV;
  int64_t len = (2 * all + kSms - 1) / kSms;
  len = len < 8 ? 8 : len;
  if (len > 0x7fffffff) return false;
  if (!ks::worth_segments(total, len)) return true;
  *seg_chunks = static_cast<int32_t>(len);
  *slots = packed ? total / len + N : N * ((total + len - 1) / len);
  return true;
}

bool workspace_bytes(int64_t N, int64_t T, bool packed, int64_t HV, bool training, int64_t* bytes, int64_t* records = nullptr) {
  int64_t slots, recs, seg_slots, seg_bytes = 0;
  int32_t seg_chunks;
  if (!chunk_slots(N, T, packed, &slots) || !mul_ok(slots, HV, &recs) || recs > 0x7fffffffLL ||
      !mul_ok(recs, training ? ks::Record::kTraining : ks::Record::kForward, bytes) || __builtin_add_overflow(*bytes, ks::kWsHeader, bytes) ||
      !segments(N, T, packed, HV, &seg_chunks, &seg_slots))
    return false;
  if (records) *records = *bytes;
  if (seg_chunks > 0 && (!mul_ok(seg_slots, HV, &seg_bytes) || seg_bytes > 0x7fffffffLL / 2 ||
                         !mul_ok(seg_bytes, 2 * ks::kK * ks::kV * static_cast<int64_t>(sizeof(float)), &seg_bytes)))
    return false;
  return !__builtin_add_overflow(*bytes, seg_bytes, bytes);
}

kda_status check_rows(const void* p, int64_t stride, int64_t width, int64_t rows, uintptr_t align, int64_t mult) {
  if (rows > 0 && p == nullptr) return KDA_ERR_INVALID_ARG;
  if (stride < width) return KDA_ERR_INVALID_ARG;
  if (!aligned(p, align) || stride % mult != 0) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

#define KDA_TRY(x)                        \
  do {                                    \
    const kda_status st_ = (x);           \
    if (st_ != KDA_OK) return st_;        \
  } while (0)

// Checks what both calls share and fills the kernels' parameters.
kda_status common(const kda_scan_args& a, bool training, ks::ScanParams* p, int64_t* slots, int64_t* seg_slots, int64_t* rows) {
  if (a.N < 0 || a.T < 0 || a.HV < 0 || a.workspace_bytes < 0 || a.num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (a.HV < 1 || a.K != ks::kK || a.V != ks::kV) return KDA_ERR_UNSUPPORTED;
  const bool packed = a.cu_seqlens != nullptr;
  int64_t need, units, records;
  if (!mul_ok(a.N, packed ? 1 : a.T, rows)) return KDA_ERR_UNSUPPORTED;
  if (packed) *rows = a.T;
  if (!chunk_slots(a.N, a.T, packed, slots) || !workspace_bytes(a.N, a.T, packed, a.HV, training, &need, &records) ||
      !mul_ok(a.N, a.HV, &units) || units > 0x7fffffffLL || a.N > 0x7fffffffLL || *rows > INT64_MAX / (a.HV * ks::kK * 8))
    return KDA_ERR_UNSUPPORTED;
  if (packed && a.T > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;  // int32 offsets
  const int64_t hk = a.HV * ks::kK, hv = a.HV * ks::kV;
  KDA_TRY(check_rows(a.q, a.q_row_stride, hk, *rows, 16, 8));
  KDA_TRY(check_rows(a.k, a.k_row_stride, hk, *rows, 16, 8));
  KDA_TRY(check_rows(a.v, a.v_row_stride, hv, *rows, 16, 8));
  KDA_TRY(check_rows(a.g, a.g_row_stride, hk, *rows, 4, 1));
  KDA_TRY(check_rows(a.beta, a.beta_row_stride, a.HV, *rows, 4, 1));
  if (a.workspace == nullptr || a.workspace_bytes < need) return KDA_ERR_INVALID_ARG;
  if (!aligned(a.workspace, 16) || !aligned(a.initial_state, 16) || !aligned(a.final_state, 16) ||
      !aligned(a.cu_seqlens, 4) || !aligned(a.slot_idx, 4))
    return KDA_ERR_MISALIGNED;
  if (a.slot_idx != nullptr && a.num_slots <= 0) return KDA_ERR_INVALID_ARG;
  *p = ks::ScanParams{};
  p->q = static_cast<const __nv_bfloat16*>(a.q), p->q_ts = a.q_row_stride;
  p->k = static_cast<const __nv_bfloat16*>(a.k), p->k_ts = a.k_row_stride;
  p->v = static_cast<const __nv_bfloat16*>(a.v), p->v_ts = a.v_row_stride;
  p->g = a.g, p->g_ts = a.g_row_stride;
  p->beta = a.beta, p->beta_ts = a.beta_row_stride;
  p->cu = a.cu_seqlens;
  p->s_in = a.initial_state;
  p->ws = static_cast<unsigned char*>(a.workspace);
  p->rec_bytes = training ? ks::Record::kTraining : ks::Record::kForward;
  p->tokens = *rows, p->T = a.T, p->HV = a.HV;
  p->N = static_cast<int32_t>(a.N);
  p->seq_chunks = static_cast<int32_t>(packed ? 0 : (a.T + ks::kC - 1) / ks::kC);
  p->scale = a.scale;
  p->save = training;
  segments(a.N, a.T, packed, a.HV, &p->seg_chunks, seg_slots);
  if (p->seg_chunks > 0) {
    p->seq_segs = static_cast<int32_t>(packed ? 0 : (p->seq_chunks + p->seg_chunks - 1) / p->seg_chunks);
    p->seg_state = reinterpret_cast<float*>(p->ws + records);
    p->seg_map = p->seg_state + *seg_slots * a.HV * ks::kK * ks::kV;
  }
  return KDA_OK;
}

// The inputs' extents, for the overlap checks.
struct Inputs {
  Rows r[9];
};
Inputs inputs_of(const kda_scan_args& a, int64_t rows) {
  const int64_t hk = a.HV * ks::kK, hv = a.HV * ks::kV, blocks = a.slot_idx ? a.num_slots : a.N;
  return Inputs{{Rows{a.q, rows, a.q_row_stride, hk, 2}, Rows{a.k, rows, a.k_row_stride, hk, 2},
                 Rows{a.v, rows, a.v_row_stride, hv, 2}, Rows{a.g, rows, a.g_row_stride, hk, 4},
                 Rows{a.beta, rows, a.beta_row_stride, a.HV, 4}, dense(a.cu_seqlens, a.N + 1, 4),
                 dense(a.slot_idx, a.N, 4), dense(a.initial_state, blocks * hk * ks::kV, 4),
                 dense(a.workspace, a.workspace_bytes, 1)}};
}

template <typename F>
bool launch(F kernel, int64_t grid, int threads, int smem, kda_stream_t stream, const ks::ScanParams& p) {
  if (grid == 0) return true;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.tokens > 0;  // without tokens the forward chains, which look up their sequence before they wait, are first
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess;
}

constexpr int kJoinGroups = ks::kV / ks::kJoinCols;

bool launch_forward(ks::ScanParams p, int64_t slots, int64_t seg_slots, kda_stream_t stream) {
  if (!launch(ks::kda_scan_prep_kernel, slots * p.HV, ks::kPrepThreads, sizeof(ks::PrepSmem), stream, p)) return false;
  if (p.seg_chunks > 0) {
    p.transitions = 1;
    if (!launch(ks::kda_scan_forward_kernel, seg_slots * p.HV * 2, ks::kChainThreads, kChainSmem, stream, p) ||
        !launch(ks::kda_scan_join_kernel<false>, p.N * p.HV * kJoinGroups, ks::kJoinThreads, 0, stream, p))
      return false;
    p.transitions = 0;
  }
  return launch(ks::kda_scan_forward_kernel, seg_slots * p.HV, ks::kChainThreads, kChainSmem, stream, p);
}
bool launch_backward(ks::ScanParams p, int64_t slots, int64_t seg_slots, kda_stream_t stream) {
  if (p.seg_chunks > 0) {
    p.transitions = 1;
    if (!launch(ks::kda_scan_backward_kernel, seg_slots * p.HV, ks::kChainThreads, kChainSmem, stream, p) ||
        !launch(ks::kda_scan_join_kernel<true>, p.N * p.HV * kJoinGroups, ks::kJoinThreads, 0, stream, p))
      return false;
    p.transitions = 0;
  }
  return launch(ks::kda_scan_backward_kernel, seg_slots * p.HV, ks::kChainThreads, kChainSmem, stream, p) &&
         launch(ks::kda_scan_grad_kernel, slots * p.HV, ks::kGradThreads, sizeof(ks::GradSmem), stream, p);
}

}  // namespace

extern "C" {

int64_t kda_scan_workspace_bytes(int64_t N, int64_t T, int32_t packed, int64_t HV, int64_t K, int64_t V, int32_t training) {
  if (N < 0 || T < 0 || HV < 1 || K != ks::kK || V != ks::kV) return -1;
  if (N == 0) return 0;
  int64_t bytes;
  return workspace_bytes(N, T, packed != 0, HV, training != 0, &bytes) ? bytes : -1;
}

kda_status kda_scan(const kda_scan_args* args, kda_stream_t stream) {
  if (args == nullptr) return KDA_ERR_INVALID_ARG;
  const kda_scan_args& a = *args;
  if (a.N == 0 && a.T >= 0 && a.HV >= 1 && a.K == ks::kK && a.V == ks::kV) return KDA_OK;  // no sequence
  ks::ScanParams p;
  int64_t slots, seg_slots, rows;
  KDA_TRY(common(a, a.save != 0, &p, &slots, &seg_slots, &rows));
  const int64_t hv = a.HV * ks::kV, state = a.HV * ks::kK * ks::kV;
  KDA_TRY(check_rows(a.out, a.out_row_stride, hv, rows, 16, 8));
  const int64_t blocks = a.slot_idx ? a.num_slots : a.N;
  int64_t elems;
  if (!mul_ok(blocks, state, &elems) || elems > INT64_MAX / 8) return KDA_ERR_UNSUPPORTED;
  const Inputs in = inputs_of(a, rows);
  const Rows out{a.out, rows, a.out_row_stride, hv, 2}, fin = dense(a.final_state, elems, 4);
  for (int i = 0; i < 9; ++i) {
    if (!disjoint(out, in.r[i])) return KDA_ERR_ALIAS;
    if (!(i == 7 && a.final_state == a.initial_state) && !disjoint(fin, in.r[i])) return KDA_ERR_ALIAS;
    if (i < 8 && !disjoint(in.r[8], in.r[i])) return KDA_ERR_ALIAS;
  }
  if (!disjoint(out, fin)) return KDA_ERR_ALIAS;
  KDA_TRY(check_device());
  if (prepare_kernels() != cudaSuccess) return KDA_ERR_CUDA;
  p.s_out = a.final_state;
  p.slot_idx = a.slot_idx;
  p.num_slots = a.num_slots;
  p.out = static_cast<__nv_bfloat16*>(a.out), p.out_ts = a.out_row_stride;
  return launch_forward(p, slots, seg_slots, stream) ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_scan_backward(const kda_scan_args* args, const kda_scan_grads* grads, kda_stream_t stream) {
  if (args == nullptr || grads == nullptr) return KDA_ERR_INVALID_ARG;
  const kda_scan_args& a = *args;
  const kda_scan_grads& d = *grads;
  if (a.N == 0 && a.T >= 0 && a.HV >= 1 && a.K == ks::kK && a.V == ks::kV) return KDA_OK;
  if (a.slot_idx != nullptr) return KDA_ERR_INVALID_ARG;
  ks::ScanParams p;
  int64_t slots, seg_slots, rows;
  KDA_TRY(common(a, true, &p, &slots, &seg_slots, &rows));
  const int64_t hk = a.HV * ks::kK, hv = a.HV * ks::kV, state = hk * ks::kV;
  KDA_TRY(check_rows(d.d_out, d.d_out_row_stride, hv, rows, 16, 8));
  KDA_TRY(check_rows(d.dq, d.dq_row_stride, hk, rows, 16, 8));
  KDA_TRY(check_rows(d.dk, d.dk_row_stride, hk, rows, 16, 8));
  KDA_TRY(check_rows(d.dv, d.dv_row_stride, hv, rows, 16, 8));
  KDA_TRY(check_rows(d.dg, d.dg_row_stride, hk, rows, 4, 1));
  KDA_TRY(check_rows(d.dbeta, d.dbeta_row_stride, a.HV, rows, 4, 1));
  if (!aligned(d.d_final_state, 16) || !aligned(d.d_initial_state, 16)) return KDA_ERR_MISALIGNED;
  const Inputs in = inputs_of(a, rows);
  const Rows more[2] = {Rows{d.d_out, rows, d.d_out_row_stride, hv, 2}, dense(d.d_final_state, a.N * state, 4)};
  const Rows outs[6] = {Rows{d.dq, rows, d.dq_row_stride, hk, 2}, Rows{d.dk, rows, d.dk_row_stride, hk, 2},
                        Rows{d.dv, rows, d.dv_row_stride, hv, 2}, Rows{d.dg, rows, d.dg_row_stride, hk, 4},
                        Rows{d.dbeta, rows, d.dbeta_row_stride, a.HV, 4}, dense(d.d_initial_state, a.N * state, 4)};
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 9; ++i)
      if (!disjoint(outs[o], in.r[i])) return KDA_ERR_ALIAS;
    for (int i = 0; i < 2; ++i)
      if (!disjoint(outs[o], more[i])) return KDA_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (!disjoint(outs[o], outs[q])) return KDA_ERR_ALIAS;
  }
  for (int i = 0; i < 8; ++i)
    if (!disjoint(in.r[8], in.r[i])) return KDA_ERR_ALIAS;
  for (int i = 0; i < 2; ++i)
    if (!disjoint(in.r[8], more[i])) return KDA_ERR_ALIAS;
  KDA_TRY(check_device());
  if (prepare_kernels() != cudaSuccess) return KDA_ERR_CUDA;
  p.d_out = static_cast<const __nv_bfloat16*>(d.d_out), p.d_out_ts = d.d_out_row_stride;
  p.d_final = d.d_final_state;
  p.dq = static_cast<__nv_bfloat16*>(d.dq), p.dq_ts = d.dq_row_stride;
  p.dk = static_cast<__nv_bfloat16*>(d.dk), p.dk_ts = d.dk_row_stride;
  p.dv = static_cast<__nv_bfloat16*>(d.dv), p.dv_ts = d.dv_row_stride;
  p.dg = d.dg, p.dg_ts = d.dg_row_stride;
  p.dbeta = d.dbeta, p.dbeta_ts = d.dbeta_row_stride;
  p.d_init = d.d_initial_state;
  if (!d.saved && !launch_forward(p, slots, seg_slots, stream)) return KDA_ERR_CUDA;  // p.out is null: states only
  return launch_backward(p, slots, seg_slots, stream) ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
