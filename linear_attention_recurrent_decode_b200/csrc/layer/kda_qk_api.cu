// kda_qk_api.cu -- C ABI of the q/k norm with rotation (include/layer/kda_qk.h).
#include "kda_layer_host.h"
#include "kda_qk_kernel.cuh"
#include "layer/kda_qk.h"

namespace {

using namespace kda_layer;
namespace ks = kdal;

#define KDA_TRY(x)                 \
  do {                             \
    const kda_status st_ = (x);    \
    if (st_ != KDA_OK) return st_; \
  } while (0)

kda_status check_rows(const void* p, int64_t stride, int64_t width, int64_t rows) {
  if (rows <= 0) return KDA_OK;
  if (p == nullptr || stride < width) return KDA_ERR_INVALID_ARG;
  if (!aligned(p, 16) || stride % 8 != 0) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride && a.width == b.width; }

// Checks a call and fills the parameters, without the split into tiles.
kda_status common(const kda_qk_args& a, bool backward, ks::QkParams* p) {
  if (a.rows < 0 || a.q.heads < 0 || a.k.heads < 0 || a.workspace_bytes < 0) return KDA_ERR_INVALID_ARG;
  if (a.norm < KDA_QK_NORM_NONE || a.norm > KDA_QK_NORM_RMS) return KDA_ERR_INVALID_ARG;
  if (a.D < 8 || a.D > 256 || a.D % 8 != 0 || a.rot < 0 || a.rot > a.D || a.rot % 16 != 0) return KDA_ERR_UNSUPPORTED;
  const kda_qk_tensor* const t[2] = {&a.q, &a.k};
  *p = ks::QkParams{};
  bool any = false, dw = false;
  for (int i = 0; i < 2; ++i) {
    int64_t items, width, elems;
    if (t[i]->heads > ks::kMaxHeads || !mul_ok(a.rows, t[i]->heads, &items) || !mul_ok(t[i]->heads, a.D, &width) ||
        !mul_ok(items, a.D, &elems) || elems >= (int64_t{1} << 51))
      return KDA_ERR_UNSUPPORTED;
    const int64_t rows = t[i]->heads > 0 ? a.rows : 0;
    any = any || (rows > 0);
    KDA_TRY(check_rows(t[i]->x, t[i]->x_row_stride, width, backward && a.norm == KDA_QK_NORM_NONE ? 0 : rows));
    KDA_TRY(check_rows(backward ? t[i]->dx : t[i]->y, backward ? t[i]->dx_row_stride : t[i]->y_row_stride, width, rows));
    if (backward) KDA_TRY(check_rows(t[i]->dy, t[i]->dy_row_stride, width, rows));
    if (a.norm == KDA_QK_NORM_NONE && t[i]->weight != nullptr) return KDA_ERR_INVALID_ARG;
    if (backward && t[i]->dweight != nullptr) {
      if (t[i]->weight == nullptr) return KDA_ERR_INVALID_ARG;
      dw = true;
    }
    if (!aligned(t[i]->weight, 16) || !aligned(t[i]->dweight, 4)) return KDA_ERR_MISALIGNED;
    ks::QkTensor& o = p->t[i];
    o.x = static_cast<const __nv_bfloat16*>(t[i]->x), o.x_ts = t[i]->x_row_stride;
    o.y = static_cast<__nv_bfloat16*>(backward ? t[i]->dx : t[i]->y);
    o.y_ts = backward ? t[i]->dx_row_stride : t[i]->y_row_stride;
    o.dy = static_cast<const __nv_bfloat16*>(t[i]->dy), o.dy_ts = t[i]->dy_row_stride;
    o.w = static_cast<const __nv_bfloat16*>(t[i]->weight);
    o.dw = backward ? t[i]->dweight : nullptr;
    o.items = items;
    o.heads = static_cast<int32_t>(t[i]->heads);
    if (o.heads > 1) {  // ceil(2^n / heads)
      o.div64 = ~uint64_t{0} / static_cast<uint64_t>(o.heads) + 1;
      o.div32 = ~uint32_t{0} / static_cast<uint32_t>(o.heads) + 1;
    }
  }
  if (a.rot > 0 && any) {
    if (a.positions == nullptr || a.inv_freq == nullptr) return KDA_ERR_INVALID_ARG;
    if (!aligned(a.positions, a.positions_64 ? 8 : 4) || !aligned(a.inv_freq, 8)) return KDA_ERR_MISALIGNED;
  }
  if (dw) {
    if (a.workspace == nullptr || a.workspace_bytes < kda_qk_workspace_bytes(a.D)) return KDA_ERR_INVALID_ARG;
    if (!aligned(a.workspace, 16)) return KDA_ERR_MISALIGNED;
  }
  // outputs against everything else
  Rows in[16], out[6];
  int ni = 0, no = 0, own[6];
  for (int i = 0; i < 2; ++i) {
    const int64_t rows = t[i]->heads > 0 ? a.rows : 0, width = t[i]->heads * a.D;
    const int x = ni;
    in[ni++] = Rows{backward && a.norm == KDA_QK_NORM_NONE ? nullptr : t[i]->x, rows, t[i]->x_row_stride, width, 2};
    if (backward) in[ni++] = Rows{t[i]->dy, rows, t[i]->dy_row_stride, width, 2};
    in[ni++] = dense(t[i]->weight, a.D, 2);
    own[no] = backward ? x + 1 : x;  // the input an output may be
    out[no++] = Rows{p->t[i].y, rows, p->t[i].y_ts, width, 2};
    if (p->t[i].dw != nullptr) own[no] = -1, out[no++] = dense(p->t[i].dw, a.D, 4);
  }
  if (a.rot > 0) {
    in[ni++] = dense(a.positions, a.rows, a.positions_64 ? 8 : 4);
    in[ni++] = dense(a.inv_freq, a.rot / 2, 8);
  }
  if (dw) own[no] = -1, out[no++] = dense(a.workspace, kda_qk_workspace_bytes(a.D), 1);
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (!(i == own[o] && same_rows(out[o], in[i])) && !disjoint(out[o], in[i])) return KDA_ERR_ALIAS;
    for (int q = 0; q < o; ++q)
      if (!disjoint(out[o], out[q])) return KDA_ERR_ALIAS;
  }
  p->pos = a.positions, p->pos64 = a.positions_64 != 0;
  p->freq = a.inv_freq;
  p->partial = static_cast<float*>(a.workspace);
  p->rows = a.rows;
  p->D = static_cast<int32_t>(a.D), p->rot = static_cast<int32_t>(a.rot);
  while ((8 << p->lanes) < a.D) ++p->lanes;
  p->norm = a.norm;
  p->eps = a.eps, p->scale = a.rope_scale;
  p->inv_d = a.norm == KDA_QK_NORM_RMS ? 1.f / static_cast<float>(a.D) : 1.f;
  return KDA_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

// Splits both tensors into tiles of vpt heads a group of threads; the shared memory of the rows' cos and sin.
int64_t split(ks::QkParams* p, int vpt) {
  const int64_t per = static_cast<int64_t>(ks::kQkThreads >> p->lanes) * vpt;
  int64_t span = 0;
  for (auto& t : p->t) {
    t.tiles = ceil_div(t.items, per);
    if (t.items > 0) {
      int64_t s = (t.heads - 1 + per - 1) / t.heads + 1;
      s = s < p->rows ? s : p->rows;
      span = s > span ? s : span;
    }
  }
  return span * (p->rot / 2) * static_cast<int64_t>(sizeof(float2));
}
// Heads a thread takes: the measured best for large calls (see the kernels) once that still leaves two tiles an SM,
// else one, which spreads few heads over more SMs.
constexpr int kForwardVpt = 4, kBackwardVpt = 2;
int pick_vpt(ks::QkParams* p, int most) {
  split(p, most);
  return p->t[0].tiles + p->t[1].tiles >= 2 * sm_count() ? most : 1;
}

template <typename F>
bool launch(F kernel, dim3 grid, int threads, int64_t smem, kda_stream_t stream, const ks::QkParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess;
}

template <ks::QkRotate ROT, int LANES>
bool launch_lanes(bool backward, int vpt, unsigned grid, int64_t smem, kda_stream_t stream, const ks::QkParams& p) {
  if (backward) {
    const int64_t red = p.t[0].dw || p.t[1].dw ? static_cast<int64_t>(ks::kQkThreads >> LANES) * p.D * 4 : 0;  // dw's sums
    smem = smem > red ? smem : red;
    return vpt == 1 ? launch(ks::kda_qk_backward_kernel<ROT, LANES, 1>, dim3(grid), ks::kQkThreads, smem, stream, p)
                    : launch(ks::kda_qk_backward_kernel<ROT, LANES, kBackwardVpt>, dim3(grid), ks::kQkThreads, smem, stream, p);
  }
  return vpt == 1 ? launch(ks::kda_qk_forward_kernel<ROT, LANES, 1>, dim3(grid), ks::kQkThreads, smem, stream, p)
                  : launch(ks::kda_qk_forward_kernel<ROT, LANES, kForwardVpt>, dim3(grid), ks::kQkThreads, smem, stream, p);
}
template <ks::QkRotate ROT>
bool launch_rotate(bool backward, int vpt, unsigned grid, int64_t smem, kda_stream_t stream, const ks::QkParams& p) {
  switch (p.lanes) {
    case 0: return launch_lanes<ROT, 0>(backward, vpt, grid, smem, stream, p);
    case 1: return launch_lanes<ROT, 1>(backward, vpt, grid, smem, stream, p);
    case 2: return launch_lanes<ROT, 2>(backward, vpt, grid, smem, stream, p);
    case 3: return launch_lanes<ROT, 3>(backward, vpt, grid, smem, stream, p);
    case 4: return launch_lanes<ROT, 4>(backward, vpt, grid, smem, stream, p);
    default: return launch_lanes<ROT, 5>(backward, vpt, grid, smem, stream, p);
  }
}
bool launch_qk(const kda_qk_args& a, bool backward, int vpt, int64_t grid, int64_t smem, kda_stream_t stream, const ks::QkParams& p) {
  const unsigned n = static_cast<unsigned>(grid);
  if (a.rot == 0) return launch_rotate<ks::kQkNone>(backward, vpt, n, smem, stream, p);
  return a.interleaved ? launch_rotate<ks::kQkInterleaved>(backward, vpt, n, smem, stream, p)
                       : launch_rotate<ks::kQkHalves>(backward, vpt, n, smem, stream, p);
}

}  // namespace

extern "C" {

int64_t kda_qk_workspace_bytes(int64_t D) {
  if (D < 8 || D > 256 || D % 8 != 0) return -1;
  return static_cast<int64_t>(ks::kQkMaxCtas) * D * static_cast<int64_t>(sizeof(float));
}

kda_status kda_qk_norm_rope(const kda_qk_args* args, kda_stream_t stream) {
  if (args == nullptr) return KDA_ERR_INVALID_ARG;
  ks::QkParams p;
  KDA_TRY(common(*args, false, &p));
  if (p.t[0].items + p.t[1].items == 0) return KDA_OK;
  KDA_TRY(check_device());
  const int vpt = pick_vpt(&p, kForwardVpt);
  const int64_t smem = split(&p, vpt), grid = p.t[0].tiles + p.t[1].tiles;
  if (grid > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  return launch_qk(*args, false, vpt, grid, smem, stream, p) ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_qk_norm_rope_backward(const kda_qk_args* args, kda_stream_t stream) {
  if (args == nullptr) return KDA_ERR_INVALID_ARG;
  ks::QkParams p;
  KDA_TRY(common(*args, true, &p));
  const bool dw = p.t[0].dw != nullptr || p.t[1].dw != nullptr;
  if (p.t[0].items + p.t[1].items == 0 && !dw) return KDA_OK;
  KDA_TRY(check_device());
  const int vpt = pick_vpt(&p, kBackwardVpt);
  const int64_t smem = split(&p, vpt);
  // as many blocks as run at once, by the tensors' shares of the tiles
  const int64_t fit = ks::kQkBackwardCtas * sm_count(), most = fit < ks::kQkMaxCtas - 2 ? fit : ks::kQkMaxCtas - 2;
  const int64_t tiles = p.t[0].tiles + p.t[1].tiles;
  for (auto& t : p.t)
    t.ctas = static_cast<int32_t>(tiles <= most ? t.tiles
                                                : (t.tiles == 0 ? 0 : 1 + static_cast<int64_t>(static_cast<double>(t.tiles) / tiles * (most - 2))));
  const int64_t grid = p.t[0].ctas + p.t[1].ctas;
  if (grid > 0 && !launch_qk(*args, true, vpt, grid, smem, stream, p)) return KDA_ERR_CUDA;
  if (dw && !launch(ks::kda_qk_weight_kernel, dim3(static_cast<unsigned>((p.D + 31) / 32), 2), 1024, 0, stream, p)) return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"
