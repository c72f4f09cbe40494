// C ABI of the norm and of the dense feed-forward block: argument checks,
// workspace, tensor maps, launch sequences.
//
//   forward:  gate/up products + activation -> hid;  hid x down
//   backward: dy x down + activation gradient -> dg, du, hid;
//             dg x gate + du x up -> dx, dg^T x, du^T x, dy^T hid in one launch
#include <cmath>
#include <new>

#include "../../include/lmoe_ffn.h"
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "tmap.h"

using namespace lmoe;

struct lmoe_ffn_ctx {
  lmoe_ffn_config cfg;
  lmoe_ffn_weights w;
  int device = 0;               // where the workspace lies
  int ctas = 0;                 // resident CTAs of the pair kernels
  FfnSplitLimits split = {};
  void* pool = nullptr;
  int* err = nullptr;
  void *hid = nullptr, *dg = nullptr, *du = nullptr;
  // K contiguous, boxes of 64 K values x 128 and 64 rows; MXFP8: 128 K values x 96 and 64 rows
  CUtensorMap gate[2], up[2], down[2];
  CUtensorMap gate_n, up_n, down_n;   // the same memory as N contiguous operands, boxes of 64 x 64
  // MXFP8 blocks: hid holds codes; scale atoms of x, hid and the weights
  // (for tiles of 192 and of 128 rows)
  uint8_t *x_sf = nullptr, *hid_sf = nullptr, *gu_sf[2] = {}, *down_sf[2] = {};
  CUtensorMap m_x_sf, m_hid_sf, m_gu_sf[2], m_down_sf[2];
  int launches = 0;
};

namespace {

// A failed call is reported here; the runtime's copy of the error is cleared,
// so that the caller's next check of its own launches does not find it.
lmoe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return LMOE_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? LMOE_ERR_OOM : LMOE_ERR_CUDA;
}
#define FFN_TRY(expr)                              \
  do {                                             \
    const cudaError_t e_ = (expr);                 \
    if (e_ != cudaSuccess) return cuda_status(e_); \
  } while (0)

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool usable(const void* p) { return p && aligned16(p); }
// The stream of a call, which may be NULL, is one of the current device: the
// handle's memory has to lie there.
bool on_its_device(lmoe_ffn_handle h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}
int ceil_div(int a, int b) { return (a + b - 1) / b; }

// K-contiguous bf16 operand [rows][K]: boxes of 64 K values x `box` rows.
bool map_k(CUtensorMap* m, const void* base, int K, int rows, long long ld, int box = 128) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, K, rows, 2 * ld, 64, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}
// The transposed use of [K][N]: boxes of 64 N values x 64 K rows.
bool map_n(CUtensorMap* m, const void* base, int N, int K, long long ld) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, N, K, 2 * ld, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

// MXFP8 codes [rows][K]: boxes of 128 K values x `box` rows.
bool map_mx(CUtensorMap* m, const void* base, int K, int rows, int box) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, K, rows, K, 128, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale atoms (512 bytes each), `box` at a time.
bool map_atoms(CUtensorMap* m, const void* base, size_t bytes, int box) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 128, bytes / 512, 512, 128, box,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Rows that one copy of the tokens brings, of the `rows` that a stage waits for:
// all of them, but half in the self-test of the waits.
int token_rows(int rows, bool whole) { return whole ? rows : rows / 2; }

// Weight-streaming passes: x (or hid) and the weights of one pass.  `whole`
// maps split K into 64-wide chunks as an outer dimension.
bool skinny_maps(FfnSkinnyParams& p, const void* a, long long lda, const void* w0, const void* w1, int K, int tb) {
  constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t k = K, row = 2 * k, rows = p.rows, M = p.M, T = p.T;
  p.whole = K % 64 == 0;
  if (w1) {      // two boxes of half a tile's rows each, side by side
    if (!make_tmap_2d(&p.b, dt, w0, k, M, row, 64, rows, sw) || !make_tmap_2d(&p.b_up, dt, w1, k, M, row, 64, rows, sw))
      return false;
  } else if (!(p.whole ? make_tmap_3d(&p.b, dt, w0, 64, M, k / 64, row, 128, 64, rows, p.kc, sw)
                       : make_tmap_2d(&p.b, dt, w0, k, M, row, 64, rows, sw))) {
    return false;
  }
  return p.whole ? make_tmap_3d(&p.a, dt, a, 64, T, k / 64, 2 * lda, 128, 64, tb, p.kc, sw)
                 : make_tmap_2d(&p.a, dt, a, k, T, 2 * lda, 64, tb, sw);
}

lmoe_status norm_args(int T, int d, const void* w, float eps, bool mx) {
  if (T < 0 || d < 1 || !usable(w) || !(eps >= 0.0f) || std::isinf(eps)) return LMOE_ERR_INVALID_ARG;
  if (d % (mx ? 32 : 8) != 0 || d > kNormMaxWidth) return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}
lmoe_status row_args(const void* p, int64_t ld, int d) {
  if (!usable(p) || ld < d) return LMOE_ERR_INVALID_ARG;
  return ld % 8 == 0 ? LMOE_OK : LMOE_ERR_UNSUPPORTED;
}
#define FFN_TRY_STATUS(expr)            \
  do {                                  \
    const lmoe_status s_ = (expr);      \
    if (s_ != LMOE_OK) return s_;       \
  } while (0)

// whole: false in the self-test.
lmoe_status forward(lmoe_ffn_handle h, const void* x, int64_t ldx, int T, void* out, void* gate, void* up, bool whole,
                    cudaStream_t stream) {
  if (!h || !on_its_device(h) || T < 0 || T > h->cfg.max_tokens) return LMOE_ERR_INVALID_ARG;
  if (h->cfg.wfmt != LMOE_FFN_W_BF16) return LMOE_ERR_UNSUPPORTED;
  h->launches = 0;
  if (T == 0) return LMOE_OK;
  const int d = h->cfg.d_model, F = h->cfg.d_ff;
  FFN_TRY_STATUS(row_args(x, ldx, d));
  if (!usable(out) || (gate == nullptr) != (up == nullptr) || !aligned16(gate) || !aligned16(up))
    return LMOE_ERR_INVALID_ARG;
  // Up to 72 tokens stream the weights (ffn_skinny.cu), larger batches run on
  // pair tiles, K split where they are few.  Streaming against pair tiles, 64,
  // 72 and 80 tokens, weights from HBM: widths 7168 and 6144 55.2, 56.0 and 60.8 us
  // against 60.6, 60.9 and 61.0 us; 7168 and 2048 24.3, 24.9 and 26.4 us against
  // 26.0, 26.6 and 26.7 us; 2048 and 2048 13.7, 14.3 and 15.3 us against 14.0, 14.8
  // and 14.8 us.  One limit serves all widths, too high a one for blocks of few
  // weights: 1152 and 864 9.0, 9.6 and 10.0 us against 8.8, 9.7 and 9.7 us; 512 and
  // 512 7.8, 8.4 and 8.5 us against 7.6, 8.3 and 8.3 us; 256 and 256 lose at any
  // number (8 tokens 6.8 us against 6.2 us, 72 tokens 9.4 us against 7.6 us).
  if (T <= kSkinnyMaxTokens) {
    FfnSkinnyParams g = {}, n = {};
    g.T = n.T = T;
    g.M = F;
    n.M = d;
    g.chunks = ceil_div(d, 64);
    n.chunks = ceil_div(F, 64);
    if (ffn_skinny_plan(g, true) && ffn_skinny_plan(n, false)) {
      g.b1 = h->cfg.situ_beta;
      g.b2 = h->cfg.situ_linear_beta;
      g.err = n.err = h->err;
      g.out = h->hid;
      g.save_g = gate;
      g.save_u = up;
      n.out = out;
      if (!skinny_maps(g, x, ldx, h->w.gate, h->w.up, d, token_rows(g.tb, whole)) ||
          !skinny_maps(n, h->hid, F, h->w.down, nullptr, F, n.tb))
        return LMOE_ERR_CUDA;
      FFN_TRY(launch_ffn_skinny(g, true, h->cfg.act == LMOE_ACT_SWIGLU, stream));
      FFN_TRY(launch_ffn_skinny(n, false, 0, stream));
      h->launches = 2;
      return LMOE_OK;
    }
  }
  FfnPairParams p = {};
  p.b1 = h->cfg.situ_beta;
  p.b2 = h->cfg.situ_linear_beta;
  p.act = h->cfg.act == LMOE_ACT_SWIGLU;
  p.err = h->err;
  p.nprod = 1;
  p.M[0] = T;
  p.N[0] = F;
  p.nkb = ceil_div(d, 64);
  p.out[0] = h->hid;
  p.out[1] = gate;
  p.out[2] = up;
  if (!map_k(&p.a[0], x, d, T, ldx, token_rows(128, whole))) return LMOE_ERR_CUDA;
  int splits = ffn_split_plan(p, kFfnGateUp, h->split);
  if (splits > 1) {
    p.b[0] = h->gate[1];
    p.b[1] = h->up[1];
    FFN_TRY(launch_ffn_split(kFfnGateUp, p, splits, stream));
    p.early = 1;
  } else {
    const int tn = ffn_pair_tiles(p, kFfnGateUp, h->ctas);
    p.b[0] = h->gate[tn == 128];
    p.b[1] = h->up[tn == 128];
    p.b_half[0] = h->gate[1];
    p.b_half[1] = h->up[1];
    FFN_TRY(launch_ffn_pair(kFfnGateUp, p, tn, h->ctas, stream));
  }
  p.N[0] = d;
  p.nkb = ceil_div(F, 64);
  p.out[0] = out;
  if (!map_k(&p.a[0], h->hid, F, T, F)) return LMOE_ERR_CUDA;
  splits = ffn_split_plan(p, kFfnPlain, h->split);
  if (splits > 1) {
    p.b[0] = h->down[1];
    FFN_TRY(launch_ffn_split(kFfnPlain, p, splits, stream));
  } else {
    p.early = 0;
    const int tn = ffn_pair_tiles(p, kFfnPlain, h->ctas);
    p.b[0] = h->down[tn == 128];
    p.b_half[0] = h->down[1];
    FFN_TRY(launch_ffn_pair(kFfnPlain, p, tn, h->ctas, stream));
  }
  h->launches = 2;
  return LMOE_OK;
}

lmoe_status forward_mx(lmoe_ffn_handle h, const uint8_t* x, const uint8_t* x_scales, int T, void* out, bool whole,
                       cudaStream_t stream) {
  if (!h || !on_its_device(h) || T < 0 || T > h->cfg.max_tokens) return LMOE_ERR_INVALID_ARG;
  if (h->cfg.wfmt != LMOE_FFN_W_MXFP8) return LMOE_ERR_UNSUPPORTED;
  h->launches = 0;
  if (T == 0) return LMOE_OK;
  if (!usable(x) || !usable(x_scales) || !usable(out)) return LMOE_ERR_INVALID_ARG;
  const int d = h->cfg.d_model, F = h->cfg.d_ff;
  FfnMxSkinnyParams g = {}, n = {};
  g.T = n.T = T;
  g.M = F;
  n.M = d;
  g.nkb = ceil_div(d, 128);
  n.nkb = ceil_div(F, 128);
  if (ffn_mx_skinny_plan(g, true) && ffn_mx_skinny_plan(n, false)) {
    g.b1 = h->cfg.situ_beta;
    g.b2 = h->cfg.situ_linear_beta;
    g.err = n.err = h->err;
    g.kblks = d / 32;
    g.b[0] = h->gate[1];
    g.b[1] = h->up[1];
    g.sfb = h->m_gu_sf[1];
    g.row_sf = x_scales;
    g.out = h->hid;
    g.out_sf = h->hid_sf;
    n.b[0] = h->down[1];
    n.sfb = h->m_down_sf[1];
    n.row_sf = h->hid_sf;
    n.out = out;
    if (!map_mx(&g.a, x, d, T, token_rows(g.tb, whole)) || !map_mx(&n.a, h->hid, F, T, n.tb)) return LMOE_ERR_CUDA;
    FFN_TRY(launch_ffn_mx_skinny(g, true, h->cfg.act == LMOE_ACT_SWIGLU, stream));
    FFN_TRY(launch_ffn_mx_skinny(n, false, 0, stream));
    h->launches = 2;
    return LMOE_OK;
  }
  FFN_TRY(launch_mx_row_atoms(x_scales, T, d, h->x_sf, stream));
  FfnMxParams p = {};
  p.b1 = h->cfg.situ_beta;
  p.b2 = h->cfg.situ_linear_beta;
  p.act = h->cfg.act == LMOE_ACT_SWIGLU;
  p.err = h->err;
  p.sfa = h->m_x_sf;
  p.out = h->hid;
  p.out_sf = h->hid_sf;
  p.out_nkb = ceil_div(F, 128);
  p.M = T;
  p.N = F;
  p.nkb = ceil_div(d, 128);
  int tn = ffn_mx_tiles(p, true, h->ctas), i = tn == kMxTileN[1];
  p.b[0] = h->gate[i];
  p.b[1] = h->up[i];
  p.sfb = h->m_gu_sf[i];
  if (!map_mx(&p.a, x, d, T, token_rows(128, whole))) return LMOE_ERR_CUDA;
  FFN_TRY(launch_ffn_mx_pair(p, true, tn, h->ctas, stream));
  p.sfa = h->m_hid_sf;
  p.out = out;
  p.wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;   // d is a multiple of 32
  p.N = d;
  p.nkb = ceil_div(F, 128);
  tn = ffn_mx_tiles(p, false, h->ctas);
  i = tn == kMxTileN[1];
  p.b[0] = h->down[i];
  p.sfb = h->m_down_sf[i];
  if (!map_mx(&p.a, h->hid, F, T, 128)) return LMOE_ERR_CUDA;
  FFN_TRY(launch_ffn_mx_pair(p, false, tn, h->ctas, stream));
  h->launches = 3;
  return LMOE_OK;
}

}  // namespace

extern "C" {

lmoe_status lmoe_add_rms_norm(const void* x, int64_t ldx, const void* r, int64_t ldr, lmoe_stream_type stream_type,
                              int T, int d, const void* w, float eps, void* h, void* y, lmoe_norm_out fmt,
                              uint8_t* scale, cudaStream_t stream) {
  if ((fmt != LMOE_NORM_OUT_BF16 && fmt != LMOE_NORM_OUT_MXFP8) ||
      (stream_type != LMOE_STREAM_BF16 && stream_type != LMOE_STREAM_FP32))
    return LMOE_ERR_INVALID_ARG;
  const bool mx = fmt == LMOE_NORM_OUT_MXFP8;
  FFN_TRY_STATUS(norm_args(T, d, w, eps, mx));
  if (T == 0) return LMOE_OK;
  FFN_TRY_STATUS(row_args(x, ldx, d));
  if (r) {
    FFN_TRY_STATUS(row_args(r, ldr, d));
    if (!usable(h)) return LMOE_ERR_INVALID_ARG;
  }
  if (!usable(y) || (mx && !scale)) return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_add_rms_norm(x, ldx, r, ldr, stream_type == LMOE_STREAM_FP32, T, d, w, eps, h, y,
                                         mx ? scale : nullptr, 0, stream));
}

lmoe_status lmoe_add_rms_norm_backward_workspace(int T, int d, size_t* bytes) {
  if (!bytes || T < 0 || d < 1) return LMOE_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > kNormMaxWidth) return LMOE_ERR_UNSUPPORTED;
  *bytes = T == 0 ? 0 : 4 * rms_norm_bwd_partials(T, d);
  return LMOE_OK;
}

lmoe_status lmoe_add_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* dh,
                                       int64_t lddh, lmoe_stream_type stream_type, int T, int d, const void* w,
                                       float eps, void* dx, float* dw, void* ws, size_t ws_bytes,
                                       cudaStream_t stream) {
  if (stream_type != LMOE_STREAM_BF16 && stream_type != LMOE_STREAM_FP32) return LMOE_ERR_INVALID_ARG;
  FFN_TRY_STATUS(norm_args(T, d, w, eps, false));
  if (!usable(dw)) return LMOE_ERR_INVALID_ARG;
  if (T == 0) return cuda_status(cudaMemsetAsync(dw, 0, 4 * static_cast<size_t>(d), stream));
  FFN_TRY_STATUS(row_args(dy, lddy, d));
  FFN_TRY_STATUS(row_args(h, ldh, d));
  if (dh) FFN_TRY_STATUS(row_args(dh, lddh, d));
  if (!usable(dx) || !usable(ws) || ws_bytes < 4 * rms_norm_bwd_partials(T, d)) return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_rms_norm_bwd(dy, lddy, h, ldh, dh, lddh, stream_type == LMOE_STREAM_FP32, T, d, w, eps,
                                         dx, static_cast<float*>(ws), dw, 0, stream));
}

lmoe_status lmoe_add_rms_norm_selftest_timeout(int backward, const void* x, int T, int d, const void* w, void* y,
                                               float* dw, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FFN_TRY_STATUS(norm_args(T, d, w, 0.0f, false));
  FFN_TRY_STATUS(row_args(x, d, d));
  if (T < 1 || !usable(y)) return LMOE_ERR_INVALID_ARG;
  if (!backward) {
    // fewer values may take the form that waits for nothing
    if (static_cast<long long>(T) * d < 1 << 23) return LMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_add_rms_norm(x, d, nullptr, d, false, T, d, w, 0.0f, nullptr, y, nullptr, 16, stream));
  }
  if (!usable(dw) || !usable(ws) || ws_bytes < 4 * rms_norm_bwd_partials(T, d)) return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_rms_norm_bwd(x, d, x, d, nullptr, d, false, T, d, w, 0.0f, y, static_cast<float*>(ws), dw,
                                         16, stream));
}

lmoe_status lmoe_ffn_create(const lmoe_ffn_config* cfg, const lmoe_ffn_weights* w, cudaStream_t stream,
                            lmoe_ffn_handle* out) {
  if (!out) return LMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || !w) return LMOE_ERR_INVALID_ARG;
  const int d = cfg->d_model, F = cfg->d_ff;
  if (d < 1 || F < 1 || cfg->max_tokens < 1 || (cfg->act != LMOE_ACT_SITU && cfg->act != LMOE_ACT_SWIGLU) ||
      (cfg->wfmt != LMOE_FFN_W_BF16 && cfg->wfmt != LMOE_FFN_W_MXFP8) || (cfg->training != 0 && cfg->training != 1))
    return LMOE_ERR_INVALID_ARG;
  if (cfg->act == LMOE_ACT_SITU && !(cfg->situ_beta > 0.0f && cfg->situ_linear_beta > 0.0f &&
                                     std::isfinite(cfg->situ_beta) && std::isfinite(cfg->situ_linear_beta)))
    return LMOE_ERR_INVALID_ARG;
  const bool mx = cfg->wfmt == LMOE_FFN_W_MXFP8;
  if (!usable(w->gate) || !usable(w->up) || !usable(w->down)) return LMOE_ERR_INVALID_ARG;
  if (mx && (!usable(w->gate_s) || !usable(w->up_s) || !usable(w->down_s))) return LMOE_ERR_INVALID_ARG;
  if (d % (mx ? 32 : 8) || F % (mx ? 32 : 8) || (mx && cfg->training)) return LMOE_ERR_UNSUPPORTED;
  int dev = 0, major = 0, minor = 0;
  FFN_TRY(cudaGetDevice(&dev));
  FFN_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  FFN_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  if (major != 10 || minor != 3) return LMOE_ERR_UNSUPPORTED;
  lmoe_ffn_ctx* h = new (std::nothrow) lmoe_ffn_ctx;
  if (!h) return LMOE_ERR_OOM;
  h->cfg = *cfg;
  h->w = *w;
  h->device = dev;
  const size_t Tm = cfg->max_tokens, T256 = (Tm + 255) / 256 * 256;
  const auto pad = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t act_bytes = pad(Tm * F * (mx ? 1 : 2));
  // scale atoms: 512 bytes for 128 rows x 128 values
  const size_t kd = ceil_div(d, 128), kf = ceil_div(F, 128);
  const size_t x_sf = T256 / 128 * kd * 512, hid_sf = T256 / 128 * kf * 512;
  // the weights' atoms for both tile widths: two atoms for 192 rows, one for 128
  const int per[2] = {1024, 512};
  size_t gu_sf[2], down_sf[2], w_sf = 0;
  int gu_tiles[2], down_tiles[2];
  for (int i = 0; i < 2; ++i) {
    gu_tiles[i] = ceil_div(F, kMxTileN[i] / 2);
    down_tiles[i] = ceil_div(d, kMxTileN[i]);
    gu_sf[i] = gu_tiles[i] * kd * per[i];
    down_sf[i] = down_tiles[i] * kf * per[i];
    w_sf += gu_sf[i] + down_sf[i];
  }
  const size_t bytes = 256 + act_bytes * (cfg->training ? 3 : 1) + (mx ? x_sf + hid_sf + w_sf : 0);
  cudaError_t e = ffn_pair_ctas(&h->ctas);
  if (e == cudaSuccess) e = ffn_split_limits(&h->split);
  if (e == cudaSuccess) e = cudaMalloc(&h->pool, bytes);
  // the error flag, and the bytes of the scale atoms that nothing writes
  if (e == cudaSuccess) e = cudaMemsetAsync(h->pool, 0, 256, stream);
  if (e == cudaSuccess && mx)
    e = cudaMemsetAsync(static_cast<uint8_t*>(h->pool) + 256 + act_bytes, 0, x_sf + hid_sf, stream);
  if (e != cudaSuccess) {
    lmoe_ffn_destroy(h);
    return cuda_status(e);
  }
  uint8_t* base = static_cast<uint8_t*>(h->pool);
  h->err = reinterpret_cast<int*>(base);
  h->hid = base + 256;
  bool ok;
  if (mx) {
    h->x_sf = base + 256 + act_bytes;
    h->hid_sf = h->x_sf + x_sf;
    ok = map_atoms(&h->m_x_sf, h->x_sf, x_sf, 1) && map_atoms(&h->m_hid_sf, h->hid_sf, hid_sf, 1);
    uint8_t* at = h->hid_sf + hid_sf;
    for (int i = 0; i < 2 && ok && e == cudaSuccess; ++i) {
      const int box = kMxTileN[i] / 2;
      h->gu_sf[i] = at;
      h->down_sf[i] = at + gu_sf[i];
      at += gu_sf[i] + down_sf[i];
      e = launch_mx_weight_atoms(w->gate_s, w->up_s, F, d, kMxTileN[i], gu_tiles[i], h->gu_sf[i], stream);
      if (e == cudaSuccess)
        e = launch_mx_weight_atoms(w->down_s, nullptr, d, F, kMxTileN[i], down_tiles[i], h->down_sf[i], stream);
      ok = map_mx(&h->gate[i], w->gate, d, F, box) && map_mx(&h->up[i], w->up, d, F, box) &&
           map_mx(&h->down[i], w->down, F, d, box) && map_atoms(&h->m_gu_sf[i], h->gu_sf[i], gu_sf[i], per[i] / 512) &&
           map_atoms(&h->m_down_sf[i], h->down_sf[i], down_sf[i], per[i] / 512);
    }
  } else {
    h->dg = base + 256 + act_bytes;
    h->du = base + 256 + 2 * act_bytes;
    ok = true;
    for (int i = 0; i < 2; ++i)
      ok = ok && map_k(&h->gate[i], w->gate, d, F, d, 128 >> i) && map_k(&h->up[i], w->up, d, F, d, 128 >> i) &&
           map_k(&h->down[i], w->down, F, d, F, 128 >> i);
    ok = ok && map_n(&h->gate_n, w->gate, d, F, d) && map_n(&h->up_n, w->up, d, F, d) &&
         map_n(&h->down_n, w->down, F, d, F);
  }
  // calls on other streams may follow: the workspace is ready when this returns
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || !ok) {
    lmoe_ffn_destroy(h);
    return e != cudaSuccess ? cuda_status(e) : LMOE_ERR_CUDA;
  }
  *out = h;
  return LMOE_OK;
}

lmoe_status lmoe_ffn_destroy(lmoe_ffn_handle h) {
  if (!h) return LMOE_OK;
  cudaError_t e = cudaSuccess;
  if (h->pool) e = cudaFree(h->pool);   // waits for the device
  delete h;
  return cuda_status(e);
}

lmoe_status lmoe_ffn_forward(lmoe_ffn_handle h, const void* x, int64_t ldx, int T, void* out, void* gate, void* up,
                             cudaStream_t stream) {
  return forward(h, x, ldx, T, out, gate, up, true, stream);
}

lmoe_status lmoe_ffn_backward(lmoe_ffn_handle h, const void* x, int64_t ldx, const void* gate, const void* up,
                              const void* dy, int64_t lddy, int T, void* dx, void* dwg, void* dwu, void* dwd,
                              cudaStream_t stream) {
  if (!h || !on_its_device(h) || T < 0 || T > h->cfg.max_tokens) return LMOE_ERR_INVALID_ARG;
  if (h->cfg.wfmt != LMOE_FFN_W_BF16 || !h->cfg.training) return LMOE_ERR_UNSUPPORTED;
  h->launches = 0;
  const int d = h->cfg.d_model, F = h->cfg.d_ff;
  if (!aligned16(dx) || !aligned16(dwg) || !aligned16(dwu) || !aligned16(dwd)) return LMOE_ERR_INVALID_ARG;
  if (T == 0) {
    for (void* w : {dwg, dwu, dwd})
      if (w) FFN_TRY(cudaMemsetAsync(w, 0, 2 * static_cast<size_t>(d) * F, stream));
    return LMOE_OK;
  }
  FFN_TRY_STATUS(row_args(x, ldx, d));
  FFN_TRY_STATUS(row_args(dy, lddy, d));
  if (!usable(gate) || !usable(up)) return LMOE_ERR_INVALID_ARG;
  if (!dx && !dwg && !dwu && !dwd) return LMOE_OK;

  FfnPairParams p = {};
  p.b1 = h->cfg.situ_beta;
  p.b2 = h->cfg.situ_linear_beta;
  p.act = h->cfg.act == LMOE_ACT_SWIGLU;
  p.err = h->err;
  // dhid = dy down, and its activation gradient
  p.nprod = 1;
  p.b[0] = h->down_n;
  p.in_g = gate;
  p.in_u = up;
  p.out[0] = h->dg;
  p.out[1] = h->du;
  p.out[2] = h->hid;
  p.M[0] = T;
  p.N[0] = F;
  p.nkb = ceil_div(d, 64);
  if (!map_k(&p.a[0], dy, d, T, lddy)) return LMOE_ERR_CUDA;
  int splits = ffn_split_plan(p, kFfnDHid, h->split);
  if (splits > 1) {
    FFN_TRY(launch_ffn_split(kFfnDHid, p, splits, stream));
  } else {
    FFN_TRY(launch_ffn_pair(kFfnDHid, p, ffn_pair_tiles(p, kFfnDHid, h->ctas), h->ctas, stream));
  }
  h->launches = 1;
  // the gradients: dx = [dg | du] [gate ; up], dw = dg^T x, du^T x, dy^T hid, in one launch unless dx is split
  FfnPairParams w = p;
  w.nprod = 0;
  bool ok = true;
  if (dx) {
    w.M[0] = T;
    w.N[0] = d;
    w.out[0] = dx;
    w.cat = 1;
    w.nkb_cat = ceil_div(F, 64);
    w.b[0] = h->gate_n;
    w.b_cat = h->up_n;
    ok = map_k(&w.a[0], h->dg, F, T, F) && map_k(&w.a_cat, h->du, F, T, F);
    w.nprod = 1;
    w.early = splits > 1;      // behind a split dhid
    splits = ffn_split_plan(w, kFfnGrads, h->split);
    if (splits > 1) {
      p = w;
      w.nprod = w.cat = 0;
    }
  }
  const bool apart = p.cat;    // p is dx, w the rest
  const auto add_dw = [&](const void* a, long long lda, int M, const void* b, long long ldb, int N, void* out) {
    const int i = w.nprod++;
    w.M[i] = M;
    w.N[i] = N;
    w.out[i] = out;
    return map_n(&w.a[i], a, M, T, lda) && map_n(&w.b[i], b, N, T, ldb);
  };
  if (dwg) ok = ok && add_dw(h->dg, F, F, x, ldx, d, dwg);
  if (dwu) ok = ok && add_dw(h->du, F, F, x, ldx, d, dwu);
  if (dwd) ok = ok && add_dw(dy, lddy, d, h->hid, F, F, dwd);
  if (!ok) return LMOE_ERR_CUDA;
  w.nkb = ceil_div(T, 64);
  w.early = apart;      // the weight gradients run beside dx
  const int tn = w.nprod > 0 ? ffn_pair_tiles(w, kFfnGrads, h->ctas) : 0;
  if (apart) {
    // Two splits rather than four where dx then leaves the weight gradients the
    // CTAs that they take: 256 tokens at 768 x 768 14.1 us against 15.8 us.
    const int tiles = p.tile_end[0], others = w.nprod > 0 ? ffn_pair_grid(w, h->ctas) : 0;
    if (splits == 4 && 8 * tiles + others > h->ctas && 4 * tiles + others <= h->ctas) splits = 2;
    FFN_TRY(launch_ffn_split(kFfnGrads, p, splits, stream));
    ++h->launches;
  }
  if (w.nprod > 0) {
    FFN_TRY(launch_ffn_pair(kFfnGrads, w, tn, h->ctas, stream));
    ++h->launches;
  }
  return LMOE_OK;
}

lmoe_status lmoe_ffn_forward_mx(lmoe_ffn_handle h, const uint8_t* x, const uint8_t* x_scales, int T, void* out,
                                cudaStream_t stream) {
  return forward_mx(h, x, x_scales, T, out, true, stream);
}

lmoe_status lmoe_ffn_selftest_timeout(lmoe_ffn_handle h, const void* x, const uint8_t* x_scales, int T, void* out,
                                      cudaStream_t stream) {
  if (!h || T < 1) return LMOE_ERR_INVALID_ARG;
  if (h->cfg.wfmt == LMOE_FFN_W_MXFP8)
    return forward_mx(h, static_cast<const uint8_t*>(x), x_scales, T, out, false, stream);
  return forward(h, x, h->cfg.d_model, T, out, nullptr, nullptr, false, stream);
}

lmoe_status lmoe_ffn_sync_status(lmoe_ffn_handle h, cudaStream_t stream) {
  if (!h || !on_its_device(h)) return LMOE_ERR_INVALID_ARG;
  FFN_TRY(cudaStreamSynchronize(stream));
  int flag = 0;
  FFN_TRY(cudaMemcpy(&flag, h->err, sizeof(flag), cudaMemcpyDeviceToHost));
  if (flag == 0) return LMOE_OK;
  FFN_TRY(cudaMemset(h->err, 0, sizeof(flag)));
  return LMOE_ERR_TIMEOUT;
}

int lmoe_ffn_last_launch_count(lmoe_ffn_handle h) { return h ? h->launches : 0; }

}  // extern "C"
