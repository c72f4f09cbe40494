// C ABI of the norms on both sides of a block, of the product with bias, activation
// and residual, and of the AdamW step: argument checks, workspaces, tensor maps,
// launch sequences.
#include <cmath>
#include <new>
#include <vector>

#include "../../include/lmoe_block.h"
#include "block_internal.h"
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "tmap.h"

using namespace lmoe;

struct lmoe_linear_ctx {
  lmoe_linear_config cfg;
  const void *w, *bias;
  int device = 0;               // where the workspace lies
  int ctas = 0;                 // resident CTAs of the pair kernels
  FfnSplitLimits split = {};
  void* pool = nullptr;
  int *err = nullptr, *done = nullptr;
  float* part = nullptr;
  void* dz = nullptr;
  CUtensorMap w_k[2];           // K contiguous, boxes of 64 K values x 128 and 64 rows
  CUtensorMap w_n;              // the same memory as an N contiguous operand, boxes of 64 x 64
  int launches = 0;
};

struct lmoe_adamw_ctx {
  lmoe_adamw_config cfg;
  int device = 0;
  void* pool = nullptr;
  std::vector<AdamTensor> tensors;
  std::vector<int> chunks;      // of each tensor
  AdamTensor* dev = nullptr;
  int *owner = nullptr, *done = nullptr;
  int vectors = 1;              // of a chunk
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
#define BLOCK_TRY(expr)                            \
  do {                                             \
    const cudaError_t e_ = (expr);                 \
    if (e_ != cudaSuccess) return cuda_status(e_); \
  } while (0)
#define BLOCK_TRY_STATUS(expr)          \
  do {                                  \
    const lmoe_status s_ = (expr);      \
    if (s_ != LMOE_OK) return s_;       \
  } while (0)

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool usable(const void* p) { return p && aligned16(p); }
int ceil_div(int a, int b) { return (a + b - 1) / b; }
lmoe_status row_args(const void* p, int64_t ld, int d) {
  if (!usable(p) || ld < d) return LMOE_ERR_INVALID_ARG;
  return ld % 8 == 0 ? LMOE_OK : LMOE_ERR_UNSUPPORTED;
}
// The stream of a call, which may be NULL, is one of the current device: the
// handle's memory has to lie there.
template <class H>
bool on_its_device(const H* h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}
lmoe_status this_device(int* dev) {
  int major = 0, minor = 0;
  BLOCK_TRY(cudaGetDevice(dev));
  BLOCK_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev));
  BLOCK_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev));
  return major == 10 && minor == 3 ? LMOE_OK : LMOE_ERR_UNSUPPORTED;
}

// K-contiguous bf16 operand [rows][K]: boxes of 64 K values x `box` rows.
bool map_k(CUtensorMap* m, const void* base, int K, int rows, long long ld, int box = 128) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, K, rows, 2 * ld, 64, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}
// The transposed use of [K][N]: boxes of 64 N values x 64 K rows.
bool map_n(CUtensorMap* m, const void* base, int N, int K, long long ld) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, N, K, 2 * ld, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

// ------------------------------------------------------------------- norms
lmoe_status norm_args(const lmoe_gated_norm_args* a, bool mx) {
  if (!a || a->T < 0 || a->d < 1 || !usable(a->w_post) || !usable(a->w_next) || !(a->eps >= 0.0f) ||
      std::isinf(a->eps) || !std::isfinite(a->stream_scale) || !std::isfinite(a->branch_scale) ||
      (a->stream_type != LMOE_STREAM_BF16 && a->stream_type != LMOE_STREAM_FP32) || a->gate_type < LMOE_GATE_NONE ||
      a->gate_type > LMOE_GATE_TOKEN)
    return LMOE_ERR_INVALID_ARG;
  if (a->d % (mx ? 32 : 8) != 0 || a->d > kGatedNormMaxWidth) return LMOE_ERR_UNSUPPORTED;
  if (a->gate_type == LMOE_GATE_CHANNEL && !usable(a->gate)) return LMOE_ERR_INVALID_ARG;
  if (a->T == 0) return LMOE_OK;
  BLOCK_TRY_STATUS(row_args(a->y, a->ldy, a->d));
  BLOCK_TRY_STATUS(row_args(a->stream, a->lds, a->d));
  if (a->gate_type == LMOE_GATE_TOKEN) BLOCK_TRY_STATUS(row_args(a->gate, a->ldgate, a->d));
  return LMOE_OK;
}
GatedNorm norm_of(const lmoe_gated_norm_args* a) {
  GatedNorm g = {};
  g.y = a->y;
  g.stream = a->stream;
  g.gate = a->gate_type == LMOE_GATE_NONE ? nullptr : a->gate;
  g.w_post = a->w_post;
  g.w_next = a->w_next;
  g.ldy = a->ldy;
  g.lds = a->lds;
  g.ldg = a->ldgate;
  g.T = a->T;
  g.d = a->d;
  g.fp32 = a->stream_type == LMOE_STREAM_FP32;
  g.gate_type = a->gate_type;
  g.a = a->stream_scale;
  g.b = a->branch_scale;
  g.eps = a->eps;
  return g;
}

// ------------------------------------------------------------------ linear
// whole: false in the self-test, whose copies of the tokens bring half of the rows
// that a stage waits for.
lmoe_status linear_forward(lmoe_linear_handle h, const void* x, int64_t ldx, int T, const void* res, int64_t ldr,
                           lmoe_stream_type type, void* out, void* pre, bool whole, cudaStream_t stream) {
  if (!h || !on_its_device(h) || T < 0 || T > h->cfg.max_tokens ||
      (type != LMOE_STREAM_BF16 && type != LMOE_STREAM_FP32))
    return LMOE_ERR_INVALID_ARG;
  if (T > kMostRows) return LMOE_ERR_UNSUPPORTED;
  h->launches = 0;
  if (T == 0) return LMOE_OK;
  const int K = h->cfg.d_in, N = h->cfg.d_out;
  BLOCK_TRY_STATUS(row_args(x, ldx, K));
  if (res) BLOCK_TRY_STATUS(row_args(res, ldr, N));
  if (!usable(out) || !aligned16(pre)) return LMOE_ERR_INVALID_ARG;
  LinearEpilogue lin = {};
  lin.bias = h->bias;
  lin.res = res;
  lin.ldr = ldr;
  lin.fp32 = res && type == LMOE_STREAM_FP32;
  lin.act = h->cfg.act;
  const auto token_rows = [&](int rows) { return whole ? rows : rows / 2; };
  // Up to 72 tokens stream the weights (up to 128 where that splits a long K), larger
  // batches run on pair tiles, K split where they are few: the feed-forward block's kernels.
  if (T <= kSkinnyWideTokens) {
    FfnSkinnyParams p = {};
    p.T = T;
    p.M = N;
    p.chunks = ceil_div(K, 64);
    if (ffn_skinny_plan(p, false, kSkinnyWideTokens)) {
      constexpr CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
      constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
      const uint64_t k = K, row = 2 * k;
      p.whole = K % 64 == 0;
      const bool ok =
          p.whole ? make_tmap_3d(&p.b, dt, h->w, 64, N, k / 64, row, 128, 64, p.rows, p.kc, sw) &&
                        make_tmap_3d(&p.a, dt, x, 64, T, k / 64, 2 * ldx, 128, 64, token_rows(p.tb), p.kc, sw)
                  : make_tmap_2d(&p.b, dt, h->w, k, N, row, 64, p.rows, sw) &&
                        make_tmap_2d(&p.a, dt, x, k, T, 2 * ldx, 64, token_rows(p.tb), sw);
      if (!ok) return LMOE_ERR_CUDA;
      p.out = out;
      p.save_g = pre;
      p.lin = lin;
      p.err = h->err;
      BLOCK_TRY(launch_linear_skinny(p, stream));
      h->launches = 1;
      return LMOE_OK;
    }
  }
  FfnPairParams p = {};
  p.err = h->err;
  p.lin = lin;
  p.nprod = 1;
  p.M[0] = T;
  p.N[0] = N;
  p.nkb = ceil_div(K, 64);
  p.out[0] = out;
  p.out[1] = pre;
  if (!map_k(&p.a[0], x, K, T, ldx, token_rows(128))) return LMOE_ERR_CUDA;
  const int splits = ffn_split_plan(p, kFfnLinear, h->split);
  if (splits > 1) {
    p.b[0] = h->w_k[1];
    BLOCK_TRY(launch_ffn_split(kFfnLinear, p, splits, stream));
  } else {
    const int tn = ffn_pair_tiles(p, kFfnLinear, h->ctas);
    p.b[0] = h->w_k[tn == 128];
    p.b_half[0] = h->w_k[1];
    BLOCK_TRY(launch_ffn_pair(kFfnLinear, p, tn, h->ctas, stream));
  }
  h->launches = 1;
  return LMOE_OK;
}

// ------------------------------------------------------------------- AdamW
constexpr int64_t kAdamMaxValues = int64_t{1} << 40;

lmoe_status tensor_args(const lmoe_adamw_tensor& t, bool mx) {
  if (t.n < 0 || t.first % 32 != 0 || (t.param_fp32 != 0 && t.param_fp32 != 1) || (t.param_fp32 && t.master) ||
      !(t.weight_decay >= 0.0f) || std::isinf(t.weight_decay))
    return LMOE_ERR_INVALID_ARG;
  if (t.n == 0) return LMOE_OK;
  if (!usable(t.param) || !aligned16(t.master) || !usable(t.m) || !usable(t.v) ||
      (mx && (!t.m_scale || !t.v_scale)))
    return LMOE_ERR_INVALID_ARG;
  return t.n > kAdamMaxValues ? LMOE_ERR_UNSUPPORTED : LMOE_OK;
}

}  // namespace

extern "C" {

lmoe_status lmoe_gated_add_norm(const lmoe_gated_norm_args* a, void* h_out, void* o, lmoe_norm_out fmt,
                                uint8_t* scale, cudaStream_t stream) {
  if (fmt != LMOE_NORM_OUT_BF16 && fmt != LMOE_NORM_OUT_MXFP8) return LMOE_ERR_INVALID_ARG;
  const bool mx = fmt == LMOE_NORM_OUT_MXFP8;
  BLOCK_TRY_STATUS(norm_args(a, mx));
  if (a->T == 0) return LMOE_OK;
  if (!usable(h_out) || !usable(o) || (mx && !scale)) return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_gated_norm(norm_of(a), h_out, o, mx ? scale : nullptr, stream));
}

lmoe_status lmoe_gated_add_norm_backward_workspace(int T, int d, size_t* bytes) {
  if (!bytes || T < 0 || d < 1) return LMOE_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > kGatedNormMaxWidth) return LMOE_ERR_UNSUPPORTED;
  *bytes = 4 * gated_norm_bwd_partials(T, d);
  return LMOE_OK;
}

lmoe_status lmoe_gated_add_norm_backward(const lmoe_gated_norm_args* a, const void* go, int64_t ldgo, const void* gh,
                                         int64_t ldgh, void* dy, void* dr, float* dw_post, float* dw_next, void* dgate,
                                         void* ws, size_t ws_bytes, cudaStream_t stream) {
  BLOCK_TRY_STATUS(norm_args(a, false));
  const bool channel = a->gate_type == LMOE_GATE_CHANNEL;
  if (!usable(dw_post) || !usable(dw_next) || (channel && !usable(dgate))) return LMOE_ERR_INVALID_ARG;
  if (a->T == 0) {
    const size_t n = 4 * static_cast<size_t>(a->d);
    BLOCK_TRY(cudaMemsetAsync(dw_post, 0, n, stream));
    BLOCK_TRY(cudaMemsetAsync(dw_next, 0, n, stream));
    if (channel) BLOCK_TRY(cudaMemsetAsync(dgate, 0, n, stream));
    return LMOE_OK;
  }
  BLOCK_TRY_STATUS(row_args(go, ldgo, a->d));
  if (gh) BLOCK_TRY_STATUS(row_args(gh, ldgh, a->d));
  if (!usable(dy) || !usable(dr) || (a->gate_type == LMOE_GATE_TOKEN && !usable(dgate)) || !usable(ws) ||
      ws_bytes < 4 * gated_norm_bwd_partials(a->T, a->d))
    return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_gated_norm_bwd(norm_of(a), go, ldgo, gh, ldgh, dy, dr, dw_post, dw_next, dgate,
                                           static_cast<float*>(ws), stream));
}

lmoe_status lmoe_gated_add_norm_selftest_timeout(int backward, const void* x, int T, int d, const void* w, void* out0,
                                                 void* out1, float* dw, void* ws, size_t ws_bytes,
                                                 cudaStream_t stream) {
  lmoe_gated_norm_args a = {};
  a.T = T;
  a.d = d;
  a.y = a.stream = x;
  a.ldy = a.lds = d;
  a.w_post = a.w_next = w;
  a.stream_scale = a.branch_scale = 1.0f;
  BLOCK_TRY_STATUS(norm_args(&a, false));
  if (T < 1 || !usable(out0) || !usable(out1)) return LMOE_ERR_INVALID_ARG;
  GatedNorm g = norm_of(&a);
  g.unsent = 16;
  if (!backward) return cuda_status(launch_gated_norm(g, out0, out1, nullptr, stream));
  if (!usable(dw) || !usable(ws) || ws_bytes < 4 * gated_norm_bwd_partials(T, d)) return LMOE_ERR_INVALID_ARG;
  return cuda_status(launch_gated_norm_bwd(g, x, d, nullptr, 0, out0, out1, dw, dw + d, nullptr,
                                           static_cast<float*>(ws), stream));
}

lmoe_status lmoe_linear_create(const lmoe_linear_config* cfg, const void* w, const void* bias, cudaStream_t stream,
                               lmoe_linear_handle* out) {
  if (!out) return LMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg) return LMOE_ERR_INVALID_ARG;
  const int K = cfg->d_in, N = cfg->d_out;
  if (K < 1 || N < 1 || cfg->max_tokens < 1 || cfg->act < LMOE_LINEAR_NONE || cfg->act > LMOE_LINEAR_GELU ||
      (cfg->training != 0 && cfg->training != 1) || !usable(w) || !aligned16(bias))
    return LMOE_ERR_INVALID_ARG;
  if (K % 8 || N % 8 || K > kMostRows || N > kMostRows) return LMOE_ERR_UNSUPPORTED;
  int dev = 0;
  BLOCK_TRY_STATUS(this_device(&dev));
  lmoe_linear_ctx* h = new (std::nothrow) lmoe_linear_ctx;
  if (!h) return LMOE_ERR_OOM;
  h->cfg = *cfg;
  h->w = w;
  h->bias = bias;
  h->device = dev;
  const auto pad = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t done = pad(4 * linear_dz_tiles(N)), part = pad(4 * linear_dz_partials(N));
  const size_t dz = pad(2 * static_cast<size_t>(cfg->max_tokens) * N);
  cudaError_t e = ffn_pair_ctas(&h->ctas);
  if (e == cudaSuccess) e = ffn_split_limits(&h->split);
  if (e == cudaSuccess) e = cudaMalloc(&h->pool, 256 + (cfg->training ? done + part + dz : 0));
  // the error flag and the counters
  if (e == cudaSuccess) e = cudaMemsetAsync(h->pool, 0, 256 + (cfg->training ? done : 0), stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);      // calls on other streams may follow
  const bool ok = e == cudaSuccess && map_k(&h->w_k[0], w, K, N, K) && map_k(&h->w_k[1], w, K, N, K, 64) &&
                  map_n(&h->w_n, w, K, N, K);
  if (!ok) {
    lmoe_linear_destroy(h);
    return e != cudaSuccess ? cuda_status(e) : LMOE_ERR_CUDA;
  }
  uint8_t* base = static_cast<uint8_t*>(h->pool);
  h->err = reinterpret_cast<int*>(base);
  h->done = reinterpret_cast<int*>(base + 256);
  h->part = reinterpret_cast<float*>(base + 256 + done);
  h->dz = base + 256 + done + part;
  *out = h;
  return LMOE_OK;
}

lmoe_status lmoe_linear_forward(lmoe_linear_handle h, const void* x, int64_t ldx, int T, const void* res, int64_t ldr,
                                lmoe_stream_type type, void* out, void* pre, cudaStream_t stream) {
  return linear_forward(h, x, ldx, T, res, ldr, type, out, pre, true, stream);
}

lmoe_status lmoe_linear_selftest_timeout(lmoe_linear_handle h, const void* x, int T, void* out, cudaStream_t stream) {
  if (!h || T < 1) return LMOE_ERR_INVALID_ARG;
  return linear_forward(h, x, h->cfg.d_in, T, nullptr, 0, LMOE_STREAM_BF16, out, nullptr, false, stream);
}

lmoe_status lmoe_linear_backward(lmoe_linear_handle h, const void* x, int64_t ldx, const void* dy, int64_t lddy,
                                 lmoe_stream_type type, const void* pre, int T, void* dx, void* dw, float* dbias,
                                 cudaStream_t stream) {
  if (!h || !on_its_device(h) || T < 0 || T > h->cfg.max_tokens ||
      (type != LMOE_STREAM_BF16 && type != LMOE_STREAM_FP32))
    return LMOE_ERR_INVALID_ARG;
  if (!h->cfg.training || T > kMostRows) return LMOE_ERR_UNSUPPORTED;
  h->launches = 0;
  const int K = h->cfg.d_in, N = h->cfg.d_out, act = h->cfg.act;
  if (!aligned16(dx) || !aligned16(dw) || !aligned16(dbias)) return LMOE_ERR_INVALID_ARG;
  if (T == 0) {
    if (dw) BLOCK_TRY(cudaMemsetAsync(dw, 0, 2 * static_cast<size_t>(K) * N, stream));
    if (dbias) BLOCK_TRY(cudaMemsetAsync(dbias, 0, 4 * static_cast<size_t>(N), stream));
    return LMOE_OK;
  }
  BLOCK_TRY_STATUS(row_args(x, ldx, K));
  BLOCK_TRY_STATUS(row_args(dy, lddy, N));
  if (act != LMOE_LINEAR_NONE && !usable(pre)) return LMOE_ERR_INVALID_ARG;
  if (!dx && !dw && !dbias) return LMOE_OK;
  const bool fp32 = type == LMOE_STREAM_FP32;
  // dz is dy itself where nothing changes it
  const bool made = (act != LMOE_LINEAR_NONE || fp32) && (dx || dw);
  const void* dz = made ? h->dz : dy;
  const int64_t lddz = made ? N : lddy;
  if (made || dbias) {
    BLOCK_TRY(launch_linear_dz(dy, lddy, fp32, act == LMOE_LINEAR_NONE ? nullptr : pre, act, T, N,
                               made ? h->dz : nullptr, dbias, h->part, h->done, stream));
    h->launches = 1;
  }
  const bool beside = dbias && !made;      // the sums run beside the products
  // dx = dz W and dw = dz^T x in one launch, unless dx is split
  FfnPairParams w = {}, p = {};
  w.err = h->err;
  int splits = 1;
  bool ok = true;
  if (dx) {
    w.nprod = 1;
    w.M[0] = T;
    w.N[0] = K;
    w.out[0] = dx;
    w.cat = 1;
    w.nkb_cat = w.nkb_dx = ceil_div(N, 64);
    w.b[0] = h->w_n;
    w.early = beside ? 2 : 0;
    ok = map_k(&w.a[0], dz, N, T, lddz);
    splits = ffn_split_plan(w, kFfnGrads, h->split);
    if (splits > 1) {
      p = w;
      w.nprod = w.cat = 0;
    }
  }
  if (dw) {
    const int i = w.nprod++;
    w.M[i] = N;
    w.N[i] = K;
    w.out[i] = dw;
    ok = ok && map_n(&w.a[i], dz, N, T, lddz) && map_n(&w.b[i], x, K, T, ldx);
  }
  if (!ok) return LMOE_ERR_CUDA;
  w.nkb = ceil_div(T, 64);
  w.early = beside || splits > 1;      // dw runs beside dx
  const int tn = w.nprod > 0 ? ffn_pair_tiles(w, kFfnGrads, h->ctas) : 0;
  if (splits > 1) {
    // as in the feed-forward block: two splits rather than four where dx then leaves dw the CTAs that it takes
    const int tiles = p.tile_end[0], others = w.nprod > 0 ? ffn_pair_grid(w, h->ctas) : 0;
    if (splits == 4 && 8 * tiles + others > h->ctas && 4 * tiles + others <= h->ctas) splits = 2;
    BLOCK_TRY(launch_ffn_split(kFfnGrads, p, splits, stream));
    ++h->launches;
  }
  if (w.nprod > 0) {
    BLOCK_TRY(launch_ffn_pair(kFfnGrads, w, tn, h->ctas, stream));
    ++h->launches;
  }
  return LMOE_OK;
}

lmoe_status lmoe_linear_sync_status(lmoe_linear_handle h, cudaStream_t stream) {
  if (!h || !on_its_device(h)) return LMOE_ERR_INVALID_ARG;
  BLOCK_TRY(cudaStreamSynchronize(stream));
  int flag = 0;
  BLOCK_TRY(cudaMemcpy(&flag, h->err, sizeof(flag), cudaMemcpyDeviceToHost));
  if (flag == 0) return LMOE_OK;
  BLOCK_TRY(cudaMemset(h->err, 0, sizeof(flag)));
  return LMOE_ERR_TIMEOUT;
}

int lmoe_linear_last_launch_count(lmoe_linear_handle h) { return h ? h->launches : 0; }

lmoe_status lmoe_linear_destroy(lmoe_linear_handle h) {
  if (!h) return LMOE_OK;
  cudaError_t e = cudaSuccess;
  if (h->pool) e = cudaFree(h->pool);   // waits for the device
  delete h;
  return cuda_status(e);
}

lmoe_status lmoe_adamw_create(const lmoe_adamw_config* cfg, const lmoe_adamw_tensor* tensors, int count,
                              cudaStream_t stream, lmoe_adamw_handle* out) {
  if (!out) return LMOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg || !tensors || count < 1 || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) ||
      !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(cfg->eps >= 0.0) || std::isinf(cfg->eps) ||
      (cfg->states != LMOE_ADAMW_FP32 && cfg->states != LMOE_ADAMW_MXFP8) || !cfg->step || !aligned(cfg->step, 8))
    return LMOE_ERR_INVALID_ARG;
  const bool mx = cfg->states == LMOE_ADAMW_MXFP8;
  int64_t all = 0;
  for (int i = 0; i < count; ++i) {
    BLOCK_TRY_STATUS(tensor_args(tensors[i], mx));
    all += tensors[i].n;
    if (all > kAdamMaxValues) return LMOE_ERR_UNSUPPORTED;
  }
  int dev = 0;
  BLOCK_TRY_STATUS(this_device(&dev));
  lmoe_adamw_ctx* h = new (std::nothrow) lmoe_adamw_ctx;
  if (!h) return LMOE_ERR_OOM;
  h->cfg = *cfg;
  h->device = dev;
  h->vectors = adamw_vectors(all, mx);
  const int64_t chunk = static_cast<int64_t>(h->vectors) * kAdamVector;
  std::vector<int> owner;
  try {
    for (int i = 0; i < count; ++i) {
      const lmoe_adamw_tensor& t = tensors[i];
      if (i % kAdamTensors == 0) h->chunks.push_back(static_cast<int>(owner.size()));      // a launch begins
      const int base = h->chunks.back();
      AdamTensor a = {};
      a.param = t.param;
      a.master = t.master;
      a.m = t.m;
      a.v = t.v;
      a.m_scale = t.m_scale;
      a.v_scale = t.v_scale;
      a.n = t.n;
      a.first = t.first;
      a.decay = t.weight_decay;
      a.fp32 = t.param_fp32;
      a.chunk0 = static_cast<int>(owner.size()) - base;
      h->tensors.push_back(a);
      owner.resize(owner.size() + static_cast<size_t>((t.n + chunk - 1) / chunk), i % kAdamTensors);
    }
    h->chunks.push_back(static_cast<int>(owner.size()));
  } catch (const std::bad_alloc&) {
    delete h;
    return LMOE_ERR_OOM;
  }
  const size_t table = (sizeof(AdamTensor) * h->tensors.size() + 255) / 256 * 256;
  cudaError_t e = cudaMalloc(&h->pool, 256 + table + 4 * owner.size());
  uint8_t* base = static_cast<uint8_t*>(h->pool);
  if (e == cudaSuccess) e = cudaMemsetAsync(base, 0, 256, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(base + 256, h->tensors.data(), sizeof(AdamTensor) * h->tensors.size(), cudaMemcpyHostToDevice,
                        stream);
  if (e == cudaSuccess && !owner.empty())
    e = cudaMemcpyAsync(base + 256 + table, owner.data(), 4 * owner.size(), cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);      // `owner` ends here
  if (e != cudaSuccess) {
    lmoe_adamw_destroy(h);
    return cuda_status(e);
  }
  h->done = reinterpret_cast<int*>(base);
  h->dev = reinterpret_cast<AdamTensor*>(base + 256);
  h->owner = reinterpret_cast<int*>(base + 256 + table);
  *out = h;
  return LMOE_OK;
}

lmoe_status lmoe_adamw_step(lmoe_adamw_handle h, const void* const* grads, const uint8_t* grad_fp32, float lr,
                            const float* lr_opt, const float* grad_scale_opt, cudaStream_t stream) {
  if (!h || !on_its_device(h) || !grads || !(lr >= 0.0f) || std::isinf(lr) || !aligned(lr_opt, 4) ||
      !aligned(grad_scale_opt, 4))
    return LMOE_ERR_INVALID_ARG;
  const int count = static_cast<int>(h->tensors.size());
  for (int i = 0; i < count; ++i)
    if (!aligned16(grads[i])) return LMOE_ERR_INVALID_ARG;
  h->launches = 0;
  const int launches = static_cast<int>(h->chunks.size()) - 1;
  AdamParams p;
  p.done = h->done;
  p.step = reinterpret_cast<long long*>(h->cfg.step);
  p.lr = lr;
  p.lr_dev = lr_opt;
  p.scale_dev = grad_scale_opt;
  p.beta1 = static_cast<float>(h->cfg.beta1);
  p.beta2 = static_cast<float>(h->cfg.beta2);
  p.rest1 = static_cast<float>(1.0 - h->cfg.beta1);
  p.rest2 = static_cast<float>(1.0 - h->cfg.beta2);
  p.log1 = static_cast<float>(std::log(h->cfg.beta1));
  p.log2 = static_cast<float>(std::log(h->cfg.beta2));
  p.eps = static_cast<float>(h->cfg.eps);
  p.seed = adamw_mix(h->cfg.seed);
  for (int l = 0; l < launches; ++l) {
    const int first = l * kAdamTensors;
    p.tensors = h->dev + first;
    p.owner = h->owner + h->chunks[l];
    p.chunks = h->chunks[l + 1] - h->chunks[l];
    p.vectors = h->vectors;
    p.last = l == launches - 1;
    for (int i = 0; i < kAdamTensors; ++i) {
      const bool there = first + i < count;
      if (i % 32 == 0) p.fp32[i / 32] = 0;
      p.grads[i] = there ? grads[first + i] : nullptr;
      if (there && grad_fp32 && grad_fp32[first + i]) p.fp32[i / 32] |= 1u << (i % 32);
    }
    if (p.chunks == 0 && !p.last) continue;
    BLOCK_TRY(launch_adamw(p, h->cfg.states == LMOE_ADAMW_MXFP8, stream));
    ++h->launches;
  }
  return LMOE_OK;
}

int lmoe_adamw_last_launch_count(lmoe_adamw_handle h) { return h ? h->launches : 0; }

lmoe_status lmoe_adamw_destroy(lmoe_adamw_handle h) {
  if (!h) return LMOE_OK;
  cudaError_t e = cudaSuccess;
  if (h->pool) e = cudaFree(h->pool);   // waits for the device
  delete h;
  return cuda_status(e);
}

}  // extern "C"
