// Residual addition with RMS normalisation, forward and backward.
//
//   h = r + x (in r's type),  y = w h rho,  rho = 1 / sqrt(mean(h^2) + eps)
//   dx = rho (w dy - h rho^2 mean(w dy h)) + dh,   dw = sum over rows of dy h rho
//
// Both passes move each value once and do a few operations on it: HBM bounds
// them.  A row is held in registers by a group of whole warps (16-byte
// vectors, VPT of them per thread) between the reduction and the output, so
// nothing is read twice.  Sums and the norm are fp32; the only roundings are
// those of the stored outputs.
#include "common.cuh"
#include "lmoe_internal.h"

namespace lmoe {
namespace {

// Eight consecutive values, as stored.
template <class T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

constexpr int kMaxRowWarps = 32;

// Sum over the `warps` warps of a row group; every thread gets it.  `slot`:
// the group's kMaxRowWarps floats of shared memory, used once per barrier.
__device__ __forceinline__ float group_sum(float v, int warps, float* slot) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int w = (threadIdx.x >> 5) % warps;
  if ((threadIdx.x & 31) == 0) slot[w] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < warps ? slot[threadIdx.x & 31] : 0.0f;
  return warp_sum(s);
}

struct NormParams {
  const __nv_bfloat16* x;
  const void* r;        // residual or null
  const __nv_bfloat16* w;
  void* h;              // r + x, written when r is given
  void* y;              // bf16 values or E4M3 codes
  uint8_t* scale;       // E8M0 per 32 values (MX output)
  long long ldx, ldr;
  int T, d, warps;      // warps per row
  float eps;
};

// R: type of the residual stream (bf16 or fp32); HAS_R: a residual is added;
// MX: output E4M3 codes with an E8M0 scale per 32 values.
template <class R, bool HAS_R, bool MX, int VPT>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float slots[kMaxRowWarps];
  const int group = (threadIdx.x >> 5) / p.warps;              // rows of the CTA
  const int groups = blockDim.x / (32 * p.warps);
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  const long long row = static_cast<long long>(blockIdx.x) * groups + group;
  const bool live = row < p.T;
  griddep_launch();
  griddep_wait();
  float v[VPT][8];
  Vec8<__nv_bfloat16> wv[VPT];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    wv[i].zero();
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (live && c < p.d) {
      Vec8<__nv_bfloat16> xv;
      xv.load(p.x + row * p.ldx + c);
      wv[i].load(p.w + c);
      xv.get(v[i]);
      if constexpr (HAS_R) {
        Vec8<R> rv;
        float f[8];
        rv.load(static_cast<const R*>(p.r) + row * p.ldr + c);
        rv.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += v[i][j];
        rv.set(f);       // the sum in the stream's type is what is stored and normalised
        rv.store(static_cast<R*>(p.h) + row * p.d + c);
        rv.get(v[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
  ss = group_sum(ss, p.warps, slots + (p.warps == 1 ? 0 : group * p.warps));
  const float rho = rsqrtf(ss / static_cast<float>(p.d) + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    float f[8];
    wv[i].get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= v[i][j] * rho;
    if constexpr (MX) {
      // a 32-value block is four consecutive lanes' vectors
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(fabsf(f[j])));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      // an infinity or NaN (exponent field 255) makes the block NaN: E8M0 byte 255
      const uint32_t s = m >= 0x7F800000u ? 255u : e4m3_block_scale(__uint_as_float(m));
      const float inv = s == 255u ? 1.0f : e8m0_to_f32(254u - s);
      uint32_t q[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j >> 2] |= static_cast<uint32_t>(f32_to_e4m3(f[j] * inv)) << (8 * (j & 3));
      if (live && c < p.d) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.d + c) = make_uint2(q[0], q[1]);
        if ((threadIdx.x & 3) == 0) p.scale[row * (p.d >> 5) + (c >> 5)] = static_cast<uint8_t>(s);
      }
    } else if (live && c < p.d) {
      Vec8<__nv_bfloat16> o;
      o.set(f);
      o.store(static_cast<__nv_bfloat16*>(p.y) + row * p.d + c);
    }
  }
}

struct NormBwdParams {
  const __nv_bfloat16* dy;
  const void* h;
  const void* dh;       // gradient along the residual stream, or null
  const __nv_bfloat16* w;
  void* dx;
  float* part;          // [gridDim.x * groups][d] partial sums of dw
  long long lddy, ldh, lddh;
  int T, d, warps;
  float eps;
};

// One CTA takes rows blockIdx.x * groups + group, + gridDim.x * groups, ...:
// the column sums of dw stay in its registers until the last row.
template <class R, bool HAS_DH, int VPT>
__global__ void __launch_bounds__(512) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float slots[2][2][kMaxRowWarps];
  const int group = (threadIdx.x >> 5) / p.warps;
  const int groups = blockDim.x / (32 * p.warps);
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  griddep_launch();
  griddep_wait();
  Vec8<__nv_bfloat16> wv[VPT];
  float acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    wv[i].zero();
    if (c < p.d) wv[i].load(p.w + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  int flip = 0;
  for (long long row0 = static_cast<long long>(blockIdx.x) * groups; row0 < p.T;
       row0 += static_cast<long long>(gridDim.x) * groups, flip ^= 1) {
    const long long row = row0 + group;
    const bool live = row < p.T;
    Vec8<__nv_bfloat16> gv[VPT];
    Vec8<R> hv[VPT], ev[VPT];
    float ss = 0.0f, sc = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      gv[i].zero();
      hv[i].zero();
      if (live && c < p.d) {
        gv[i].load(p.dy + row * p.lddy + c);
        hv[i].load(static_cast<const R*>(p.h) + row * p.ldh + c);
        if constexpr (HAS_DH) ev[i].load(static_cast<const R*>(p.dh) + row * p.lddh + c);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float g[8], h[8], w[8];
      gv[i].get(g);
      hv[i].get(h);
      wv[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += h[j] * h[j];
        sc += g[j] * w[j] * h[j];
      }
    }
    // two sums behind one barrier; the slots alternate between rows, so the
    // next row's writes cannot meet this row's reads
    ss = warp_sum(ss);
    sc = warp_sum(sc);
    if (p.warps > 1) {
      const int wi = (threadIdx.x >> 5) - group * p.warps, lane = threadIdx.x & 31;
      float* s0 = slots[flip][0] + group * p.warps;
      float* s1 = slots[flip][1] + group * p.warps;
      if (lane == 0) s0[wi] = ss, s1[wi] = sc;
      __syncthreads();
      ss = warp_sum(lane < p.warps ? s0[lane] : 0.0f);
      sc = warp_sum(lane < p.warps ? s1[lane] : 0.0f);
    }
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const float rho = rsqrtf(ss / static_cast<float>(p.d) + p.eps);
    const float k = rho * rho * (sc * inv_d);
    if (live) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (t + i * stride) * 8;
        if (c >= p.d) continue;
        float g[8], h[8], w[8], e[8], o[8];
        gv[i].get(g);
        hv[i].get(h);
        wv[i].get(w);
        if constexpr (HAS_DH) ev[i].get(e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = rho * (w[j] * g[j] - h[j] * k);
          if constexpr (HAS_DH) o[j] += e[j];
          acc[i][j] += g[j] * (h[j] * rho);
        }
        Vec8<R> ov;
        ov.set(o);
        ov.store(static_cast<R*>(p.dx) + row * p.d + c);
      }
    }
  }
  float* part = p.part + (static_cast<size_t>(blockIdx.x) * groups + group) * p.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    if (c < p.d) {
      reinterpret_cast<float4*>(part + c)[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      reinterpret_cast<float4*>(part + c)[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// dw[c] = sum of part[0..n)[c], in a fixed order: thread (x, y) adds rows y,
// y + 32, ... of its four columns, and the 32 sums are added in order.
constexpr int kSumCols = 8, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows) sum_rows_kernel(const float* part, int n, int d, float* out) {
  __shared__ float4 s[kSumRows][kSumCols];
  griddep_launch();
  griddep_wait();
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int c = (blockIdx.x * kSumCols + x) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
#pragma unroll 4
    for (int r = y; r < n; r += kSumRows) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<size_t>(r) * d + c);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  s[y][x] = a;
  __syncthreads();
  if (y == 0 && c < d) {
    for (int r = 1; r < kSumRows; ++r) {
      const float4 v = s[r][x];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    *reinterpret_cast<float4*>(out + c) = a;
  }
}

// Row layout: vectors per thread, warps per row, rows per CTA.
struct RowPlan {
  int vpt, warps, groups;
};
RowPlan row_plan(int d, int max_threads) {
  RowPlan r;
  const int nvec = d / 8;
  r.vpt = nvec <= max_threads ? 1 : nvec <= 2 * max_threads ? 2 : 4;
  const int threads = (nvec + r.vpt - 1) / r.vpt;
  r.warps = (threads + 31) / 32;
  r.groups = r.warps >= 8 ? 1 : 8 / r.warps;
  return r;
}

template <class R, bool HAS_R, bool MX>
cudaError_t launch_fwd(const NormParams& p, const RowPlan& r, cudaStream_t s) {
  const dim3 grid((p.T + r.groups - 1) / r.groups), block(32 * r.warps * r.groups);
  switch (r.vpt) {
    case 1: return launch_pdl(add_rms_norm_kernel<R, HAS_R, MX, 1>, grid, block, 0, s, p);
    case 2: return launch_pdl(add_rms_norm_kernel<R, HAS_R, MX, 2>, grid, block, 0, s, p);
    default: return launch_pdl(add_rms_norm_kernel<R, HAS_R, MX, 4>, grid, block, 0, s, p);
  }
}

template <class R, bool HAS_DH>
cudaError_t launch_bwd(const NormBwdParams& p, const RowPlan& r, int grid, cudaStream_t s) {
  const dim3 block(32 * r.warps * r.groups);
  switch (r.vpt) {
    case 1: return launch_pdl(rms_norm_bwd_kernel<R, HAS_DH, 1>, dim3(grid), block, 0, s, p);
    case 2: return launch_pdl(rms_norm_bwd_kernel<R, HAS_DH, 2>, dim3(grid), block, 0, s, p);
    default: return launch_pdl(rms_norm_bwd_kernel<R, HAS_DH, 4>, dim3(grid), block, 0, s, p);
  }
}

constexpr int kBwdCtas = 304;    // two CTAs for each SM
int bwd_grid(int T, const RowPlan& r) {
  const int need = (T + r.groups - 1) / r.groups;
  return need < kBwdCtas ? need : kBwdCtas;
}
RowPlan bwd_plan(int d) { return row_plan(d, 512); }

}  // namespace

size_t rms_norm_bwd_partials(int T, int d) {
  const RowPlan r = bwd_plan(d);
  return static_cast<size_t>(bwd_grid(T, r)) * r.groups * d;
}

cudaError_t launch_add_rms_norm(const void* x, long long ldx, const void* r, long long ldr, bool r_fp32, int T, int d,
                                const void* w, float eps, void* h, void* y, uint8_t* scale, cudaStream_t s) {
  NormParams p = {};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.r = r;
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.h = h;
  p.y = y;
  p.scale = scale;
  p.ldx = ldx;
  p.ldr = ldr;
  p.T = T;
  p.d = d;
  p.eps = eps;
  const RowPlan pl = row_plan(d, 1024);
  p.warps = pl.warps;
  if (!r) return scale ? launch_fwd<float, false, true>(p, pl, s) : launch_fwd<float, false, false>(p, pl, s);
  if (r_fp32) return scale ? launch_fwd<float, true, true>(p, pl, s) : launch_fwd<float, true, false>(p, pl, s);
  return scale ? launch_fwd<__nv_bfloat16, true, true>(p, pl, s) : launch_fwd<__nv_bfloat16, true, false>(p, pl, s);
}

cudaError_t launch_rms_norm_bwd(const void* dy, long long lddy, const void* h, long long ldh, const void* dh,
                                long long lddh, bool h_fp32, int T, int d, const void* w, float eps, void* dx,
                                float* part, float* dw, cudaStream_t s) {
  NormBwdParams p = {};
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.h = h;
  p.dh = dh;
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.dx = dx;
  p.part = part;
  p.lddy = lddy;
  p.ldh = ldh;
  p.lddh = lddh;
  p.T = T;
  p.d = d;
  p.eps = eps;
  const RowPlan pl = bwd_plan(d);
  p.warps = pl.warps;
  const int grid = bwd_grid(T, pl);
  cudaError_t e;
  if (h_fp32)
    e = dh ? launch_bwd<float, true>(p, pl, grid, s) : launch_bwd<float, false>(p, pl, grid, s);
  else
    e = dh ? launch_bwd<__nv_bfloat16, true>(p, pl, grid, s) : launch_bwd<__nv_bfloat16, false>(p, pl, grid, s);
  if (e != cudaSuccess) return e;
  const int cols = 4 * kSumCols;
  return launch_pdl(sum_rows_kernel, dim3((d + cols - 1) / cols), dim3(kSumCols * kSumRows), 0, s,
                    static_cast<const float*>(part), grid * pl.groups, d, dw);
}

}  // namespace lmoe
