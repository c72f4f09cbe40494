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
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "moe_common.cuh"
#include "norm_vec.cuh"

namespace lmoe {
namespace {

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
  int groups, stages;   // ring form: rows at a time, rows in flight for each
  int unsent;           // bytes of a row that are waited for and never copied: 0, or 16 in the self-test of the waits
  float eps;
};
// Ring forms: compute warps of a CTA at most, rows in flight of a group, shared
// memory.  Many vectors per thread leave fewer warps their registers: a thread
// has 64 with 28 warps and the copying one, 128 with 15.
constexpr int kRingMaxWarps = 28, kRingMaxStages = 8;
constexpr int ring_warps(int vpt) { return vpt <= 2 ? kRingMaxWarps : 15; }
constexpr int kRingSmem = 208 * 1024;
static_assert(10 * kNormMaxWidth <= kRingSmem, "a row of the widest types fits");

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
  for (int i = 0; i < VPT; ++i) write_vec<MX>(p.y, p.scale, p.d, row, (t + i * stride) * 8, live, v[i], wv[i], rho);
}

// The forward pass on many rows: one CTA per SM, each group of warps taking
// every (gridDim.x * groups)-th row from a ring of shared memory that a warp
// of its own fills by bulk copies, several rows ahead; a slot is free again as
// soon as its row is in registers.
template <class R, bool HAS_R, bool MX, int VPT>
__global__ void __launch_bounds__(32 * ring_warps(VPT) + 32)
    add_rms_norm_ring_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRingMaxWarps * kRingMaxStages], empty[kRingMaxWarps * kRingMaxStages];
  __shared__ float slots[2][kRingMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / p.warps;                      // == groups: the copying warp
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  const uint32_t x_bytes = 2 * p.d, r_bytes = HAS_R ? sizeof(R) * p.d : 0, row_bytes = x_bytes + r_bytes;
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  if (threadIdx.x < p.groups * p.stages) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], p.warps);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch();
  griddep_wait();
  if (warp == p.groups * p.warps) {
    if (lane < p.groups) {   // lane g feeds group g
      int s = 0;
      uint32_t phase = 1;    // the first round of the ring finds its slots empty
      bool ok = true;
      for (long long row = static_cast<long long>(blockIdx.x) * p.groups + lane; row < p.T; row += step) {
        const int b = lane * p.stages + s;
        if (!(ok = mbar_wait(&empty[b], phase))) break;
        uint8_t* dst = ring + static_cast<size_t>(b) * row_bytes;
        mbar_arrive_expect_tx(&full[b], row_bytes + p.unsent);
        bulk_g2s(dst, p.x + row * p.ldx, x_bytes, &full[b]);
        if constexpr (HAS_R) bulk_g2s(dst + x_bytes, static_cast<const R*>(p.r) + row * p.ldr, r_bytes, &full[b]);
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      if (__builtin_expect(!ok, 0)) let_copies_land();
    }
    return;
  }
  Vec8<__nv_bfloat16> wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    wv[i].zero();
    if (c < p.d) wv[i].load(p.w + c);
  }
  const float inv_d = 1.0f / static_cast<float>(p.d);
  int s = 0, flip = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (long long row = static_cast<long long>(blockIdx.x) * p.groups + group; row < p.T; row += step, flip ^= 1) {
    const int b = group * p.stages + s;
    ok = ok && mbar_wait(&full[b], phase);
    const uint8_t* src = ring + static_cast<size_t>(b) * row_bytes;
    float v[VPT][8], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      if (c < p.d) {
        Vec8<__nv_bfloat16> xv;
        xv.load(reinterpret_cast<const __nv_bfloat16*>(src) + c);
        xv.get(v[i]);
        if constexpr (HAS_R) {
          Vec8<R> rv;
          float f[8];
          rv.load(reinterpret_cast<const R*>(src + x_bytes) + c);
          rv.get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] += v[i][j];
          rv.set(f);
          rv.store(static_cast<R*>(p.h) + row * p.d + c);
          rv.get(v[i]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    }
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&empty[b]);
    if (++s == p.stages) s = 0, phase ^= 1;
    // a bounded wait that ran out on any lane (no handle carries an error flag) makes this row and the group's next
    // ones NaN by their sums
    ss = warp_sum(ok ? ss : __int_as_float(0x7FC00000));
    if (p.warps > 1) {       // the slots alternate between rows
      float* at = slots[flip] + group * p.warps;
      if (lane == 0) at[warp - group * p.warps] = ss;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * p.warps) : "memory");
      ss = warp_sum(lane < p.warps ? at[lane] : 0.0f);
    }
    const float rho = rsqrtf(ss * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) write_vec<MX>(p.y, p.scale, p.d, row, (t + i * stride) * 8, true, v[i], wv[i], rho);
  }
  if (__builtin_expect(!ok, 0)) let_copies_land();
}

struct NormBwdParams {
  const __nv_bfloat16* dy;
  const void* h;
  const void* dh;       // gradient along the residual stream, or null
  const __nv_bfloat16* w;
  void* dx;
  float* part;          // [gridDim.x][d] partial sums of dw
  long long lddy, ldh, lddh;
  int T, d, warps, groups, stages;   // warps per row, rows at a time, rows in flight for each
  int unsent;           // as in the forward pass
  float eps;
};
template <class R, bool HAS_DH, int VPT>
__global__ void __launch_bounds__(32 * ring_warps(VPT) + 32)
    rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kRingMaxWarps * kRingMaxStages], empty[kRingMaxWarps * kRingMaxStages];
  __shared__ float slots[2][2][kRingMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / p.warps;                      // == groups: the copying warp
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  const uint32_t dy_bytes = 2 * p.d, h_bytes = sizeof(R) * p.d;
  const uint32_t row_bytes = dy_bytes + h_bytes * (HAS_DH ? 2 : 1);
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  if (threadIdx.x < p.groups * p.stages) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], p.warps);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch();
  griddep_wait();
  if (warp == p.groups * p.warps) {
    // lane g feeds group g
    if (lane < p.groups) {
      int s = 0;
      uint32_t phase = 1;       // the first round of the ring finds its slots empty
      bool ok = true;
      for (long long row = static_cast<long long>(blockIdx.x) * p.groups + lane; row < p.T; row += step) {
        const int b = lane * p.stages + s;
        if (!(ok = mbar_wait(&empty[b], phase))) break;
        uint8_t* dst = ring + static_cast<size_t>(b) * row_bytes;
        mbar_arrive_expect_tx(&full[b], row_bytes + p.unsent);
        bulk_g2s(dst, p.dy + row * p.lddy, dy_bytes, &full[b]);
        bulk_g2s(dst + dy_bytes, static_cast<const R*>(p.h) + row * p.ldh, h_bytes, &full[b]);
        if constexpr (HAS_DH)
          bulk_g2s(dst + dy_bytes + h_bytes, static_cast<const R*>(p.dh) + row * p.lddh, h_bytes, &full[b]);
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      if (__builtin_expect(!ok, 0)) let_copies_land();
    }
    return;
  }
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
  const float inv_d = 1.0f / static_cast<float>(p.d);
  int s = 0, flip = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (long long row = static_cast<long long>(blockIdx.x) * p.groups + group; row < p.T; row += step, flip ^= 1) {
    const int b = group * p.stages + s;
    ok = ok && mbar_wait(&full[b], phase);
    const uint8_t* src = ring + static_cast<size_t>(b) * row_bytes;
    const __nv_bfloat16* dy = reinterpret_cast<const __nv_bfloat16*>(src);
    const R* h = reinterpret_cast<const R*>(src + dy_bytes);
    const R* dh = reinterpret_cast<const R*>(src + dy_bytes + h_bytes);
    float ss = 0.0f, sc = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      if (c >= p.d) continue;
      Vec8<__nv_bfloat16> gv;
      Vec8<R> hv;
      float g[8], x[8], w[8];
      gv.load(dy + c);
      hv.load(h + c);
      gv.get(g);
      hv.get(x);
      wv[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += x[j] * x[j];
        sc += g[j] * w[j] * x[j];
      }
    }
    // two sums behind one barrier of the group; the slots alternate between
    // rows, so the next row's writes cannot meet this row's reads.  A bounded wait
    // that ran out on any lane (no handle carries an error flag) makes this row,
    // the group's next ones and so dw NaN by their sums.
    ss = warp_sum(ok ? ss : __int_as_float(0x7FC00000));
    sc = warp_sum(sc);
    if (p.warps > 1) {
      float* s0 = slots[flip][0] + group * p.warps;
      float* s1 = slots[flip][1] + group * p.warps;
      if (lane == 0) s0[warp - group * p.warps] = ss, s1[warp - group * p.warps] = sc;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * p.warps) : "memory");
      ss = warp_sum(lane < p.warps ? s0[lane] : 0.0f);
      sc = warp_sum(lane < p.warps ? s1[lane] : 0.0f);
    }
    const float rho = rsqrtf(ss * inv_d + p.eps);
    const float k = rho * rho * (sc * inv_d);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      if (c >= p.d) continue;
      Vec8<__nv_bfloat16> gv;
      Vec8<R> hv, ev, ov;
      float g[8], x[8], w[8], e[8], o[8];
      gv.load(dy + c);
      hv.load(h + c);
      if constexpr (HAS_DH) ev.load(dh + c);
      gv.get(g);
      hv.get(x);
      wv[i].get(w);
      if constexpr (HAS_DH) ev.get(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = rho * (w[j] * g[j] - x[j] * k);
        if constexpr (HAS_DH) o[j] += e[j];
        acc[i][j] += g[j] * (x[j] * rho);
      }
      ov.set(o);
      ov.store(static_cast<R*>(p.dx) + row * p.d + c);
    }
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&empty[b]);
    if (++s == p.stages) s = 0, phase ^= 1;
  }
  if (__builtin_expect(!ok, 0)) let_copies_land();      // before the sums take the ring's place, or the CTA leaves
  // One row of partial sums per CTA: its groups' sums meet in the ring, once
  // all of them are done with it, and are added in order.
  float* const out = p.part + static_cast<size_t>(blockIdx.x) * p.d;
  float* part = out;
  const int threads = 32 * p.warps * p.groups;
  if (p.groups > 1) {
    asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory");
    part = reinterpret_cast<float*>(ring) + group * p.d;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    if (c < p.d) {
      reinterpret_cast<float4*>(part + c)[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      reinterpret_cast<float4*>(part + c)[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
  if (p.groups > 1) {
    asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory");
    for (int c = threadIdx.x; c < p.d; c += threads) {
      float v = 0.0f;
      for (int g = 0; g < p.groups; ++g) v += reinterpret_cast<const float*>(ring)[g * p.d + c];
      out[c] = v;
    }
  }
}

// dw[c] = sum of part[0..n)[c], in a fixed order: thread (x, y) adds rows y,
// y + 32, ... of its four columns; then the four y of a warp, then the warps.
constexpr int kSumCols = 8, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows) sum_rows_kernel(const float* part, int n, int d, float* out) {
  __shared__ float4 s[kSumRows / 4][kSumCols];
  griddep_launch();
  griddep_wait();
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int c = (blockIdx.x * kSumCols + x) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
#pragma unroll 5
    for (int r = y; r < n; r += kSumRows) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<size_t>(r) * d + c);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
#pragma unroll
  for (int o = kSumCols; o < 32; o *= 2) {
    a.x += __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
    a.y += __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
    a.z += __shfl_xor_sync(0xFFFFFFFFu, a.z, o);
    a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, o);
  }
  if (y % 4 == 0) s[y / 4][x] = a;
  __syncthreads();
  if (y == 0 && c < d) {
#pragma unroll
    for (int r = 1; r < kSumRows / 4; ++r) {
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

constexpr int kRingCtas = 152;       // one per SM

template <class R, bool HAS_R, bool MX, int VPT>
cudaError_t launch_ring(NormParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, add_rms_norm_ring_kernel<R, HAS_R, MX, VPT>, kRingSmem);
  if (e != cudaSuccess) return e;
  const int row = p.d * (2 + (HAS_R ? static_cast<int>(sizeof(R)) : 0));
  p.groups = ring_warps(VPT) / p.warps;
  const int fit = kRingSmem / row;                 // rows of the ring; d <= kNormMaxWidth: two at least
  if (p.groups > fit) p.groups = fit;
  p.stages = fit / p.groups < kRingMaxStages ? fit / p.groups : kRingMaxStages;
  if (p.groups < 1 || p.stages < 1) return cudaErrorInvalidValue;
  return launch_pdl(add_rms_norm_ring_kernel<R, HAS_R, MX, VPT>, dim3(kRingCtas), dim3(32 * (p.warps * p.groups + 1)),
                    static_cast<size_t>(p.groups) * p.stages * row, s, p);
}

template <class R, bool HAS_R, bool MX>
cudaError_t launch_fwd(NormParams& p, cudaStream_t s) {
  // From about two million values on the ring form: 512 rows of 7168 4.4 us
  // against 5.4 us, 8192 rows 75 us against 79 us (6.2 TB/s; MXFP8 73 us against
  // 82 us), but 333 rows of 3584 3.0 us against 2.7 us.
  const long long n = static_cast<long long>(p.T) * p.d;
  if (n >= 1 << 21 && p.d <= 8192) {
    const RowPlan r = row_plan(p.d, 512);
    p.warps = r.warps;
    return r.vpt == 1 ? launch_ring<R, HAS_R, MX, 1>(p, s) : launch_ring<R, HAS_R, MX, 2>(p, s);
  }
  // Wider rows later (512 rows of 9216 as MXFP8 8.1 us against 7.4 us, 2048 rows
  // 26.9 us against 31.1 us; 2048 rows of 16384 45 us against 52 us), and not
  // those of an fp32 stream, of which the ring holds few (2048 rows of 16384 70 us
  // against 67 us).
  if constexpr (!(HAS_R && sizeof(R) == 4)) {
    if (n >= 1 << 23 && p.d > 8192) {
      p.warps = (p.d / 8 + 32 * 5 - 1) / (32 * 5);
      return launch_ring<R, HAS_R, MX, 5>(p, s);
    }
  }
  // One vector per thread up to 8192 values (8192 rows of 7168: 79 us against
  // 90 us with two), four beyond (2048 rows of 16384: 51 us against 57 us).
  const RowPlan r = row_plan(p.d, p.d <= 8192 ? 1024 : 512);
  p.warps = r.warps;
  const dim3 grid((p.T + r.groups - 1) / r.groups), block(32 * r.warps * r.groups);
  return r.vpt == 1 ? launch_pdl(add_rms_norm_kernel<R, HAS_R, MX, 1>, grid, block, 0, s, p)
                    : launch_pdl(add_rms_norm_kernel<R, HAS_R, MX, 4>, grid, block, 0, s, p);
}

// Backward: warps of a row, rows at a time and in flight, and how many CTAs.
struct BwdPlan {
  int vpt, warps, groups, stages, grid;
};
BwdPlan bwd_plan(int T, int d, int row) {
  // One vector per thread for narrow rows, four or five for wide ones: fewer
  // warps meet at a row's barrier, and more rows are worked on at once.  4096
  // rows of a bf16 stream with dh, 1 / 4 vectors: 11.3 / 11.6 us at 1152 values,
  // 18.6 / 18.3 us at 2560, 23.6 / 24.4 us at 3584, 28.3 / 26.5 us at 4096 (without
  // dh 10.6 / 10.7, 17.5 / 17.8, 22.8 / 20.3 and 25.9 / 22.5 us); at 7168, 2 / 4:
  // 42.6 / 42.3 us (36.7 / 33.4 us).  2048 rows of 16384, 4 / 5: 58.9 / 51.2 us.
  const int vpt = d <= 2560 ? 1 : d <= 8192 ? 4 : 5;
  const int warps = (d / 8 + 32 * vpt - 1) / (32 * vpt);
  BwdPlan b = {vpt, warps, ring_warps(vpt) / warps, 0, 1};
  // Each group has two rows in flight at least, where they fit: fp32 stream with
  // dh, 4096 rows of 7168, one group of two 66.6 us against two of one 83.9 us.
  const int fit = kRingSmem / row;
  if (b.groups > fit / 2) b.groups = fit > 1 ? fit / 2 : 1;
  b.stages = fit / b.groups < kRingMaxStages ? fit / b.groups : kRingMaxStages;
  const int need = (T - 1) / b.groups + 1;
  b.grid = need < kRingCtas ? need : kRingCtas;
  return b;
}

template <class R, bool HAS_DH, int VPT>
cudaError_t launch_bwd_vpt(const NormBwdParams& p, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, rms_norm_bwd_kernel<R, HAS_DH, VPT>, kRingSmem);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(p.groups) * p.stages * p.d * (2 + sizeof(R) * (HAS_DH ? 2 : 1));
  return launch_pdl(rms_norm_bwd_kernel<R, HAS_DH, VPT>, dim3(grid), dim3(32 * (p.warps * p.groups + 1)), smem, s, p);
}
template <class R, bool HAS_DH>
cudaError_t launch_bwd(NormBwdParams& p, const BwdPlan& b, cudaStream_t s) {
  switch (b.vpt) {
    case 1: return launch_bwd_vpt<R, HAS_DH, 1>(p, b.grid, s);
    case 4: return launch_bwd_vpt<R, HAS_DH, 4>(p, b.grid, s);
    default: return launch_bwd_vpt<R, HAS_DH, 5>(p, b.grid, s);
  }
}

}  // namespace

size_t rms_norm_bwd_partials(int T, int d) {
  return static_cast<size_t>(T < kRingCtas ? T : kRingCtas) * d;
}

cudaError_t launch_add_rms_norm(const void* x, long long ldx, const void* r, long long ldr, bool r_fp32, int T, int d,
                                const void* w, float eps, void* h, void* y, uint8_t* scale, int unsent, cudaStream_t s) {
  NormParams p = {};
  p.unsent = unsent;
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
  if (!r) return scale ? launch_fwd<float, false, true>(p, s) : launch_fwd<float, false, false>(p, s);
  if (r_fp32) return scale ? launch_fwd<float, true, true>(p, s) : launch_fwd<float, true, false>(p, s);
  return scale ? launch_fwd<__nv_bfloat16, true, true>(p, s) : launch_fwd<__nv_bfloat16, true, false>(p, s);
}

cudaError_t launch_rms_norm_bwd(const void* dy, long long lddy, const void* h, long long ldh, const void* dh,
                                long long lddh, bool h_fp32, int T, int d, const void* w, float eps, void* dx,
                                float* part, float* dw, int unsent, cudaStream_t s) {
  NormBwdParams p = {};
  p.unsent = unsent;
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
  const BwdPlan b = bwd_plan(T, d, d * (2 + (h_fp32 ? 4 : 2) * (dh ? 2 : 1)));
  if (b.stages < 1) return cudaErrorInvalidValue;      // not for d <= kNormMaxWidth
  p.warps = b.warps;
  p.groups = b.groups;
  p.stages = b.stages;
  cudaError_t e;
  if (h_fp32)
    e = dh ? launch_bwd<float, true>(p, b, s) : launch_bwd<float, false>(p, b, s);
  else
    e = dh ? launch_bwd<__nv_bfloat16, true>(p, b, s) : launch_bwd<__nv_bfloat16, false>(p, b, s);
  if (e != cudaSuccess) return e;
  const int cols = 4 * kSumCols;
  return launch_pdl(sum_rows_kernel, dim3((d + cols - 1) / cols), dim3(kSumCols * kSumRows), 0, s,
                    static_cast<const float*>(part), b.grid, d, dw);
}

}  // namespace lmoe
