// The norms on both sides of a block with its gate and residual scale, forward
// and backward; y is the block's output, r the residual stream.
//
//   n = w1 y rho1,  h = a r + b g n (in r's type),  o = w2 h rho2,  rho = 1 / sqrt(mean(.^2) + eps)
//   gH = gh + rho2 (w2 go - h k),          k = rho2^2 mean(w2 go h)
//   dr = a gH,  q = b g gH,  dg = b n gH
//   dy = rho1 (w1 q - y rho1^2 mean(w1 q y)),  dw1 = sum over rows of q y rho1,  dw2 = of go h rho2
//
// HBM bounds both: each value moves once (8192 rows of 7168 forward 73.3 us, 6.4 TB/s;
// 4096 rows backward 65.1 us with the 4 us of the sums over rows, 5.8 TB/s before
// them).  One CTA per SM, whose groups of warps take every (gridDim.x * groups)-th
// row from a ring of shared memory that a warp of its own fills by bulk copies, several
// rows ahead.  The forward pass reduces twice, since h is normalised as stored.  The
// backward pass reduces once: the mean of w1 q y is linear in gH, so with u = b w1 g y
//   sum w1 q y = rho2 (sum u w2 go - k sum u h) + sum u gh
// and its three sums meet with those of h^2, y^2 and w2 go h.  Sums and norms are fp32;
// the only roundings are those of the stored outputs.
#include "block_internal.h"
#include "common.cuh"
#include "ffn_act.cuh"
#include "lmoe_internal.h"
#include "moe_common.cuh"
#include "norm_vec.cuh"

namespace lmoe {
namespace {

constexpr int kCtas = 152;               // one per SM
constexpr int kMaxWarps = 28, kMaxStages = 8;
// Compute warps of a CTA at most, by vectors per thread; one more copies.
constexpr int fwd_warps(int vpt) { return vpt == 1 ? kMaxWarps : vpt == 2 ? 19 : 15; }
// The backward pass: 96 registers with 20 warps, 128 with 16, 168 with 12.
constexpr int bwd_warps(int vpt) { return vpt == 1 ? 19 : vpt == 2 ? 15 : 11; }
// Shared memory of a CTA's ring.  Three rows of 7168 values of a bf16 stream's backward pass with a gate for each token
// take 210 KB: 80 us for 4096 of them; with two in the ring 117 us.
constexpr int kRing = 218 * 1024;
constexpr float kNan = __builtin_nanf("");

struct Params {
  const __nv_bfloat16 *y, *gate, *w1, *w2, *go;
  const void *s, *gh;     // stream (forward r, backward h), gradient along it
  void *h, *o;            // forward
  uint8_t* scale;
  void *dy, *dr, *dgate;  // backward
  float* part;            // [gridDim.x][2][d] partial sums: of go h rho2, and of the branch's
  long long ldy, lds, ldg, ldgo, ldgh;
  int T, d, warps, groups, stages;   // warps of a row, rows at a time, rows in flight of each
  int unsent;
  float a, b, eps;
};

// Eight consecutive values as stored, read and written as pairs: a thread does its
// arithmetic on two values at a time.
template <class T>
struct Pairs;
template <>
struct Pairs<__nv_bfloat16> {
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ F2 get(int j) const { return bf16_both(w[j]); }
  __device__ void set(int j, F2 v) { w[j] = pack_bf16(v); }
};
template <>
struct Pairs<float> {
  F2 v[4];
  __device__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = {a.x, a.y}, v[1] = {a.z, a.w}, v[2] = {b.x, b.y}, v[3] = {b.z, b.w};
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  __device__ void zero() { v[0] = v[1] = v[2] = v[3] = F2{0.0f, 0.0f}; }
  __device__ F2 get(int j) const { return v[j]; }
  __device__ void set(int j, F2 x) { v[j] = x; }
};
__device__ __forceinline__ float total(F2 v) { return v.x + v.y; }

// o of one vector as MXFP8: w2 h rho2 as codes, with the scale of its 32-value block, four
// consecutive lanes' vectors.
template <class H>
__device__ __forceinline__ void write_mx(const Params& p, long long row, int c, const H& h,
                                         const Vec8<__nv_bfloat16>& w2, float rho2) {
  const uint32_t w[4] = {w2.v.x, w2.v.y, w2.v.z, w2.v.w};
  F2 f[4];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = vmul(vmul(h.get(j), splat<F2>(rho2)), bf16_both(w[j]));
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(f[j].x)), "f"(fabsf(f[j].y)));
  }
  uint32_t top = __float_as_uint(m);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // an infinity or NaN (exponent field 255) makes the block NaN: E8M0 byte 255
  const uint32_t s = top >= 0x7F800000u ? 255u : e4m3_block_scale(__uint_as_float(top));
  const float inv = s == 255u ? 1.0f : e8m0_to_f32(254u - s);
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const F2 v = vmul(f[j], splat<F2>(inv));
    q[j] = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  }
  if (c < p.d) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.o) + row * p.d + c) =
        make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    if ((threadIdx.x & 3) == 0) p.scale[row * (p.d >> 5) + (c >> 5)] = static_cast<uint8_t>(s);
  }
}

// Barrier of the warps of a row.
__device__ __forceinline__ void group_sync(int group, int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * warps) : "memory");
}

// The sums over a warp's lanes of eight values, value lane / 4 in each lane: half of the
// values go to the other half of the lanes, then a quarter to the other quarter ...
__device__ __forceinline__ float sum_eight(const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + 4], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + 2], 8);
  }
  const bool up = lane & 4;
  float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xFFFFFFFFu, c, 2);
  return c + __shfl_xor_sync(0xFFFFFFFFu, c, 1);
}

// b w1 with the channels' gate, if there is one, at column c.
__device__ __forceinline__ void branch_weights(Pairs<float>& o, const __nv_bfloat16* w1, const __nv_bfloat16* gate,
                                               float b, int c) {
  Pairs<__nv_bfloat16> w, g;
  w.load(w1 + c);
  if (gate) g.load(gate + c);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const F2 v = vmul(w.get(j), splat<F2>(b));
    o.set(j, gate ? vmul(v, g.get(j)) : v);
  }
}

// TOKEN: the gate is a row for each token; else it is part of the weights kept in
// registers.
template <class R, bool TOKEN, bool MX, int VPT>
__global__ void __launch_bounds__(32 * fwd_warps(VPT) + 32) gated_norm_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxWarps * kMaxStages], empty[kMaxWarps * kMaxStages];
  __shared__ float slots[2][kMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / p.warps;                      // == groups: the copying warp
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  const uint32_t y_bytes = 2 * p.d, s_bytes = sizeof(R) * p.d, row_bytes = y_bytes * (TOKEN ? 2 : 1) + s_bytes;
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
      int st = 0;
      uint32_t phase = 1;    // the first round of the ring finds its slots empty
      bool ok = true;
      for (long long row = static_cast<long long>(blockIdx.x) * p.groups + lane; row < p.T; row += step) {
        const int i = lane * p.stages + st;
        if (!(ok = mbar_wait(&empty[i], phase))) break;
        uint8_t* dst = ring + static_cast<size_t>(i) * row_bytes;
        mbar_arrive_expect_tx(&full[i], row_bytes + p.unsent);
        bulk_g2s(dst, p.y + row * p.ldy, y_bytes, &full[i]);
        bulk_g2s(dst + y_bytes, static_cast<const R*>(p.s) + row * p.lds, s_bytes, &full[i]);
        if constexpr (TOKEN) bulk_g2s(dst + y_bytes + s_bytes, p.gate + row * p.ldg, y_bytes, &full[i]);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
      if (__builtin_expect(!ok, 0)) let_copies_land();
    }
    return;
  }
  Pairs<float> w1[VPT];          // b w1, with the channels' gate
  Vec8<__nv_bfloat16> w2[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    w2[i].zero();
    w1[i].zero();
    if (c < p.d) {
      w2[i].load(p.w2 + c);
      branch_weights(w1[i], p.w1, TOKEN ? nullptr : p.gate, p.b, c);
    }
  }
  const float inv_d = 1.0f / static_cast<float>(p.d);
  int st = 0;
  uint32_t phase = 0;
  bool ok = true;
  // Sum over the row's warps.  The two sums of a row have slots of their own, so
  // that between a read and the next write of a slot lies the other one's barrier.
  const auto row_sum = [&](float v, float* slot) {
    v = warp_sum(v);
    if (p.warps == 1) return v;
    slot += group * p.warps;
    if (lane == 0) slot[warp - group * p.warps] = v;
    group_sync(group, p.warps);
    return warp_sum(lane < p.warps ? slot[lane] : 0.0f);
  };
  for (long long row = static_cast<long long>(blockIdx.x) * p.groups + group; row < p.T; row += step) {
    const int b = group * p.stages + st;
    ok = ok && mbar_wait(&full[b], phase);
    const uint8_t* src = ring + static_cast<size_t>(b) * row_bytes;
    Pairs<__nv_bfloat16> yv[VPT];
    F2 s2 = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      yv[i].zero();
      if (c < p.d) yv[i].load(reinterpret_cast<const __nv_bfloat16*>(src) + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = vfma(yv[i].get(j), yv[i].get(j), s2);
    }
    // a bounded wait that ran out on any lane (no handle carries an error flag) makes this row and the group's next
    // ones NaN by their sums
    float ss = row_sum(ok ? total(s2) : kNan, slots[0]);
    const float rho1 = rsqrtf(ss * inv_d + p.eps);
    Pairs<R> v[VPT];
    s2 = F2{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      v[i].zero();
      if (c < p.d) {
        Pairs<R> rv;
        Pairs<__nv_bfloat16> gv;
        rv.load(reinterpret_cast<const R*>(src + y_bytes) + c);
        if constexpr (TOKEN) gv.load(reinterpret_cast<const __nv_bfloat16*>(src + y_bytes + s_bytes) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          F2 f = vmul(vmul(yv[i].get(j), splat<F2>(rho1)), w1[i].get(j));
          if constexpr (TOKEN) f = vmul(f, gv.get(j));
          v[i].set(j, vfma(rv.get(j), splat<F2>(p.a), f));      // in the stream's type: what is stored and normalised
        }
        v[i].store(static_cast<R*>(p.h) + row * p.d + c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = vfma(v[i].get(j), v[i].get(j), s2);
    }
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&empty[b]);
    if (++st == p.stages) st = 0, phase ^= 1;
    ss = row_sum(total(s2), slots[1]);
    const float rho2 = rsqrtf(ss * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      if constexpr (MX) {
        write_mx(p, row, c, v[i], w2[i], rho2);
      } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[2 * j] = v[i].get(j).x, f[2 * j + 1] = v[i].get(j).y;
        write_vec<false>(p.o, nullptr, p.d, row, c, true, f, w2[i], rho2);
      }
    }
  }
  if (__builtin_expect(!ok, 0)) let_copies_land();
}

// GATE: lmoe_gate_type.  A row's sums are reduced while its warps already add up the next
// row's: they meet at an mbarrier that nobody waits at in vain (one row after the other
// behind a barrier of its warps, 4096 x 7168: 79.6 us).
template <class R, int GATE, bool HAS_GH, int VPT>
__global__ void __launch_bounds__(32 * bwd_warps(VPT) + 32) gated_norm_bwd_kernel(const __grid_constant__ Params p) {
  constexpr bool kToken = GATE == 2;
  // A warp writes row n + 3's sums only once every warp has read row n - 1's: it has seen
  // row n + 1's complete, and a warp reads n - 1's before it gives n + 1's.
  constexpr int kSums = 6, kPitch = 8, kSlots = 4;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxWarps * kMaxStages], empty[kMaxWarps * kMaxStages], met[kMaxWarps][kSlots];
  __shared__ __align__(16) float slots[kSlots][kMaxWarps * kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / p.warps;                      // == groups: the copying warp
  const int t = threadIdx.x - group * 32 * p.warps, stride = 32 * p.warps;
  const uint32_t y_bytes = 2 * p.d, s_bytes = sizeof(R) * p.d;
  // go, y, h, gh, gate
  const uint32_t h_at = 2 * y_bytes, gh_at = h_at + s_bytes, gate_at = gh_at + (HAS_GH ? s_bytes : 0);
  const uint32_t row_bytes = gate_at + (kToken ? y_bytes : 0);
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  if (threadIdx.x < p.groups * p.stages) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], p.warps);
  }
  if (threadIdx.x < p.groups * kSlots) mbar_init(&met[threadIdx.x / kSlots][threadIdx.x % kSlots], p.warps);
  fence_mbar_init();
  __syncthreads();
  griddep_launch();
  griddep_wait();
  if (warp == p.groups * p.warps) {
    if (lane < p.groups) {   // lane g feeds group g
      int st = 0;
      uint32_t phase = 1;    // the first round of the ring finds its slots empty
      bool ok = true;
      for (long long row = static_cast<long long>(blockIdx.x) * p.groups + lane; row < p.T; row += step) {
        const int i = lane * p.stages + st;
        if (!(ok = mbar_wait(&empty[i], phase))) break;
        uint8_t* dst = ring + static_cast<size_t>(i) * row_bytes;
        mbar_arrive_expect_tx(&full[i], row_bytes + p.unsent);
        bulk_g2s(dst, p.go + row * p.ldgo, y_bytes, &full[i]);
        bulk_g2s(dst + y_bytes, p.y + row * p.ldy, y_bytes, &full[i]);
        bulk_g2s(dst + h_at, static_cast<const R*>(p.s) + row * p.lds, s_bytes, &full[i]);
        if constexpr (HAS_GH) bulk_g2s(dst + gh_at, static_cast<const R*>(p.gh) + row * p.ldgh, s_bytes, &full[i]);
        if constexpr (kToken) bulk_g2s(dst + gate_at, p.gate + row * p.ldg, y_bytes, &full[i]);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
      if (__builtin_expect(!ok, 0)) let_copies_land();
    }
    return;
  }
  Pairs<float> w1[VPT];                  // b w1, with the channels' gate
  Pairs<__nv_bfloat16> w2[VPT];
  Pairs<float> acc_next[VPT], acc[VPT];  // sums of go h rho2, and of y rho1 gH (a token's gate: times b gate)
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    w1[i].zero();
    w2[i].zero();
    acc_next[i].zero();
    acc[i].zero();
    if (c < p.d) {
      Pairs<__nv_bfloat16> v;
      branch_weights(w1[i], p.w1, GATE == 1 ? p.gate : nullptr, p.b, c);
      v.load(p.w2 + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) w2[i].set(j, v.get(j));
    }
  }
  // Eight values of a row at column c.
  struct Row {
    Pairs<__nv_bfloat16> go, y, g;
    Pairs<R> h, gh;
  };
  const auto load = [&](const uint8_t* src, int c, Row& r) {
    r.go.load(reinterpret_cast<const __nv_bfloat16*>(src) + c);
    r.y.load(reinterpret_cast<const __nv_bfloat16*>(src + y_bytes) + c);
    r.h.load(reinterpret_cast<const R*>(src + h_at) + c);
    if constexpr (HAS_GH) r.gh.load(reinterpret_cast<const R*>(src + gh_at) + c);
    if constexpr (kToken) r.g.load(reinterpret_cast<const __nv_bfloat16*>(src + gate_at) + c);
  };
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const long long row0 = static_cast<long long>(blockIdx.x) * p.groups + group;
  const int rows = row0 < p.T ? static_cast<int>((p.T - row0 + step - 1) / step) : 0;
  bool ok = true;
  int st1 = 0, st2 = 0;      // ring slots of the row that is added up and of the one that is finished
  uint32_t phase1 = 0;
  const auto sums = [&](int n) {
    const int b = group * p.stages + st1;
    ok = ok && mbar_wait(&full[b], phase1);
    if (++st1 == p.stages) st1 = 0, phase1 ^= 1;
    const uint8_t* src = ring + static_cast<size_t>(b) * row_bytes;
    F2 s2[kSums] = {};       // of h^2, w2 go h, y^2, u w2 go, u h, u gh, with u = b w1 g y
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      if (c >= p.d) continue;
      Row r;
      load(src, c, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 y = r.y.get(j), h = r.h.get(j), wg = vmul(w2[i].get(j), r.go.get(j));
        F2 u = vmul(w1[i].get(j), y);
        if constexpr (kToken) u = vmul(u, r.g.get(j));
        s2[0] = vfma(h, h, s2[0]);
        s2[1] = vfma(wg, h, s2[1]);
        s2[2] = vfma(y, y, s2[2]);
        s2[3] = vfma(u, wg, s2[3]);
        s2[4] = vfma(u, h, s2[4]);
        if constexpr (HAS_GH) s2[5] = vfma(u, r.gh.get(j), s2[5]);
      }
    }
    float s[kPitch] = {};
#pragma unroll
    for (int k = 0; k < kSums; ++k) s[k] = total(s2[k]);
    // Narrow rows have few warps and wait for these sums' latency, wide ones for their
    // instructions: 512 values 11.2 us so, 12.4 us by sum_eight; 8192 values 73.9 and 71.1 us.
    float* const at = slots[n % kSlots] + warp * kPitch;
    if constexpr (VPT == 1) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) s[k] = warp_sum(s[k]);
      if (lane == 0) {
        *reinterpret_cast<float4*>(at) = make_float4(s[0], s[1], s[2], s[3]);
        *reinterpret_cast<float2*>(at + 4) = make_float2(s[4], s[5]);
      }
    } else {
      const float mine = sum_eight(s);
      if (lane % 4 == 0) at[lane / 4] = mine;
      __syncwarp();
    }
    if (lane == 0) mbar_arrive(&met[group][n % kSlots]);
  };
  const auto finish = [&](int n) {
    ok = ok && mbar_wait(&met[group][n % kSlots], n / kSlots & 1);
    const float* at = slots[n % kSlots] + group * p.warps * kPitch;
    float s[kSums] = {};
    if constexpr (VPT == 1) {
      for (int w = 0; w < p.warps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(at + w * kPitch);
        const float2 z = *reinterpret_cast<const float2*>(at + w * kPitch + 4);
        s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += z.x, s[5] += z.y;
      }
    } else {
      float part = 0.0f;      // of sum lane % 8
      for (int w = lane / kPitch; w < p.warps; w += 32 / kPitch) part += at[w * kPitch + lane % kPitch];
      part += __shfl_xor_sync(0xFFFFFFFFu, part, 8);
      part += __shfl_xor_sync(0xFFFFFFFFu, part, 16);
#pragma unroll
      for (int k = 0; k < kSums; ++k) s[k] = __shfl_sync(0xFFFFFFFFu, part, k);
    }
    // A bounded wait that ran out on this lane (no handle carries an error flag) makes its
    // values of this row and the next ones, and its sums over rows, NaN by these.
    if (!ok) s[0] = s[2] = kNan;
    const float rho2 = rsqrtf(s[0] * inv_d + p.eps), rho1 = rsqrtf(s[2] * inv_d + p.eps);
    const float k2 = rho2 * rho2 * (s[1] * inv_d);
    const float k1 = rho1 * rho1 * ((rho2 * (s[3] - k2 * s[4]) + s[5]) * inv_d);
    const int b = group * p.stages + st2;
    if (++st2 == p.stages) st2 = 0;
    const uint8_t* src = ring + static_cast<size_t>(b) * row_bytes;
    const long long row = row0 + n * step;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * stride) * 8;
      if (c >= p.d) continue;
      Row r;
      load(src, c, r);
      Pairs<R> dr;
      Pairs<__nv_bfloat16> dy, dg;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 go = r.go.get(j), y = r.y.get(j), h = r.h.get(j);
        const F2 hr = vmul(h, splat<F2>(rho2));
        F2 gH = vfma(hr, splat<F2>(-k2), vmul(vmul(w2[i].get(j), go), splat<F2>(rho2)));
        if constexpr (HAS_GH) gH = vadd(gH, r.gh.get(j));
        dr.set(j, vmul(gH, splat<F2>(p.a)));
        const F2 n = vmul(y, splat<F2>(rho1)), wH = vmul(w1[i].get(j), gH);      // b w1 (g) gH
        const F2 wq = kToken ? vmul(wH, r.g.get(j)) : wH;
        dy.set(j, vfma(wq, splat<F2>(rho1), vmul(n, splat<F2>(-k1))));
        if constexpr (kToken) dg.set(j, vmul(wH, n));
        acc_next[i].set(j, vfma(go, hr, acc_next[i].get(j)));
        acc[i].set(j, vfma(n, kToken ? vmul(gH, vmul(r.g.get(j), splat<F2>(p.b))) : gH, acc[i].get(j)));
      }
      dr.store(static_cast<R*>(p.dr) + row * p.d + c);
      dy.store(static_cast<__nv_bfloat16*>(p.dy) + row * p.d + c);
      if constexpr (kToken) dg.store(static_cast<__nv_bfloat16*>(p.dgate) + row * p.d + c);
    }
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&empty[b]);
  };
  const bool ahead = p.stages > 2;      // the next row is there while the one behind it is on its way
  if (rows > 0) sums(0);
  for (int n = 0; n < rows; ++n) {
    if (ahead && n + 1 < rows) sums(n + 1);
    finish(n);
    if (!ahead && n + 1 < rows) sums(n + 1);
  }
  if (__builtin_expect(!ok, 0)) let_copies_land();      // before the sums take the ring's place, or the CTA leaves
  // Two rows of partial sums per CTA: its groups' sums meet in the ring, once all of
  // them are done with it, and are added in order.
  float* const out = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.d;
  float* part = out;
  const int threads = 32 * p.warps * p.groups;
  if (p.groups > 1) {
    asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory");
    part = reinterpret_cast<float*>(ring) + group * 2 * p.d;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * stride) * 8;
    if (c < p.d) {
      acc_next[i].store(part + c);
      acc[i].store(part + p.d + c);
    }
  }
  if (p.groups > 1) {
    asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory");
    for (int c = threadIdx.x; c < 2 * p.d; c += threads) {
      float v = 0.0f;
      for (int g = 0; g < p.groups; ++g) v += reinterpret_cast<const float*>(ring)[g * 2 * p.d + c];
      out[c] = v;
    }
  }
}

// The sums over rows, of part[0..n)[2][d] in a fixed order: thread (x, y) adds rows y,
// y + 32, ... of its four columns; then the four y of a warp, then the warps.
// blockIdx.y: which of the two; the branch's S becomes dw1 = b g S and dg = b w1 S
// (a token's gate: dw1 = S).
constexpr int kSumCols = 8, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows)
    gated_sums_kernel(const float* part, int n, int d, float* dw1, float* dw2, float* dg, const __nv_bfloat16* w1,
                      const __nv_bfloat16* gate, float b) {
  __shared__ float4 s[kSumRows / 4][kSumCols];
  griddep_launch();
  griddep_wait();
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int c = (blockIdx.x * kSumCols + x) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
    part += blockIdx.y * d + c;
#pragma unroll 5
    for (int r = y; r < n; r += kSumRows) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<size_t>(r) * 2 * d);
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
  if (y != 0 || c >= d) return;
#pragma unroll
  for (int r = 1; r < kSumRows / 4; ++r) {
    const float4 v = s[r][x];
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
  }
  if (blockIdx.y == 0) {
    *reinterpret_cast<float4*>(dw2 + c) = a;
    return;
  }
  const float v[4] = {a.x, a.y, a.z, a.w};
  float o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = gate ? b * __bfloat162float(gate[c + j]) * v[j] : b * v[j];
  *reinterpret_cast<float4*>(dw1 + c) = make_float4(o[0], o[1], o[2], o[3]);
  if (dg) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = b * __bfloat162float(w1[c + j]) * v[j];
    *reinterpret_cast<float4*>(dg + c) = make_float4(o[0], o[1], o[2], o[3]);
  }
}

struct Plan {
  int vpt, warps, groups, stages, grid;
  size_t smem;
};
// most: compute warps of a CTA; row: bytes of a row in the ring; sums: floats of a group's
// sums over rows, which meet in the ring.  False where not even one row fits.
bool plan(Plan& r, int T, int d, int vpt, int most, int row, int sums) {
  r.vpt = vpt;
  r.warps = (d / 8 + 32 * vpt - 1) / (32 * vpt);
  r.groups = most / r.warps;
  const int fit = kRing / row;
  if (r.groups > fit / 2) r.groups = fit > 1 ? fit / 2 : 1;      // each has two rows in flight at least, where they fit
  r.stages = fit / r.groups < kMaxStages ? fit / r.groups : kMaxStages;
  const int need = (T - 1) / r.groups + 1;
  r.grid = need < kCtas ? need : kCtas;
  const size_t ring = static_cast<size_t>(r.groups) * r.stages * row;
  const size_t met = r.groups > 1 ? static_cast<size_t>(r.groups) * sums * 4 : 0;
  r.smem = ring > met ? ring : met;
  return r.groups >= 1 && r.stages >= 1 && r.smem <= kRing;
}

// Vectors per thread.  8192 rows forward, 1 / 2 / 4, in us:
//                              2560          4096          5120           6144           7168        8192 wide
//   bf16                     30/30/29      51/44/45      58/68/60       65/70/65       73/78/81      -/88/96
//   bf16, gate               38/36/38      55/57/56      69/74/69       88/89/82     104/102/95      -/113/125
//   fp32                     46/44/45      69/68/73      78/84/91       95/94/108    120/112/124     -/132/129
//   fp32, gate               52/50/51      74/82/81      89/104/101   118/123/122    142/142/133     -/160/140
//   to MXFP8                 33/30/35      58/43/53      65/71/60       73/73/78       82/80/87      -/82/137
//   bf16, gate, to MXFP8     36/32/40      61/49/67      68/74/77       77/77/99      85/85/112      -/95/170
//   fp32, to MXFP8           43/40/43      74/62/67      84/87/79      99/98/100    110/106/115      -/119/180
//   fp32, gate, to MXFP8     48/50/46      79/80/69      93/89/89    107/100/101    120/112/145      -/141/150
// (gate: of each token; 3584 wide within 6%, but for four to MXFP8.)  So two, except where another number is ahead:
// rows over 4608 up to 5120 wide have ten of the 19 warps that two vectors take, one row at a time, and are faster with
// one (20 of 28 warps) or four (three rows of five); bf16 rows to bf16, of which little is held, with one, unless that
// leaves 10 to 13 of 28 warps without a row; tokens' gates as the table has it, onto fp32 from 4096 rows on (1024 rows
// 5120 wide 16.2/-/14.8 us, 2048 26.8/-/25.8 us, 4096 47.0/-/50.1 us).  Few rows want many threads each: 333 rows 7168
// wide 6.4/6.8/6.7 us, 8192 wide 7.0/7.4 us with two and four, 10.2/10.6 us onto fp32 with a gate.
int forward_vectors(const GatedNorm& g, bool token, bool mx) {
  const int d = g.d;
  if (d <= 2048 || (g.T < 1024 && d <= 7168)) return 1;
  if (g.T < 1024) return 2;
  if (token && g.fp32 && mx) return d <= 5120 ? 4 : 2;
  if (token && !mx && d > 3584) return g.fp32 ? (d >= 4096 && d <= 6144 && g.T >= 4096 ? 1 : 4) : d <= 7168 ? 4 : 2;
  if (d > 4608 && d <= 5120) return mx && !token ? 4 : 1;
  return mx || token || g.fp32 || (d > 3584 && d <= 4608) || d > 7168 ? 2 : 1;
}
// 4096 rows backward, 1 / 2 / 3: 1024 wide 15.6 / 17.7 / 20.5 us, 2048 27.5 / 26.5 / 31.3
// us, 3584 48.4 / 40.2 / 42.6 us, 7168 - / 66.4 / 67.6 us.  Two take up to 7680 values.
int backward_vectors(int d) { return d <= 1536 ? 1 : d <= 512 * bwd_warps(2) ? 2 : 3; }

template <class... KArgs>
cudaError_t launch(std::atomic<uint64_t>& limit, void (*kernel)(KArgs...), const Plan& r, const Params& p,
                   cudaStream_t s) {
  const cudaError_t e = allow_smem(limit, kernel, kRing);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(r.grid), dim3(32 * (r.warps * r.groups + 1)), r.smem, s, p);
}

template <class R, bool TOKEN, bool MX>
cudaError_t forward(const Params& p, const Plan& r, cudaStream_t s) {
  static std::atomic<uint64_t> limit[3];
  return r.vpt == 1   ? launch(limit[0], gated_norm_kernel<R, TOKEN, MX, 1>, r, p, s)
         : r.vpt == 2 ? launch(limit[1], gated_norm_kernel<R, TOKEN, MX, 2>, r, p, s)
                      : launch(limit[2], gated_norm_kernel<R, TOKEN, MX, 4>, r, p, s);
}
template <class R>
cudaError_t forward(const Params& p, const Plan& r, bool token, bool mx, cudaStream_t s) {
  if (token) return mx ? forward<R, true, true>(p, r, s) : forward<R, true, false>(p, r, s);
  return mx ? forward<R, false, true>(p, r, s) : forward<R, false, false>(p, r, s);
}

template <class R, int GATE, bool HAS_GH>
cudaError_t backward(const Params& p, const Plan& r, cudaStream_t s) {
  static std::atomic<uint64_t> limit[3];
  return r.vpt == 1   ? launch(limit[0], gated_norm_bwd_kernel<R, GATE, HAS_GH, 1>, r, p, s)
         : r.vpt == 2 ? launch(limit[1], gated_norm_bwd_kernel<R, GATE, HAS_GH, 2>, r, p, s)
                      : launch(limit[2], gated_norm_bwd_kernel<R, GATE, HAS_GH, 3>, r, p, s);
}
template <class R, int GATE>
cudaError_t backward(const Params& p, const Plan& r, cudaStream_t s) {
  return p.gh ? backward<R, GATE, true>(p, r, s) : backward<R, GATE, false>(p, r, s);
}
template <class R>
cudaError_t backward(const Params& p, const Plan& r, int gate, cudaStream_t s) {
  return gate == 0 ? backward<R, 0>(p, r, s) : gate == 1 ? backward<R, 1>(p, r, s) : backward<R, 2>(p, r, s);
}

Params params(const GatedNorm& g, const Plan& r) {
  Params p = {};
  p.y = static_cast<const __nv_bfloat16*>(g.y);
  p.s = g.stream;
  p.gate = static_cast<const __nv_bfloat16*>(g.gate);
  p.w1 = static_cast<const __nv_bfloat16*>(g.w_post);
  p.w2 = static_cast<const __nv_bfloat16*>(g.w_next);
  p.ldy = g.ldy;
  p.lds = g.lds;
  p.ldg = g.ldg;
  p.T = g.T;
  p.d = g.d;
  p.a = g.a;
  p.b = g.b;
  p.eps = g.eps;
  p.unsent = g.unsent;
  p.warps = r.warps;
  p.groups = r.groups;
  p.stages = r.stages;
  return p;
}

}  // namespace

size_t gated_norm_bwd_partials(int T, int d) { return static_cast<size_t>(T < kCtas ? T : kCtas) * 2 * d; }

cudaError_t launch_gated_norm(const GatedNorm& g, void* h, void* o, uint8_t* scale, cudaStream_t s) {
  Plan r;
  const bool token = g.gate_type == 2;
  const int vpt = forward_vectors(g, token, scale != nullptr), row = g.d * (2 + (g.fp32 ? 4 : 2) + (token ? 2 : 0));
  if (!plan(r, g.T, g.d, vpt, fwd_warps(vpt), row, 0)) return cudaErrorInvalidValue;
  Params p = params(g, r);
  p.h = h;
  p.o = o;
  p.scale = scale;
  return g.fp32 ? forward<float>(p, r, token, scale != nullptr, s)
                : forward<__nv_bfloat16>(p, r, token, scale != nullptr, s);
}

cudaError_t launch_gated_norm_bwd(const GatedNorm& g, const void* go, long long ldgo, const void* gh, long long ldgh,
                                  void* dy, void* dr, float* dw_post, float* dw_next, void* dgate, float* part,
                                  cudaStream_t s) {
  Plan r;
  const bool token = g.gate_type == 2, channel = g.gate_type == 1;
  const int sb = g.fp32 ? 4 : 2, row = g.d * (4 + sb * (gh ? 2 : 1) + (token ? 2 : 0)), vpt = backward_vectors(g.d);
  if (!plan(r, g.T, g.d, vpt, bwd_warps(vpt), row, 2 * g.d)) return cudaErrorInvalidValue;
  Params p = params(g, r);
  p.go = static_cast<const __nv_bfloat16*>(go);
  p.ldgo = ldgo;
  p.gh = gh;
  p.ldgh = ldgh;
  p.dy = dy;
  p.dr = dr;
  p.dgate = token ? dgate : nullptr;
  p.part = part;
  const cudaError_t e = g.fp32 ? backward<float>(p, r, g.gate_type, s) : backward<__nv_bfloat16>(p, r, g.gate_type, s);
  if (e != cudaSuccess) return e;
  const int cols = 4 * kSumCols;
  return launch_pdl(gated_sums_kernel, dim3((g.d + cols - 1) / cols, 2), dim3(kSumCols * kSumRows), 0, s,
                    static_cast<const float*>(part), r.grid, g.d, dw_post, dw_next,
                    channel ? static_cast<float*>(dgate) : static_cast<float*>(nullptr), p.w1,
                    channel ? p.gate : static_cast<const __nv_bfloat16*>(nullptr), token ? 1.0f : g.b);
}

}  // namespace lmoe
