// One AdamW step over many tensors.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// HBM bounds it: 28 bytes a value with fp32 states, a master and a bf16 gradient,
// about 10 with MXFP8 states and no master.  A CTA takes a chunk of one or several times
// 2048 values of one tensor; a thread holds eight consecutive values, four lanes a block
// of 32 with its scales.  All arithmetic is fp32.  Measured on 132 million values: 534 us
// with masters and fp32 states (6.9 TB/s), 416 us for bf16 weights; with MXFP8 states 326
// us with masters (6.5 TB/s), 265 us for bf16 weights (5.0 TB/s), which what is left of
// the decoding, mixing and encoding, about 65 instructions a value, bounds.
//
// Roundings: a bf16 weight to nearest beside an fp32 master; without one, and for
// MXFP8 states, stochastically, since a step's change is mostly far below a step of
// the format (b2 = 0.999 changes sqrt(v) by 0.05%, an E4M3 step is 6 to 12%) and would
// be lost by rounding to nearest.  v is stored by its root, whose exponents span half
// the range (a v below 2^-126 counts as zero there): the 18 binades of a block of E4M3
// codes then hold values of v 2^35 apart.
#include "block_internal.h"
#include "common.cuh"
#include "ffn_act.cuh"
#include "lmoe_internal.h"
#include "norm_vec.cuh"

namespace lmoe {
namespace {

constexpr int kThreads = 256;
static_assert(kAdamVector == 8 * kThreads, "eight values of each thread");
static_assert(sizeof(AdamParams) <= 4096, "kernel parameters");

__host__ __device__ __forceinline__ uint32_t mix_rest(uint32_t x) {
  x *= 0x9E9F34A5u;
  x ^= x >> 15;
  x *= 0xBB3A919Bu;
  return x ^ (x >> 16);
}
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) { return mix_rest(x ^ (x >> 16)); }

// The largest of m, |x| and |y|; a NaN wins.
__device__ __forceinline__ float max_abs(float m, float x, float y) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(x)), "f"(fabsf(y)));
  return m;
}
__device__ __forceinline__ float fast_sqrt(float x) {
  asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float fast_rcp(float x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
// Two values as bf16, rounded stochastically: the low half of r is added below x's bits,
// the high half below y's, and the rest is cut off.  A NaN stays one.
__device__ __forceinline__ uint32_t stochastic_bf16(float x, float y, uint32_t r) {
  uint32_t d;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(d) : "f"(y), "f"(x), "r"(r));
  return d;
}

// Eight values as stored, in words: eight of fp32, four of bf16, two of codes; `left` of
// them are there, zeros behind them.
__device__ __forceinline__ void load_words(const float* p, int left, uint32_t (&w)[8]) {
  if (left >= 8) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < left ? __float_as_uint(p[j]) : 0u;
  }
}
__device__ __forceinline__ void load_words(const __nv_bfloat16* p, int left, uint32_t (&w)[8]) {
  if (left >= 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) w[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j % 2));
  }
}
__device__ __forceinline__ void load_words(const uint8_t* p, int left, uint32_t (&w)[2]) {
  if (left >= 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) w[j / 4] |= static_cast<uint32_t>(p[j]) << (8 * (j % 4));
  }
}
__device__ __forceinline__ void values(const uint32_t (&w)[8], bool fp32, float (&f)[8]) {
  if (fp32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
  }
}
__device__ __forceinline__ void values(const uint32_t (&w)[2], float (&f)[8]) {      // of codes, without their scale
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[j / 2] >> (16 * (j % 2))), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}
__device__ __forceinline__ float scale_of(uint32_t s) {
  return s == 255u ? __int_as_float(0x7FC00000) : e8m0_to_f32(s);
}
__device__ __forceinline__ void store(float* p, int left, const float (&f)[8]) {
  if (left >= 8) {
    Vec8<float> v;
    v.set(f);
    v.store(p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = f[j];
  }
}
__device__ __forceinline__ void store(__nv_bfloat16* p, int left, const uint32_t (&w)[4]) {
  if (left >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) reinterpret_cast<uint16_t*>(p)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
  }
}
__device__ __forceinline__ void store(uint8_t* p, int left, const uint32_t (&w)[2]) {
  if (left >= 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
  }
}

// Eight values as E4M3 codes, rounded stochastically by 20 bits of their words, and the
// scale of their block of four lanes.  Multiplied by 2^-120 a value in units of its scale
// has E4M3's exponents in fp32, its subnormals among fp32's (2^-9 becomes 2^-129, 20 bits
// above the last one), so the code lies in bits 20..26 whatever the value, and rounding
// is one addition below them.  ROOT: no sign, and what is not zero stays so, however far
// below the block's maximum (at 2^-38 of it the product with `down` is zero).
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(float (&f)[8], const uint32_t (&word)[8], uint32_t (&codes)[2]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) m = max_abs(m, f[j], f[j + 1]);
  uint32_t top = __float_as_uint(m);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // an infinity or NaN (exponent field 255) makes the block NaN: E8M0 byte 255
  const uint32_t s = top >= 0x7F800000u ? 255u : e4m3_block_scale(__uint_as_float(top));
  // 2^(127 - s) 2^-120 is a normal number up to s = 133; blocks with values over 28672 are multiplied in two steps
  float down = __uint_as_float((134u - s) << 23);
  if (__builtin_expect(s > 133u, 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = f[j] * 0x1p-120f;
      f[j] = ROOT && f[j] != 0.0f ? fmaxf(x, 0x1p-149f) : x;
    }
    down = s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[4], x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = word[4 * i + j], a = __float_as_uint(fabsf(f[4 * i + j]) * down);
      c[j] = (a + (ROOT ? w & 0xFFFFFu : w >> 12)) >> 20;
      if (ROOT && f[4 * i + j] != 0.0f) c[j] = max(c[j], 1u);
      x[j] = __float_as_uint(f[4 * i + j]);
    }
    codes[i] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    if (!ROOT) {
      const uint32_t signs = __byte_perm(__byte_perm(x[0], x[1], 0x0073), __byte_perm(x[2], x[3], 0x0073), 0x5410);
      codes[i] |= signs & 0x80808080u;
    }
  }
  return s;
}

// A chunk's tensor, and where this thread's first values of the chunk lie in it.
struct Chunk {
  const void* grad;
  void *param, *m, *v;
  float* master;
  uint8_t *m_scale, *v_scale;
  long long at, rest;           // this thread's first value; values from there to the tensor's end
  unsigned long long first;
  float decay;                  // -lr weight_decay
  bool grad_fp32, fp32, rounded;
};

// Eight values of a thread as read, in words.
template <bool MX>
struct Held {
  uint32_t g[8], w[8];
  uint32_t m[MX ? 2 : 8], v[MX ? 2 : 8], ms, vs;
};

// Vector i of a thread lies i * kAdamVector values behind its first one.  FULL: all of the CTA's
// threads have eight values there.
template <bool MX, bool FULL>
__device__ __forceinline__ int left_of(const Chunk& c, int i) {
  if (FULL) return 8;
  const long long r = c.rest - i * kAdamVector;
  return r >= 8 ? 8 : r > 0 ? static_cast<int>(r) : 0;
}
template <bool MX, bool FULL>
__device__ __forceinline__ void load(const Chunk& c, int i, Held<MX>& h) {
  const long long at = c.at + i * kAdamVector;
  const int left = left_of<MX, FULL>(c, i);
  if (c.grad_fp32)
    load_words(static_cast<const float*>(c.grad) + at, left, h.g);
  else
    load_words(static_cast<const __nv_bfloat16*>(c.grad) + at, left, h.g);
  if (c.rounded)
    load_words(static_cast<const __nv_bfloat16*>(c.param) + at, left, h.w);
  else
    load_words((c.fp32 ? static_cast<const float*>(c.param) : c.master) + at, left, h.w);
  if constexpr (MX) {
    load_words(static_cast<const uint8_t*>(c.m) + at, left, h.m);
    load_words(static_cast<const uint8_t*>(c.v) + at, left, h.v);
    h.ms = left ? c.m_scale[at >> 5] : 0;
    h.vs = left ? c.v_scale[at >> 5] : 0;
  } else {
    load_words(static_cast<const float*>(c.m) + at, left, h.m);
    load_words(static_cast<const float*>(c.v) + at, left, h.v);
  }
}

// Copies of a vector's words, of each thread for itself.
struct Staged {
  uint4 g[2][kThreads], w[2][kThreads];
  uint2 m[kThreads], v[kThreads];
};
template <int N>
__device__ __forceinline__ void copy(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait_all_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void fetch(const Chunk& c, int i, Staged& s, uint32_t& ms, uint32_t& vs) {
  const long long at = c.at + i * kAdamVector;
  const int t = threadIdx.x;
  const char* g = static_cast<const char*>(c.grad) + (at << (c.grad_fp32 ? 2 : 1));
  copy<16>(&s.g[0][t], g);
  if (c.grad_fp32) copy<16>(&s.g[1][t], g + 16);
  if (c.rounded) {
    copy<16>(&s.w[0][t], static_cast<const __nv_bfloat16*>(c.param) + at);
  } else {
    const float* w = (c.fp32 ? static_cast<const float*>(c.param) : c.master) + at;
    copy<16>(&s.w[0][t], w);
    copy<16>(&s.w[1][t], w + 4);
  }
  copy<8>(&s.m[t], static_cast<const uint8_t*>(c.m) + at);
  copy<8>(&s.v[t], static_cast<const uint8_t*>(c.v) + at);
  ms = c.m_scale[at >> 5];
  vs = c.v_scale[at >> 5];
}
__device__ __forceinline__ void take(const Chunk& c, const Staged& s, Held<true>& h) {
  const int t = threadIdx.x;
  const auto put = [&](uint32_t (&w)[8], const uint4 (&from)[2][kThreads], bool both) {
    const uint4 a = from[0][t];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    if (both) {
      const uint4 b = from[1][t];
      w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  };
  put(h.g, s.g, c.grad_fp32);
  put(h.w, s.w, !c.rounded);
  h.m[0] = s.m[t].x, h.m[1] = s.m[t].y;
  h.v[0] = s.v[t].x, h.v[1] = s.v[t].y;
}

// Factors of a step: lr, -lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t), of the gradients.
struct Factors {
  float lr, k1, k2, scale;
  uint32_t key;
};

template <bool MX, bool FULL>
__device__ __forceinline__ void update(const AdamParams& p, const Factors& f, const Chunk& c, int i,
                                       const Held<MX>& h) {
  const long long at = c.at + i * kAdamVector;
  const int left = left_of<MX, FULL>(c, i);
  float g[8], m[8], v[8], w[8], root[8];
  values(h.g, c.grad_fp32, g);
  values(h.w, !c.rounded, w);
  float b1 = p.beta1;
  if constexpr (MX) {
    values(h.m, m);
    values(h.v, v);
    b1 *= scale_of(h.ms);
    const float s = scale_of(h.vs);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      F2 r = vmul(F2{v[j], v[j + 1]}, splat<F2>(s));
      r = vmul(r, r);
      v[j] = r.x, v[j + 1] = r.y;
    }
  } else {
    values(h.m, true, m);
    values(h.v, true, v);
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const F2 g2 = vmul(F2{g[j], g[j + 1]}, splat<F2>(f.scale));
    const F2 m2 = vfma(F2{m[j], m[j + 1]}, splat<F2>(b1), vmul(g2, splat<F2>(p.rest1)));
    const F2 v2 = vfma(F2{v[j], v[j + 1]}, splat<F2>(p.beta2), vmul(vmul(g2, g2), splat<F2>(p.rest2)));
    root[j] = fast_sqrt(v2.x), root[j + 1] = fast_sqrt(v2.y);
    const F2 d = vfma(F2{root[j], root[j + 1]}, splat<F2>(f.k2), splat<F2>(p.eps));
    const F2 u = vmul(m2, splat<F2>(f.k1));
    // The step and the decay are added first, and then the weight once: 1 - lr weight_decay would round the decay to
    // fp32's grid below one, the same way for every weight (1e-7 would be 1.2e-7, 2e-8 nothing).
    const F2 w1 = {w[j], w[j + 1]}, step = vfma(w1, splat<F2>(c.decay), vmul(u, F2{fast_rcp(d.x), fast_rcp(d.y)}));
    const F2 w2 = vadd(w1, step);
    m[j] = m2.x, m[j + 1] = m2.y, v[j] = v2.x, v[j + 1] = v2.y, w[j] = w2.x, w[j + 1] = w2.y;
  }
  uint32_t word[8];
  if (MX || c.rounded) {
    const unsigned long long n = c.first + at;
    const uint32_t hi = static_cast<uint32_t>(n >> 32);
    // n is a multiple of eight: the numbers n + j differ in their last bits only, and share mix's first step
    const uint32_t x0 = static_cast<uint32_t>(n) ^ (hi ? mix(f.key + hi) : f.key), x1 = x0 ^ (x0 >> 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) word[j] = mix_rest(x1 ^ j);
  }
  if (c.fp32) {
    store(static_cast<float*>(c.param) + at, left, w);
  } else {
    uint32_t b[4];
    if (c.rounded) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = stochastic_bf16(w[2 * j], w[2 * j + 1], __byte_perm(word[2 * j], word[2 * j + 1], 0x6521));
    } else {
      store(c.master + at, left, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = pack_bf16(w[2 * j], w[2 * j + 1]);
    }
    store(static_cast<__nv_bfloat16*>(c.param) + at, left, b);
  }
  if constexpr (MX) {
    uint32_t q[2];
    const uint32_t ms = encode<false>(m, word, q);
    store(static_cast<uint8_t*>(c.m) + at, left, q);
    const uint32_t vs = encode<true>(root, word, q);
    store(static_cast<uint8_t*>(c.v) + at, left, q);
    if (left && (threadIdx.x & 3) == 0) {
      c.m_scale[at >> 5] = static_cast<uint8_t>(ms);
      c.v_scale[at >> 5] = static_cast<uint8_t>(vs);
    }
  } else {
    store(static_cast<float*>(c.m) + at, left, m);
    store(static_cast<float*>(c.v) + at, left, v);
  }
}

// The values of one chunk.
template <bool MX>
__device__ __forceinline__ void work(const AdamParams& p, const Factors& f, int chunk, Staged (&staged)[MX ? 2 : 1]) {
  const int id = p.owner[chunk];
  Chunk c;
  c.grad = p.grads[id];
  if (!c.grad) return;
  const AdamTensor& x = p.tensors[id];
  c.param = x.param;
  c.m = x.m;
  c.v = x.v;
  c.master = x.master;
  c.m_scale = x.m_scale;
  c.v_scale = x.v_scale;
  c.first = x.first;
  c.decay = -f.lr * x.decay;
  c.grad_fp32 = p.fp32[id >> 5] >> (id & 31) & 1u;
  c.fp32 = x.fp32;
  c.rounded = !x.fp32 && !x.master;
  const long long from = static_cast<long long>(chunk - x.chunk0) * p.vectors * kAdamVector, all = x.n - from;
  c.at = from + 8 * threadIdx.x;
  c.rest = all - 8 * threadIdx.x;
  Held<MX> h;
  if (all < static_cast<long long>(p.vectors) * kAdamVector) {
#pragma unroll 1
    for (int i = 0; i < p.vectors && i * kAdamVector < all; ++i) {
      load<MX, false>(c, i, h);
      update<MX, false>(p, f, c, i, h);
    }
  } else if constexpr (MX) {
    // Much arithmetic for few bytes: the next values are on their way meanwhile, by copies
    // into shared memory that each thread makes for itself (bf16 weights: with loads
    // alone 366 us instead of 264 us).
    uint32_t ms, vs, ms1 = 0, vs1 = 0;
    fetch(c, 0, staged[0], ms, vs);
    copies_end_group();
#pragma unroll 1
    for (int i = 0; i < p.vectors; ++i) {
      if (i + 1 < p.vectors) fetch(c, i + 1, staged[(i + 1) & 1], ms1, vs1);
      copies_end_group();
      copies_wait_all_but_one();
      take(c, staged[i & 1], h);
      h.ms = ms, h.vs = vs;
      update<MX, true>(p, f, c, i, h);
      ms = ms1, vs = vs1;
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < p.vectors; ++i) {
      load<MX, true>(c, i, h);
      update<MX, true>(p, f, c, i, h);
    }
  }
}

template <bool MX>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ AdamParams p) {
  __shared__ Staged staged[MX ? 2 : 1];
  griddep_launch();
  griddep_wait();
  const long long t = *p.step + 1;
  Factors f;
  f.lr = p.lr_dev ? *p.lr_dev : p.lr;
  f.scale = p.scale_dev ? *p.scale_dev : 1.0f;
  // 1 - beta^t without the cancellation at small t
  f.k1 = f.lr / expm1f(static_cast<float>(t) * p.log1);
  f.k2 = 1.0f / sqrtf(-expm1f(static_cast<float>(t) * p.log2));
  f.key = mix(p.seed + static_cast<uint32_t>(t));
  if (blockIdx.x < p.chunks) work<MX>(p, f, blockIdx.x, staged);
  // The last CTA of the step's last launch counts it: every CTA has read the count by then.
  if (p.last) {
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.done, 1) == static_cast<int>(gridDim.x) - 1) {
      *p.done = 0;
      *p.step = t;
    }
  }
}

}  // namespace

uint32_t adamw_mix(uint32_t x) { return mix(x); }
// CTAs are handed out by the hardware, one chunk each: with CTAs that stay and take every
// n-th chunk 132 million values with fp32 states and masters take 570 us and more instead
// of 529 us.  MXFP8 states want chunks long enough that the step's factors and the first
// fetch do not count (1, 4, 8 and 16 vectors: 377, 281, 264 and 263 us, with masters 421,
// 328, 327 and 336 us), fp32 states one or two (bf16 weights 439 and 417 us; with masters
// 529 and 533 us); few values come first in giving each SM several chunks.
int adamw_vectors(int64_t values, bool mx) {
  const int64_t v = values / kAdamVector / (152 * 16), most = mx ? 8 : 2;
  return static_cast<int>(v < 1 ? 1 : v > most ? most : v);
}

cudaError_t launch_adamw(const AdamParams& p, bool mx, cudaStream_t s) {
  const dim3 grid(p.chunks < 1 ? 1 : p.chunks);      // without chunks the step is counted all the same
  return mx ? launch_pdl(adamw_kernel<true>, grid, dim3(kThreads), 0, s, p)
            : launch_pdl(adamw_kernel<false>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace lmoe
