// Gated activations of the dense feed-forward block and their derivatives,
// fp32.  SiTU-GLU: a(g) = b1 tanh(g/b1) sigma(g), v(u) = b2 tanh(u/b2);
// SwiGLU: a(g) = g sigma(g), v(u) = u.  hid = a v, dg = dhid v a'(g),
// du = dhid a v'(u).
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace lmoe {

// The arithmetic on one value or, where a thread has two side by side, on both
// by one instruction (fma.rn.f32x2 and its kin).  With six special-function
// calls for each SiTU-GLU value one at a time, the epilogue of a short product
// took longer than the product.
struct F2 {
  float x, y;
};
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 vmul(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 vadd(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 vfma(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
template <class V>
__device__ __forceinline__ V splat(float c);
template <>
__device__ __forceinline__ float splat<float>(float c) { return c; }
template <>
__device__ __forceinline__ F2 splat<F2>(float c) { return {c, c}; }
__device__ __forceinline__ float vex2(float a) {       // 2^a
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ F2 vex2(F2 a) { return {vex2(a.x), vex2(a.y)}; }
__device__ __forceinline__ float vrcp(float a) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ F2 vrcp(F2 a) { return {vrcp(a.x), vrcp(a.y)}; }
__device__ __forceinline__ float vmin(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ F2 vmin(F2 a, F2 b) { return {fminf(a.x, b.x), fminf(a.y, b.y)}; }
__device__ __forceinline__ float minus_abs(float a) { return -fabsf(a); }
__device__ __forceinline__ F2 minus_abs(F2 a) { return {-fabsf(a.x), -fabsf(a.y)}; }
// far with the sign of x for |x| >= 1/4, else (and for a NaN) near
__device__ __forceinline__ float by_size(float x, float near, float far) {
  return fabsf(x) >= 0.25f ? copysignf(far, x) : near;
}
__device__ __forceinline__ F2 by_size(F2 x, F2 near, F2 far) {
  return {by_size(x.x, near.x, far.x), by_size(x.y, near.y, far.y)};
}

constexpr float kLog2E = 1.44269504f;
template <class V>
__device__ __forceinline__ V sigmoid(V x) {
  return vrcp(vadd(vex2(vmul(x, splat<V>(-kLog2E))), splat<V>(1.0f)));
}
// sigma(x), and 1 - sigma(x) as e^-x sigma(x): from the rounded sigma alone its
// tail would be lost (e^-x stops at 2^126, where sigma is zero).
template <class V>
__device__ __forceinline__ V sigmoid(V x, V& rest) {
  const V e = vex2(vmul(x, splat<V>(-kLog2E))), s = vrcp(vadd(e, splat<V>(1.0f)));
  rest = vmul(vmin(e, splat<V>(0x1p126f)), s);
  return s;
}
// tanh of two values to ~1e-6 relative: with e = e^-2|x|, 2/(1 + e) - 1, both
// quotients from one reciprocal, and the odd Taylor polynomial through x^9 near
// zero, where that difference cancels (at |x| = 0.25 the next term is 4e-9 of
// tanh; the quotient form there is off ~9e-7).
template <class V>
__device__ __forceinline__ V tanh_near(V x) {
  const V x2 = vmul(x, x);
  V p = vfma(x2, splat<V>(62.0f / 2835), splat<V>(-17.0f / 315));
  p = vfma(x2, p, splat<V>(2.0f / 15));
  p = vfma(x2, p, splat<V>(-1.0f / 3));
  return vfma(vmul(x, x2), p, x);
}
template <class V>
struct Tanh {
  V t, e, h;      // tanh x, e^-2|x|, 2/(1 + e)
};
template <class V>
__device__ __forceinline__ void tanh_both(V x, V y, Tanh<V>& tx, Tanh<V>& ty) {
  const V k = splat<V>(2.0f * kLog2E), one = splat<V>(1.0f), two = splat<V>(2.0f), minus = splat<V>(-1.0f);
  tx.e = vex2(minus_abs(vmul(x, k)));
  ty.e = vex2(minus_abs(vmul(y, k)));
  const V a = vadd(tx.e, one), b = vadd(ty.e, one), r = vmul(vrcp(vmul(a, b)), two);
  tx.h = vmul(b, r);
  ty.h = vmul(a, r);
  tx.t = by_size(x, tanh_near(x), vadd(tx.h, minus));
  ty.t = by_size(y, tanh_near(y), vadd(ty.h, minus));
}
// 1 - tanh^2 = 4 e / (1 + e)^2.  From the rounded tanh it would be 1% off at
// |x| = 6 and nothing but rounding from 8 on.
template <class V>
__device__ __forceinline__ V tanh_slope(const Tanh<V>& t) { return vmul(vmul(t.e, t.h), t.h); }

struct GluCaps {
  float b1, b2, r1, r2;   // caps and their reciprocals
};

template <int ACT, class V>
__device__ __forceinline__ V glu_hidden(V g, V u, const GluCaps& c) {
  const V s = sigmoid(g);
  if constexpr (ACT == 1) return vmul(vmul(g, s), u);
  Tanh<V> tg, tu;
  tanh_both(vmul(g, splat<V>(c.r1)), vmul(u, splat<V>(c.r2)), tg, tu);
  return vmul(vmul(splat<V>(c.b1), vmul(tg.t, s)), vmul(splat<V>(c.b2), tu.t));
}

struct GluGrad {
  F2 hid, dg, du;
};
template <int ACT>
__device__ __forceinline__ GluGrad glu_grad(F2 g, F2 u, F2 dhid, const GluCaps& c) {
  GluGrad o;
  if constexpr (ACT == 1) {
    const F2 s = sigmoid(g), rest = vfma(s, splat<F2>(-1.0f), splat<F2>(1.0f)), a = vmul(g, s);
    o.hid = vmul(a, u);
    o.dg = vmul(vmul(dhid, u), vfma(a, rest, s));
    o.du = vmul(dhid, a);
  } else {
    F2 rest;
    const F2 s = sigmoid(g, rest);
    Tanh<F2> tg, tu;
    tanh_both(vmul(g, splat<F2>(c.r1)), vmul(u, splat<F2>(c.r2)), tg, tu);
    const F2 a = vmul(splat<F2>(c.b1), vmul(tg.t, s)), v = vmul(splat<F2>(c.b2), tu.t);
    const F2 dtg = tanh_slope(tg), dtu = tanh_slope(tu);
    o.hid = vmul(a, v);
    o.dg = vmul(vmul(dhid, v), vfma(a, rest, vmul(dtg, s)));
    o.du = vmul(vmul(dhid, a), dtu);
  }
  return o;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack_bf16(F2 v) { return pack_bf16(v.x, v.y); }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ F2 bf16_both(uint32_t v) { return {bf16_lo(v), bf16_hi(v)}; }
// Values 2j and 2j + 1 of 32 (as bits).
__device__ __forceinline__ F2 pair_at(const uint32_t (&v)[32], int j) {
  return {__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])};
}

// 32 fp32 values (as bits) -> bf16.
__device__ __forceinline__ void pack32(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
}

// 32 bf16 columns of this thread's row, as far as `left` (a multiple of 8)
// goes; `wide`: rows start on 32-byte boundaries, and whole sectors move per
// instruction.
__device__ __forceinline__ void store32(__nv_bfloat16* dst, const uint32_t (&w)[16], int left, bool wide) {
#pragma unroll
  for (int i = 0; i < 16; i += 8) {
    if (wide && left >= 2 * i + 16) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 2 * i), "r"(w[i]),
                   "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                   "r"(w[i + 7])
                   : "memory");
    } else {
      if (left >= 2 * i + 8) *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      if (left >= 2 * i + 16)
        *reinterpret_cast<uint4*>(dst + 2 * i + 8) = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    }
  }
}

// A warp's 32 rows of 64 bf16 columns, lane = row, to the matrix [.][ld] at dst,
// of which `rows` and `cols` (a multiple of 8) are left, by way of `buf` (4 KB of
// shared memory), so that eight lanes store a row's 128 bytes side by side.  In
// `buf` a 16-byte chunk's place depends on its row: no two of eight lanes meet in
// a bank.  Against store32, 256 tokens at 7168 x 2048, all gradients: 64.1 us, 67.6 us.
__device__ __forceinline__ void store_rows(uint8_t* buf, const uint32_t (&w)[32], __nv_bfloat16* dst, int ld, int rows,
                                           int cols) {
  const int lane = threadIdx.x & 31, ch = lane & 7;
  const auto at = [&](int row, int c) { return reinterpret_cast<uint4*>(buf + 128 * row + 16 * (c ^ (row & 7))); };
#pragma unroll
  for (int j = 0; j < 8; ++j) *at(lane, j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + lane / 8;
    const uint4 v = *at(row, ch);
    if (row < rows && 8 * ch < cols) *reinterpret_cast<uint4*>(dst + static_cast<size_t>(row) * ld + 8 * ch) = v;
  }
  __syncwarp();
}

}  // namespace lmoe
