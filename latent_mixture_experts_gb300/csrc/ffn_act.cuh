// Gated activations of the dense feed-forward block and their derivatives,
// fp32.  SiTU-GLU: a(g) = b1 tanh(g/b1) sigma(g), v(u) = b2 tanh(u/b2);
// SwiGLU: a(g) = g sigma(g), v(u) = u.  hid = a v, dg = dhid v a'(g),
// du = dhid a v'(u).
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace lmoe {

// tanh to ~1e-6 relative: 1 - 2/(e^2x + 1), and the odd Taylor polynomial
// through x^9 near zero, where that difference cancels (at |x| = 0.25 the
// next term is 4e-9 of tanh; the quotient form there is off ~2.5e-7).
__device__ __forceinline__ float tanh_acc(float x) {
  const float x2 = x * x;
  const float p =
      x * (1.0f + x2 * (-1.0f / 3 + x2 * (2.0f / 15 + x2 * (-17.0f / 315 + x2 * (62.0f / 2835)))));
  const float q = 1.0f - __fdividef(2.0f, __expf(2.0f * x) + 1.0f);
  return fabsf(x) < 0.25f ? p : q;
}

struct GluCaps {
  float b1, b2, r1, r2;   // caps and their reciprocals
};

template <int ACT>
__device__ __forceinline__ float glu_hidden(float g, float u, const GluCaps& c) {
  const float s = sigmoid_fast(g);
  if constexpr (ACT == 1) return g * s * u;
  return c.b1 * tanh_acc(g * c.r1) * s * (c.b2 * tanh_acc(u * c.r2));
}

struct GluGrad {
  float hid, dg, du;
};
template <int ACT>
__device__ __forceinline__ GluGrad glu_grad(float g, float u, float dhid, const GluCaps& c) {
  const float s = sigmoid_fast(g);
  GluGrad o;
  if constexpr (ACT == 1) {
    const float a = g * s;
    o.hid = a * u;
    o.dg = dhid * u * (s + a * (1.0f - s));
    o.du = dhid * a;
  } else {
    const float tg = tanh_acc(g * c.r1), tu = tanh_acc(u * c.r2);
    const float a = c.b1 * tg * s, v = c.b2 * tu;
    o.hid = a * v;
    o.dg = dhid * v * ((1.0f - tg * tg) * s + a * (1.0f - s));
    o.du = dhid * a * (1.0f - tu * tu);
  }
  return o;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

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
}  // namespace lmoe
