// Activations of the product with an epilogue, and their derivatives, fp32.
#pragma once
#include <type_traits>

#include "ffn_act.cuh"

namespace lmoe {

// ACT: lmoe_linear_act.
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3;

// f(std::integral_constant<int, act>): the choice once, outside of f's loops.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    default: f(std::integral_constant<int, kActNone>());
  }
}

__device__ __forceinline__ void set_pair(uint32_t (&v)[32], int j, F2 x) {
  v[2 * j] = __float_as_uint(x.x);
  v[2 * j + 1] = __float_as_uint(x.y);
}

// A warp's 32 rows of 32 fp32 columns, lane = row, through `buf` (4 KB): after turn_rows every lane
// may take four consecutive columns of any row.  A 16-byte chunk's place depends on its row, as in
// store_rows; a __syncwarp() ends the use of buf.
__device__ __forceinline__ float4* turned_at(uint8_t* buf, int row, int ch) {
  return reinterpret_cast<float4*>(buf + 128 * row + 16 * (ch ^ (row & 7)));
}
__device__ __forceinline__ void turn_rows(uint8_t* buf, const uint32_t (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *turned_at(buf, lane, j) = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                           __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
  __syncwarp();
}
__device__ __forceinline__ float4 turned(uint8_t* buf, int row, int ch) { return *turned_at(buf, row, ch); }

// The other way: a warp's 32 rows of 64 bf16 columns, of which `rows` and `cols` are there,
// eight lanes on a row's 128 bytes; by way of `buf` each lane then has its own row, 16 bytes at
// a time.
__device__ __forceinline__ void load_rows(uint4 (&r)[8], const __nv_bfloat16* src, long long ld, int rows, int cols) {
  const int sub = threadIdx.x >> 3 & 3, ch = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + sub;
    r[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && 8 * ch < cols) r[i] = *reinterpret_cast<const uint4*>(src + row * ld + 8 * ch);
  }
}
__device__ __forceinline__ void rows_in(uint8_t* buf, const uint4 (&r)[8]) {
  const int sub = threadIdx.x >> 3 & 3, ch = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + sub;
    *reinterpret_cast<uint4*>(buf + 128 * row + 16 * (ch ^ (row & 7))) = r[i];
  }
  __syncwarp();
}
__device__ __forceinline__ uint4 own_row(const uint8_t* buf, int j) {
  const int row = threadIdx.x & 31;
  return *reinterpret_cast<const uint4*>(buf + 128 * row + 16 * (j ^ (row & 7)));
}

// 1/2 (1 + tanh(u)) = sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGelu2A = 1.5957691216057308f, kGeluB = 0.044715f;
__device__ __forceinline__ float relu(float z) { return z <= 0.0f ? 0.0f : z; }      // a NaN stays one
template <int ACT>
__device__ __forceinline__ F2 linear_act(F2 z) {
  if constexpr (ACT == kActRelu) return {relu(z.x), relu(z.y)};
  if constexpr (ACT == kActSilu) return vmul(z, sigmoid(z));
  if constexpr (ACT == kActGelu) {
    const F2 z2 = vmul(z, z), k = vfma(z2, splat<F2>(kGelu2A * kGeluB), splat<F2>(kGelu2A));
    return vmul(z, sigmoid(vmul(z, k)));
  }
  return z;
}

// The derivative; a NaN stays one.  Beyond 16 silu's and gelu's terms are 0 or 1 within fp32 (gelu's) or
// need no product of a huge and a zero factor.
__device__ __forceinline__ float step(float z) { return z <= 0.0f ? 0.0f : z > 0.0f ? 1.0f : z; }
template <int ACT>
__device__ __forceinline__ F2 linear_slope(F2 z) {
  if constexpr (ACT == kActRelu) return {step(z.x), step(z.y)};
  if constexpr (ACT == kActSilu) {
    F2 rest;
    const F2 s = sigmoid(z, rest);
    return vmul(s, vfma(z, rest, splat<F2>(1.0f)));
  }
  if constexpr (ACT == kActGelu) {
    const auto limit = [](float x) { return fabsf(x) > 16.0f ? copysignf(16.0f, x) : x; };      // a NaN stays one
    z = {limit(z.x), limit(z.y)};
    const F2 z2 = vmul(z, z), k = vfma(z2, splat<F2>(kGelu2A * kGeluB), splat<F2>(kGelu2A));
    F2 rest;
    const F2 s = sigmoid(vmul(z, k), rest);
    const F2 dk = vfma(z2, splat<F2>(3.0f * kGelu2A * kGeluB), splat<F2>(kGelu2A));
    return vmul(s, vfma(vmul(z, rest), dk, splat<F2>(1.0f)));
  }
  return splat<F2>(1.0f);
}

}  // namespace lmoe
