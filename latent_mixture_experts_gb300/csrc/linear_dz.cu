// What the backward pass of a product with an epilogue does before its products:
// dz = dy act'(z), rounded to bf16 for them (a bf16 MMA takes bf16 operands), and
// dbias, the sums of the unrounded dz over rows.  One pass: HBM bounds it.  A thread
// holds eight columns, the eight warps of a CTA take its rows in turn; the CTAs' sums
// are added, in order, by the last one of their columns to finish.
#include "block_internal.h"
#include "lmoe_internal.h"
#include "linear_act.cuh"
#include "norm_vec.cuh"

namespace lmoe {
namespace {

constexpr int kWarps = 8, kCols = 256;      // of a CTA
// Rows that a warp has in flight (4096 tokens at 512 x 2048, gelu's slope, and 1000 at 3584 x 3584, whole backward
// pass: two rows 36.7 and 43.3 us, four 39.3 and 41.8 us, eight 41.7 and 41.5 us; 64 tokens at 7168 x 2048 26.0, 24.4
// and 23.5 us).
constexpr int kAhead = 8;
// A thread's running sums hold at most 64 rows; each 64 of them go to a compensated sum
// (Kahan) in shared memory, so that a gradient is within 2^-17 of the size of its terms
// whatever T is: one after the other a million rows of 512 values were off by 2^-15.
constexpr int kFold = 64 / kAhead;

struct Params {
  const void* dy;
  const __nv_bfloat16* z;
  __nv_bfloat16* dz;
  float *dbias, *part;      // part [gridDim.y][gridDim.x][kCols]
  int* done;                // [gridDim.x], 0 between calls
  long long lddy;
  int T, d, rows;           // rows of a CTA
  int apart;                // the products do not read what this kernel writes
};

template <class Y, int ACT>
__global__ void __launch_bounds__(32 * kWarps, 2) linear_dz_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float sums[kWarps][kCols], rest[kWarps][kCols];
  __shared__ int last;
  if (p.apart) {      // who follows may begin, not only be there, once everything before this kernel has finished
    griddep_wait();
    griddep_launch();
  } else {
    griddep_launch();
    griddep_wait();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * kCols + 8 * lane;
  const int end = min(p.T, (static_cast<int>(blockIdx.y) + 1) * p.rows);
  float acc[8] = {};
  // Adds acc to this thread's sums in shared memory; `rest` is what their last bits have lost.
  float *const total = &sums[warp][8 * lane], *const lost = &rest[warp][8 * lane];
  int n = 0;
  bool folded = false;
  const auto fold = [&] {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = folded ? total[j] : 0.0f, y = acc[j] - (folded ? lost[j] : 0.0f), t = s + y;
      total[j] = t;
      lost[j] = fabsf(t) < __int_as_float(0x7F800000) ? (t - s) - y : 0.0f;      // an infinity stays one
      acc[j] = 0.0f;
    }
    folded = true;
    n = 0;
  };
  if (c < p.d) {
    for (int r0 = blockIdx.y * p.rows + warp; r0 < end; r0 += kAhead * kWarps) {
      Vec8<Y> yv[kAhead];
      Vec8<__nv_bfloat16> zv[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kWarps;
        yv[i].zero();
        zv[i].zero();
        if (r < end) {
          yv[i].load(static_cast<const Y*>(p.dy) + r * p.lddy + c);
          if constexpr (ACT != kActNone) zv[i].load(p.z + static_cast<size_t>(r) * p.d + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kWarps;
        float y[8], z[8];
        yv[i].get(y);
        zv[i].get(z);
        if constexpr (ACT != kActNone) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const F2 g = vmul(F2{y[j], y[j + 1]}, linear_slope<ACT>(F2{z[j], z[j + 1]}));
            y[j] = g.x, y[j + 1] = g.y;
          }
        }
        if (r < end) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += y[j];
          if (p.dz) {
            Vec8<__nv_bfloat16> o;
            o.set(y);
            o.store(p.dz + static_cast<size_t>(r) * p.d + c);
          }
        }
      }
      if (++n == kFold && p.dbias) fold();
    }
  }
  if (!p.dbias) return;
  Vec8<float> v;
  if (folded) {
    fold();
  } else {
    v.set(acc);
    v.store(total);
  }
  __syncthreads();
  const int x = threadIdx.x, col = blockIdx.x * kCols + x;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sums[w][x];
  if (gridDim.y == 1) {
    if (col < p.d) p.dbias[col] = s;
    return;
  }
  const size_t step = static_cast<size_t>(gridDim.x) * kCols;
  p.part[blockIdx.y * step + col] = s;
  __threadfence();
  __syncthreads();
  if (x == 0) last = atomicAdd(&p.done[blockIdx.x], 1) == static_cast<int>(gridDim.y) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // Each warp adds every eighth part of all columns, its loads in flight together; then the warps' sums.
  float t[8] = {};
#pragma unroll
  for (int k = 0; k < kLinearMaxParts / kWarps; ++k) {
    const int r = warp + k * kWarps;
    if (r < static_cast<int>(gridDim.y)) {
      const float4* at = reinterpret_cast<const float4*>(p.part + r * step + c);
      const float4 a = __ldcg(at), b = __ldcg(at + 1);
      t[0] += a.x, t[1] += a.y, t[2] += a.z, t[3] += a.w, t[4] += b.x, t[5] += b.y, t[6] += b.z, t[7] += b.w;
    }
  }
  v.set(t);
  v.store(&sums[warp][8 * lane]);
  __syncthreads();
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sums[w][x];
  if (col < p.d) p.dbias[col] = s;
  if (x == 0) p.done[blockIdx.x] = 0;
}

template <class Y>
cudaError_t launch(const Params& p, int act, dim3 grid, cudaStream_t s) {
  const dim3 block(32 * kWarps);
  switch (act) {
    case kActRelu: return launch_pdl(linear_dz_kernel<Y, kActRelu>, grid, block, 0, s, p);
    case kActSilu: return launch_pdl(linear_dz_kernel<Y, kActSilu>, grid, block, 0, s, p);
    case kActGelu: return launch_pdl(linear_dz_kernel<Y, kActGelu>, grid, block, 0, s, p);
    default: return launch_pdl(linear_dz_kernel<Y, kActNone>, grid, block, 0, s, p);
  }
}

// CTAs along the rows: about four for each SM, each warp with eight rows at least, and
// not more sums than the last CTA adds in a microsecond or two.
int row_ctas(int T, int d) {
  const int tiles = (d + kCols - 1) / kCols;
  int n = 608 / tiles;
  if (n > (T + 63) / 64) n = (T + 63) / 64;
  return n > kLinearMaxParts ? kLinearMaxParts : n < 1 ? 1 : n;
}

}  // namespace

size_t linear_dz_tiles(int d) { return static_cast<size_t>((d + kCols - 1) / kCols); }
size_t linear_dz_partials(int d) { return linear_dz_tiles(d) * kCols * kLinearMaxParts; }

cudaError_t launch_linear_dz(const void* dy, long long lddy, bool fp32, const void* z, int act, int T, int d, void* dz,
                             float* dbias, float* part, int* done, cudaStream_t s) {
  Params p = {};
  p.dy = dy;
  p.lddy = lddy;
  p.z = static_cast<const __nv_bfloat16*>(z);
  p.dz = static_cast<__nv_bfloat16*>(dz);
  p.dbias = dbias;
  p.part = part;
  p.done = done;
  p.T = T;
  p.d = d;
  p.apart = dz == nullptr;
  const int n = row_ctas(T, d);
  p.rows = (T + n - 1) / n;
  const dim3 grid(static_cast<unsigned>(linear_dz_tiles(d)), (T + p.rows - 1) / p.rows);
  return fp32 ? launch<float>(p, act, grid, s) : launch<__nv_bfloat16>(p, act, grid, s);
}

}  // namespace lmoe
