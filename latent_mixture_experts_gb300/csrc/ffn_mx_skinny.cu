// The MXFP8 feed-forward passes on small batches (up to 48 tokens), bound by
// streaming the weights' codes and scales once from HBM.
//
// As in the bf16 form, tokens are the MMA's M rows, weight rows its N columns
// (128: one whole scale atom for each 128-wide K block), and a cluster splits
// K.  Each CTA finishes a share of the tokens with all of the tile's features,
// so that a warp holds a whole 32-value block of the hidden activation when it
// encodes it.  The scales of the tokens are put into
// shared memory once, for all of the CTA's K range: x's by the epilogue's
// warps, which are idle then, from rows as the caller has them; hid's by one
// bulk copy.  MXFP8 weights do not change while the handle lives, so both
// passes load their first stages before they wait for the kernel before them.
#include "ffn_act.cuh"
#include "ffn_internal.h"
#include "issue.cuh"
#include "lmoe_internal.h"

namespace lmoe {
namespace {

// Warps: 0 = TMA, 1 = MMA, 2-5 read the sums out of tensor memory; all finish
// them, ten of them for more than 16 tokens.
constexpr int kThreads = 192, kManyThreads = 320, kManyTokens = 16;
constexpr int kN = kMxSkinnyN, kHalf = kN / 2;
constexpr int kB = kN * 128;             // codes of a 128-wide K block
constexpr int kMaxStages = 8;            // 8 columns of scales each, beside 128 of sums
constexpr int kTmem = 256, kSfCols = 8;
constexpr int kSfb = 512;
constexpr int kMxSkinnySmem = 110 * 1024;   // two CTAs on an SM
constexpr int kPitch = kN + 4;           // floats of a token's partial sums: 16-byte rows, four banks apart
// Up to here rather than the pair tiles: 40, 48 and 56 tokens at widths 7168 and
// 6144 take 34.2, 35.9 and 37.4 us here and 35.4, 35.6 and 35.9 us there, at 7168 and
// 2048 19.0, 20.0 and 21.1 us and 23.3, 23.2 and 23.1 us, at 512 and 3584 10.3, 11.4 and
// 12.2 us and 13.3, 13.4 and 13.5 us.  One limit for all widths, too high a one where
// both are 2048 or less: 48 tokens at 2048 and 2048 14.4 us here and 13.7 us there, at
// 768 and 768 10.5 us and 9.9 us, at 256 and 256 11.7 us and 8.6 us.  16 tokens at 7168
// and 6144: 29.8 us, 4.6 TB/s of weights.
constexpr int kMxSkinnyMaxTokens = 48;
static_assert(kN + kMaxStages * kSfCols <= kTmem, "tensor memory");

template <bool GU, int ACT>
__global__ void __launch_bounds__(kManyThreads) ffn_mx_skinny_kernel(const __grid_constant__ FfnMxSkinnyParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done, rows_ready;
  __shared__ uint32_t tmem_base;
  __shared__ int lost;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform
  const int rank = static_cast<int>(cluster_rank());
  const int tile = static_cast<int>(blockIdx.x) / p.splits;
  const int first = rank * p.nkb / p.splits, steps = (rank + 1) * p.nkb / p.splits - first;
  // stage: A rows, B rows; behind the ring the B scales, the tokens' scales and the partial sums
  const int a_bytes = p.tb * 128;
  uint8_t* sb = sm + p.stages * a_bytes;
  uint8_t* sfb = sb + p.stages * kB;
  uint8_t* sfa = sm + p.sfa_at;
  float* recv = reinterpret_cast<float*>(sm + p.recv);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    lost = 0;
    mbar_init(&rows_ready, GU ? blockDim.x / 32 - 2 : 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(&tmem_base, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!p.reuse_ring) cluster_arrive();
  const uint32_t tacc = tmem_base;
  griddep_launch();
  if (warp != 0) griddep_wait();

  if (warp == 0) {
    auto load_b = [&](int i, int s) {
      const int kb = first + i;
      uint8_t* dst = sb + s * kB;
      if constexpr (GU) {
        w_load_2d(dst, &p.b[0], &full[s], kb * 128, tile * kHalf);
        w_load_2d(dst + kHalf * 128, &p.b[1], &full[s], kb * 128, tile * kHalf);
      } else {
        w_load_2d(dst, &p.b[0], &full[s], kb * 128, tile * kN);
        w_load_2d(dst + kHalf * 128, &p.b[0], &full[s], kb * 128, tile * kN + kHalf);
      }
      w_load_2d(sfb + s * kSfb, &p.sfb, &full[s], 0, tile * p.nkb + kb);
    };
    const int pre = steps < p.stages ? steps : p.stages;
    for (int i = 0; i < pre; ++i) {
      w_arrive_expect_tx(&full[i], a_bytes + kB + kSfb);
      load_b(i, i);
    }
    griddep_wait();
    for (int i = 0; i < pre; ++i) w_load_2d(sm + i * a_bytes, &p.a, &full[i], (first + i) * 128, 0);
    if (!GU) {
      w_arrive_expect_tx(&rows_ready, steps * 512);
      w_bulk_load(sfa, p.row_sf + static_cast<size_t>(first) * 512, steps * 512, &rows_ready);
    }
    int s = pre == p.stages ? 0 : pre;
    uint32_t phase = 0;
    for (int i = pre; i < steps; ++i) {
      if (!warp_wait(&empty[s], phase, p.err)) break;
      w_arrive_expect_tx(&full[s], a_bytes + kB + kSfb);
      load_b(i, s);
      w_load_2d(sm + s * a_bytes, &p.a, &full[s], (first + i) * 128, 0);
      if (++s == p.stages) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {
    const uint64_t a_desc = sdesc_sw128(smem_u32(sm)), b_desc = sdesc_sw128(smem_u32(sb));
    const uint64_t sa_desc = sdesc_noswz(smem_u32(sfa), 16, 128), sb_desc = sdesc_noswz(smem_u32(sfb), 16, 128);
    int s = 0;
    uint32_t phase = 0;
    bool ok = warp_wait(&rows_ready, 0, p.err);
    for (int i = 0; i < steps && ok; ++i) {
      if (!(ok = warp_wait(&full[s], phase, p.err))) break;
      tc_fence_after();
      const uint64_t ad = a_desc + static_cast<uint32_t>(s * a_bytes >> 4), bd = b_desc + s * (kB >> 4);
      const uint32_t sf = tacc + kN + s * kSfCols;
      w_copy_atom(sf, sa_desc + 32 * i);
      w_copy_atom(sf + 4, sb_desc + 32 * s);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w_mma_mx(tacc, ad + 2 * k, bd + 2 * k, idesc_mxf8f6f4(128, kN, 0, 0, k, k), sf, sf + 4, (i | k) != 0);
      w_commit(&empty[s]);
      if (++s == p.stages) s = 0, phase ^= 1;
    }
    if (ok) w_commit(&done);
  } else if constexpr (GU) {
    // x's scales of this K range, from rows [T][K/32] to the MMA's image
    const int t0 = threadIdx.x - 64;
    for (int e = t0; e < p.T * steps; e += static_cast<int>(blockDim.x) - 64) {
      const int row = e / steps, i = e - row * steps, blk = 4 * (first + i);
      const uint8_t* src = p.row_sf + static_cast<size_t>(row) * p.kblks + blk;
      uint32_t w = 0;
      if (p.kblks % 4 == 0) {
        w = *reinterpret_cast<const uint32_t*>(src);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (blk + k < p.kblks) w |= static_cast<uint32_t>(src[k]) << (8 * k);
      }
      *reinterpret_cast<uint32_t*>(sfa + i * 512 + sf_atom_offset(row, 0)) = w;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&rows_ready);
  }
  __syncwarp();

  const bool ok = mbar_wait(&done, 0, p.err, kErrTimeout);
  if (__builtin_expect(!ok, 0)) let_copies_land();
  tc_fence_after();
  __syncwarp();
  if (p.reuse_ring) cluster_arrive();
  cluster_wait();
  if (__builtin_expect(!ok, 0)) cluster_lost(&lost, p.splits);
  __syncwarp();
  // Token t is finished by CTA t / per: its row of partial sums goes to that
  // CTA's shared memory, one block [per][kPitch] for each source rank.
  const int per = (p.T + p.splits - 1) / p.splits;
  const int q = warp & 3, t = 32 * q + lane;
  if (warp >= 2 && warp < 6 && 32 * q < p.T) {
    const int owner = t < p.T ? t / per : 0;
    const uint32_t dst = map_rank(recv, owner) + 4 * ((rank * per + t - owner * per) * kPitch);
#pragma unroll 1
    for (int c = 0; c < kN; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem_addr(tacc, 32 * q, c), v);
      tmem_ld_wait();
      if (t < p.T)
#pragma unroll
        for (int j = 0; j < 32; j += 4) st_cluster4(dst + 4 * (c + j), v + j);
      __syncwarp();      // lanes part at the stores; whole warps load
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tacc, kTmem);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  const int tok0 = rank * per, ntok = min(per, p.T - tok0);
  if (__builtin_expect(lost, 0)) {      // sums that are not whole become NaN by their first part
    for (int e = threadIdx.x; e < per * kPitch; e += blockDim.x) recv[e] = __int_as_float(0x7FC00000);
    __syncthreads();
  }
  if constexpr (GU) {
    // one warp for each token and block of 32 features, lane = feature
    constexpr int kBlocks = kHalf / 32;
    const GluCaps caps = {p.b1, p.b2, 1.0f / p.b1, 1.0f / p.b2};
    for (int e = warp; e < kBlocks * ntok; e += blockDim.x / 32) {
      const int i = e / kBlocks, c = 32 * (e - kBlocks * i), f = tile * kHalf + c;
      if (f >= p.M) continue;
      float g = 0.f, u = 0.f;
      for (int r = 0; r < p.splits; ++r) {
        const float* src = recv + (r * per + i) * kPitch + c + lane;
        g += src[0];
        u += src[kHalf];
      }
      const float h = glu_hidden<ACT>(g, u, caps);
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h)));
      // an infinity or NaN makes the block NaN: E8M0 byte 255
      const uint32_t s = m >= 0x7F800000u ? 255u : e4m3_block_scale(__uint_as_float(m));
      const int row = tok0 + i;
      static_cast<uint8_t*>(p.out)[static_cast<size_t>(row) * p.M + f + lane] =
          f32_to_e4m3(h * (s == 255u ? 1.0f : e8m0_to_f32(254u - s)));
      if (lane == 0)
        p.out_sf[static_cast<size_t>(f >> 7) * 512 + sf_atom_offset(row, (f >> 5) & 3)] = static_cast<uint8_t>(s);
    }
  } else {
    for (int e = threadIdx.x; e < ntok * kHalf; e += blockDim.x) {
      const int i = e / kHalf, c = 2 * (e - i * kHalf), f = tile * kN + c;
      if (f >= p.M) continue;
      float2 v = make_float2(0.f, 0.f);
      for (int r = 0; r < p.splits; ++r) {
        const float2 a = *reinterpret_cast<const float2*>(recv + (r * per + i) * kPitch + c);
        v.x += a.x, v.y += a.y;
      }
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(tok0 + i) * p.M + f) =
          pack_bf16(v.x, v.y);
    }
  }
}

template <bool GU, int ACT>
cudaError_t launch(const FfnMxSkinnyParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, ffn_mx_skinny_kernel<GU, ACT>, kMxSkinnySmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(ffn_mx_skinny_kernel<GU, ACT>, dim3(p.tiles * p.splits),
                            dim3(p.T > kManyTokens ? kManyThreads : kThreads), kMxSkinnySmem,
                            p.splits, s, p);
}

}  // namespace

bool ffn_mx_skinny_plan(FfnMxSkinnyParams& p, bool gate_up) {
  if (p.T > kMxSkinnyMaxTokens) return false;
  p.tiles = gate_up ? (p.M + kHalf - 1) / kHalf : (p.M + kN - 1) / kN;
  p.tb = (p.T + 7) / 8 * 8;
  // as in the bf16 form, in 128-wide K blocks
  p.splits = 1;
  for (int n = 2; n <= kSkinnyMaxSplits; n *= 2) {
    const int ctas = p.tiles * p.splits, left = p.nkb / n;
    if (n > p.nkb || !((ctas < 110 && left >= 2) || (ctas < 150 && left >= 6))) break;
    p.splits = n;
  }
  const int budget = kMxSkinnySmem - 1024;
  const int sfa = (p.nkb + p.splits - 1) / p.splits * 512;
  const int recv = 4 * p.splits * ((p.T + p.splits - 1) / p.splits) * kPitch;
  // the partial sums meet behind the ring, or over it where room behind would cost a stage
  const int stage = p.tb * 128 + kB + kSfb;
  p.reuse_ring = (budget - sfa - recv) / stage < (budget - sfa) / stage;
  const int ring = (budget - sfa - (p.reuse_ring ? 0 : recv)) / 1024 * 1024;
  p.stages = ring / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.sfa_at = ring;
  p.recv = p.reuse_ring ? 0 : ring + sfa;
  // the MMA reads 128 token rows from the last stage's A on
  const int a_end = p.stages * p.tb * 128 + (128 - p.tb) * 128;
  return p.stages >= 2 && recv <= budget && a_end <= budget;
}

cudaError_t launch_ffn_mx_skinny(const FfnMxSkinnyParams& p, bool gate_up, int act, cudaStream_t s) {
  if (!gate_up) return launch<false, 0>(p, s);
  return act == 1 ? launch<true, 1>(p, s) : launch<true, 0>(p, s);
}

}  // namespace lmoe
