// The products of the dense feed-forward block where the pair tiles of
// ffn_gemm.cu would leave half of the SMs idle: the same 256 x 128 tile of a
// CTA pair, with K split over the pairs of a cluster.
//
// What a pair loads for its tile, 24 KB of shared memory per CTA and 64-wide K
// block at about 64 bytes a clock, bounds such calls; two or four pairs each
// load a part of K.  Their partial sums meet in distributed shared memory: each
// pair finishes 1 / S of the tile's columns, adding the parts in the pairs'
// order.
//
// Warps: 0 = TMA, 1 = MMA (the even CTA of a pair); then all eight read the sums
// out of tensor memory (lane quarter warp % 4, column half warp / 4) and finish
// the joined ones, columns along threads.
#include "ffn_act.cuh"
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "issue.cuh"

namespace lmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kA = 16384, kB = 8192, kStage = kA + kB;   // 128 rows of A, 64 of B, x 64 bf16
constexpr int kStages = 6;
constexpr int kTN = 128;              // columns of a tile: gate and up of 64 features, or output features
constexpr int kPitch = 129;           // 16-byte units between quads of columns: no two of eight in the same banks
constexpr int kSmem = kStages * kStage + kTN / 4 * kPitch * 16 + 1024;

// MODE: FfnMode, kFfnGrads for dx.  S: pairs of a cluster.
template <int MODE, int ACT, int S>
__global__ void __launch_bounds__(kThreads) ffn_split_kernel(const __grid_constant__ FfnPairParams p) {
  constexpr bool kBMn = MODE == kFfnDHid || MODE == kFfnGrads, kGu = MODE == kFfnGateUp, kDx = MODE == kFfnGrads;
  constexpr int kQuads = kTN / 4 / S;              // of columns, that a CTA finishes (gate/up: of both kinds)
  constexpr int kOwn = kGu ? kQuads / 2 : kQuads;  // quads of output features among them
  constexpr int kEach = 128 * kOwn / kThreads;     // of a thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ uint64_t full[kStages], empty[kStages], done;
  __shared__ uint32_t tmem_base;
  __shared__ int lost;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform
  const uint32_t crank = cluster_rank(), rank = crank & 1, leader = crank & ~1u;
  const int split = static_cast<int>(crank >> 1);
  const int tile = static_cast<int>(blockIdx.x) / (2 * S), tm = (p.M[0] + 255) / 256;
  const int n = tile / tm, m0 = (tile - n * tm) * 256 + 128 * static_cast<int>(rank);
  const int nkb = kDx ? 2 * p.nkb_cat : p.nkb;
  const int kb0 = split * nkb / S, steps = (split + 1) * nkb / S - kb0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    lost = 0;
    fence_mbar_init();
  }
  __syncwarp();
  cluster_sync();
  if (warp == 1) {      // under the first loads
    tmem_alloc_pair(&tmem_base, kTN);
    tmem_relinquish_pair();
  }
  // The dependents are let in only after everything before this kernel has
  // finished: where they are this file's, they may read weights at once.
  const bool producer = warp == 0;
  if (!(producer && p.early)) {
    griddep_wait();
    griddep_launch();
  }

  if (producer) {
    const uint32_t bar0 = map_rank(&full[0], leader);
    const auto load_b = [&](int i, int s) {
      const bool second = kDx && kb0 + i >= p.nkb_cat;      // the concatenation's second half
      const int k0 = (second ? kb0 + i - p.nkb_cat : kb0 + i) * 64;
      uint8_t* dst = sm + s * kStage + kA;
      const uint32_t bar = bar0 + 8 * s;
      if constexpr (kGu)        // gate rows in the even CTA, up rows in the odd one
        w_load_2d_pair(dst, &p.b[rank], bar, k0, n * (kTN / 2));
      else if constexpr (kBMn)
        w_load_2d_pair(dst, second ? &p.b_cat : &p.b[0], bar, n * kTN + 64 * static_cast<int>(rank), k0);
      else
        w_load_2d_pair(dst, &p.b[0], bar, k0, n * kTN + 64 * static_cast<int>(rank));
    };
    const auto load_a = [&](int i, int s) {
      const bool second = kDx && kb0 + i >= p.nkb_cat;
      const int k0 = (second ? kb0 + i - p.nkb_cat : kb0 + i) * 64;
      w_load_2d_pair(sm + s * kStage, second ? &p.a_cat : &p.a[0], bar0 + 8 * s, k0, m0);
    };
    const int pre = steps < kStages ? steps : kStages;
    for (int i = 0; i < pre; ++i) {
      if (rank == 0) w_arrive_expect_tx(&full[i], 2 * kStage);
      load_b(i, i);
    }
    if (p.early) {
      griddep_wait();
      griddep_launch();
    }
    for (int i = 0; i < pre; ++i) load_a(i, i);
    int s = 0;
    uint32_t phase = 0;
    for (int i = kStages; i < steps; ++i) {
      if (!warp_wait(&empty[s], phase, p.err)) break;
      if (rank == 0) w_arrive_expect_tx(&full[s], 2 * kStage);
      load_b(i, s);
      load_a(i, s);
      if (++s == kStages) s = 0, phase ^= 1;
    }
  } else if (warp == 1 && rank == 0) {
    const uint32_t base = smem_u32(sm), tacc = tmem_base;
    const uint64_t a_desc = sdesc_sw128(base);
    const uint64_t b_desc = kBMn ? sdesc_sw128_mn(base + kA, 8192) : sdesc_sw128(base + kA);
    const uint32_t idesc = idesc_bf16(256, kTN) | (kBMn ? kIdescBMajorMn : 0u);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      if (!(ok = warp_wait(&full[s], phase, p.err))) break;
      tc_fence_after();
      // descriptors count 16-byte units: a step of 16 along K is 32 bytes of a
      // K-contiguous row, or 16 rows of 128 bytes
      const uint64_t ad = a_desc + s * (kStage >> 4), bd = b_desc + s * (kStage >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w_mma_bf16_pair(tacc, ad + 2 * k, bd + k * (kBMn ? 128 : 2), idesc, (i | k) != 0);
      w_commit_pair(&empty[s], leader);
      if (++s == kStages) s = 0, phase ^= 1;
    }
    if (ok) w_commit_pair(&done, leader);
  }
  __syncwarp();

  // This thread's outputs: rows e / kOwn, quads of features e % kOwn of the CTA's.
  const int N = p.N[0], f0 = kGu ? n * (kTN / 2) + split * 4 * kOwn : n * kTN + split * 4 * kOwn;
  uint2 gv[kEach], uv[kEach];
  if constexpr (MODE == kFfnDHid) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = threadIdx.x + i * kThreads, row = m0 + e / kOwn, f = f0 + 4 * (e % kOwn);
      gv[i] = uv[i] = make_uint2(0, 0);
      if (row < p.M[0] && f < N) {
        const size_t at = static_cast<size_t>(row) * N + f;
        gv[i] = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.in_g) + at);
        uv[i] = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.in_u) + at);
      }
    }
  }

  // The products are done, and so the ring's loads.
  __syncthreads();      // tmem_base
  const uint32_t tacc = tmem_base;
  const bool ok = mbar_wait_cluster(&done, 0, p.err, kErrTimeout);
  if (__builtin_expect(!ok, 0)) {
    let_copies_land();
    cluster_lost(&lost, 2 * S);
  }
  tc_fence_after();
  __syncwarp();
  uint8_t* recv = sm + kStages * kStage;
  // The partial sums (lane = row) to the CTA of the same side in the pair that
  // owns the columns: quad q of source r at (r kQuads + q) kPitch + row, in 16 bytes.
  const int q = warp & 3;
  if (m0 + 32 * q < p.M[0]) {
#pragma unroll 1
    for (int c = kTN / 2 * (warp >> 2); c < kTN / 2 * ((warp >> 2) + 1); c += 32) {
      uint32_t v[32];
      tmem_ld32(tacc + (static_cast<uint32_t>(32 * q) << 16) + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const int up = kGu && c + j >= kTN / 2, f4 = (c + j - (up ? kTN / 2 : 0)) / 4, o = f4 / kOwn;
        const int quad = split * kQuads + f4 - o * kOwn + (up ? kOwn : 0);
        st_cluster4(map_rank(recv, 2 * o + rank) + 16 * (quad * kPitch + 32 * q + lane), v + j);
      }
    }
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tacc, kTN);
  }
  cluster_arrive();      // neither CTA leaves while the other still frees the pair's columns

  const GluCaps caps = {p.b1, p.b2, 1.0f / p.b1, 1.0f / p.b2};
  const float4* part = reinterpret_cast<const float4*>(recv);
  if (__builtin_expect(lost, 0)) {      // sums that are not whole become NaN by their first part
    const float nan = __int_as_float(0x7FC00000);
    for (int e = threadIdx.x; e < 128 * kQuads; e += kThreads)
      reinterpret_cast<float4*>(recv)[e / 128 * kPitch + e % 128] = make_float4(nan, nan, nan, nan);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / kOwn, quad = e % kOwn, row = m0 + r, f = f0 + 4 * quad;
    if (row >= p.M[0] || f >= N) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const float4 a = part[(k * kQuads + quad) * kPitch + r];
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      if constexpr (kGu) {
        const float4 b = part[(k * kQuads + kOwn + quad) * kPitch + r];
        w.x += b.x, w.y += b.y, w.z += b.z, w.w += b.w;
      }
    }
    const size_t at = static_cast<size_t>(row) * N + f;
    const auto put = [&](void* out, uint32_t lo, uint32_t hi) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint2(lo, hi);
    };
    if constexpr (kGu) {
      put(p.out[0], pack_bf16(glu_hidden<ACT>(F2{v.x, v.y}, F2{w.x, w.y}, caps)),
          pack_bf16(glu_hidden<ACT>(F2{v.z, v.w}, F2{w.z, w.w}, caps)));
      if (p.out[1]) {
        put(p.out[1], pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        put(p.out[2], pack_bf16(w.x, w.y), pack_bf16(w.z, w.w));
      }
    } else if constexpr (MODE == kFfnDHid) {
      const GluGrad a = glu_grad<ACT>(bf16_both(gv[i].x), bf16_both(uv[i].x), F2{v.x, v.y}, caps);
      const GluGrad b = glu_grad<ACT>(bf16_both(gv[i].y), bf16_both(uv[i].y), F2{v.z, v.w}, caps);
      put(p.out[0], pack_bf16(a.dg), pack_bf16(b.dg));
      put(p.out[1], pack_bf16(a.du), pack_bf16(b.du));
      put(p.out[2], pack_bf16(a.hid), pack_bf16(b.hid));
    } else {
      put(p.out[0], pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
  }
  __syncwarp();
  cluster_wait();
}

template <int MODE, int ACT, int S>
cudaError_t launch(const FfnPairParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, ffn_split_kernel<MODE, ACT, S>, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(ffn_split_kernel<MODE, ACT, S>, dim3(2 * S * p.tile_end[0]), dim3(kThreads), kSmem, 2 * S,
                            s, p);
}
template <int MODE, int ACT>
cudaError_t launch(const FfnPairParams& p, int splits, cudaStream_t s) {
  return splits == 2 ? launch<MODE, ACT, 2>(p, s) : launch<MODE, ACT, 4>(p, s);
}

}  // namespace

int ffn_split_plan(FfnPairParams& p, FfnMode mode, const FfnSplitLimits& l) {
  const int width = mode == kFfnGateUp ? kTN / 2 : kTN;
  p.tile_end[0] = (p.M[0] + 255) / 256 * ((p.N[0] + width - 1) / width);
  const int tiles = p.tile_end[0], nkb = mode == kFfnGrads ? 2 * p.nkb_cat : p.nkb;
  const bool bwd = mode == kFfnDHid || mode == kFfnGrads;
  // Split while all clusters run at once and a pair keeps two K blocks.  Whole
  // tiles, two, two or four splits: 256 tokens at 256 x 256 forward 10.0 us, 9.0 us,
  // backward 15.4 us, 12.0 us; at 2048 x 1024 15.9 us, 13.1 us, 12.5 us and 26.7 us,
  // 23.0 us, 19.8 us; 1003 tokens at 1152 x 864 backward 25.3 us, 24.6 us.  Four of
  // 12 blocks (768 x 768): forward 11.5 us against 10.5 us, but backward 15.6 us
  // against 16.7 us.
  if (tiles <= l.clusters4 && nkb >= (bwd ? 8 : 16)) return 4;
  return tiles <= l.clusters2 && nkb >= 4 ? 2 : 1;
}

cudaError_t launch_ffn_split(FfnMode mode, const FfnPairParams& p, int splits, cudaStream_t s) {
  const bool sw = p.act == 1;
  switch (mode) {
    case kFfnGateUp: return sw ? launch<kFfnGateUp, 1>(p, splits, s) : launch<kFfnGateUp, 0>(p, splits, s);
    case kFfnPlain: return launch<kFfnPlain, 0>(p, splits, s);
    case kFfnDHid: return sw ? launch<kFfnDHid, 1>(p, splits, s) : launch<kFfnDHid, 0>(p, splits, s);
    case kFfnGrads: return launch<kFfnGrads, 0>(p, splits, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t ffn_split_limits(FfnSplitLimits* l) {
  const auto query = [](auto kernel, int ctas, int* n) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
  };
  const cudaError_t e = query(ffn_split_kernel<kFfnPlain, 0, 2>, 4, &l->clusters2);
  return e != cudaSuccess ? e : query(ffn_split_kernel<kFfnPlain, 0, 4>, 8, &l->clusters4);
}

}  // namespace lmoe
