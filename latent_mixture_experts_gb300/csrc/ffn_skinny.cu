// The feed-forward block's two forward passes on small batches (bf16), where
// streaming the weights once from HBM bounds the time.
//
// Tokens are the MMA's M rows (rows past the batch are whatever shared memory
// holds, and only reach output rows that nobody reads), weight rows its N
// columns.  A cluster of up to 8 CTAs owns `rows` consecutive output features
// and splits K; its partial sums are joined through distributed shared memory,
// in rank order, by all of its CTAs: one token at widths 7168 and 2048 takes
// 20 us, against 32 us with narrow tiles over the whole of K (an MMA reads its
// 128 token rows whatever its width).  The gate and up rows of the same
// features lie side by side in a stage, each by a copy of its own.  (One tensor
// map over both matrices, with a dimension that steps from one to the other,
// would save half of the copies, but its copies also bring in memory behind the
// first matrix, 80 KB for one of 2 KB, that need not be there: an illegal access.
// Copies by maps of one matrix stayed within its 4 KB blocks, 188 maps measured.)
// A ring of about 100 KB per CTA puts two CTAs on an SM, and lets the down
// pass's CTAs load their first weights while the gate/up pass's last ones
// finish.  One token at 7168 and 6144: 47 to 48 us, 5.5 TB/s of weights.
#include "ffn_act.cuh"
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "issue.cuh"

namespace lmoe {
namespace {

// Warps: 0 = TMA, 1 = MMA; 0-3 read the sums out of tensor memory; all finish
// them, eight of them for more than 16 tokens (64 tokens at 7168 x 2048: 24.4 us
// against 25.1 us with four; one token 20.2 us against 20.0 us).
constexpr int kThreads = 128, kManyThreads = 256, kManyTokens = 16;
// MMA columns, the weight rows of a tile.  Wider tiles cost fewer MMAs, narrower
// ones fewer bytes of partial sums: one token at widths 7168 and 6144 takes
// 45.5 us with 128 columns, 46.4 us with 64 and 61 us with 32; at 7168 and 2048
// 20.6 us, 20.0 us and 23.6 us; 64 tokens there 29 us, 25 us and 26 us.
constexpr int kCols = 64;

// GU: gate and up rows of 32 features -> act(g, u); else 64 output features of
// one matrix.
template <bool GU, int ACT>
__global__ void __launch_bounds__(kManyThreads) ffn_skinny_kernel(const __grid_constant__ FfnSkinnyParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ uint64_t full[kSkinnyMaxStages], empty[kSkinnyMaxStages], done;
  __shared__ uint32_t tmem_base;
  __shared__ int lost;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform
  constexpr int N = kCols, rows = GU ? N / 2 : N;     // features of the cluster
  const int rank = static_cast<int>(cluster_rank());  // K split of this CTA
  const int f0 = static_cast<int>(blockIdx.x) / p.splits * rows;   // first feature
  const int a_chunk = p.tb * 128, b_chunk = N * 128;  // bytes of one 64-wide K chunk
  const int a_slot = a_chunk * p.kc, b_slot = b_chunk * p.kc;
  uint8_t* sb = sm + p.stages * a_slot;
  const int all = (p.chunks + p.kc - 1) / p.kc;
  const int first = rank * all / p.splits, steps = (rank + 1) * all / p.splits - first;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    lost = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, N);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();      // every CTA of the cluster runs before another one writes to it
  const uint32_t tacc = tmem_base;
  const bool producer = warp == 0;
  // The dependents are let in only after everything before this kernel has
  // finished: the down pass may then read its weights at once.
  if (GU || !producer) {
    griddep_wait();
    griddep_launch();
  }

  if (producer) {
    auto load_b = [&](int i, int s) {
      i += first;
      uint8_t* dst = sb + s * b_slot;
      if (!GU && p.whole) {
        w_load_3d(dst, &p.b, &full[s], 0, f0, i * p.kc);
      } else {
        for (int c = 0; c < p.kc; ++c) {
          w_load_2d(dst + c * b_chunk, &p.b, &full[s], (i * p.kc + c) * 64, f0);
          if constexpr (GU) w_load_2d(dst + c * b_chunk + (b_chunk >> 1), &p.b_up, &full[s], (i * p.kc + c) * 64, f0);
        }
      }
    };
    auto load_a = [&](int i, int s) {
      i += first;
      uint8_t* dst = sm + s * a_slot;
      if (p.whole) {
        w_load_3d(dst, &p.a, &full[s], 0, 0, i * p.kc);
      } else {
        for (int c = 0; c < p.kc; ++c) w_load_2d(dst + c * a_chunk, &p.a, &full[s], (i * p.kc + c) * 64, 0);
      }
    };
    const int pre = steps < p.stages ? steps : p.stages;
    for (int i = 0; i < pre; ++i) {
      w_arrive_expect_tx(&full[i], a_slot + b_slot);
      load_b(i, i);
      if (GU) load_a(i, i);
    }
    if (!GU) {                     // the tokens come from the kernel before
      griddep_wait();
      griddep_launch();
      for (int i = 0; i < pre; ++i) load_a(i, i);
    }
    int s = pre == p.stages ? 0 : pre;
    uint32_t phase = 0;
    for (int i = pre; i < steps; ++i) {
      if (!warp_wait(&empty[s], phase, p.err)) break;
      w_arrive_expect_tx(&full[s], a_slot + b_slot);
      load_b(i, s);
      load_a(i, s);
      if (++s == p.stages) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(128, N);
    const uint64_t a_desc = sdesc_sw128(smem_u32(sm)), b_desc = sdesc_sw128(smem_u32(sb));
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      if (!(ok = warp_wait(&full[s], phase, p.err))) break;
      tc_fence_after();
      // descriptors count 16-byte units
      uint64_t ad = a_desc + static_cast<uint32_t>(s * a_slot >> 4);
      uint64_t bd = b_desc + static_cast<uint32_t>(s * b_slot >> 4);
      for (int c = 0; c < p.kc; ++c) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w_mma_bf16(tacc, ad + 2 * k, bd + 2 * k, idesc, (i | c | k) != 0);
        ad += a_chunk >> 4;
        bd += b_chunk >> 4;
      }
      w_commit(&empty[s]);
      if (++s == p.stages) s = 0, phase ^= 1;
    }
    if (ok) w_commit(&done);
  }
  __syncwarp();

  // Each CTA of the cluster finishes fs = rows / splits of the features: the
  // partial sums (lane = token) go straight into its shared memory, one block
  // [token][fs columns, GU: gate then up] per source rank, and are added in
  // rank order by all of its threads, features along threads.
  const bool ok = mbar_wait(&done, 0, p.err, kErrTimeout);
  if (__builtin_expect(!ok, 0)) let_copies_land();
  tc_fence_after();
  __syncwarp();
  cluster_wait();
  if (__builtin_expect(!ok, 0)) cluster_lost(&lost, p.splits);
  __syncwarp();
  const int lfs = 31 - __clz(rows / p.splits), fs = 1 << lfs;
  const int pitch = N / p.splits + 4;   // 16-byte rows, four banks apart
  float* recv = reinterpret_cast<float*>(sm + p.recv);
  const int row = 32 * warp;
  if (warp < 4 && row < p.T) {      // warp-uniform
    const uint32_t at = 4 * ((rank * p.T + row + lane) * pitch);
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem_addr(tacc, row, c), v);
      tmem_ld_wait();
      if (row + lane < p.T)
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          // four columns have one owner; its block holds fs gate columns, then fs up columns
          const int up = GU && c + j >= rows, f = c + j - (up ? rows : 0), o = f >> lfs;
          st_cluster4(map_rank(recv, o) + at + 4 * (f - o * fs + (up ? fs : 0)), v + j);
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tacc, N);
  cluster_arrive();
  cluster_wait();
  const GluCaps caps = {p.b1, p.b2, 1.0f / p.b1, 1.0f / p.b2};
  if (__builtin_expect(lost, 0)) {      // sums that are not whole become NaN by their first part
    for (int e = threadIdx.x; e < p.T * pitch; e += blockDim.x) recv[e] = __int_as_float(0x7FC00000);
    __syncthreads();
  }
  const int shift = lfs - 1;        // log2 of the pairs of features
  const int f1 = f0 + rank * fs, left = p.M - f1;
  for (int e = threadIdx.x; e < p.T << shift; e += blockDim.x) {
    const int t = e >> shift, f = 2 * (e - (t << shift));
    if (f >= left) continue;
    float2 v = make_float2(0.f, 0.f), w = v;
    for (int r = 0; r < p.splits; ++r) {
      const float* src = recv + (r * p.T + t) * pitch + f;
      const float2 a = *reinterpret_cast<const float2*>(src);
      v.x += a.x, v.y += a.y;
      if constexpr (GU) {
        const float2 b = *reinterpret_cast<const float2*>(src + fs);
        w.x += b.x, w.y += b.y;
      }
    }
    const size_t at = static_cast<size_t>(t) * p.M + f1 + f;
    if constexpr (GU) {
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at) =
          pack_bf16(glu_hidden<ACT>(F2{v.x, v.y}, F2{w.x, w.y}, caps));
      if (p.save_g) {
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.save_g) + at) = pack_bf16(v.x, v.y);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.save_u) + at) = pack_bf16(w.x, w.y);
      }
    } else {
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + at) = pack_bf16(v.x, v.y);
    }
  }
}

template <bool GU, int ACT>
cudaError_t launch(const FfnSkinnyParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, ffn_skinny_kernel<GU, ACT>, kSkinnySmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(ffn_skinny_kernel<GU, ACT>, dim3((p.M + p.rows - 1) / p.rows * p.splits),
                            dim3(p.T > kManyTokens ? kManyThreads : kThreads), kSkinnySmem, p.splits, s, p);
}

}  // namespace

bool ffn_skinny_plan(FfnSkinnyParams& p, bool gate_up) {
  if (p.T > kSkinnyMaxTokens) return false;
  constexpr int N = kCols;
  p.rows = gate_up ? N / 2 : N;
  const int tiles = (p.M + p.rows - 1) / p.rows;
  p.tb = (p.T + 7) / 8 * 8;
  const int chunk = (p.tb + N) * 128;
  p.kc = chunk <= 12 * 1024 ? 2 : 1;    // K chunks of a stage: up to 24 KB
  const int all = (p.chunks + p.kc - 1) / p.kc;
  // Split K until there is a CTA for most SMs, and on to two for each while
  // that leaves a CTA 12 chunks of K or more (a CTA's fixed costs against what
  // it streams: at 2048 x 2048 two splits of the gate/up pass 9.1 us, four
  // 10.5 us; at 7168 x 2048 22.0 us and 20.1 us).
  p.splits = 1;
  for (int s = 2; s <= kSkinnyMaxSplits; s *= 2) {
    const int ctas = tiles * p.splits, left = p.chunks / s;
    if (s > all || !((ctas < 110 && left >= 4) || (ctas < 150 && left >= 12))) break;
    p.splits = s;
  }
  const int budget = kSkinnySmem - 1024;
  const int recv = 4 * p.T * (N + 4 * p.splits);
  p.recv = (budget - recv) / 1024 * 1024;
  p.stages = p.recv / (chunk * p.kc);      // four at least
  if (p.stages > kSkinnyMaxStages) p.stages = kSkinnyMaxStages;
  // the joined sums, and the MMA's reads of up to 128 rows from the last chunk, stay inside
  const int a_end = p.stages * p.kc * p.tb * 128 + (128 - p.tb) * 128;
  return p.stages >= 2 && a_end <= budget;
}

cudaError_t launch_ffn_skinny(const FfnSkinnyParams& p, bool gate_up, int act, cudaStream_t s) {
  if (!gate_up) return launch<false, 0>(p, s);
  return act == 1 ? launch<true, 1>(p, s) : launch<true, 0>(p, s);
}

}  // namespace lmoe
