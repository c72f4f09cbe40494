// The feed-forward block on MXFP8 operands (E4M3 codes, one E8M0 scale per 32
// values along K): kind::mxf8f6f4 block-scaled tcgen05, scales applied by the
// tensor cores, fp32 accumulation, on 256 x 192 tiles of CTA pairs (256 x 128
// where those leave pairs idle).
//
// The structure is that of the bf16 pair tiles.  N = 192 rather than 256: two
// accumulators and seven stages' scales (12 columns each) fit tensor memory,
// so the epilogue still runs under the next tile's products; 96 gate and 96
// up rows keep the hidden activation's 32-value blocks inside a tile, and the
// thread that holds a row encodes them without talking to others.
//
// Scales live in memory in the image that the block-scaled MMA wants
// ("atoms": 512 bytes for 128 rows x 4 blocks) and come with the operands;
// the MMA thread copies them on to tensor memory (tcgen05.cp) ahead of each
// stage's products (4096 tokens of 7168 x 6144, when one lane still issued the
// loads and products: 553 us, against 964 us with a set of warps that moved them
// by tcgen05.st and 564 us with three sets).
// The weights' atoms are laid out once, when the handle is made; the hidden
// activation's are written by the gate/up epilogue; x's by a small kernel in
// front.
#include "ffn_act.cuh"
#include "ffn_internal.h"
#include "issue.cuh"
#include "lmoe_internal.h"

namespace lmoe {
namespace {

// TN: weight rows of a tile, 192 or 128.
template <int TN>
struct MxCfg {
  static constexpr int kHalf = TN / 2;                     // B rows of each CTA
  static constexpr int kA = 128 * 128, kB = kHalf * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kAtoms = (TN + 127) / 128;          // scale atoms of B
  static constexpr int kSf = 512 * (1 + kAtoms);
  static constexpr int kStages = TN == 192 ? 7 : 8;
  static constexpr int kSmem = kStages * (kStage + kSf) + 1024;
  static constexpr int kSfCols = 4 * (1 + kAtoms), kSfBase = 2 * TN;
  static_assert(kStage % 1024 == 0 && kSmem <= 227 * 1024 && kSfBase + kStages * kSfCols <= 512, "budgets");
};
constexpr int kThreads = 320;                        // TMA, MMA, 8 epilogue warps: two for each lane quarter
constexpr int kTmemBarrier = 1;                      // tmem_base is there for the epilogue warps
// Short runs of 4096 tokens at 7168 x 6144, before the power limit sets in (358 us in
// long ones): 307 us; 8 rows 312 us, 4 rows 319 us.
constexpr int kTileRows = 16;

__device__ __forceinline__ void tile_of(const FfnMxParams& p, int i, int& m, int& n) {
  const int tm = p.tiles / p.tiles_n;
  const int g = i / (kTileRows * p.tiles_n), r = i - g * kTileRows * p.tiles_n;
  const int rows = min(kTileRows, tm - g * kTileRows);
  m = g * kTileRows + r % rows;
  n = r / rows;
}

// One 32-value block of the hidden activation: codes to memory, scale byte
// to its place in the atom.
__device__ __forceinline__ void store_hidden_block(const float (&h)[32], uint8_t* codes, uint8_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(fabsf(h[j])));
  const uint32_t s = m >= 0x7F800000u ? 255u : e4m3_block_scale(__uint_as_float(m));
  const float inv = s == 255u ? 1.0f : e8m0_to_f32(254u - s);
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(h[4 * j] * inv, h[4 * j + 1] * inv), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(h[4 * j + 2] * inv, h[4 * j + 3] * inv), __NV_SATFINITE,
                                                 __NV_E4M3);
    q[j] = lo | (hi << 16);
  }
  reinterpret_cast<uint4*>(codes)[0] = make_uint4(q[0], q[1], q[2], q[3]);
  reinterpret_cast<uint4*>(codes)[1] = make_uint4(q[4], q[5], q[6], q[7]);
  *scale = static_cast<uint8_t>(s);
}

// Byte of block `kblk` of `row` in scale atoms [row / 128][nkb][512].
__device__ __forceinline__ size_t atom_byte(int row, int kblk, int nkb) {
  return (static_cast<size_t>(row >> 7) * nkb + (kblk >> 2)) * 512 + sf_atom_offset(row & 127, kblk & 3);
}

template <bool GU, int ACT, int TN>
__global__ void __launch_bounds__(kThreads, 1) ffn_mx_pair_kernel(const __grid_constant__ FfnMxParams p) {
  using C = MxCfg<TN>;
  constexpr int kStages = C::kStages, kStage = C::kStage, kSf = C::kSf, kHalfN = C::kHalf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint8_t* sf = sm + kStages * kStage;
  // full, acc_empty: used in the even CTA; the others in both
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform
  const int rank = static_cast<int>(cluster_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);     // the epilogue warps of both CTAs
    }
    fence_mbar_init();
  }
  __syncwarp();
  cluster_sync();
  griddep_launch();
  if (warp == 1) {      // under the first loads
    tmem_alloc_pair(&tmem_base, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (warp != 0) griddep_wait();
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;

  if (warp == 0) {
    uint32_t it = 0;
    bool ok = true;
    for (int i = first; i < p.tiles && ok; i += pairs) {
      int m, n;
      tile_of(p, i, m, n);
      const int m0 = m * 256 + 128 * rank;
      const int atom_a = (2 * m + rank) * p.nkb, atom_b = C::kAtoms * n * p.nkb;
      const auto load_b = [&](int kb, uint32_t s) {
        if (rank == 0) w_arrive_expect_tx(&full[s], 2 * (kStage + kSf));
        const uint32_t bar = map_rank(&full[s], 0);
        uint8_t* sb = sm + s * kStage + C::kA;
        if constexpr (GU)      // gate rows in the even CTA, up rows in the odd one
          w_load_2d_pair(sb, &p.b[rank], bar, kb * 128, n * kHalfN);
        else
          w_load_2d_pair(sb, &p.b[0], bar, kb * 128, n * TN + rank * kHalfN);
        w_load_2d_pair(sf + s * kSf + 512, &p.sfb, bar, 0, atom_b + C::kAtoms * kb);   // both CTAs need all N scales
      };
      // weights do not change: the first stages' are on their way while the kernel before finishes
      const int pre = i == first ? (p.nkb < kStages ? p.nkb : kStages) : 0;
      if (i == first) {
        for (int kb = 0; kb < pre; ++kb) load_b(kb, kb);
        griddep_wait();
      }
      for (int kb = 0; kb < p.nkb; ++kb, ++it) {
        const uint32_t s = it % kStages;
        if (it >= kStages && !warp_wait(&empty[s], ((it / kStages) - 1) & 1, p.err)) {
          ok = false;
          break;
        }
        if (kb >= pre) load_b(kb, s);
        const uint32_t bar = map_rank(&full[s], 0);
        w_load_2d_pair(sm + s * kStage, &p.a, bar, kb * 128, m0);
        w_load_2d_pair(sf + s * kSf, &p.sfa, bar, 0, atom_a + kb);
      }
    }
    // every stage has been read before the pair may leave; after a wait that
    // ran out, the copies in flight get a millisecond to land
    const uint32_t used = it < kStages ? it : kStages;
    for (uint32_t j = it - used; j < it && ok; ++j) ok = warp_wait(&empty[j % kStages], (j / kStages) & 1, p.err);
    if (!ok) let_copies_land();
  } else if (warp == 1) {
    named_arrive(kTmemBarrier, kThreads - 32);
    if (rank == 0) {
      const uint32_t tbase = tmem_base;
      const uint64_t a_desc = sdesc_sw128(smem_u32(sm)), b_desc = sdesc_sw128(smem_u32(sm) + C::kA);
      const uint64_t sf_desc = sdesc_noswz(smem_u32(sf), 16, 128);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int i = first; i < p.tiles && ok; i += pairs, ++n) {
        const uint32_t b = n & 1, use = n >> 1;
        if (use > 0 && !warp_wait(&acc_empty[b], (use - 1) & 1, p.err)) break;
        tc_fence_after();
        const uint32_t d = tbase + b * TN;
        for (int kb = 0; kb < p.nkb; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!warp_wait(&full[s], (it / kStages) & 1, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a_desc + s * (kStage >> 4), bd = b_desc + s * (kStage >> 4);
          const uint64_t sd = sf_desc + s * (kSf >> 4);
          const uint32_t sfa = tbase + C::kSfBase + s * C::kSfCols;
#pragma unroll
          for (int k = 0; k < 1 + C::kAtoms; ++k) w_copy_atom_pair(sfa + 4 * k, sd + 32 * k);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w_mma_mx_pair(d, ad + 2 * k, bd + 2 * k, idesc_mxf8f6f4(256, TN, 0, 0, k, k), sfa, sfa + 4,
                          (kb | k) != 0);
          w_commit_pair(&empty[s]);
        }
        if (ok) w_commit_pair(&acc_full[b]);
      }
    }
  } else {
    named_sync(kTmemBarrier, kThreads - 32);
    tc_fence_after();
    const uint32_t tbase = tmem_base;
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t remote_empty[2] = {map_rank(&acc_empty[0], 0), map_rank(&acc_empty[1], 0)};
    const GluCaps caps = {p.b1, p.b2, 1.0f / p.b1, 1.0f / p.b2};
    uint32_t cnt = 0;
    for (int i = first; i < p.tiles; i += pairs, ++cnt) {
      const uint32_t b = cnt & 1;
      const bool ok = mbar_wait_cluster(&acc_full[b], (cnt >> 1) & 1, p.err, kErrTimeout);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      int m, n;
      tile_of(p, i, m, n);
      const int row0 = m * 256 + 128 * rank + 32 * q, row = row0 + lane;
      const uint32_t acc = tbase + b * TN + (static_cast<uint32_t>(32 * q) << 16);
      if (row0 < p.M) {
        if constexpr (GU) {
          constexpr int kFirst = (kHalfN / 32 + 1) / 2 * 32;   // two of three 32-value blocks, or one of two
#pragma unroll 1
          for (int c = kFirst * half; c < (half ? kHalfN : kFirst); c += 32) {
            const int f = n * kHalfN + c;
            if (f >= p.N) break;
            uint32_t g[32], u[32];
            tmem_ld32(acc + c, g);
            tmem_ld32(acc + kHalfN + c, u);
            tmem_ld_wait();
            float h[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const F2 v = glu_hidden<ACT>(pair_at(g, j), pair_at(u, j), caps);
              h[2 * j] = v.x;
              h[2 * j + 1] = v.y;
            }
            if (row < p.M)
              store_hidden_block(h, static_cast<uint8_t*>(p.out) + static_cast<size_t>(row) * p.N + f,
                                 p.out_sf + atom_byte(row, f >> 5, p.out_nkb));
            __syncwarp();      // lanes part at the last rows; whole warps load
          }
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(row) * p.N + n * TN;
#pragma unroll 1
          for (int c = kHalfN * half; c < kHalfN * (half + 1); c += 32) {
            const int left = p.N - n * TN - c;
            if (left <= 0) break;
            uint32_t v[32], w[16];
            tmem_ld32(acc + c, v);
            tmem_ld_wait();
            pack32(v, w);
            if (row < p.M) store32(dst + c, w, left, p.wide);
            __syncwarp();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(b ? remote_empty[1] : remote_empty[0]);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
  cluster_sync();
}

// x's scales [T][K/32] -> atoms.  One thread per row and group of 4 blocks.
__global__ void mx_row_atoms_kernel(const uint8_t* __restrict__ s, int T, int kblks, int nkb,
                                    uint8_t* __restrict__ out) {
  griddep_launch();
  griddep_wait();
  const long long n = static_cast<long long>(T) * nkb;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int row = static_cast<int>(i / nkb), g = static_cast<int>(i - static_cast<long long>(row) * nkb);
    const uint8_t* src = s + static_cast<size_t>(row) * kblks + 4 * g;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (4 * g + k < kblks) w |= static_cast<uint32_t>(src[k]) << (8 * k);
    *reinterpret_cast<uint32_t*>(out + atom_byte(row, 4 * g, nkb)) = w;
  }
}

// Weight scales -> atoms [tile][nkb][width / 128 rounded up][512].  Tile row
// r < width: with `up`, gate row width/2 * tile + r, then the up rows of the
// same features; else row width * tile + r of the one matrix.  Rows past the
// end and blocks past kblks get zeros.
__global__ void mx_weight_atoms_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ up, int rows,
                                       int kblks, int nkb, int width, int tiles, uint8_t* __restrict__ out) {
  const int atoms = (width + 127) / 128, half = width / 2;
  const long long n = static_cast<long long>(tiles) * nkb * atoms * 128;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int r = static_cast<int>(i % (atoms * 128));
    const long long tk = i / (atoms * 128);
    const int g = static_cast<int>(tk % nkb), t = static_cast<int>(tk / nkb);
    const uint8_t* src = a;
    int row = t * width + r;
    if (up) {
      row = t * half + (r < half ? r : r - half);
      if (r >= half) src = up;
    }
    uint32_t w = 0;
    if (r < width && row < rows)
      for (int k = 0; k < 4; ++k)
        if (4 * g + k < kblks) w |= static_cast<uint32_t>(src[static_cast<size_t>(row) * kblks + 4 * g + k]) << (8 * k);
    *reinterpret_cast<uint32_t*>(out + (tk * atoms + (r >> 7)) * 512 + sf_atom_offset(r & 127, 0)) = w;
  }
}

template <bool GU, int ACT, int TN>
cudaError_t launch_tn(const FfnMxParams& p, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, ffn_mx_pair_kernel<GU, ACT, TN>, MxCfg<TN>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(ffn_mx_pair_kernel<GU, ACT, TN>, dim3(2 * p.tiles < ctas ? 2 * p.tiles : ctas),
                            dim3(kThreads), MxCfg<TN>::kSmem, 2, s, p);
}
template <bool GU, int ACT>
cudaError_t launch(const FfnMxParams& p, int tn, int ctas, cudaStream_t s) {
  return tn == 192 ? launch_tn<GU, ACT, 192>(p, ctas, s) : launch_tn<GU, ACT, 128>(p, ctas, s);
}

int ew_blocks(long long n) {
  const long long b = (n + 255) / 256;
  return static_cast<int>(b < 152 * 8 ? (b ? b : 1) : 152 * 8);
}

}  // namespace

cudaError_t launch_mx_row_atoms(const uint8_t* s, int T, int K, uint8_t* out, cudaStream_t stream) {
  const int nkb = (K + 127) / 128;
  return launch_pdl(mx_row_atoms_kernel, dim3(ew_blocks(static_cast<long long>(T) * nkb)), dim3(256), 0, stream, s, T,
                    K / 32, nkb, out);
}

cudaError_t launch_mx_weight_atoms(const uint8_t* a, const uint8_t* up, int rows, int K, int width, int tiles,
                                   uint8_t* out, cudaStream_t stream) {
  const int nkb = (K + 127) / 128;
  mx_weight_atoms_kernel<<<ew_blocks(256ll * tiles * nkb), 256, 0, stream>>>(a, up, rows, K / 32, nkb, width, tiles,
                                                                             out);
  return cudaGetLastError();
}

int ffn_mx_tiles(FfnMxParams& p, bool gate_up, int ctas) {
  const auto rounds = [&](int tn) {
    const int width = gate_up ? tn / 2 : tn;
    p.tiles_n = (p.N + width - 1) / width;
    p.tiles = (p.M + 255) / 256 * p.tiles_n;
    return (p.tiles + ctas / 2 - 1) / (ctas / 2);
  };
  // With all SMs busy a 128-row tile takes 0.76 of a 192-row one's time (4096
  // tokens at 7168 x 6144, short runs: 360 us against 307 us); where both leave pairs idle
  // the narrow ones win (300 tokens at 1152 x 864: 13.4 us against 15.8 us).
  const int narrow = rounds(128), wide = rounds(192);      // leaves the wide tiling in p
  if (wide <= 0.76f * narrow) return 192;
  rounds(128);
  return 128;
}

cudaError_t launch_ffn_mx_pair(const FfnMxParams& p, bool gate_up, int tn, int ctas, cudaStream_t s) {
  if (!gate_up) return launch<false, 0>(p, tn, ctas, s);
  return p.act == 1 ? launch<true, 1>(p, tn, ctas, s) : launch<true, 0>(p, tn, ctas, s);
}

}  // namespace lmoe
