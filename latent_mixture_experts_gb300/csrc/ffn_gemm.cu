// The products of the dense feed-forward block on large batches: bf16, fp32
// accumulation in tensor memory, one 256 x 256 output tile per pair of CTAs
// (256 x 128 where those leave pairs idle, for the whole grid or its last wave:
// half the products and half the epilogue of a tile, but half as much again to
// load for each product).
//
// A pair shares one tcgen05.mma (cta_group::2, M = 256, N = 256): each CTA
// stages 128 rows of A and 128 of B, so a 64-wide K block costs 32 KB of
// shared memory per CTA for 256 x 256 x 64 products - two thirds of the
// bytes per product of a single CTA's 128 x 256 tile, which the
// shared-memory fill would bound.  The ring holds six such blocks; two
// 256-column accumulators fill tensor memory, so the epilogue of one tile
// runs under the products of the next.  Grid: one CTA per SM, tiles handed
// out statically, eight tile rows at a time so that concurrent tiles share
// their operands in L2.
//
// Operands reach shared memory by TMA in the order they have in memory: rows
// along K ("K contiguous") or, for the backward products, along M or N,
// which the MMA descriptors express, so nothing is transposed or copied.
//
// Warps: 0 = TMA, 1 = MMA (even CTA), 2..9 = epilogue (TMEM lane quarter
// warp % 4; the first four take the left half of the columns, the others the
// right half).
#include "ffn_act.cuh"
#include "ffn_internal.h"
#include "lmoe_internal.h"
#include "issue.cuh"
#include "linear_act.cuh"

namespace lmoe {
namespace {

constexpr int kEpiPairWarps = 8;             // two for each TMEM lane quarter
constexpr int kRowsBuf = 4096;               // each one's for turning its rows: 32 rows x 64 bf16
// TN: columns of a tile.
template <int TN>
struct PairCfg {
  static constexpr int kA = 16384;           // 128 rows x 64 bf16
  static constexpr int kB = TN / 2 * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = TN == 256 ? 6 : 8;
  static constexpr int kSmem = kStages * kStage + kEpiPairWarps * kRowsBuf + 1024;
};
constexpr int kPairThreads = 64 + 32 * kEpiPairWarps;
constexpr int kTmemBarrier = 1;              // tmem_base is there for the epilogue warps
// Tile rows of one raster group (4096 tokens at 7168 x 6144, backward, in short
// runs, before the power limit sets in: 1155 us; with 4 rows 1175 us, with 16 rows
// 1176 us.  In long ones 1325 us).
constexpr int kTileRows = 8;

// narrow: half a wide tile, at the end of the wide grid; n counts half tiles.
struct Tile {
  int prod, m, n;
  bool narrow;
};
// The tiles of a pair, round by round: item `round` of pair `pair` of `pairs`, -1
// for none in this round, -2 at the end.  Tiles are dealt out in turn, except
// that a dx tile counts for `delta` of the weight gradients' (their K ranges
// differ): the pairs that get one more dx tile sit out delta - 1 rounds.
__device__ __forceinline__ int item_of(const FfnPairParams& p, int total, int round, int pair, int pairs) {
  const int k1 = p.n1 / pairs, r = p.n1 - k1 * pairs;
  if (round < k1) return round * pairs + pair;
  round -= k1;
  int i;
  if (r == 0) {
    i = round * pairs + pair;
  } else if (round < p.delta) {
    if (pair < r) return round == 0 ? k1 * pairs + pair : -1;
    i = round * (pairs - r) + pair - r;
  } else {
    i = p.delta * (pairs - r) + (round - p.delta) * pairs + pair;
  }
  i += p.n1;
  return i < total ? i : -2;
}

__device__ __forceinline__ Tile tile_of(const FfnPairParams& p, int i) {
  Tile t;
  t.narrow = i >= p.full;
  const int sub = t.narrow ? (i - p.full) & 1 : 0;
  if (t.narrow) i = p.full + ((i - p.full) >> 1);
  t.prod = 0;
  while (t.prod + 1 < p.nprod && i >= p.tile_end[t.prod]) ++t.prod;
  const int first = t.prod ? p.tile_end[t.prod - 1] : 0;
  const int tn = p.tiles_n[t.prod], tm = (p.tile_end[t.prod] - first) / tn;
  i -= first;
  const int g = i / (kTileRows * tn), r = i - g * kTileRows * tn;
  const int rows = min(kTileRows, tm - g * kTileRows);
  t.m = g * kTileRows + r % rows;
  t.n = r / rows;
  if (t.narrow) t.n = 2 * t.n + sub;
  return t;
}

// 32 columns of this thread's row, zeros past `left`.
__device__ __forceinline__ void load32(const __nv_bfloat16* src, uint32_t (&w)[16], int left) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    uint4 a = make_uint4(0, 0, 0, 0);
    if (left >= 2 * i + 8) a = *reinterpret_cast<const uint4*>(src + 2 * i);
    w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
  }
}
// The warp's 32 rows of half a tile's columns, from the CTA's TN-column
// accumulator at `acc`.  N is a multiple of 8, so a row ends on a 16-byte
// boundary.  `ready`: waits for the accumulator; what the epilogue reads from
// memory is requested before, and then one step ahead.
template <int MODE, int ACT, int TN, class Ready>
__device__ __forceinline__ bool epilogue_rows(const FfnPairParams& p, const Tile& t, uint32_t acc, int row0, int half,
                                              uint8_t* buf, Ready ready) {
  const GluCaps caps = {p.b1, p.b2, 1.0f / p.b1, 1.0f / p.b2};
  const int row = threadIdx.x & 31, rows = p.M[t.prod] - row0;
  const bool row_ok = row < rows;
  const auto out = [&](int i, size_t at) { return static_cast<__nv_bfloat16*>(p.out[i]) + at; };
  if constexpr (MODE == kFfnGateUp) {
    constexpr int kF = TN / 2;      // features of a tile
    const int n0 = t.n * kF, N = p.N[0];
    const size_t at = static_cast<size_t>(row0 + row) * N + n0;
    if (!ready()) return false;
#pragma unroll 1
    for (int c = kF / 2 * half; c < kF / 2 * (half + 1); c += 32) {
      const int left = N - n0 - c;
      if (left <= 0) break;
      uint32_t g[32], u[32], w[16];
      tmem_ld32(acc + c, g);
      tmem_ld32(acc + kF + c, u);
      tmem_ld_wait();
      if (p.out[1] && row_ok) {
        pack32(g, w);
        store32(out(1, at + c), w, left, p.wide);
        pack32(u, w);
        store32(out(2, at + c), w, left, p.wide);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack_bf16(glu_hidden<ACT>(pair_at(g, j), pair_at(u, j), caps));
      if (row_ok) store32(out(0, at + c), w, left, p.wide);
      __syncwarp();      // lanes part at the last rows; whole warps load
    }
  } else {
    const int n0 = t.n * TN, N = p.N[t.prod], c0 = TN / 2 * half;
    if constexpr (MODE == kFfnDHid) {
      const size_t at = static_cast<size_t>(row0 + row) * N + n0;
      const __nv_bfloat16* gp = static_cast<const __nv_bfloat16*>(p.in_g) + at;
      const __nv_bfloat16* up = static_cast<const __nv_bfloat16*>(p.in_u) + at;
      uint32_t g[16], u[16], v[32];
      load32(gp + c0, g, row_ok ? N - n0 - c0 : 0);
      load32(up + c0, u, row_ok ? N - n0 - c0 : 0);
      if (!ready()) return false;
#pragma unroll 1
      for (int c = c0; c < c0 + TN / 2; c += 32) {
        const int left = N - n0 - c;
        if (left <= 0) break;
        tmem_ld32(acc + c, v);
        uint32_t g1[16], u1[16];
        const int next = row_ok && c + 32 < c0 + TN / 2 ? left - 32 : 0;
        load32(gp + c + 32, g1, next);
        load32(up + c + 32, u1, next);
        __syncwarp();      // lanes part at the last rows; whole warps load and wait
        tmem_ld_wait();
        uint32_t h[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const GluGrad x = glu_grad<ACT>(bf16_both(g[j]), bf16_both(u[j]), pair_at(v, j), caps);
          g[j] = pack_bf16(x.dg);
          u[j] = pack_bf16(x.du);
          h[j] = pack_bf16(x.hid);
        }
        if (row_ok) {
          store32(out(0, at + c), g, left, p.wide);
          store32(out(1, at + c), u, left, p.wide);
          store32(out(2, at + c), h, left, p.wide);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          g[j] = g1[j];
          u[j] = u1[j];
        }
        __syncwarp();
      }
    } else if constexpr (MODE == kFfnLinear) {
      const size_t at = static_cast<size_t>(row0) * N + n0;
      // Each lane keeps the bias of four of the warp's columns, there before the products are;
      // loads of all of them by every lane, behind the products, took 0.7 us of every 64 columns.
      uint2 bias = make_uint2(0, 0);
      if (p.lin.bias && 4 * row < TN / 2 && n0 + c0 + 4 * row < N)
        bias = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.lin.bias) + n0 + c0 + 4 * row);
      const auto add_bias = [&](uint32_t (&v)[32], int c) {
        if (!p.lin.bias) return;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t b = __shfl_sync(0xFFFFFFFFu, j % 2 ? bias.y : bias.x, (c - c0) / 4 + j / 2);
          set_pair(v, j, vadd(pair_at(v, j), bf16_both(b)));
        }
      };
      const auto activate = [&](uint32_t (&v)[32]) {
        with_act(p.lin.act, [&](auto A) {
#pragma unroll
          for (int j = 0; j < 16; ++j) set_pair(v, j, linear_act<A.value>(pair_at(v, j)));
        });
      };
      if (p.lin.fp32) {
        // 32 columns at a time are turned in shared memory, so that eight lanes read a row's
        // residuals and write its sums side by side (with each lane on a row of its own 1000
        // tokens at 3584 x 3584 took 39.1 us, so 26.7 us).
        const int sub = threadIdx.x >> 3 & 3, ch = threadIdx.x & 7;
        float4 r[8];
        const auto fetch = [&](int c) {
          const int left = c < c0 + TN / 2 ? N - n0 - c : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * i + sub < rows && 4 * ch < left)
              r[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.lin.res) +
                                                      static_cast<size_t>(row0 + 4 * i + sub) * p.lin.ldr + n0 + c +
                                                      4 * ch);
          }
        };
        fetch(c0);
        if (!ready()) return false;
#pragma unroll 1
        for (int c = c0; c < c0 + TN / 2; c += 32) {
          const int left = N - n0 - c;
          if (left <= 0) break;
          uint32_t v[32];
          tmem_ld32(acc + c, v);
          tmem_ld_wait();
          add_bias(v, c);
          if (p.out[1] && row_ok) {
            uint32_t w[16];
            pack32(v, w);
            store32(out(1, at + c + static_cast<size_t>(row) * N), w, left, p.wide);
          }
          activate(v);
          turn_rows(buf, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (4 * i + sub >= rows || 4 * ch >= left) continue;
            const float4 x = turned(buf, 4 * i + sub, ch);
            *reinterpret_cast<float4*>(static_cast<float*>(p.out[0]) + at + static_cast<size_t>(4 * i + sub) * N + c +
                                       4 * ch) = make_float4(x.x + r[i].x, x.y + r[i].y, x.z + r[i].z, x.w + r[i].w);
          }
          fetch(c + 32);
          __syncwarp();
        }
        return true;
      }
      // bf16 residuals come in as the sums leave, 64 columns at a time by way of `buf`,
      // requested one step ahead (the same tokens 23.3 us, without a residual 21.6 us).
      uint4 r[8];
      const auto fetch = [&](int c) {
        if (p.lin.res)
          load_rows(r, static_cast<const __nv_bfloat16*>(p.lin.res) + static_cast<size_t>(row0) * p.lin.ldr + n0 + c,
                    p.lin.ldr, rows, c < c0 + TN / 2 ? N - n0 - c : 0);
      };
      fetch(c0);
      if (!ready()) return false;
#pragma unroll 1
      for (int c = c0; c < c0 + TN / 2; c += 64) {
        const int left = N - n0 - c;
        if (left <= 0) break;
        uint32_t v[2][32], w[32];
        tmem_ld32(acc + c, v[0]);
        tmem_ld32(acc + c + 32, v[1]);
        tmem_ld_wait();
        add_bias(v[0], c);
        add_bias(v[1], c + 32);
        if (p.out[1]) {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = pack_bf16(pair_at(v[j / 16], j % 16));
          store_rows(buf, w, out(1, at + c), N, rows, left);
        }
        activate(v[0]);
        activate(v[1]);
        if (p.lin.res) {
          rows_in(buf, r);
          fetch(c + 64);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 x = own_row(buf, j);
            const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = 4 * j + k;
              w[i] = pack_bf16(vadd(pair_at(v[i / 16], i % 16), bf16_both(q[k])));
            }
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = pack_bf16(pair_at(v[j / 16], j % 16));
        }
        store_rows(buf, w, out(0, at + c), N, rows, left);
      }
    } else {
      const size_t at = static_cast<size_t>(row0) * N + n0;
      if (!ready()) return false;
#pragma unroll 1
      for (int c = c0; c < c0 + TN / 2; c += 64) {
        const int left = N - n0 - c;
        if (left <= 0) break;
        uint32_t v[2][32], w[32];
        tmem_ld32(acc + c, v[0]);
        tmem_ld32(acc + c + 32, v[1]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = pack_bf16(pair_at(v[j / 16], j % 16));
        store_rows(buf, w, out(t.prod, at + c), N, rows, left);
      }
    }
  }
  return true;
}

template <int MODE, int ACT, int TN>
__global__ void __launch_bounds__(kPairThreads, 1) ffn_pair_kernel(const __grid_constant__ FfnPairParams p) {
  constexpr bool kBMn = MODE == kFfnDHid || MODE == kFfnGrads;
  using C = PairCfg<TN>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiPairWarps);      // the epilogue warps of both CTAs
    }
    fence_mbar_init();
  }
  __syncwarp();
  cluster_sync();
  if (warp == 1) {      // under the first loads
    tmem_alloc_pair(&tmem_base, 2 * TN);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (!p.early) {
    griddep_launch();
    griddep_wait();
  }
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
  const int total = 2 * p.tile_end[p.nprod - 1] - p.full;   // wide tiles, then halves

  if (warp == 0) {
    uint32_t it = 0;
    bool ok = true;
    for (int round = 0; ok; ++round) {
      const int i = item_of(p, total, round, first, pairs);
      if (i == -1) continue;
      if (i < 0) break;
      const Tile t = tile_of(p, i);
      const int m0 = t.m * 256 + 128 * static_cast<int>(rank);
      const bool dx = MODE == kFfnGrads && p.cat && t.prod == 0, a_mn = MODE == kFfnGrads && !dx;
      const int nkb = dx ? p.nkb_dx : p.nkb;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t s = it % kStages;
        if (it >= kStages && !warp_wait(&empty[s], ((it / kStages) - 1) & 1, p.err)) {
          ok = false;
          break;
        }
        const bool half = TN == 256 && t.narrow;
        if (rank == 0) w_arrive_expect_tx(&full[s], 2 * (half ? C::kA + C::kB / 2 : C::kStage));
        const uint32_t bar = map_rank(&full[s], 0);
        uint8_t* sa = sm + s * C::kStage;
        uint8_t* sb = sa + C::kA;
        const bool second = dx && kb >= p.nkb_cat;      // the concatenation's second half
        const int k0 = (second ? kb - p.nkb_cat : kb) * 64;
        const CUtensorMap* A = second ? &p.a_cat : &p.a[t.prod];
        const CUtensorMap* Bm = second ? &p.b_cat : &p.b[t.prod];
        if (a_mn) {
          w_load_2d_pair(sa, A, bar, m0, k0);
          w_load_2d_pair(sa + 8192, A, bar, m0 + 64, k0);
        } else {
          w_load_2d_pair(sa, A, bar, k0, m0);
        }
        if constexpr (MODE == kFfnGateUp) {   // gate rows in the even CTA, up rows in the odd one
          if (half)
            w_load_2d_pair(sb, &p.b_half[rank], bar, k0, t.n * (TN / 4));
          else
            w_load_2d_pair(sb, &p.b[rank], bar, k0, t.n * (TN / 2));
        } else if constexpr (kBMn) {
          const int width = half ? TN / 2 : TN, n0 = t.n * width + width / 2 * static_cast<int>(rank);
          w_load_2d_pair(sb, Bm, bar, n0, k0);
          if (TN == 256 && !half) w_load_2d_pair(sb + 8192, Bm, bar, n0 + 64, k0);
        } else {
          if (half)
            w_load_2d_pair(sb, &p.b_half[0], bar, k0, t.n * (TN / 2) + TN / 4 * static_cast<int>(rank));
          else
            w_load_2d_pair(sb, Bm, bar, k0, t.n * TN + TN / 2 * static_cast<int>(rank));
        }
      }
    }
    // Every stage has been read by the MMAs (and so every copy has landed)
    // before the pair may leave; if a wait ran out, the copies in flight get a
    // millisecond to land.
    const uint32_t used = it < kStages ? it : kStages;
    for (uint32_t j = it - used; j < it && ok; ++j) ok = warp_wait(&empty[j % kStages], (j / kStages) & 1, p.err);
    if (!ok) let_copies_land();
  } else if (warp == 1) {
    named_arrive(kTmemBarrier, kPairThreads - 32);
    if (rank == 0) {
      const uint32_t tbase = tmem_base;
      const uint32_t base = smem_u32(sm);
      const uint64_t b_desc = kBMn ? sdesc_sw128_mn(base + C::kA, 8192) : sdesc_sw128(base + C::kA);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int round = 0; ok; ++round) {
        const int i = item_of(p, total, round, first, pairs);
        if (i == -1) continue;
        if (i < 0) break;
        const uint32_t b = n & 1, use = n >> 1;
        ++n;
        if (use > 0 && !warp_wait(&acc_empty[b], (use - 1) & 1, p.err)) break;
        tc_fence_after();
        const uint32_t d = tbase + b * TN;
        const bool dx = MODE == kFfnGrads && p.cat && tile_of(p, i).prod == 0, a_mn = MODE == kFfnGrads && !dx;
        const int nkb = dx ? p.nkb_dx : p.nkb;
        const uint32_t idesc = idesc_bf16(256, TN == 256 && i >= p.full ? TN / 2 : TN) | (a_mn ? kIdescAMajorMn : 0u) |
                               (kBMn ? kIdescBMajorMn : 0u);
        // descriptors count 16-byte units: a step of 16 along K is 32 bytes of a
        // K-contiguous row, or 16 rows of 128 bytes
        const uint64_t a_desc = a_mn ? sdesc_sw128_mn(base, 8192) : sdesc_sw128(base);
        const uint32_t a_step = a_mn ? 128 : 2;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!warp_wait(&full[s], (it / kStages) & 1, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a_desc + s * (C::kStage >> 4), bd = b_desc + s * (C::kStage >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w_mma_bf16_pair(d, ad + k * a_step, bd + k * (kBMn ? 128 : 2), idesc, (kb | k) != 0);
          w_commit_pair(&empty[s]);
        }
        if (ok) w_commit_pair(&acc_full[b]);
      }
    }
  } else {
    named_sync(kTmemBarrier, kPairThreads - 32);
    tc_fence_after();
    const uint32_t tbase = tmem_base;
    const int q = warp & 3;
    uint8_t* buf = sm + kStages * C::kStage + (warp - 2) * kRowsBuf;
    const uint32_t remote_empty[2] = {map_rank(&acc_empty[0], 0), map_rank(&acc_empty[1], 0)};
    uint32_t n = 0;
    for (int round = 0;; ++round) {
      const int i = item_of(p, total, round, first, pairs);
      if (i == -1) continue;
      if (i < 0) break;
      const uint32_t b = n & 1, use = n >> 1;
      ++n;
      const auto ready = [&] {
        const bool ok = mbar_wait_cluster(&acc_full[b], use & 1, p.err, kErrTimeout);
        tc_fence_after();
        return __all_sync(0xFFFFFFFFu, ok) != 0;
      };
      const Tile t = tile_of(p, i);
      const int row0 = t.m * 256 + 128 * static_cast<int>(rank) + 32 * q;
      const uint32_t acc = tbase + b * TN + (static_cast<uint32_t>(32 * q) << 16);
      const int half = (warp - 2) >> 2;
      bool ok;
      if (row0 >= p.M[t.prod])
        ok = ready();
      else if (TN == 256 && t.narrow)
        ok = epilogue_rows<MODE, ACT, 128>(p, t, acc, row0, half, buf, ready);
      else
        ok = epilogue_rows<MODE, ACT, TN>(p, t, acc, row0, half, buf, ready);
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(b ? remote_empty[1] : remote_empty[0]);
    }
  }
  if (p.early) {      // what follows this kernel follows the one in front too
    griddep_wait();
    griddep_launch();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 2 * TN);
  cluster_sync();      // neither CTA leaves while the other still frees the pair's columns
}

template <int MODE, int ACT, int TN>
cudaError_t launch_tn(const FfnPairParams& p, int ctas, cudaStream_t s) {
  using C = PairCfg<TN>;
  static std::atomic<uint64_t> limit;
  const cudaError_t e = allow_smem(limit, ffn_pair_kernel<MODE, ACT, TN>, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(ffn_pair_kernel<MODE, ACT, TN>, dim3(ffn_pair_grid(p, ctas)), dim3(kPairThreads), C::kSmem,
                            2, s, p);
}
template <int MODE, int ACT>
cudaError_t launch(const FfnPairParams& p, int tn, int ctas, cudaStream_t s) {
  return tn == 256 ? launch_tn<MODE, ACT, 256>(p, ctas, s) : launch_tn<MODE, ACT, 128>(p, ctas, s);
}

}  // namespace

int ffn_pair_tiles(FfnPairParams& p, FfnMode mode, int ctas) {
  const auto tiles = [&](int tn) {
    int n = 0;
    const int width = mode == kFfnGateUp ? tn / 2 : tn;
    for (int i = 0; i < p.nprod; ++i) {
      p.tiles_n[i] = (p.N[i] + width - 1) / width;
      n += (p.M[i] + 255) / 256 * p.tiles_n[i];
      p.tile_end[i] = n;
    }
    return n;
  };
  // activations: 1 where every output row starts on a 32-byte boundary
  p.wide = p.N[0] % 16 == 0;
  for (int i = 0; i < 3; ++i) p.wide = p.wide && reinterpret_cast<uintptr_t>(p.out[i]) % 32 == 0;
  // With all SMs busy a narrow tile takes 0.55 to 0.58 of a wide one's time
  // (4096 tokens at 7168 x 6144, short runs: forward 601 us against 546 us), of the
  // gradients' 0.67 (backward 1500 us against 1155 us); 1003 tokens at 1152 x 864,
  // which leave half of the wide grid idle: forward 16.8 us against 22.8 us.  A last
  // round of wide tiles that fills at most half of the pairs is cut into halves.
  // Tiles cost their K blocks, and eight of them at least: 256 tokens at 5120 x
  // 3584, backward, 64.4 us; with 14 at least 72.0 us.
  const float ratio = mode == kFfnGrads ? 0.67f : 0.57f;
  const auto cost = [](int nkb) { return static_cast<float>(nkb < 6 ? 8 : nkb + 2); };
  const int pairs = ctas / 2;
  const float c2 = cost(p.nkb), c1 = p.cat ? cost(p.nkb_dx) : c2;
  p.delta = c1 > c2 ? static_cast<int>(c1 / c2 + 0.5f) : 1;
  int rest = 0, cut = 0;
  const auto rounds = [&](int tn) {          // of a pair, in c2; rest: the tiles of the last one
    const int all = tiles(tn);
    p.n1 = p.cat ? p.tile_end[0] : 0;
    const int k1 = p.n1 / pairs, r = p.n1 % pairs, slots = all - p.n1 + r * p.delta, n = slots / pairs;
    rest = slots % pairs;
    cut = tn == 256 && rest > 0 && 2 * rest <= pairs && rest <= all - p.n1 && n >= (r > 0 ? p.delta : k1 > 0 ? 0 : 1);
    const float others = n + (rest == 0 ? 0.0f : cut ? ratio : 1.0f), dx = r > 0 ? c1 / c2 : 0.0f;
    return k1 * c1 / c2 + (others > dx ? others : dx);
  };
  const float narrow = ratio * rounds(128), wide = rounds(256);   // leaves the wide tiling in p
  if (narrow < wide) {
    rounds(128);
    p.full = p.tile_end[p.nprod - 1];
    return 128;
  }
  p.full = p.tile_end[p.nprod - 1] - (cut ? rest : 0);
  return 256;
}

int ffn_pair_grid(const FfnPairParams& p, int ctas) {
  const int tiles = 2 * p.tile_end[p.nprod - 1] - p.full;
  return 2 * tiles < ctas ? 2 * tiles : ctas;
}

cudaError_t launch_ffn_pair(FfnMode mode, const FfnPairParams& p, int tn, int ctas, cudaStream_t s) {
  const bool sw = p.act == 1;
  switch (mode) {
    case kFfnGateUp: return sw ? launch<kFfnGateUp, 1>(p, tn, ctas, s) : launch<kFfnGateUp, 0>(p, tn, ctas, s);
    case kFfnPlain: return launch<kFfnPlain, 0>(p, tn, ctas, s);
    case kFfnLinear: return launch<kFfnLinear, 0>(p, tn, ctas, s);
    case kFfnDHid: return sw ? launch<kFfnDHid, 1>(p, tn, ctas, s) : launch<kFfnDHid, 0>(p, tn, ctas, s);
    case kFfnGrads: return launch<kFfnGrads, 0>(p, tn, ctas, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t ffn_pair_ctas(int* ctas) {
  cudaError_t e = cudaFuncSetAttribute(ffn_pair_kernel<kFfnPlain, 0, 256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PairCfg<256>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = PairCfg<256>::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, ffn_pair_kernel<kFfnPlain, 0, 256>, &cfg);
  if (e != cudaSuccess) return e;
  *ctas = 2 * (n > 0 ? n : 1);
  return cudaSuccess;
}

}  // namespace lmoe
