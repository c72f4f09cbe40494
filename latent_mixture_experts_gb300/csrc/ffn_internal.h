// Interfaces between the feed-forward block's C ABI and its kernels, and of
// the norm kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace lmoe {

// ---------------------------------------------------------------- RMS norm
constexpr int kNormMaxWidth = 16384;
// Floats of `part` that launch_rms_norm_bwd needs.
size_t rms_norm_bwd_partials(int T, int d);
// r null: h = x is not written.  scale set: y is E4M3 codes with E8M0 scales.
// unsent: 0; 16 in the self-test, whose rows then never are complete.
cudaError_t launch_add_rms_norm(const void* x, long long ldx, const void* r, long long ldr, bool r_fp32, int T, int d,
                                const void* w, float eps, void* h, void* y, uint8_t* scale, int unsent,
                                cudaStream_t s);
cudaError_t launch_rms_norm_bwd(const void* dy, long long lddy, const void* h, long long ldh, const void* dh,
                                long long lddh, bool h_fp32, int T, int d, const void* w, float eps, void* dx,
                                float* part, float* dw, int unsent, cudaStream_t s);

// What the bf16 products of a block hand on is rounded to bf16, because a bf16 MMA
// takes bf16 operands: hid in the forward pass, dg, du and hid in the backward
// pass (the saved g and u as well).  One rounding each, of an fp32 value.
//
// ------------------------------------------------------ pair-tile bf16 GEMM
// C[M][N] (bf16) = A B^T on tiles of CTA pairs, 256 rows x 256 or 128 columns.
enum FfnMode {
  kFfnGateUp = 0,   // A = x, B = gate | up rows of half a tile's features; out0 = act(g, u), out1/out2 = g, u when set
  kFfnPlain = 1,    // A, B stored K contiguous; out0
  kFfnDHid = 2,     // B stored N contiguous; out0 = dg, out1 = du, out2 = hid from in_g, in_u
  kFfnGrads = 3     // up to four products, B stored N contiguous: with `cat` first dx, A stored K contiguous, K
                    // concatenated over (a[0], b[0]) and (a_cat, b_cat); then A[i]^T B[i], A stored M contiguous
};
constexpr int kPairProducts = 4;
struct FfnPairParams {
  CUtensorMap a[kPairProducts], b[kPairProducts], a_cat, b_cat;
  CUtensorMap b_half[2];      // K-contiguous b with boxes of half as many rows
  void* out[kPairProducts];
  const void *in_g, *in_u;
  int M[kPairProducts], N[kPairProducts];   // output rows and columns of each product
  int tiles_n[kPairProducts], tile_end[kPairProducts], nprod;
  int full;                   // tiles from here on are worked in halves of their columns
  int wide;                   // gate/up, dhid: output rows start on 32-byte boundaries
  int nkb;                    // 64-wide K blocks
  int cat, nkb_cat;           // kFfnGrads: the first product is dx, of 2 * nkb_cat K blocks
  // What the kernel in front lets this one, which starts once everything
  // before that kernel has finished: read b (split form), or do all of its work
  // (pair form) before that kernel has finished.
  int early;
  int n1, delta;              // its tiles, and how many of the others one of them counts for
  float b1, b2;
  int act;
  int* err;
};
// Chooses the tile width (128 or 256) for M, N, nprod and out and fills
// tiles_n, tile_end, full, n1, delta and wide; K-contiguous b maps have boxes
// of half of it, b_half (width 256) of a quarter.
int ffn_pair_tiles(FfnPairParams& p, FfnMode mode, int ctas);
int ffn_pair_grid(const FfnPairParams& p, int ctas);      // CTAs of its launch
cudaError_t launch_ffn_pair(FfnMode mode, const FfnPairParams& p, int tn, int ctas, cudaStream_t s);
// The split form, for one product of few tiles (K split over the pairs of a
// cluster; kFfnGrads: dx): fills tile_end, returns the splits, 1 where it does
// not take the shape; K-contiguous b maps have boxes of 64 rows.
struct FfnSplitLimits {
  int clusters2, clusters4;   // clusters that run at once, of two and of four pairs
};
cudaError_t ffn_split_limits(FfnSplitLimits* l);
int ffn_split_plan(FfnPairParams& p, FfnMode mode, const FfnSplitLimits& l);
cudaError_t launch_ffn_split(FfnMode mode, const FfnPairParams& p, int splits, cudaStream_t s);
// Largest number of CTAs (an even number) of the pair kernels that run at once.
cudaError_t ffn_pair_ctas(int* ctas);

// ------------------------------------------------------ small-batch passes
// out[t][f] over all tokens of a batch of at most kSkinnyMaxTokens.
constexpr int kSkinnyMaxTokens = 72;
constexpr int kSkinnyMaxStages = 16;
constexpr int kSkinnyMaxSplits = 8;    // K splits: the portable cluster size
// Two CTAs on an SM (one token at 7168 x 6144: 46.5 us; with 74 KB and three CTAs 48.6 us).
constexpr int kSkinnySmem = 110 * 1024;
struct FfnSkinnyParams {
  // whole (K a multiple of 64): a (64, T, K/64) and, down pass, b (64, features, K/64), boxes of tb / rows and kc
  // chunks; else, and gate (b) and up (b_up) always, (K, T) and (K, features), one box per 64-wide chunk
  CUtensorMap a, b, b_up;
  void *out, *save_g, *save_u;
  int T, M;            // tokens; features of the output
  int rows;            // features of a cluster
  int tb;              // token rows loaded: T rounded up to 8
  int chunks, kc;      // 64-wide K chunks; chunks of a stage
  int stages;
  int splits;          // CTAs of a cluster, over K
  int recv;            // where in shared memory the partial sums meet, behind the ring
  int whole;
  float b1, b2;
  int* err;
};
// Fills rows, splits, tb, kc and stages from T, M and chunks; false where the
// kernel does not take the shape.
bool ffn_skinny_plan(FfnSkinnyParams& p, bool gate_up);
cudaError_t launch_ffn_skinny(const FfnSkinnyParams& p, bool gate_up, int act, cudaStream_t s);

// ------------------------------------------------------------ MXFP8 passes
// Weight rows of a tile: half gate and half up rows, or output features.
constexpr int kMxTileN[2] = {192, 128};
struct FfnMxParams {
  CUtensorMap a, b[2];          // codes, boxes of 128 K values x 128 rows (a) or half a tile's (b)
  CUtensorMap sfa, sfb;         // scale atoms [row / 128][nkb], [tile][nkb][2 or 1] of 128 words; boxes of 1, 2 or 1
  void* out;                    // gate/up: hidden codes [M][N]; else bf16 [M][N]
  uint8_t* out_sf;              // gate/up: the hidden activation's atoms
  int out_nkb;
  int M, N;                     // tokens, output features
  int tiles_n, tiles, nkb;      // nkb: 128-wide K blocks
  int wide;                     // bf16 output rows start on 32-byte boundaries
  float b1, b2;
  int act;
  int* err;
};
// Chooses the tile width for M and N and fills tiles_n and tiles.
int ffn_mx_tiles(FfnMxParams& p, bool gate_up, int ctas);
cudaError_t launch_ffn_mx_pair(const FfnMxParams& p, bool gate_up, int tn, int ctas, cudaStream_t s);
// Scales [T][K/32] -> atoms; bytes of blocks past K/32 keep the zeros that the
// buffer is created with where a group of four is not begun.
cudaError_t launch_mx_row_atoms(const uint8_t* s, int T, int K, uint8_t* out, cudaStream_t stream);
// Weight scales [rows][K/32] (with `up`: gate and up) -> atoms of tiles of
// `width` (192 or 128) rows.
cudaError_t launch_mx_weight_atoms(const uint8_t* a, const uint8_t* up, int rows, int K, int width, int tiles,
                                   uint8_t* out, cudaStream_t stream);

// Small batches: K split over clusters, as in the bf16 form.
constexpr int kMxSkinnyN = kMxTileN[1];
struct FfnMxSkinnyParams {
  CUtensorMap a, b[2], sfb;     // codes: boxes of 128 K values x tb and 64 rows; the weights' atoms [tile][nkb]
  const uint8_t* row_sf;        // gate/up: x's scales [T][kblks]; else hid's atoms
  void* out;
  uint8_t* out_sf;              // gate/up: hid's atoms
  int T, M, nkb, kblks;         // tokens, output features, 128- and 32-wide K blocks
  int tiles, splits, stages, tb;
  int sfa_at, recv, reuse_ring; // where in shared memory the tokens' scales lie and the partial sums meet
  float b1, b2;
  int* err;
};
// Fills the tiling from T, M and nkb; false where the kernel does not take the shape.
bool ffn_mx_skinny_plan(FfnMxSkinnyParams& p, bool gate_up);
cudaError_t launch_ffn_mx_skinny(const FfnMxSkinnyParams& p, bool gate_up, int act, cudaStream_t s);

}  // namespace lmoe
