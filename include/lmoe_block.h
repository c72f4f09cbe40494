/*
 * lmoe_block — what a decoder block runs next to lmoe_ffn.h, in training and
 * in serving: the norms on both sides of a block with its gate and residual
 * scale, a matrix product with bias, activation and residual, each with its
 * backward pass, and the AdamW step over all weights.  One GB300 (sm_103a).
 * C ABI, conventions of lmoe_ffn.h: device pointers, row-major nn.Linear
 * [out][in] weights, raw bf16, stream-ordered asynchronous calls, argument
 * errors reported synchronously with nothing launched, no host
 * synchronisation unless stated.  Row strides ("ld...") are in elements;
 * outputs are packed.  Unless stated every pointer is 16-byte aligned, and
 * every width and stride is such that rows start on 16-byte boundaries (bf16:
 * multiples of 8).  MXFP8 tensors are those of lmoe_ffn.h.
 */
#ifndef LMOE_BLOCK_H
#define LMOE_BLOCK_H

#include "lmoe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------- norms on both sides of a block */
/* What a block's branch is multiplied by besides branch_scale. */
typedef enum {
  LMOE_GATE_NONE = 0,
  LMOE_GATE_CHANNEL = 1,   /* one row [d] for all tokens (a learned scale per channel) */
  LMOE_GATE_TOKEN = 2      /* [T][d] */
} lmoe_gate_type;

/* y: the block's output, bf16 [T][d]; stream [T][d] (`stream_type`): forward the
 * residual stream r, backward the stored h.  gate bf16; ldgate for TOKEN only.
 * w_post, w_next bf16 [d]: norms of the block's output and of what the next block
 * reads. */
typedef struct {
  int T, d;
  const void* y;
  int64_t ldy;
  const void* stream;
  int64_t lds;
  lmoe_stream_type stream_type;
  lmoe_gate_type gate_type;
  const void* gate;
  int64_t ldgate;
  const void* w_post;
  const void* w_next;
  float stream_scale, branch_scale;   /* a, s */
  float eps;                          /* of both norms */
} lmoe_gated_norm_args;

/* Per row of d values:
 *   n = w_post y / sqrt(mean(y^2) + eps)
 *   h = a r + s gate n            [T][d], packed, r's type: rounded once to that
 *                                 type, which is also the value that is normalised
 *   o = w_next h / sqrt(mean(h^2) + eps)    bf16 [T][d], or MXFP8 codes [T][d] with
 *                                 scales [T][d/32]
 * In place: h_out may be the stream (lds = d), o (bf16) may be y (ldy = d).
 * Errors: INVALID_ARG (NULL or misaligned pointer, T < 0, eps negative or not
 * finite, a scale not finite, strides < d, bad enum; MXFP8 without scales),
 * UNSUPPORTED (d not a multiple of 8 - of 32 for MXFP8 - or over 8192, a stride not
 * a multiple of 8), CUDA.  T = 0 is a no-op.  A bounded wait of the kernel that
 * runs out leaves NaN in the rows of h and o. */
LMOE_API lmoe_status lmoe_gated_add_norm(const lmoe_gated_norm_args* args, void* h_out, void* o,
                                         lmoe_norm_out out_format, uint8_t* o_scale, cudaStream_t stream);

/* Backward, `stream` of the arguments being h, from go bf16 [T][d] (gradient of o)
 * and gh_opt [T][d] (h's type; of h along the stream, or NULL):
 *   gH  = gh + rho2 (w_next go - h rho2^2 mean(w_next go h)),  rho2 = 1/sqrt(mean(h^2) + eps)
 *   dr  = a gH                                   [T][d], packed, h's type
 *   q   = s gate gH
 *   dy  = rho1 (w_post q - y rho1^2 mean(w_post q y)),         rho1 = 1/sqrt(mean(y^2) + eps)
 *                                                bf16 [T][d], packed
 *   dw_post = sum over rows of q y rho1,  dw_next = sum of go h rho2      fp32 [d]
 *   dgate: CHANNEL fp32 [d], the sum over rows of s n gH; TOKEN bf16 [T][d], packed,
 *          s n gH; NONE: not written, may be NULL
 * dr may be gh (ldgh = d), dy may be go (ldgo = d) or y (ldy = d).  The sums over
 * rows are added in an order that depends on T, d, the types and which of gate and gh
 * there are, in fp32, T / 152 of them one after the other.  T = 0 writes zero sums.  workspace: lmoe_gated_add_norm_backward_workspace bytes, contents
 * irrelevant.  A bounded wait that runs out leaves NaN in its rows and in the sums.
 * Errors as above. */
LMOE_API lmoe_status lmoe_gated_add_norm_backward_workspace(int T, int d, size_t* bytes);
LMOE_API lmoe_status lmoe_gated_add_norm_backward(const lmoe_gated_norm_args* args, const void* go_bf16, int64_t ldgo,
                                                  const void* gh_opt, int64_t ldgh, void* dy, void* dr,
                                                  float* dw_post, float* dw_next, void* dgate, void* workspace,
                                                  size_t workspace_bytes, cudaStream_t stream);

/* Self-test of the bounded waits (2 s each): the same calls, packed and bf16, with rows of
 * which 16 bytes are waited for that no copy brings, on x in place of every input
 * row; gate NONE.  Forward (backward == 0): out0 = h, out1 = o.  Backward: out0 =
 * dy, out1 = dr, dw (fp32 [2][d]) = dw_post, dw_next.  All of it is NaN. */
LMOE_API lmoe_status lmoe_gated_add_norm_selftest_timeout(int backward, const void* x_bf16, int T, int d,
                                                          const void* w_bf16, void* out0, void* out1, float* dw_opt,
                                                          void* workspace_opt, size_t workspace_bytes,
                                                          cudaStream_t stream);

/* ------------------- product with bias, activation and residual */
typedef enum {
  LMOE_LINEAR_NONE = 0,
  LMOE_LINEAR_RELU = 1,
  LMOE_LINEAR_SILU = 2,   /* z sigmoid(z) */
  LMOE_LINEAR_GELU = 3    /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
} lmoe_linear_act;

/*   z = x W^T + b,   y = act(z) + r
 * Products accumulate in fp32; z, act and the sum are fp32 and y is rounded once.
 * d_in and d_out multiples of 8; they and T at most 2^30. */
typedef struct {
  int d_in;
  int d_out;
  lmoe_linear_act act;
  int max_tokens;          /* largest T of any call */
  int training;            /* 1: allocate what lmoe_linear_backward needs */
} lmoe_linear_config;

typedef struct lmoe_linear_ctx* lmoe_linear_handle;

/* w bf16 [d_out][d_in], bias_opt bf16 [d_out] or NULL.  Borrowed: they stay valid
 * while the handle lives, are read anew by every call, and may be updated in place
 * between calls (in stream order).  Errors: INVALID_ARG (NULL, misaligned, sizes < 1,
 * bad enum), UNSUPPORTED (shapes above; not an sm_103 GPU), OOM, CUDA.  Synchronises
 * `stream`.  *out is NULL on error.  One handle is used by one stream at a time, and
 * belongs to the device that is current here: the calls below return INVALID_ARG
 * while another one is (destroy excepted). */
LMOE_API lmoe_status lmoe_linear_create(const lmoe_linear_config* cfg, const void* w_bf16, const void* bias_opt,
                                        cudaStream_t stream, lmoe_linear_handle* out);

/* x bf16 [T][d_in] (stride ldx) -> out [T][d_out], packed, in the residual's type
 * (`stream_type`), without a residual bf16.  residual_opt [T][d_out] (stride ldr).
 * pre_opt bf16 [T][d_out]: z for the backward pass.  out may be the residual
 * (ldr = d_out), and may not overlap x.  T = 0 is a no-op. */
LMOE_API lmoe_status lmoe_linear_forward(lmoe_linear_handle h, const void* x_bf16, int64_t ldx, int T,
                                         const void* residual_opt, int64_t ldr, lmoe_stream_type stream_type,
                                         void* out, void* pre_opt, cudaStream_t stream);

/* Gradients from x, dy [T][d_out] (stride lddy, `dy_type`; the residual's gradient is
 * dy itself) and, unless act is NONE, the stored z (bf16 [T][d_out]):
 *   dz = dy act'(z)
 *   dx = dz W bf16 [T][d_in],  dw = dz^T x bf16 [d_out][d_in],  dbias = sum of dz over
 *   rows, fp32 [d_out]
 * overwritten; any of the three may be NULL and is then not computed.  dz is rounded to
 * bf16 for the products, also where it is an fp32 dy itself (not for dbias).  The gradients may not overlap an input, the
 * weight or one another.  The same inputs and the same gradients asked for give the
 * same bits.  T = 0 writes zero dw and dbias. */
LMOE_API lmoe_status lmoe_linear_backward(lmoe_linear_handle h, const void* x_bf16, int64_t ldx, const void* dy,
                                          int64_t lddy, lmoe_stream_type dy_type, const void* pre_opt, int T,
                                          void* dx_opt, void* dw_opt, float* dbias_opt, cudaStream_t stream);

/* As lmoe_ffn_sync_status, lmoe_ffn_selftest_timeout (packed x, no residual),
 * lmoe_ffn_last_launch_count and lmoe_ffn_destroy. */
LMOE_API lmoe_status lmoe_linear_sync_status(lmoe_linear_handle h, cudaStream_t stream);
LMOE_API lmoe_status lmoe_linear_selftest_timeout(lmoe_linear_handle h, const void* x_bf16, int T, void* out_bf16,
                                                  cudaStream_t stream);
LMOE_API int lmoe_linear_last_launch_count(lmoe_linear_handle h);
LMOE_API lmoe_status lmoe_linear_destroy(lmoe_linear_handle h);

/* ------------------------------------------------------- AdamW step */
/*   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g,    v = beta2 v + (1 - beta2) g^2
 *   w = w (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * for every value of every tensor, in fp32 (the root of a v below 2^-126 is zero; the
 * root and the division are the card's approximations, each within 2^-22 of its value).
 * What w changes by, the decay and the step together, is summed first and added to w
 * once.  t: the number of the step, kept on the device.  What is stored in fewer bits
 * after that:
 *   - a bf16 weight with an fp32 master: the master's value rounded to nearest;
 *   - a bf16 weight without one: rounded stochastically, so that updates far smaller
 *     than a step of the weight still arrive in the mean (down to fp32's last bit of it);
 *   - MXFP8 states: m, and sqrt(v) in place of v (half the range of exponents), rounded
 *     stochastically: rounded to nearest they would never decay (a factor of 0.999 is
 *     less than half a step).  A root that is not zero is not rounded to zero: m is
 *     divided by it.  A block with an infinity or NaN becomes NaN (scale 255).
 * Stochastic rounding adds the top of a random word to what is cut off, and cuts.  The
 * word of value i in step t is mix(i ^ mix(mix(seed) + t)), of 32 bits (from the 2^32-th
 * value on with mix(key + (i >> 32)) in place of key = mix(mix(seed) + t)), i counting
 * from the tensor's `first`:
 *   mix(x): x ^= x >> 16; x *= 0x9E9F34A5; x ^= x >> 15; x *= 0xBB3A919B; x ^= x >> 16
 * (odd multipliers taken for this function, from no published one: a change of any bit of
 * x changes each bit of the word for half of the x, within 0.002 of a million of them).
 * Weights use its bits 8..23 (below bf16's), m bits 12..31, sqrt(v) bits 0..19 (the 20
 * bits below an E4M3 step). */
typedef enum { LMOE_ADAMW_FP32 = 0, LMOE_ADAMW_MXFP8 = 1 } lmoe_adamw_states;

typedef struct {
  void* param;             /* bf16, or fp32 with param_fp32 */
  int param_fp32;
  float* master;           /* fp32 [n] of a bf16 weight, or NULL */
  void* m;                 /* fp32 [n], or codes [n] */
  void* v;                 /* fp32 [n], or codes of sqrt(v) [n] */
  uint8_t* m_scale;        /* MXFP8: [ceil(n / 32)], any alignment */
  uint8_t* v_scale;
  int64_t n;
  uint64_t first;          /* number of its first value, a multiple of 32 */
  float weight_decay;
} lmoe_adamw_tensor;

typedef struct {
  double beta1, beta2, eps;
  lmoe_adamw_states states;
  uint32_t seed;
  int64_t* step;           /* on the device: steps done so far; 8-byte aligned.  A step counts it up. */
} lmoe_adamw_config;

typedef struct lmoe_adamw_ctx* lmoe_adamw_handle;

/* tensors [count] is copied; what it points to is borrowed.  Zero states are all bytes
 * zero.  Errors: INVALID_ARG (NULL or misaligned pointer, count < 1, n < 0, beta outside
 * [0, 1), eps or weight_decay negative or not finite, `first` not a multiple of 32, a
 * master of an fp32 weight, bad enum), UNSUPPORTED (over 2^40 values, not an sm_103 GPU),
 * OOM, CUDA.  Synchronises `stream`.  *out is NULL on error.  One handle is used by one
 * stream at a time, and belongs to the device that is current here. */
LMOE_API lmoe_status lmoe_adamw_create(const lmoe_adamw_config* cfg, const lmoe_adamw_tensor* tensors, int count,
                                       cudaStream_t stream, lmoe_adamw_handle* out);

/* One step.  grads [count], an array on the host (read before the call returns): device
 * pointers, packed; bf16, or fp32 where grad_fp32_opt[i] != 0 (NULL: all bf16).  A
 * tensor whose gradient is NULL is left as it is.  lr_opt, grad_scale_opt: one fp32 value
 * each on the device, read by the step; without lr_opt `lr` is used, without
 * grad_scale_opt 1.  A step may be captured into a graph: each replay is a step.
 * Errors: INVALID_ARG (as above; lr not finite or negative), CUDA. */
LMOE_API lmoe_status lmoe_adamw_step(lmoe_adamw_handle h, const void* const* grads, const uint8_t* grad_fp32_opt,
                                     float lr, const float* lr_opt, const float* grad_scale_opt,
                                     cudaStream_t stream);

/* Kernels the last call on this handle launched. */
LMOE_API int lmoe_adamw_last_launch_count(lmoe_adamw_handle h);
/* Synchronises the device and releases the handle.  NULL is accepted. */
LMOE_API lmoe_status lmoe_adamw_destroy(lmoe_adamw_handle h);

#ifdef __cplusplus
}
#endif
#endif /* LMOE_BLOCK_H */
