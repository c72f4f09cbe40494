/*
 * lmoe_ffn — what a decoder needs around the MoE layer of lmoe.h: the
 * residual addition with RMS normalisation that makes a feed-forward layer's
 * input, and the dense gated feed-forward block (a model's non-expert layers,
 * or the shared MLP by itself), each with its backward pass; and both in
 * MXFP8 for serving.  One GB300 (sm_103a).  C ABI, conventions of lmoe.h:
 * device pointers, row-major nn.Linear [out][in] weights, raw bf16,
 * stream-ordered asynchronous calls, argument errors reported synchronously
 * with nothing launched, no host synchronisation unless stated.
 *
 * Row strides ("ld...") are in elements; outputs are packed.  Unless stated
 * every pointer is 16-byte aligned and every width and stride is such that
 * rows start on 16-byte boundaries (bf16: multiples of 8).
 *
 * MXFP8 tensors (OCP microscaling): E4M3 codes uint8 [rows][K] and one E8M0
 * scale byte per 32 consecutive values, uint8 [rows][K/32]; a value is
 * code * 2^(scale - 127).  Encoding takes the smallest power of two that
 * keeps the block's largest magnitude within 448, rounding codes to nearest
 * even; a block with an infinity or NaN gets scale 255 (NaN).
 */
#ifndef LMOE_FFN_H
#define LMOE_FFN_H

#include "lmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------- RMS norm */
typedef enum { LMOE_NORM_OUT_BF16 = 0, LMOE_NORM_OUT_MXFP8 = 1 } lmoe_norm_out;
typedef enum { LMOE_STREAM_BF16 = 0, LMOE_STREAM_FP32 = 1 } lmoe_stream_type;

/* h = r + x, y = w h / sqrt(mean(h^2) + eps), per row of d values.
 *   x bf16 [T][d] (stride ldx); r [T][d] (stride ldr) the residual stream in
 *   bf16 or fp32 (`stream_type`), or NULL: h = x and h_out is not written.
 *   h_out [T][d], packed, r's type: the sum rounded once to that type, which
 *   is also the value that is normalised.  w bf16 [d].
 *   y: bf16 [T][d], or MXFP8 codes [T][d] with scales [T][d/32].
 * In place: h_out may be r (ldr = d), y (bf16) may be x (ldx = d).
 * Errors: INVALID_ARG (NULL or misaligned pointer, T < 0, eps negative or
 * not finite, strides < d; r without h_out; MXFP8 without scales),
 * UNSUPPORTED (d not a multiple of 8 - of 32 for MXFP8 - or over 16384, a
 * stride not a multiple of 8), CUDA.  T = 0 is a no-op. */
LMOE_API lmoe_status lmoe_add_rms_norm(const void* x_bf16, int64_t ldx, const void* r_opt, int64_t ldr,
                                       lmoe_stream_type stream_type, int T, int d, const void* w_bf16, float eps,
                                       void* h_out, void* y, lmoe_norm_out out_format, uint8_t* y_scale,
                                       cudaStream_t stream);

/* Backward: from dy bf16 [T][d] and the stored h (`stream_type`):
 *   rho = 1/sqrt(mean(h^2) + eps)
 *   dx = rho (w dy - h rho^2 mean(w dy h)) + dh   [T][d], packed, h's type:
 *        the gradient of x and of r alike
 *   dw = sum over rows of dy h rho                fp32 [d]
 * dh_opt [T][d] (h's type): the gradient that reaches h along the residual
 * stream, or NULL.  dx may be dh (lddh = d).  workspace: 16-byte aligned,
 * lmoe_add_rms_norm_backward_workspace bytes, contents irrelevant.  The sums
 * over rows are added in an order that depends on T, d, the types and whether
 * dh is given only.
 * T = 0 writes dw = 0.  A bounded wait of the kernel that runs out (there is
 * no handle to report it by) leaves NaN in dw and dx, in the forward pass in
 * the rows of y.  Errors as above. */
LMOE_API lmoe_status lmoe_add_rms_norm_backward_workspace(int T, int d, size_t* bytes);
LMOE_API lmoe_status lmoe_add_rms_norm_backward(const void* dy_bf16, int64_t lddy, const void* h, int64_t ldh,
                                                const void* dh_opt, int64_t lddh, lmoe_stream_type stream_type,
                                                int T, int d, const void* w_bf16, float eps, void* dx, float* dw,
                                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Self-test of the norm kernels' bounded waits (2 s each): a pass over packed
 * bf16 x [T][d] of whose rows 16 bytes are waited for that no copy brings, so
 * that all waits run out.  Forward: all of y [T][d] is NaN.  backward != 0: x is
 * dy and h, y is dx, and both y and dw are NaN.  Errors as above, and UNSUPPORTED for a
 * forward pass on fewer than 2^23 values; T >= 1. */
LMOE_API lmoe_status lmoe_add_rms_norm_selftest_timeout(int backward, const void* x_bf16, int T, int d,
                                                        const void* w_bf16, void* y_bf16, float* dw_opt,
                                                        void* workspace_opt, size_t workspace_bytes,
                                                        cudaStream_t stream);

/* ------------------------------------------- dense gated feed-forward */
typedef enum { LMOE_FFN_W_BF16 = 0, LMOE_FFN_W_MXFP8 = 1 } lmoe_ffn_wfmt;

/*   g = x W_gate^T,  u = x W_up^T,  hid = a(g) v(u),  y = hid W_down^T
 *   SiTU-GLU: a = b1 tanh(g/b1) sigmoid(g), v = b2 tanh(u/b2)
 *   SwiGLU:   a = g sigmoid(g),             v = u
 * Products accumulate in fp32; hid is rounded to bf16 (MXFP8 blocks: encoded
 * as MXFP8) between the two passes.
 * Shapes: d_model and d_ff multiples of 8 (MXFP8: of 32); they and T at most 2^30. */
typedef struct {
  int d_model;
  int d_ff;
  lmoe_act act;
  float situ_beta;         /* b1 > 0 (SiTU) */
  float situ_linear_beta;  /* b2 > 0 (SiTU) */
  lmoe_ffn_wfmt wfmt;
  int max_tokens;          /* largest T of any call */
  int training;            /* 1: allocate what lmoe_ffn_backward needs (bf16 only) */
} lmoe_ffn_config;

/* gate, up [d_ff][d_model], down [d_model][d_ff]: bf16, or MXFP8 codes with
 * *_s scales.  Borrowed: they stay valid while the handle lives.  bf16
 * weights are read anew by every call, so an optimizer may update them in
 * place between calls (in stream order); MXFP8 weights do not change after
 * lmoe_ffn_create, which lays their scales out for the tensor cores. */
typedef struct {
  const void* gate;
  const void* up;
  const void* down;
  const uint8_t* gate_s;
  const uint8_t* up_s;
  const uint8_t* down_s;
} lmoe_ffn_weights;

typedef struct lmoe_ffn_ctx* lmoe_ffn_handle;

/* Errors: INVALID_ARG (NULL, misaligned, sizes < 1, bad enum, caps not
 * positive), UNSUPPORTED (shapes above; training with MXFP8; not an sm_103
 * GPU), OOM, CUDA.  Synchronises `stream`.  *out is NULL on error.  One handle
 * is used by one stream at a time, and belongs to the device that is current
 * here: the calls below return INVALID_ARG while another one is (destroy
 * excepted). */
LMOE_API lmoe_status lmoe_ffn_create(const lmoe_ffn_config* cfg, const lmoe_ffn_weights* w, cudaStream_t stream,
                                     lmoe_ffn_handle* out);

/* x bf16 [T][d_model] (stride ldx) -> out bf16 [T][d_model].  gate_opt and
 * up_opt bf16 [T][d_ff], both or neither: g and u for the backward pass.
 * out may not overlap x.  T = 0 is a no-op. */
LMOE_API lmoe_status lmoe_ffn_forward(lmoe_ffn_handle h, const void* x_bf16, int64_t ldx, int T, void* out_bf16,
                                      void* gate_opt, void* up_opt, cudaStream_t stream);

/* Gradients from x, the saved g and u (bf16 [T][d_ff]) and dy bf16
 * [T][d_model] (stride lddy): dx [T][d_model], dw_gate and dw_up
 * [d_ff][d_model], dw_down [d_model][d_ff], bf16, overwritten; any of the
 * four may be NULL and is then not computed.  dg, du and hid are rounded to
 * bf16 between the products; dhid is fp32.  The gradients may not overlap an
 * input, a weight or one another.  The same inputs and the same gradients asked
 * for give the same bits.
 * T = 0 writes zero weight gradients. */
LMOE_API lmoe_status lmoe_ffn_backward(lmoe_ffn_handle h, const void* x_bf16, int64_t ldx, const void* gate,
                                       const void* up, const void* dy_bf16, int64_t lddy, int T, void* dx_opt,
                                       void* dw_gate_opt, void* dw_up_opt, void* dw_down_opt, cudaStream_t stream);

/* The block on MXFP8 operands (handles with LMOE_FFN_W_MXFP8): x_codes
 * [T][d_model], x_scales [T][d_model/32] -> out bf16 [T][d_model]. */
LMOE_API lmoe_status lmoe_ffn_forward_mx(lmoe_ffn_handle h, const uint8_t* x_codes, const uint8_t* x_scales, int T,
                                         void* out_bf16, cudaStream_t stream);

/* Synchronise `stream` and return the first deferred error (a CUDA error, or
 * TIMEOUT of a kernel's bounded wait); clears the kernel-side flag.  What the
 * calls up to a TIMEOUT wrote is not valid; where a product's partial sums are
 * joined, outputs of sums that are not whole are NaN. */
LMOE_API lmoe_status lmoe_ffn_sync_status(lmoe_ffn_handle h, cudaStream_t stream);

/* Self-test of the bounded waits: a forward pass on packed x (MXFP8: codes and
 * scales) of whose rows each copy of the first product brings only half, so
 * that its waits run out, after 2 s each, and lmoe_ffn_sync_status returns
 * TIMEOUT.  The handle stays usable.  Errors as of the forward calls; T >= 1. */
LMOE_API lmoe_status lmoe_ffn_selftest_timeout(lmoe_ffn_handle h, const void* x, const uint8_t* x_scales_opt, int T,
                                               void* out_bf16, cudaStream_t stream);

/* Kernels the last call on this handle launched. */
LMOE_API int lmoe_ffn_last_launch_count(lmoe_ffn_handle h);

/* Synchronises the device and releases the workspace.  NULL is accepted. */
LMOE_API lmoe_status lmoe_ffn_destroy(lmoe_ffn_handle h);

#ifdef __cplusplus
}
#endif
#endif /* LMOE_FFN_H */
