/*
 * ipttt_block.h: C ABI of the operators around the fast-weight layer, exported
 * by libipttt next to include/ipttt.h: what the rest of a residual block of a
 * model with such layers computes.
 *
 *   layer norm            the norm in front of a layer, with the residual add
 *   gated recurrence      a linear token mixer whose state is one vector per
 *                         sequence, carried like the layer's fast weight
 *   gated feed-forward    the plain gated MLP of the layers that keep W_o fixed
 *
 * each with its backward pass. Like the layer's own calls, these borrow every
 * pointer, allocate nothing on the device, run on the given HIP stream (NULL:
 * the null stream) without synchronising the host, validate every argument
 * before any device work and report errors as ipttt_status with
 * ipttt_last_error(). They keep no state: distinct calls are independent unless
 * they share a workspace, which must then be ordered by the caller. Results do
 * not depend on what the workspace or the outputs hold beforehand, and repeat
 * bit for bit (no atomics in sums) on the same device.
 *
 * Types. IPTTT_F32 or IPTTT_BF16 for activations and weights. Sums, norms,
 * statistics and recurrent states are fp32; bf16 outputs are rounded once, to
 * nearest even. Row and token strides are in elements, at least the width d
 * (so a tensor may be a slice of a wider one), and may be odd; pointers need
 * the alignment of their element type, except where a call says 16 bytes.
 * Outputs must not overlap inputs unless said otherwise. In bf16 the feed-forward
 * block also rounds what passes from one of its products to the next.
 */
#ifndef IPTTT_BLOCK_H
#define IPTTT_BLOCK_H

#include "ipttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm -----------------------------------------------------------
 *   h = round(x + r)                      (r NULL: h is x and is not written)
 *   mean = sum(x + r) / d, rstd = (sum((x + r - mean)^2) / d + eps)^-1/2
 *   y = (x + r - mean) rstd gamma + beta
 * of n rows of width d; the statistics and y come from the unrounded sum. */
typedef struct {
  int32_t d;          /* 1 .. 16384                                        */
  ipttt_dtype dtype;  /* of x, r, h, y, gamma, beta and their gradients dx */
  float eps;          /* >= 0                                              */
  const void *gamma;  /* [d] or NULL (ones)                                */
  const void *beta;   /* [d] or NULL (zeros)                               */
} ipttt_norm_desc;

/* h, y: [n][d] dense; mean, rstd: [n] fp32, or both NULL. h is required
 * exactly when r is given. n == 0 is a successful no-op. */
ipttt_status ipttt_norm_forward(const ipttt_norm_desc *desc, const void *x, int64_t x_stride,
                                const void *r, int64_t r_stride, int64_t n, void *h, void *y,
                                float *mean, float *rstd, void *hip_stream);

/* Gradients from dy = dL/dy and dh = dL/dh through the residual stream (NULL:
 * zero), with q = dy gamma and xh = (h - mean) rstd:
 *   dx = (q - sum(q) / d - xh sum(q xh) / d) rstd + dh   [n][d] dense
 *   dgamma = sum over rows of dy xh, dbeta = sum of dy   [d] fp32, each may be NULL
 * dx is the gradient of x and of r. n == 0 writes zero dgamma and dbeta. */
size_t ipttt_norm_backward_workspace_bytes(const ipttt_norm_desc *desc, int64_t n);
ipttt_status ipttt_norm_backward(const ipttt_norm_desc *desc, const void *h, int64_t h_stride,
                                 const float *mean, const float *rstd, const void *dy,
                                 int64_t dy_stride, const void *dh, int64_t dh_stride, int64_t n,
                                 void *dx, float *dgamma, float *dbeta, void *workspace,
                                 size_t workspace_bytes, void *hip_stream);

/* ---- gated linear recurrence ------------------------------------------------
 * For each sequence and each of d channels, with gate logits g and values v:
 *   f_t = 1 / (1 + e^-g_t)
 *   h_t = f_t h_{t-1} + (1 - f_t) v_t,   h_{-1} = h0
 * starts[t] != 0 marks the first token of a packed document: h_{t-1} counts as
 * zero there, whatever it holds (the layer's reset of W at document starts). A
 * state that is not finite stays so until then, but an infinite one may become NaN
 * where gates forget it (their product over 16 tokens can be zero in fp32).
 * lens[n] (clamped to 0 .. seq_len) ends sequence n: past it nothing is read
 * for the result, outputs are zero, and the last state is the one after token
 * lens[n] - 1 (h0 for length zero). */
typedef struct {
  void *p;            /* element (n, t, c) is p[n * seq_stride + t * tok_stride + c] */
  int64_t seq_stride;
  int64_t tok_stride;
} ipttt_view;

typedef struct {
  int32_t batch;
  int32_t d;          /* 1 .. 65536                                            */
  int64_t seq_len;
  ipttt_dtype dtype;  /* of g, v, h and of the gradients dh, dg, dv             */
  ipttt_view g, v;    /* read                                                  */
  ipttt_view h;       /* written by the forward, read by the backward          */
  const uint8_t *starts; /* [batch][seq_len] or NULL                            */
  const int32_t *lens;   /* [batch], device memory, or NULL                     */
  const float *h0;       /* [batch][d] or NULL (zero)                           */
} ipttt_recurrence;

/* Inside a long sequence blocks of tokens wait for the state of the blocks before
 * them, which run already. The wait is bounded: one that were to last a second
 * (another stream writing to the call's workspace, say) ends in NaN results, which
 * the status, long returned by then, does not show. */

/* Workspace of the forward and of the backward (the same), 0 if a size is
 * invalid; short sequences need none and get a minimum. Pointers in `r` are
 * not read. The workspace must be 256-byte aligned. */
size_t ipttt_recurrence_workspace_bytes(const ipttt_recurrence *r);

/* h_last: [batch][d] or NULL; it must not be h0 (the step's may). */
ipttt_status ipttt_recurrence_forward(const ipttt_recurrence *r, float *h_last, void *workspace,
                                      size_t workspace_bytes, void *hip_stream);

/* One token for each sequence: seq_len must be 1, h0 is the state before it
 * (NULL: zero) and state receives the one after it; state may be h0 itself. */
ipttt_status ipttt_recurrence_step(const ipttt_recurrence *r, float *state, void *hip_stream);

/* Gradients from dh = dL/dh and dh_last = dL/dh_last ([batch][d], NULL: zero).
 * With D_t = dh_t + (f_{t+1} D_{t+1}, 0 before a document start; dh_last after
 * the last token):
 *   dv_t = (1 - f_t) D_t,  dg_t = D_t (h_{t-1} - v_t) f_t (1 - f_t)
 *   dh0 = f_0 D_0 (0 at a document start), [batch][d] or NULL
 * h is the forward's output. dg and dv are zero past a sequence's length; they
 * overlap neither each other nor an input. */
ipttt_status ipttt_recurrence_backward(const ipttt_recurrence *r, const ipttt_view *dh,
                                       const float *dh_last, const ipttt_view *dg,
                                       const ipttt_view *dv, float *dh0, void *workspace,
                                       size_t workspace_bytes, void *hip_stream);

/* ---- gated feed-forward block -----------------------------------------------
 *   a = x W_g, u = x W_u, z = SiLU(a) * u, y = z W_d
 * for n tokens. Weights are output-major, as the layer's: w_gate, w_up
 * [d_ff][d], w_down [d][d_ff], 16-byte aligned. In bf16, z and the backward's dA
 * and dU are rounded to bf16 as operands of the products they enter, which run on
 * bf16 MFMA with fp32 accumulation; in fp32 every product keeps fp32 accuracy
 * (a result whose operands are not all finite is not finite, but may be NaN
 * where the formula has an infinity). Any d, d_ff; multiples of 64 avoid copies
 * of the operands. */
typedef struct {
  int32_t d;          /* 1 .. 65536  */
  int32_t d_ff;       /* 1 .. 262144 */
  ipttt_dtype dtype;
  const void *w_gate, *w_up, *w_down;
} ipttt_ff_desc;

/* a, u: [n][d_ff] fp32, dense, both given to save the pre-activations for the
 * backward or both NULL; 16-byte aligned. y rows are y_stride apart. n <= 2^24.
 * n == 0 is a successful no-op. The workspace must be 256-byte aligned. */
size_t ipttt_ff_workspace_bytes(const ipttt_ff_desc *desc, int64_t n);
ipttt_status ipttt_ff_forward(const ipttt_ff_desc *desc, const void *x, int64_t x_stride,
                              int64_t n, void *y, int64_t y_stride, float *a, float *u,
                              void *workspace, size_t workspace_bytes, void *hip_stream);

/* Gradients, all in the descriptor's type, overwritten. dx rows are dx_stride
 * apart; the weights' gradients have the weights' layouts (16-byte aligned).
 * n == 0 writes zero weight gradients. */
typedef struct {
  void *dx;
  int64_t dx_stride;
  void *dw_gate, *dw_up, *dw_down;
} ipttt_ff_grads;

size_t ipttt_ff_backward_workspace_bytes(const ipttt_ff_desc *desc, int64_t n);
ipttt_status ipttt_ff_backward(const ipttt_ff_desc *desc, const void *x, int64_t x_stride,
                               const float *a, const float *u, const void *dy, int64_t dy_stride,
                               int64_t n, const ipttt_ff_grads *grads, void *workspace,
                               size_t workspace_bytes, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* IPTTT_BLOCK_H */
