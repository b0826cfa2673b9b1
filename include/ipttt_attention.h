/*
 * ipttt_attention.h: C ABI of the attention operators beside the fast-weight
 * layer, exported by libipttt next to include/ipttt.h and include/ipttt_block.h:
 * a block whose MLP is the layer keeps its attention as it is.
 *
 *   head norm             norms of queries and keys for each head and the rotation
 *                         by position in one pass; the serving form also writes the
 *                         new keys and values into a paged cache
 *   attention             over packed prompts: causal or not, a sliding window,
 *                         grouped heads, keys from before the queries
 *   attention step        one new token of each sequence over the paged cache
 *
 * The first two with their backward pass. The calls keep to the rules of
 * include/ipttt_block.h: borrowed pointers, no device allocation, the given HIP
 * stream (NULL: the null stream), no host synchronisation, every argument checked
 * before any device work, no state between calls, results that do not depend on what
 * workspace or outputs hold and that repeat bit for bit on the same device.
 *
 * Types. IPTTT_F32 or IPTTT_BF16. Norms, scores, softmax statistics and every sum
 * are fp32; bf16 results are rounded once, to nearest even. In bf16 the softmax's
 * weights, and in the backward also the scores' gradients, are rounded to bf16 as
 * operands of the products they enter (bf16 MFMA, fp32 accumulation); in fp32 the
 * products are fp32. A result whose operands are not all finite may be NaN where
 * the formula has an infinity. Keys that a query does not see have no part in its
 * result, whatever they hold. Sums are formed before they are divided, so that numbers
 * beyond the range of activations (heads to norm beyond 2^60, values beyond 2^88) may
 * overflow fp32.
 *
 * A tensor of heads is given by its strides in elements: both at least head_dim, any
 * order of the two (a slice of a fused projection, or heads outermost); channels are
 * contiguous. Pointers need the alignment of their element type, except where a call
 * says 16 bytes; rows on 16-byte boundaries (head_dim, strides) are read fastest.
 * Outputs must not overlap inputs or each other.
 */
#ifndef IPTTT_ATTENTION_H
#define IPTTT_ATTENTION_H

#include "ipttt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void *p;             /* element (t, h, c) is p[t * tok_stride + h * head_stride + c] */
  int64_t tok_stride;
  int64_t head_stride;
} ipttt_heads;

/* Keys and values of many sequences in pages of page_size tokens, both
 * [pages][k_heads][page_size][head_dim], 16-byte aligned. */
typedef struct {
  void *k, *v;
  int32_t pages;       /* 0 .. 2^31 - 1          */
  int32_t page_size;   /* 1 .. 65536             */
  int32_t k_heads, head_dim;
  ipttt_dtype dtype;
} ipttt_kv_cache;

/* Token t of sequence s is in page p[s * stride + t / page_size], at t % page_size. A
 * number outside 0 .. pages - 1 is no page: nothing is written to it, and a step
 * counts its keys as not there. */
typedef struct {
  const int32_t *p;    /* device memory           */
  int64_t stride;      /* >= width                */
  int32_t batch;       /* sequences: 0 .. 65535   */
  int32_t width;       /* pages a sequence may have, >= 0; width * page_size < 2^31 */
} ipttt_page_table;

/* ---- head norm ---------------------------------------------------------------
 * For each token and each head x of q and k, with D = head_dim and R = rotary:
 *   n = x (sum(x^2) / D + eps)^-1/2 gamma     (gamma NULL: n = x)
 *   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin), angle = pos inv_freq[i],
 * for the pairs (a, b) = (i, i + R / 2) of the first R channels, i < R / 2, or
 * (2 i, 2 i + 1) if interleaved; the other channels are n. Angles are computed in
 * 64 bits, so positions may be as far as 2^31. */
typedef struct {
  int32_t q_heads, k_heads;   /* 1 .. 1024                              */
  int32_t head_dim;           /* 1 .. 128                               */
  int32_t rotary;             /* even, 0 .. head_dim                    */
  int32_t interleaved;
  ipttt_dtype dtype;          /* of q, k, v, gammas, outputs, gradients */
  float eps;                  /* >= 0                                   */
  const void *q_gamma, *k_gamma;  /* [head_dim], or NULL: not normed     */
  const double *inv_freq;     /* [rotary / 2], device memory, 8-byte aligned */
} ipttt_headnorm_desc;

/* pos: [n] positions, device memory. n <= 2^31 - 1; n == 0 is a successful no-op. */
ipttt_status ipttt_headnorm_forward(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                    const ipttt_heads *k, const int32_t *pos, int64_t n,
                                    const ipttt_heads *q_out, const ipttt_heads *k_out,
                                    void *hip_stream);

/* The same with k's result, and v as it is, written to the cache: token t is the
 * pos[t]-th of sequence seqs[t] (NULL: of sequence t). A token whose sequence or
 * position the table does not hold is not written; its q is computed all the same (a
 * negative position marks padding). No two tokens may have the same place: it would
 * hold parts of both. */
ipttt_status ipttt_headnorm_append(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                   const ipttt_heads *k, const ipttt_heads *v, const int32_t *pos,
                                   const int32_t *seqs, int64_t n, const ipttt_heads *q_out,
                                   const ipttt_kv_cache *cache, const ipttt_page_table *table,
                                   void *hip_stream);

/* Gradients from dq = dL/dq_out and dk = dL/dk_out, with g the rotation's transpose of
 * them, r = (sum(x^2) / D + eps)^-1/2 and w = g gamma:
 *   dx = r (w - x r sum(w x r) / D)            (gamma NULL: dx = g)
 *   dgamma = sum over tokens and heads of g x r    [head_dim] fp32, each may be NULL
 * q and k are the forward's inputs. A NULL gamma's dgamma must be NULL. n == 0 writes
 * zero dgamma. The workspace must be 256-byte aligned. */
size_t ipttt_headnorm_backward_workspace_bytes(const ipttt_headnorm_desc *desc, int64_t n);
ipttt_status ipttt_headnorm_backward(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                     const ipttt_heads *k, const int32_t *pos,
                                     const ipttt_heads *dq, const ipttt_heads *dk, int64_t n,
                                     const ipttt_heads *dx_q, const ipttt_heads *dx_k,
                                     float *dq_gamma, float *dk_gamma, void *workspace,
                                     size_t workspace_bytes, void *hip_stream);

/* ---- attention over packed prompts ----------------------------------------------
 * Sequence s has queries q_offsets[s] .. q_offsets[s + 1] - 1 of n_q and keys
 * k_offsets[s] .. k_offsets[s + 1] - 1 of n_k (offsets never fall; the first counts as
 * 0, all are cut to n; both NULL: one sequence, batch 1). Query head h reads key head h / (q_heads / k_heads). With lq
 * and lk a sequence's numbers of queries and keys, query i sees keys
 *   j <= i + lk - lq                     if causal (the last query sees the last key),
 *   j > i + lk - lq - window             as well if window > 0, which must be causal,
 * and with a_j = scale q.k_j over those keys:
 *   lse = log sum exp(a_j), o = sum exp(a_j - lse) v_j.
 * A query that sees no key, and rows behind the last sequence, have o = 0 and
 * lse = -infinity. */
typedef struct {
  int32_t q_heads, k_heads;   /* q_heads a multiple of k_heads; q_heads <= 1024 */
  int32_t head_dim;           /* 1 .. 128                                       */
  int32_t batch;              /* sequences: 0 .. 65535                          */
  int32_t causal, window;
  ipttt_dtype dtype;
  float scale;                /* finite                                         */
  int64_t n_q, n_k;           /* rows of q and of k, v; up to 2^30              */
  const int32_t *q_offsets, *k_offsets;  /* [batch + 1], device memory, or NULL */
} ipttt_attention;

/* o: heads of n_q rows. lse: [q_heads][n_q] fp32, or NULL. The workspace must be 256-byte
 * aligned; pointers of desc are not read for its size. */
size_t ipttt_attention_forward_workspace_bytes(const ipttt_attention *desc);
ipttt_status ipttt_attention_forward(const ipttt_attention *desc, const ipttt_heads *q,
                                     const ipttt_heads *k, const ipttt_heads *v,
                                     const ipttt_heads *o, float *lse, void *workspace,
                                     size_t workspace_bytes, void *hip_stream);

/* Gradients from dy = dL/do, with p_j = exp(a_j - lse):
 *   dv_j = sum p_j dy, dp_j = dy.v_j, ds_j = p_j (dp_j - sum(dy o)),
 *   dq = scale sum ds_j k_j, dk_j = scale sum ds_j q,
 * the sums of dk and dv over all queries of the key head's group. o and lse are the
 * forward's. Rows that no sequence holds have zero gradients. The workspace must be
 * 256-byte aligned. */
size_t ipttt_attention_backward_workspace_bytes(const ipttt_attention *desc);
ipttt_status ipttt_attention_backward(const ipttt_attention *desc, const ipttt_heads *q,
                                      const ipttt_heads *k, const ipttt_heads *v,
                                      const ipttt_heads *o, const float *lse,
                                      const ipttt_heads *dy, const ipttt_heads *dq,
                                      const ipttt_heads *dk, const ipttt_heads *dv,
                                      void *workspace, size_t workspace_bytes, void *hip_stream);

/* ---- attention of one new token over the paged cache -----------------------------
 * o = sum exp(a_j - lse) v_j for each sequence of the table and each query head, over
 * its keys j < lens[s] (cut to 0 .. width * page_size), of these the last `window` if
 * window > 0. The new token's own key is one of them: it is appended first. No key:
 * o = 0, lse = -infinity. */
typedef struct {
  int32_t q_heads;            /* a multiple of the cache's k_heads, <= 1024 */
  int32_t window;             /* >= 0                                       */
  float scale;                /* finite                                     */
} ipttt_step_desc;

/* q, o: heads of one row a sequence. lens: [batch], device memory. lse: [batch][q_heads]
 * fp32, or NULL. The workspace must be 256-byte aligned. */
size_t ipttt_attention_step_workspace_bytes(const ipttt_step_desc *desc, const ipttt_kv_cache *cache,
                                            const ipttt_page_table *table);
ipttt_status ipttt_attention_step(const ipttt_step_desc *desc, const ipttt_heads *q,
                                  const ipttt_kv_cache *cache, const ipttt_page_table *table,
                                  const int32_t *lens, const ipttt_heads *o, float *lse,
                                  void *workspace, size_t workspace_bytes, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* IPTTT_ATTENTION_H */
