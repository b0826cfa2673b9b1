// Internal declarations of the attention operators (include/ipttt_attention.h): what
// the host side (attention.cpp) and the kernel translation units share. Not part of
// the ABI.
#pragma once

#include "../../include/ipttt_attention.h"
#include "internal.h"

namespace ipttt {

constexpr int kHeadMaxDim = 128;

// ---- head norm (kernels_heads.hip) ----------------------------------------------
struct HeadArgs {
  int hq, hk, dh, rotary;
  bool interleaved;
  float eps;
  int64_t n;
  const void *q_gamma, *k_gamma;
  const double *inv_freq;
  const int32_t *pos;
  ipttt_heads q, k;        // inputs
  ipttt_heads v;           // append
  ipttt_heads dq, dk;      // backward: gradients of the outputs
  ipttt_heads q_out, k_out;  // outputs (append: no k_out); backward: gradients of the inputs
  const int32_t *seqs;     // append, or null
  ipttt_kv_cache cache;    // append
  ipttt_page_table table;  // append
  float *dq_gamma, *dk_gamma;  // [dh] or null
  float *part;             // backward: [blocks of q and of k][dh] partial sums
};
// Blocks (and rows of partial sums) of the backward for `heads` of all its heads.
int heads_bwd_blocks(int heads, int all, int64_t n);
template <typename T>
hipError_t heads_forward(const HeadArgs &a, hipStream_t st);
template <typename T>
hipError_t heads_append(const HeadArgs &a, hipStream_t st);
template <typename T>
hipError_t heads_backward(const HeadArgs &a, hipStream_t st);

// ---- attention over packed prompts (kernels_attention.hip) --------------------------
// A tile of one sequence's rows: the first of them in the sequence, and where its queries
// and keys are.
struct TilePlace {
  int32_t first, q_start, lq, k_start, lk, pad[3];
};
struct AttnArgs {
  int hq, hk, dh, batch;
  int causal, window;
  float scale;
  int64_t n_q, n_k;
  const int32_t *q_off, *k_off;
  ipttt_heads q, k, v, o;
  float *lse;              // [hq][n_q]; or null in the forward
  ipttt_heads dy, dq, dk, dv;  // backward
  float *delta, *lse2;     // backward: [hq][n_q], sum(dy o) and lse in units of log2
  TilePlace *q_order, *k_order;  // workspace for the order of the tiles of queries, of keys
  float *part;             // and for partial dk and dv
};
// Bytes of those.
size_t attn_q_order(const ipttt_attention &d);
size_t attn_k_order(const ipttt_attention &d);
size_t attn_parts(const ipttt_attention &d);
// Whether the tiles of such a call can be counted in 31 bits.
bool attn_size_ok(int hq, int batch, int64_t n);
template <typename T>
hipError_t attn_forward(const AttnArgs &a, hipStream_t st);
template <typename T>
hipError_t attn_backward(const AttnArgs &a, hipStream_t st);

// ---- one new token over the paged cache (kernels_step.hip) --------------------------
struct StepArgs {
  int hq, window;
  float scale;
  ipttt_heads q, o;
  ipttt_kv_cache cache;
  ipttt_page_table table;
  const int32_t *lens;
  float *lse;              // [batch][hq] or null
  void *ws;
};
size_t step_workspace(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t);
template <typename T>
hipError_t step_forward(const StepArgs &a, hipStream_t st);

}  // namespace ipttt
