// Host side of the attention operators (include/ipttt_attention.h): argument checks,
// workspace planning and launches. Kernels live in kernels_heads.hip,
// kernels_attention.hip and kernels_step.hip.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "attention_internal.h"

using namespace ipttt;

namespace {

ipttt_status fail(ipttt_status s, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(s, buf);
}

ipttt_status launched(hipError_t e, const char *what) {
  if (e == hipSuccess) return IPTTT_OK;
  return fail(IPTTT_E_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define TRY(expr)                          \
  do {                                     \
    const ipttt_status _s = (expr);        \
    if (_s != IPTTT_OK) return _s;         \
  } while (0)

constexpr int kMaxHeads = 1024;
constexpr int kMaxBatch = 65535;
// Elements a tensor may span: offsets stay within 64 bits of bytes.
constexpr int64_t kMaxElems = (int64_t)1 << 60;

ipttt_status check_dtype(ipttt_dtype t) {
  if (t != IPTTT_F32 && t != IPTTT_BF16) return fail(IPTTT_E_UNSUPPORTED, "dtype=%d", (int)t);
  return IPTTT_OK;
}
size_t size_of(ipttt_dtype t) { return t == IPTTT_BF16 ? 2 : 4; }

ipttt_status check_ptr(const void *p, size_t align, const char *name) {
  if (!p) return fail(IPTTT_E_INVALID, "%s is NULL", name);
  if ((uintptr_t)p % align)
    return fail(IPTTT_E_INVALID, "%s is not %zu-byte aligned", name, align);
  return IPTTT_OK;
}
ipttt_status check_opt(const void *p, size_t align, const char *name) {
  return p ? check_ptr(p, align, name) : IPTTT_OK;
}
ipttt_status check_workspace(const void *ws, size_t have, size_t need) {
  TRY(check_ptr(ws, 256, "workspace"));
  if (have < need)
    return fail(IPTTT_E_WORKSPACE, "workspace_bytes=%zu below the %zu this call needs", have, need);
  return IPTTT_OK;
}

ipttt_status check_head_counts(int hq, int hk, int dh) {
  if (hq < 1 || hk < 1) return fail(IPTTT_E_INVALID, "q_heads=%d k_heads=%d must be > 0", hq, hk);
  if (hq > kMaxHeads || hk > kMaxHeads)
    return fail(IPTTT_E_UNSUPPORTED, "q_heads=%d k_heads=%d exceed %d", hq, hk, kMaxHeads);
  if (dh < 1) return fail(IPTTT_E_INVALID, "head_dim=%d must be > 0", dh);
  if (dh > kHeadMaxDim)
    return fail(IPTTT_E_UNSUPPORTED, "head_dim=%d exceeds %d", dh, kHeadMaxDim);
  return IPTTT_OK;
}
ipttt_status check_group(int hq, int hk) {
  if (hq % hk)
    return fail(IPTTT_E_INVALID, "q_heads=%d is no multiple of k_heads=%d", hq, hk);
  return IPTTT_OK;
}

// A tensor of n tokens x heads x dh.
ipttt_status check_heads(const ipttt_heads *x, int64_t n, int heads, int dh, ipttt_dtype t,
                         const char *name) {
  if (!x) return fail(IPTTT_E_INVALID, "%s is NULL", name);
  if (n == 0) return IPTTT_OK;  // no element
  TRY(check_ptr(x->p, size_of(t), name));
  if (n > 1 && x->tok_stride < dh)
    return fail(IPTTT_E_INVALID, "%s token stride %lld is below head_dim %d", name,
                (long long)x->tok_stride, dh);
  if (heads > 1 && x->head_stride < dh)
    return fail(IPTTT_E_INVALID, "%s head stride %lld is below head_dim %d", name,
                (long long)x->head_stride, dh);
  if ((n > 1 && x->tok_stride > kMaxElems / n) || (heads > 1 && x->head_stride > kMaxElems / heads))
    return fail(IPTTT_E_INVALID, "%s's strides are too large", name);
  return IPTTT_OK;
}
// Strides of axes with one element are never multiplied by anything but 0; whatever
// they hold they must not overflow.
ipttt_heads view(const ipttt_heads *x, int64_t n, int heads) {
  ipttt_heads v = *x;
  if (n <= 1) v.tok_stride = 0;
  if (heads <= 1) v.head_stride = 0;
  return v;
}

ipttt_status check_cache(const ipttt_kv_cache *c) {
  if (!c) return fail(IPTTT_E_INVALID, "cache is NULL");
  TRY(check_dtype(c->dtype));
  TRY(check_head_counts(c->k_heads, c->k_heads, c->head_dim));
  if (c->pages < 0) return fail(IPTTT_E_INVALID, "pages=%d must be >= 0", c->pages);
  if (c->page_size < 1) return fail(IPTTT_E_INVALID, "page_size=%d must be > 0", c->page_size);
  if (c->page_size > 65536)
    return fail(IPTTT_E_UNSUPPORTED, "page_size=%d exceeds 65536", c->page_size);
  if (c->pages > 0) {
    TRY(check_ptr(c->k, 16, "cache k"));
    TRY(check_ptr(c->v, 16, "cache v"));
  }
  return IPTTT_OK;
}
// The sizes of a table over pages of a cache, and with `pointers` its address.
ipttt_status check_table(const ipttt_page_table *t, const ipttt_kv_cache *c, bool pointers) {
  if (!t) return fail(IPTTT_E_INVALID, "table is NULL");
  if (t->batch < 0) return fail(IPTTT_E_INVALID, "batch=%d must be >= 0", t->batch);
  if (t->batch > kMaxBatch)
    return fail(IPTTT_E_UNSUPPORTED, "batch=%d exceeds %d", t->batch, kMaxBatch);
  if (t->width < 0) return fail(IPTTT_E_INVALID, "table width=%d must be >= 0", t->width);
  if ((int64_t)t->width * c->page_size > INT32_MAX)
    return fail(IPTTT_E_UNSUPPORTED, "table width=%d x page_size=%d exceeds 2^31 - 1", t->width,
                c->page_size);
  if (t->batch > 1 && (t->stride < t->width || t->stride > kMaxElems / t->batch))
    return fail(IPTTT_E_INVALID, "table stride %lld does not fit width %d", (long long)t->stride,
                t->width);
  if (pointers && t->batch > 0 && t->width > 0) TRY(check_ptr(t->p, 4, "table"));
  return IPTTT_OK;
}

// ---- head norm --------------------------------------------------------------------

ipttt_status check_headnorm(const ipttt_headnorm_desc *d, int64_t n) {
  if (!d) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_dtype(d->dtype));
  TRY(check_head_counts(d->q_heads, d->k_heads, d->head_dim));
  if (d->rotary < 0 || d->rotary > d->head_dim || d->rotary % 2)
    return fail(IPTTT_E_INVALID, "rotary=%d must be even and within head_dim=%d", d->rotary,
                d->head_dim);
  if (!(d->eps >= 0.f) || d->eps > 3.0e38f)
    return fail(IPTTT_E_INVALID, "eps must be finite and >= 0");
  if (n < 0) return fail(IPTTT_E_INVALID, "n=%lld must be >= 0", (long long)n);
  if (n > INT32_MAX) return fail(IPTTT_E_UNSUPPORTED, "n=%lld exceeds 2^31 - 1", (long long)n);
  TRY(check_opt(d->q_gamma, size_of(d->dtype), "q_gamma"));
  TRY(check_opt(d->k_gamma, size_of(d->dtype), "k_gamma"));
  if (d->rotary > 0) TRY(check_ptr(d->inv_freq, 8, "inv_freq"));
  return IPTTT_OK;
}

HeadArgs head_args(const ipttt_headnorm_desc *d, int64_t n, const ipttt_heads *q,
                   const ipttt_heads *k, const int32_t *pos) {
  HeadArgs a{};
  a.hq = d->q_heads;
  a.hk = d->k_heads;
  a.dh = d->head_dim;
  a.rotary = d->rotary;
  a.interleaved = d->interleaved != 0;
  a.eps = d->eps;
  a.n = n;
  a.q_gamma = d->q_gamma;
  a.k_gamma = d->k_gamma;
  a.inv_freq = d->inv_freq;
  a.pos = pos;
  a.q = view(q, n, a.hq);
  a.k = view(k, n, a.hk);
  return a;
}

// ---- attention ----------------------------------------------------------------------

ipttt_status check_attn_sizes(const ipttt_attention *d) {
  if (!d) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_dtype(d->dtype));
  TRY(check_head_counts(d->q_heads, d->k_heads, d->head_dim));
  TRY(check_group(d->q_heads, d->k_heads));
  if (d->batch < 0) return fail(IPTTT_E_INVALID, "batch=%d must be >= 0", d->batch);
  if (d->batch > kMaxBatch)
    return fail(IPTTT_E_UNSUPPORTED, "batch=%d exceeds %d", d->batch, kMaxBatch);
  if (d->window < 0) return fail(IPTTT_E_INVALID, "window=%d must be >= 0", d->window);
  if (d->window > 0 && !d->causal)
    return fail(IPTTT_E_INVALID, "window=%d needs causal attention", d->window);
  if (!isfinite(d->scale)) return fail(IPTTT_E_INVALID, "scale must be finite");
  if (d->n_q < 0 || d->n_k < 0)
    return fail(IPTTT_E_INVALID, "n_q=%lld n_k=%lld must be >= 0", (long long)d->n_q,
                (long long)d->n_k);
  if (d->n_q > ((int64_t)1 << 30) || d->n_k > ((int64_t)1 << 30))
    return fail(IPTTT_E_UNSUPPORTED, "n_q=%lld n_k=%lld exceed 2^30", (long long)d->n_q,
                (long long)d->n_k);
  if (!attn_size_ok(d->q_heads, d->batch, d->n_q > d->n_k ? d->n_q : d->n_k))
    return fail(IPTTT_E_UNSUPPORTED, "q_heads=%d x n=%lld exceed 2^31 tiles", d->q_heads,
                (long long)(d->n_q > d->n_k ? d->n_q : d->n_k));
  return IPTTT_OK;
}

ipttt_status check_attn(const ipttt_attention *d, const ipttt_heads *q, const ipttt_heads *k,
                        const ipttt_heads *v, const ipttt_heads *o, const float *lse) {
  TRY(check_attn_sizes(d));
  if (!d->q_offsets != !d->k_offsets)
    return fail(IPTTT_E_INVALID, "q_offsets and k_offsets must both be given or both be NULL");
  if (!d->q_offsets && d->batch != 1)
    return fail(IPTTT_E_INVALID, "batch=%d needs offsets", d->batch);
  TRY(check_opt(d->q_offsets, 4, "q_offsets"));
  TRY(check_opt(d->k_offsets, 4, "k_offsets"));
  TRY(check_heads(q, d->n_q, d->q_heads, d->head_dim, d->dtype, "q"));
  TRY(check_heads(k, d->n_k, d->k_heads, d->head_dim, d->dtype, "k"));
  TRY(check_heads(v, d->n_k, d->k_heads, d->head_dim, d->dtype, "v"));
  TRY(check_heads(o, d->n_q, d->q_heads, d->head_dim, d->dtype, "o"));
  return check_opt(lse, 4, "lse");
}

AttnArgs attn_args(const ipttt_attention *d, const ipttt_heads *q, const ipttt_heads *k,
                   const ipttt_heads *v, const ipttt_heads *o, const float *lse) {
  AttnArgs a{};
  a.hq = d->q_heads;
  a.hk = d->k_heads;
  a.dh = d->head_dim;
  a.batch = d->batch;
  a.causal = d->causal != 0;
  // No sequence has more keys than n_k: a longer window leaves out none, and one of up to 2^30
  // keeps the kernels' i + lk - lq - window within 32 bits, also where lq > lk.
  a.window = d->window < d->n_k ? d->window : (int)d->n_k;
  a.scale = d->scale;
  a.n_q = d->n_q;
  a.n_k = d->n_k;
  a.q_off = d->q_offsets;
  a.k_off = d->k_offsets;
  a.q = view(q, a.n_q, a.hq);
  a.k = view(k, a.n_k, a.hk);
  a.v = view(v, a.n_k, a.hk);
  a.o = view(o, a.n_q, a.hq);
  a.lse = const_cast<float *>(lse);
  return a;
}

ipttt_status check_step_sizes(const ipttt_step_desc *d, const ipttt_kv_cache *c,
                              const ipttt_page_table *t, bool pointers) {
  if (!d) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_cache(c));
  TRY(check_table(t, c, pointers));
  TRY(check_head_counts(d->q_heads, c->k_heads, c->head_dim));
  TRY(check_group(d->q_heads, c->k_heads));
  if (d->window < 0) return fail(IPTTT_E_INVALID, "window=%d must be >= 0", d->window);
  if (!isfinite(d->scale)) return fail(IPTTT_E_INVALID, "scale must be finite");
  return IPTTT_OK;
}

}  // namespace

extern "C" {

ipttt_status ipttt_headnorm_forward(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                    const ipttt_heads *k, const int32_t *pos, int64_t n,
                                    const ipttt_heads *q_out, const ipttt_heads *k_out,
                                    void *hip_stream) {
  TRY(check_headnorm(desc, n));
  if (n == 0) return IPTTT_OK;
  const int dh = desc->head_dim;
  TRY(check_heads(q, n, desc->q_heads, dh, desc->dtype, "q"));
  TRY(check_heads(k, n, desc->k_heads, dh, desc->dtype, "k"));
  TRY(check_heads(q_out, n, desc->q_heads, dh, desc->dtype, "q_out"));
  TRY(check_heads(k_out, n, desc->k_heads, dh, desc->dtype, "k_out"));
  TRY(check_ptr(pos, 4, "pos"));
  HeadArgs a = head_args(desc, n, q, k, pos);
  a.q_out = view(q_out, n, a.hq);
  a.k_out = view(k_out, n, a.hk);
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? heads_forward<__bf16>(a, st) : heads_forward<float>(a, st),
      "head norm launch");
}

ipttt_status ipttt_headnorm_append(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                   const ipttt_heads *k, const ipttt_heads *v, const int32_t *pos,
                                   const int32_t *seqs, int64_t n, const ipttt_heads *q_out,
                                   const ipttt_kv_cache *cache, const ipttt_page_table *table,
                                   void *hip_stream) {
  TRY(check_headnorm(desc, n));
  TRY(check_cache(cache));
  if (cache->k_heads != desc->k_heads || cache->head_dim != desc->head_dim ||
      cache->dtype != desc->dtype)
    return fail(IPTTT_E_INVALID, "the cache's heads or type are not the descriptor's");
  TRY(check_table(table, cache, true));
  if (n == 0) return IPTTT_OK;
  const int dh = desc->head_dim;
  TRY(check_heads(q, n, desc->q_heads, dh, desc->dtype, "q"));
  TRY(check_heads(k, n, desc->k_heads, dh, desc->dtype, "k"));
  TRY(check_heads(v, n, desc->k_heads, dh, desc->dtype, "v"));
  TRY(check_heads(q_out, n, desc->q_heads, dh, desc->dtype, "q_out"));
  TRY(check_ptr(pos, 4, "pos"));
  TRY(check_opt(seqs, 4, "seqs"));
  HeadArgs a = head_args(desc, n, q, k, pos);
  a.v = view(v, n, a.hk);
  a.q_out = view(q_out, n, a.hq);
  a.seqs = seqs;
  a.cache = *cache;
  a.table = *table;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? heads_append<__bf16>(a, st) : heads_append<float>(a, st),
      "head norm append launch");
}

size_t ipttt_headnorm_backward_workspace_bytes(const ipttt_headnorm_desc *desc, int64_t n) {
  if (!desc || check_head_counts(desc->q_heads, desc->k_heads, desc->head_dim) != IPTTT_OK || n < 0 ||
      n > INT32_MAX)
    return 0;
  const int all = desc->q_heads + desc->k_heads;
  const int64_t rows = heads_bwd_blocks(desc->q_heads, all, n) + heads_bwd_blocks(desc->k_heads, all, n);
  return (size_t)round_up(rows * desc->head_dim * 4, 256);
}

ipttt_status ipttt_headnorm_backward(const ipttt_headnorm_desc *desc, const ipttt_heads *q,
                                     const ipttt_heads *k, const int32_t *pos,
                                     const ipttt_heads *dq, const ipttt_heads *dk, int64_t n,
                                     const ipttt_heads *dx_q, const ipttt_heads *dx_k,
                                     float *dq_gamma, float *dk_gamma, void *workspace,
                                     size_t workspace_bytes, void *hip_stream) {
  TRY(check_headnorm(desc, n));
  TRY(check_opt(dq_gamma, 4, "dq_gamma"));
  TRY(check_opt(dk_gamma, 4, "dk_gamma"));
  if ((dq_gamma && !desc->q_gamma) || (dk_gamma && !desc->k_gamma))
    return fail(IPTTT_E_INVALID, "a gamma that is NULL has no gradient");
  if (n == 0 && !dq_gamma && !dk_gamma) return IPTTT_OK;
  const int dh = desc->head_dim;
  static const ipttt_heads none = {nullptr, 0, 0};
  if (n > 0) {
    TRY(check_heads(q, n, desc->q_heads, dh, desc->dtype, "q"));
    TRY(check_heads(k, n, desc->k_heads, dh, desc->dtype, "k"));
    TRY(check_heads(dq, n, desc->q_heads, dh, desc->dtype, "dq"));
    TRY(check_heads(dk, n, desc->k_heads, dh, desc->dtype, "dk"));
    TRY(check_heads(dx_q, n, desc->q_heads, dh, desc->dtype, "dx_q"));
    TRY(check_heads(dx_k, n, desc->k_heads, dh, desc->dtype, "dx_k"));
    TRY(check_ptr(pos, 4, "pos"));
  }
  const bool sums = dq_gamma || dk_gamma;
  if (sums)
    TRY(check_workspace(workspace, workspace_bytes, ipttt_headnorm_backward_workspace_bytes(desc, n)));
  HeadArgs a = head_args(desc, n, n ? q : &none, n ? k : &none, pos);
  if (n > 0) {
    a.dq = view(dq, n, a.hq);
    a.dk = view(dk, n, a.hk);
    a.q_out = view(dx_q, n, a.hq);
    a.k_out = view(dx_k, n, a.hk);
  }
  a.dq_gamma = dq_gamma;
  a.dk_gamma = dk_gamma;
  a.part = sums ? (float *)workspace : nullptr;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? heads_backward<__bf16>(a, st) : heads_backward<float>(a, st),
      "head norm backward launch");
}

size_t ipttt_attention_forward_workspace_bytes(const ipttt_attention *desc) {
  if (check_attn_sizes(desc) != IPTTT_OK) return 0;
  return attn_q_order(*desc);
}

ipttt_status ipttt_attention_forward(const ipttt_attention *desc, const ipttt_heads *q,
                                     const ipttt_heads *k, const ipttt_heads *v,
                                     const ipttt_heads *o, float *lse, void *workspace,
                                     size_t workspace_bytes, void *hip_stream) {
  TRY(check_attn(desc, q, k, v, o, lse));
  if (desc->n_q == 0) return IPTTT_OK;
  TRY(check_workspace(workspace, workspace_bytes, attn_q_order(*desc)));
  AttnArgs a = attn_args(desc, q, k, v, o, lse);
  a.q_order = (TilePlace *)workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? attn_forward<__bf16>(a, st) : attn_forward<float>(a, st),
      "attention launch");
}

size_t ipttt_attention_backward_workspace_bytes(const ipttt_attention *desc) {
  if (check_attn_sizes(desc) != IPTTT_OK) return 0;
  return attn_q_order(*desc) + attn_k_order(*desc) + attn_parts(*desc) +
         (size_t)round_up((int64_t)desc->q_heads * desc->n_q * 8, 256);
}

ipttt_status ipttt_attention_backward(const ipttt_attention *desc, const ipttt_heads *q,
                                      const ipttt_heads *k, const ipttt_heads *v,
                                      const ipttt_heads *o, const float *lse,
                                      const ipttt_heads *dy, const ipttt_heads *dq,
                                      const ipttt_heads *dk, const ipttt_heads *dv,
                                      void *workspace, size_t workspace_bytes, void *hip_stream) {
  TRY(check_attn(desc, q, k, v, o, lse));
  if (desc->n_q > 0 && !lse) return fail(IPTTT_E_INVALID, "lse is NULL");
  TRY(check_heads(dy, desc->n_q, desc->q_heads, desc->head_dim, desc->dtype, "dy"));
  TRY(check_heads(dq, desc->n_q, desc->q_heads, desc->head_dim, desc->dtype, "dq"));
  TRY(check_heads(dk, desc->n_k, desc->k_heads, desc->head_dim, desc->dtype, "dk"));
  TRY(check_heads(dv, desc->n_k, desc->k_heads, desc->head_dim, desc->dtype, "dv"));
  if (desc->n_q == 0 && desc->n_k == 0) return IPTTT_OK;
  TRY(check_workspace(workspace, workspace_bytes, ipttt_attention_backward_workspace_bytes(desc)));
  AttnArgs a = attn_args(desc, q, k, v, o, lse);
  a.dy = view(dy, a.n_q, a.hq);
  a.dq = view(dq, a.n_q, a.hq);
  a.dk = view(dk, a.n_k, a.hk);
  a.dv = view(dv, a.n_k, a.hk);
  a.q_order = (TilePlace *)workspace;
  a.k_order = (TilePlace *)((char *)workspace + attn_q_order(*desc));
  a.part = (float *)((char *)a.k_order + attn_k_order(*desc));
  a.delta = (float *)((char *)a.part + attn_parts(*desc));
  a.lse2 = a.delta + a.hq * a.n_q;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? attn_backward<__bf16>(a, st) : attn_backward<float>(a, st),
      "attention backward launch");
}

size_t ipttt_attention_step_workspace_bytes(const ipttt_step_desc *desc, const ipttt_kv_cache *cache,
                                            const ipttt_page_table *table) {
  ipttt_kv_cache sizes;
  if (!desc || !cache || !table) return 0;
  sizes = *cache;
  sizes.pages = 0;  // its pointers are not looked at
  if (check_step_sizes(desc, &sizes, table, false) != IPTTT_OK) return 0;
  return step_workspace(desc->q_heads, *cache, *table);
}

ipttt_status ipttt_attention_step(const ipttt_step_desc *desc, const ipttt_heads *q,
                                  const ipttt_kv_cache *cache, const ipttt_page_table *table,
                                  const int32_t *lens, const ipttt_heads *o, float *lse,
                                  void *workspace, size_t workspace_bytes, void *hip_stream) {
  TRY(check_step_sizes(desc, cache, table, true));
  if (table->batch == 0) return IPTTT_OK;
  const int n = table->batch;
  TRY(check_heads(q, n, desc->q_heads, cache->head_dim, cache->dtype, "q"));
  TRY(check_heads(o, n, desc->q_heads, cache->head_dim, cache->dtype, "o"));
  TRY(check_ptr(lens, 4, "lens"));
  TRY(check_opt(lse, 4, "lse"));
  TRY(check_workspace(workspace, workspace_bytes,
                      step_workspace(desc->q_heads, *cache, *table)));
  StepArgs a{};
  a.hq = desc->q_heads;
  a.window = desc->window;
  a.scale = desc->scale;
  a.q = view(q, n, a.hq);
  a.o = view(o, n, a.hq);
  a.cache = *cache;
  a.table = *table;
  a.lens = lens;
  a.lse = lse;
  a.ws = workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      cache->dtype == IPTTT_BF16 ? step_forward<__bf16>(a, st) : step_forward<float>(a, st),
      "attention step launch");
}

}  // extern "C"
