// Host side of the block operators (include/ipttt_block.h): argument checks,
// workspace planning and launches. Kernels live in kernels_norm.hip,
// kernels_recurrence.hip and kernels_ff.hip.
#include <stdarg.h>
#include <stdio.h>

#include "block_internal.h"

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
// A pointer that may be NULL.
ipttt_status check_opt(const void *p, size_t align, const char *name) {
  return p ? check_ptr(p, align, name) : IPTTT_OK;
}
ipttt_status check_stride(int64_t stride, int64_t width, int64_t rows, const char *name) {
  if (rows > 1 && stride < width)
    return fail(IPTTT_E_INVALID, "%s stride %lld is below the row width %lld", name,
                (long long)stride, (long long)width);
  if (rows > 1 && stride > kMaxElems / rows)
    return fail(IPTTT_E_INVALID, "%s stride %lld is too large", name, (long long)stride);
  return IPTTT_OK;
}
ipttt_status check_workspace(const void *ws, size_t have, size_t need) {
  TRY(check_ptr(ws, 256, "workspace"));
  if (have < need)
    return fail(IPTTT_E_WORKSPACE, "workspace_bytes=%zu below the %zu this call needs", have, need);
  return IPTTT_OK;
}

// ---- layer norm -----------------------------------------------------------------

ipttt_status check_norm(const ipttt_norm_desc *d, int64_t n) {
  if (!d) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_dtype(d->dtype));
  if (d->d < 1) return fail(IPTTT_E_INVALID, "d=%d must be > 0", d->d);
  if (d->d > kNormMaxD) return fail(IPTTT_E_UNSUPPORTED, "d=%d exceeds %d", d->d, kNormMaxD);
  if (!(d->eps >= 0.f) || d->eps > 3.0e38f)
    return fail(IPTTT_E_INVALID, "eps must be finite and >= 0");
  if (n < 0) return fail(IPTTT_E_INVALID, "n=%lld must be >= 0", (long long)n);
  if (n > ((int64_t)1 << 31) - 1)
    return fail(IPTTT_E_UNSUPPORTED, "n=%lld exceeds 2^31 - 1", (long long)n);
  TRY(check_opt(d->gamma, size_of(d->dtype), "gamma"));
  return check_opt(d->beta, size_of(d->dtype), "beta");
}

NormArgs norm_args(const ipttt_norm_desc *d, int64_t n) {
  NormArgs a{};
  a.d = d->d;
  a.n = n;
  a.eps = d->eps;
  a.gamma = d->gamma;
  a.beta = d->beta;
  return a;
}

// ---- recurrence -------------------------------------------------------------------

ipttt_status check_rec_sizes(const ipttt_recurrence *r) {
  if (!r) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_dtype(r->dtype));
  if (r->d < 1) return fail(IPTTT_E_INVALID, "d=%d must be > 0", r->d);
  if (r->d > (1 << 16)) return fail(IPTTT_E_UNSUPPORTED, "d=%d exceeds 65536", r->d);
  if (r->batch < 0) return fail(IPTTT_E_INVALID, "batch=%d must be >= 0", r->batch);
  if (r->batch > 65535) return fail(IPTTT_E_UNSUPPORTED, "batch=%d exceeds 65535", r->batch);
  if (r->seq_len < 0)
    return fail(IPTTT_E_INVALID, "seq_len=%lld must be >= 0", (long long)r->seq_len);
  if (r->seq_len > ((int64_t)1 << 30))
    return fail(IPTTT_E_UNSUPPORTED, "seq_len=%lld exceeds 2^30", (long long)r->seq_len);
  if (!rec_size_ok(r->batch, r->d, r->seq_len))
    return fail(IPTTT_E_UNSUPPORTED, "batch=%d x seq_len=%lld x d=%d exceed 2^31 tiles", r->batch,
                (long long)r->seq_len, r->d);
  return IPTTT_OK;
}

ipttt_status check_view(const ipttt_recurrence *r, const ipttt_view *w, const char *name) {
  if (!w) return fail(IPTTT_E_INVALID, "%s is NULL", name);
  if (r->seq_len == 0) return IPTTT_OK;  // no element
  TRY(check_ptr(w->p, size_of(r->dtype), name));
  TRY(check_stride(w->tok_stride, r->d, r->seq_len, name));
  // sequences may interleave with tokens (a token-major batch), so their
  // stride is at least a row, like the tokens'
  return check_stride(w->seq_stride, r->d, r->batch, name);
}

// Everything the forward, step and backward share.
ipttt_status check_rec(const ipttt_recurrence *r) {
  TRY(check_rec_sizes(r));
  if (r->batch == 0) return IPTTT_OK;
  TRY(check_view(r, &r->g, "g"));
  TRY(check_view(r, &r->v, "v"));
  TRY(check_view(r, &r->h, "h"));
  TRY(check_opt(r->lens, 4, "lens"));
  return check_opt(r->h0, 4, "h0");
}

RecArgs rec_args(const ipttt_recurrence *r) {
  RecArgs a{};
  a.n = r->batch;
  a.d = r->d;
  a.L = r->seq_len;
  a.g = r->g;
  a.v = r->v;
  a.h = r->h;
  a.starts = r->starts;
  a.lens = r->lens;
  a.h0 = r->h0;
  return a;
}

// ---- gated feed-forward block --------------------------------------------------------

ipttt_status check_ff_sizes(const ipttt_ff_desc *d, int64_t n) {
  if (!d) return fail(IPTTT_E_INVALID, "descriptor is NULL");
  TRY(check_dtype(d->dtype));
  if (d->d < 1 || d->d_ff < 1)
    return fail(IPTTT_E_INVALID, "d=%d d_ff=%d must be > 0", d->d, d->d_ff);
  if (d->d > (1 << 16) || d->d_ff > (1 << 18))
    return fail(IPTTT_E_UNSUPPORTED, "d=%d d_ff=%d exceed 65536 / 262144", d->d, d->d_ff);
  if (n < 0) return fail(IPTTT_E_INVALID, "n=%lld must be >= 0", (long long)n);
  if (n > (1 << 24)) return fail(IPTTT_E_UNSUPPORTED, "n=%lld exceeds 2^24", (long long)n);
  return IPTTT_OK;
}

ipttt_status check_ff(const ipttt_ff_desc *d, int64_t n) {
  TRY(check_ff_sizes(d, n));
  TRY(check_ptr(d->w_gate, 16, "w_gate"));
  TRY(check_ptr(d->w_up, 16, "w_up"));
  return check_ptr(d->w_down, 16, "w_down");
}

FfArgs ff_args(const ipttt_ff_desc *d, int64_t n) {
  FfArgs a{};
  a.d = d->d;
  a.F = d->d_ff;
  a.n = n;
  a.w_gate = d->w_gate;
  a.w_up = d->w_up;
  a.w_down = d->w_down;
  return a;
}

bool ff_sizes_ok(const ipttt_ff_desc *d, int64_t n) {
  return d && d->d >= 1 && d->d_ff >= 1 && d->d <= (1 << 16) && d->d_ff <= (1 << 18) && n >= 0 &&
         n <= (1 << 24) && (d->dtype == IPTTT_F32 || d->dtype == IPTTT_BF16);
}

}  // namespace

extern "C" {

size_t ipttt_ff_workspace_bytes(const ipttt_ff_desc *desc, int64_t n) {
  if (!ff_sizes_ok(desc, n)) return 0;
  return ff_forward_workspace((int)size_of(desc->dtype), desc->d, desc->d_ff, n);
}

ipttt_status ipttt_ff_forward(const ipttt_ff_desc *desc, const void *x, int64_t x_stride,
                              int64_t n, void *y, int64_t y_stride, float *a, float *u,
                              void *workspace, size_t workspace_bytes, void *hip_stream) {
  TRY(check_ff(desc, n));
  const size_t el = size_of(desc->dtype);
  if (!a != !u) return fail(IPTTT_E_INVALID, "a and u must both be given or both be NULL");
  if (n == 0) return IPTTT_OK;
  TRY(check_ptr(x, el, "x"));
  TRY(check_ptr(y, el, "y"));
  TRY(check_opt(a, 16, "a"));
  TRY(check_opt(u, 16, "u"));
  TRY(check_stride(x_stride, desc->d, n, "x"));
  TRY(check_stride(y_stride, desc->d, n, "y"));
  TRY(check_workspace(workspace, workspace_bytes, ipttt_ff_workspace_bytes(desc, n)));
  FfArgs p = ff_args(desc, n);
  p.x = x;
  p.x_stride = x_stride;
  p.y = y;
  p.y_stride = y_stride;
  p.a = a;
  p.u = u;
  p.ws = workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(desc->dtype == IPTTT_BF16 ? ff_forward<__bf16>(p, st) : ff_forward<float>(p, st),
                  "feed-forward launch");
}

size_t ipttt_ff_backward_workspace_bytes(const ipttt_ff_desc *desc, int64_t n) {
  if (!ff_sizes_ok(desc, n)) return 0;
  return ff_backward_workspace((int)size_of(desc->dtype), desc->d, desc->d_ff, n);
}

ipttt_status ipttt_ff_backward(const ipttt_ff_desc *desc, const void *x, int64_t x_stride,
                               const float *a, const float *u, const void *dy, int64_t dy_stride,
                               int64_t n, const ipttt_ff_grads *grads, void *workspace,
                               size_t workspace_bytes, void *hip_stream) {
  TRY(check_ff(desc, n));
  const size_t el = size_of(desc->dtype);
  if (!grads) return fail(IPTTT_E_INVALID, "grads is NULL");
  TRY(check_ptr(grads->dw_gate, 16, "dw_gate"));
  TRY(check_ptr(grads->dw_up, 16, "dw_up"));
  TRY(check_ptr(grads->dw_down, 16, "dw_down"));
  if (n > 0) {
    TRY(check_ptr(x, el, "x"));
    TRY(check_ptr(a, 16, "a"));
    TRY(check_ptr(u, 16, "u"));
    TRY(check_ptr(dy, el, "dy"));
    TRY(check_ptr(grads->dx, el, "dx"));
    TRY(check_stride(x_stride, desc->d, n, "x"));
    TRY(check_stride(dy_stride, desc->d, n, "dy"));
    TRY(check_stride(grads->dx_stride, desc->d, n, "dx"));
    TRY(check_workspace(workspace, workspace_bytes, ipttt_ff_backward_workspace_bytes(desc, n)));
  }
  FfArgs p = ff_args(desc, n);
  p.x = x;
  p.x_stride = x_stride;
  p.a = const_cast<float *>(a);
  p.u = const_cast<float *>(u);
  p.dy = dy;
  p.dy_stride = dy_stride;
  p.dx = grads->dx;
  p.dx_stride = grads->dx_stride;
  p.dw_gate = grads->dw_gate;
  p.dw_up = grads->dw_up;
  p.dw_down = grads->dw_down;
  p.ws = workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(desc->dtype == IPTTT_BF16 ? ff_backward<__bf16>(p, st) : ff_backward<float>(p, st),
                  "feed-forward backward launch");
}

ipttt_status ipttt_norm_forward(const ipttt_norm_desc *desc, const void *x, int64_t x_stride,
                                const void *r, int64_t r_stride, int64_t n, void *h, void *y,
                                float *mean, float *rstd, void *hip_stream) {
  TRY(check_norm(desc, n));
  const size_t el = size_of(desc->dtype);
  if (!r != !h) return fail(IPTTT_E_INVALID, "r and h must both be given or both be NULL");
  if (!mean != !rstd) return fail(IPTTT_E_INVALID, "mean and rstd must both be given or both be NULL");
  if (n == 0) return IPTTT_OK;
  TRY(check_ptr(x, el, "x"));
  TRY(check_ptr(y, el, "y"));
  TRY(check_opt(r, el, "r"));
  TRY(check_opt(h, el, "h"));
  TRY(check_opt(mean, 4, "mean"));
  TRY(check_opt(rstd, 4, "rstd"));
  TRY(check_stride(x_stride, desc->d, n, "x"));
  if (r) TRY(check_stride(r_stride, desc->d, n, "r"));
  NormArgs a = norm_args(desc, n);
  a.x = x;
  a.x_stride = x_stride;
  a.r = r;
  a.r_stride = r_stride;
  a.h = h;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(desc->dtype == IPTTT_BF16 ? norm_forward<__bf16>(a, st) : norm_forward<float>(a, st),
                  "norm forward launch");
}

size_t ipttt_norm_backward_workspace_bytes(const ipttt_norm_desc *desc, int64_t n) {
  if (!desc || desc->d < 1 || desc->d > kNormMaxD || n < 0) return 0;
  return (size_t)round_up((int64_t)norm_bwd_blocks(desc->d, n) * 2 * desc->d * 4, 256);
}

ipttt_status ipttt_norm_backward(const ipttt_norm_desc *desc, const void *h, int64_t h_stride,
                                 const float *mean, const float *rstd, const void *dy,
                                 int64_t dy_stride, const void *dh, int64_t dh_stride, int64_t n,
                                 void *dx, float *dgamma, float *dbeta, void *workspace,
                                 size_t workspace_bytes, void *hip_stream) {
  TRY(check_norm(desc, n));
  const size_t el = size_of(desc->dtype);
  TRY(check_opt(dgamma, 4, "dgamma"));
  TRY(check_opt(dbeta, 4, "dbeta"));
  if (n == 0 && !dgamma && !dbeta) return IPTTT_OK;
  if (n > 0) {
    TRY(check_ptr(h, el, "h"));
    TRY(check_ptr(mean, 4, "mean"));
    TRY(check_ptr(rstd, 4, "rstd"));
    TRY(check_ptr(dy, el, "dy"));
    TRY(check_opt(dh, el, "dh"));
    TRY(check_ptr(dx, el, "dx"));
    TRY(check_stride(h_stride, desc->d, n, "h"));
    TRY(check_stride(dy_stride, desc->d, n, "dy"));
    if (dh) TRY(check_stride(dh_stride, desc->d, n, "dh"));
  }
  const bool sums = dgamma || dbeta;
  if (sums)
    TRY(check_workspace(workspace, workspace_bytes, ipttt_norm_backward_workspace_bytes(desc, n)));
  NormArgs a = norm_args(desc, n);
  a.x = h;
  a.x_stride = h_stride;
  a.r = dh;
  a.r_stride = dh_stride;
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.y = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = sums ? (float *)workspace : nullptr;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(
      desc->dtype == IPTTT_BF16 ? norm_backward<__bf16>(a, st) : norm_backward<float>(a, st),
      "norm backward launch");
}

size_t ipttt_recurrence_workspace_bytes(const ipttt_recurrence *r) {
  if (!r || r->d < 1 || r->d > (1 << 16) || r->batch < 0 || r->batch > 65535 || r->seq_len < 0 ||
      r->seq_len > ((int64_t)1 << 30) || !rec_size_ok(r->batch, r->d, r->seq_len) || (r->dtype != IPTTT_F32 && r->dtype != IPTTT_BF16))
    return 0;
  return rec_workspace(r->batch, r->d, r->seq_len);
}

ipttt_status ipttt_recurrence_forward(const ipttt_recurrence *r, float *h_last, void *workspace,
                                      size_t workspace_bytes, void *hip_stream) {
  TRY(check_rec(r));
  if (r->batch == 0) return IPTTT_OK;
  TRY(check_opt(h_last, 4, "h_last"));
  if (h_last && h_last == r->h0) return fail(IPTTT_E_INVALID, "h_last must not be h0");
  TRY(check_workspace(workspace, workspace_bytes, ipttt_recurrence_workspace_bytes(r)));
  RecArgs a = rec_args(r);
  a.h_last = h_last;
  a.ws = workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(r->dtype == IPTTT_BF16 ? rec_forward<__bf16>(a, st) : rec_forward<float>(a, st),
                  "recurrence forward launch");
}

ipttt_status ipttt_recurrence_step(const ipttt_recurrence *r, float *state, void *hip_stream) {
  TRY(check_rec(r));
  if (r->seq_len != 1)
    return fail(IPTTT_E_INVALID, "seq_len=%lld must be 1 in a step", (long long)r->seq_len);
  if (r->batch == 0) return IPTTT_OK;
  TRY(check_ptr(state, 4, "state"));
  RecArgs a = rec_args(r);
  a.h_last = state;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(r->dtype == IPTTT_BF16 ? rec_step<__bf16>(a, st) : rec_step<float>(a, st),
                  "recurrence step launch");
}

ipttt_status ipttt_recurrence_backward(const ipttt_recurrence *r, const ipttt_view *dh,
                                       const float *dh_last, const ipttt_view *dg,
                                       const ipttt_view *dv, float *dh0, void *workspace,
                                       size_t workspace_bytes, void *hip_stream) {
  TRY(check_rec(r));
  if (r->batch == 0) return IPTTT_OK;
  TRY(check_view(r, dh, "dh"));
  TRY(check_view(r, dg, "dg"));
  TRY(check_view(r, dv, "dv"));
  TRY(check_opt(dh_last, 4, "dh_last"));
  TRY(check_opt(dh0, 4, "dh0"));
  if (dh0 && (dh0 == dh_last || dh0 == r->h0))
    return fail(IPTTT_E_INVALID, "dh0 must not be dh_last or h0");
  TRY(check_workspace(workspace, workspace_bytes, ipttt_recurrence_workspace_bytes(r)));
  RecArgs a = rec_args(r);
  a.dh = *dh;
  a.dg = *dg;
  a.dv = *dv;
  a.dh_last = dh_last;
  a.dh0 = dh0;
  a.ws = workspace;
  const hipStream_t st = (hipStream_t)hip_stream;
  return launched(r->dtype == IPTTT_BF16 ? rec_backward<__bf16>(a, st) : rec_backward<float>(a, st),
                  "recurrence backward launch");
}

}  // extern "C"
