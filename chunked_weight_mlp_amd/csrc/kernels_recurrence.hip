// The gated linear recurrence h_t = f_t h_{t-1} + (1 - f_t) v_t, f = sigmoid(g),
// forward and backward.
#include <algorithm>

#include "block_internal.h"

namespace ipttt {
namespace {

using blk::Pack;

// f = 1 / (1 + e^-x) and i = 1 - f = 1 / (1 + e^x), each to a few ulp: for x > 0
// i is e^-x f (1 - f would cancel), else it is 1 - f (e^-x may overflow).
__device__ __forceinline__ void gate(float x, float &f, float &i) {
  const float e = __expf(-x);
  f = __builtin_amdgcn_rcpf(1.f + e);
  i = x > 0.f ? e * f : 1.f - f;
}

// V channels from channel c of a row; channels at or past d read as zero.
template <typename T, int V>
__device__ __forceinline__ void load_ch(const T *row, int c, int d, float (&v)[V]) {
  if (c + V <= d) {
    blk::load_pack<T, V>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = c + e < d ? (float)row[c + e] : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_ch(T *row, int c, int d, const float (&v)[V]) {
  if (c + V <= d) {
    blk::store_pack<T, V>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < d) row[c + e] = (T)v[e];
  }
}

template <typename T>
__device__ __forceinline__ T *seq_of(const ipttt_view &w, int n) {
  return (T *)w.p + n * w.seq_stride;
}

__device__ __forceinline__ int64_t seq_length(const RecArgs &a, int n) {
  return a.lens ? min(max((int64_t)a.lens[n], (int64_t)0), a.L) : a.L;
}

// One thread walks V channels of one sequence from its first token to its last,
// U tokens' loads in flight.
constexpr int SEQ_V = 2, SEQ_U = 8;

template <typename T>
__global__ __launch_bounds__(64) void k_rec_seq_fwd(RecArgs a) {
  const int c = SEQ_V * (blockIdx.x * 64 + threadIdx.x), n = blockIdx.y;
  if (c >= a.d) return;
  const int64_t len = seq_length(a, n);
  const T *g = seq_of<T>(a.g, n), *v = seq_of<T>(a.v, n);
  T *h = seq_of<T>(a.h, n);
  float s[SEQ_V] = {};
  if (a.h0) load_ch<float, SEQ_V>(a.h0 + (int64_t)n * a.d, c, a.d, s);
  for (int64_t t0 = 0; t0 < len; t0 += SEQ_U) {
    float gv[SEQ_U][SEQ_V], vv[SEQ_U][SEQ_V];
    bool cut[SEQ_U];
#pragma unroll
    for (int u = 0; u < SEQ_U; ++u) {
      const int64_t t = min(t0 + u, len - 1);
      load_ch<T, SEQ_V>(g + t * a.g.tok_stride, c, a.d, gv[u]);
      load_ch<T, SEQ_V>(v + t * a.v.tok_stride, c, a.d, vv[u]);
      cut[u] = a.starts && a.starts[n * a.L + t] != 0;
    }
#pragma unroll
    for (int u = 0; u < SEQ_U; ++u) {
      if (t0 + u >= len) break;
#pragma unroll
      for (int e = 0; e < SEQ_V; ++e) {
        float f, i;
        gate(gv[u][e], f, i);
        const float b = i * vv[u][e];
        s[e] = cut[u] ? b : fmaf(f, s[e], b);
      }
      store_ch<T, SEQ_V>(h + (t0 + u) * a.h.tok_stride, c, a.d, s);
    }
  }
  if (a.h_last) store_ch<float, SEQ_V>(a.h_last + (int64_t)n * a.d, c, a.d, s);
  const float zero[SEQ_V] = {};
  for (int64_t t = len; t < a.L; ++t) store_ch<T, SEQ_V>(h + t * a.h.tok_stride, c, a.d, zero);
}

template <typename T>
__global__ __launch_bounds__(64) void k_rec_seq_bwd(RecArgs a) {
  const int c = SEQ_V * (blockIdx.x * 64 + threadIdx.x), n = blockIdx.y;
  if (c >= a.d) return;
  const int64_t len = seq_length(a, n);
  const T *g = seq_of<T>(a.g, n), *v = seq_of<T>(a.v, n), *h = seq_of<T>(a.h, n);
  const T *dh = seq_of<T>(a.dh, n);
  T *dg = seq_of<T>(a.dg, n), *dv = seq_of<T>(a.dv, n);
  float h0[SEQ_V] = {}, s[SEQ_V] = {};  // s: gradient of the state after token t
  if (a.h0) load_ch<float, SEQ_V>(a.h0 + (int64_t)n * a.d, c, a.d, h0);
  if (a.dh_last) load_ch<float, SEQ_V>(a.dh_last + (int64_t)n * a.d, c, a.d, s);
  const float zero[SEQ_V] = {};
  for (int64_t t = a.L - 1; t >= len; --t) {
    store_ch<T, SEQ_V>(dg + t * a.dg.tok_stride, c, a.d, zero);
    store_ch<T, SEQ_V>(dv + t * a.dv.tok_stride, c, a.d, zero);
  }
  for (int64_t t0 = len - 1; t0 >= 0; t0 -= SEQ_U) {
    float gv[SEQ_U][SEQ_V], vv[SEQ_U][SEQ_V], hp[SEQ_U][SEQ_V], dd[SEQ_U][SEQ_V];
    bool cut[SEQ_U];
#pragma unroll
    for (int u = 0; u < SEQ_U; ++u) {
      const int64_t t = max(t0 - u, (int64_t)0);
      load_ch<T, SEQ_V>(g + t * a.g.tok_stride, c, a.d, gv[u]);
      load_ch<T, SEQ_V>(v + t * a.v.tok_stride, c, a.d, vv[u]);
      load_ch<T, SEQ_V>(dh + t * a.dh.tok_stride, c, a.d, dd[u]);
      load_ch<T, SEQ_V>(h + max(t - 1, (int64_t)0) * a.h.tok_stride, c, a.d, hp[u]);
      cut[u] = a.starts && a.starts[n * a.L + t] != 0;
    }
#pragma unroll
    for (int u = 0; u < SEQ_U; ++u) {
      const int64_t t = t0 - u;
      if (t < 0) break;
      float og[SEQ_V], ov[SEQ_V];
#pragma unroll
      for (int e = 0; e < SEQ_V; ++e) {
        float f, i;
        gate(gv[u][e], f, i);
        const float prev = cut[u] ? 0.f : t == 0 ? h0[e] : hp[u][e];
        const float delta = dd[u][e] + s[e];
        ov[e] = i * delta;
        og[e] = delta * (prev - vv[u][e]) * (f * i);
        s[e] = cut[u] ? 0.f : f * delta;
      }
      store_ch<T, SEQ_V>(dg + t * a.dg.tok_stride, c, a.d, og);
      store_ch<T, SEQ_V>(dv + t * a.dv.tok_stride, c, a.d, ov);
    }
  }
  if (a.dh0) store_ch<float, SEQ_V>(a.dh0 + (int64_t)n * a.d, c, a.d, s);
}

}  // namespace

size_t rec_workspace(int, int, int64_t) { return 256; }

template <typename T>
hipError_t rec_step(const RecArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_rec_seq_fwd<T>, dim3((a.d + 64 * SEQ_V - 1) / (64 * SEQ_V), a.n), dim3(64), 0,
                     st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t rec_forward(const RecArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_rec_seq_fwd<T>, dim3((a.d + 64 * SEQ_V - 1) / (64 * SEQ_V), a.n), dim3(64), 0,
                     st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t rec_backward(const RecArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_rec_seq_bwd<T>, dim3((a.d + 64 * SEQ_V - 1) / (64 * SEQ_V), a.n), dim3(64), 0,
                     st, a);
  return hipGetLastError();
}

template hipError_t rec_step<float>(const RecArgs &, hipStream_t);
template hipError_t rec_step<__bf16>(const RecArgs &, hipStream_t);
template hipError_t rec_forward<float>(const RecArgs &, hipStream_t);
template hipError_t rec_forward<__bf16>(const RecArgs &, hipStream_t);
template hipError_t rec_backward<float>(const RecArgs &, hipStream_t);
template hipError_t rec_backward<__bf16>(const RecArgs &, hipStream_t);

}  // namespace ipttt
