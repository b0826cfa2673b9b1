// Internal declarations of the block operators (include/ipttt_block.h): what the
// host side (block.cpp) and the kernel translation units share. Not part of the
// ABI.
#pragma once

#include "../../include/ipttt_block.h"
#include "internal.h"

namespace ipttt {

// ---- layer norm (kernels_norm.hip) ------------------------------------------
struct NormArgs {
  int d;
  int64_t n;
  float eps;
  const void *gamma, *beta;  // [d] or null
  const void *x, *r;         // forward: x and the added r (or null); backward: h, and dh (or null)
  int64_t x_stride, r_stride;
  const void *dy;            // backward
  int64_t dy_stride;
  void *h, *y;               // forward (h only with r); backward: y is dx
  float *mean, *rstd;        // written by the forward (or null), read by the backward
  float *dgamma, *dbeta;     // [d] or null
  float *part;               // backward: [norm_blocks][2][d] partial sums
};
constexpr int kNormMaxD = 16384;
// Blocks (and rows of partial sums) of the backward.
int norm_bwd_blocks(int d, int64_t n);
template <typename T>
hipError_t norm_forward(const NormArgs &a, hipStream_t st);
template <typename T>
hipError_t norm_backward(const NormArgs &a, hipStream_t st);

// ---- gated linear recurrence (kernels_recurrence.hip) ---------------------------
struct RecArgs {
  int n, d;
  int64_t L;
  ipttt_view g, v, h;
  const uint8_t *starts;  // or null
  const int32_t *lens;    // or null
  const float *h0;        // or null
  float *h_last;          // forward, or null
  ipttt_view dh, dg, dv;  // backward
  const float *dh_last;   // or null
  float *dh0;             // or null
  void *ws;
};
// Whether the tiles of such a call can be launched and counted in 31 bits.
bool rec_size_ok(int n, int d, int64_t L);
size_t rec_workspace(int n, int d, int64_t L);
// One token per sequence (L = 1): state h0 -> h_last, which may be the same.
template <typename T>
hipError_t rec_step(const RecArgs &a, hipStream_t st);
template <typename T>
hipError_t rec_forward(const RecArgs &a, hipStream_t st);
template <typename T>
hipError_t rec_backward(const RecArgs &a, hipStream_t st);

// ---- gated feed-forward block (kernels_ff.hip) -----------------------------------
struct FfArgs {
  int d, F;
  int64_t n;
  const void *w_gate, *w_up, *w_down;
  const void *x;
  int64_t x_stride;
  void *y;  // forward
  int64_t y_stride;
  float *a, *u;    // pre-activations [n][F]: written by the forward (or null), read by the backward
  const void *dy;  // backward
  int64_t dy_stride;
  void *dx;
  int64_t dx_stride;
  void *dw_gate, *dw_up, *dw_down;
  void *ws;
};
// elem: bytes of an element (2: bf16, 4: fp32)
size_t ff_forward_workspace(int elem, int d, int F, int64_t n);
size_t ff_backward_workspace(int elem, int d, int F, int64_t n);
template <typename T>
hipError_t ff_forward(const FfArgs &a, hipStream_t st);
template <typename T>
hipError_t ff_backward(const FfArgs &a, hipStream_t st);

// ---- small helpers -------------------------------------------------------------
#ifdef __HIPCC__
namespace blk {

// A grid of at least `blocks` blocks (a launch takes fewer than 2^32 threads along
// an axis, and rows of a narrow tensor can be more), and a block's place in it.
inline dim3 grid_of(int64_t blocks) {
  const int64_t x = blocks < 1 << 20 ? blocks : 1 << 20;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t block_id() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// N consecutive elements at the alignment of one: rows of odd width or stride
// start anywhere, and the hardware's unaligned access mode serves a wide load
// at any element address.
template <typename T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_pack(const T *p, float (&v)[N]) {
  const Pack<T, N> k = *(const Pack<T, N> *)p;
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = (float)k.v[e];
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T *p, const float (&v)[N]) {
  Pack<T, N> k;
#pragma unroll
  for (int e = 0; e < N; ++e) k.v[e] = (T)v[e];
  *(Pack<T, N> *)p = k;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

}  // namespace blk
#endif

}  // namespace ipttt
