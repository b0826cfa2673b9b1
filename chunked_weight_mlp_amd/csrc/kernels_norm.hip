// Layer norm, forward (with the residual add) and backward.
//
// Both are bound by HBM: a row is read once, held in registers as fp32, and
// written once. A row of d elements is shared by WPR waves, each lane holding
// NP pieces of 8 consecutive elements. The variance is the mean of the squared
// deviations of the values held, not a difference of moments, so a large mean
// costs no accuracy.
#include <algorithm>

#include "block_internal.h"

namespace ipttt {
namespace {

using blk::load_pack;
using blk::Pack;
using blk::store_pack;
using blk::wave_sum;

// Sum over the WPR waves of a row; every thread of the row gets it. `slot` is a
// different LDS array for consecutive sums, so one barrier per sum is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *slot) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += slot[w];
  }
  return v;
}

// Two sums at once, one barrier.
template <int WPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*slot)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) {
      slot[threadIdx.x >> 6][0] = a;
      slot[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      a += slot[w][0];
      b += slot[w][1];
    }
  }
}

// 8 elements from column c of a row of d; zero at and past d. W: d is a
// multiple of 8, so a piece is whole or absent.
template <typename T, bool W>
__device__ __forceinline__ void load_cols(const T *row, int c, int d, float (&v)[8]) {
  if constexpr (W) {
    load_pack<T, 8>(row + (c < d ? c : 0), v);
    if (c >= d) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  } else if (c + 8 <= d) {
    load_pack<T, 8>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < d ? (float)row[c + e] : 0.f;
  }
}
template <typename T, bool W>
__device__ __forceinline__ void store_cols(T *row, int c, int d, const float (&v)[8]) {
  if (c + 8 <= d) {
    store_pack<T, 8>(row + c, v);
  } else if constexpr (!W) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < d) row[c + e] = (T)v[e];
  }
}

template <typename T, int WPR, int NP, bool W>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs a) {
  __shared__ float red[2][WPR];
  constexpr int RB = 4 / WPR;  // rows per block
  constexpr int TPR = 64 * WPR;
  const int tr = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RB + threadIdx.x / TPR;
  if (row >= a.n) return;  // whole rows: with WPR > 1 the block is one row
  const int d = a.d;
  const T *x = (const T *)a.x + row * a.x_stride;
  float h[NP][8];
#pragma unroll
  for (int p = 0; p < NP; ++p) load_cols<T, W>(x, 8 * (TPR * p + tr), d, h[p]);
  if (a.r) {
    const T *r = (const T *)a.r + row * a.r_stride;
    T *ho = (T *)a.h + row * d;
    float q[NP][8];
#pragma unroll
    for (int p = 0; p < NP; ++p) load_cols<T, W>(r, 8 * (TPR * p + tr), d, q[p]);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[p][e] += q[p][e];
      store_cols<T, W>(ho, 8 * (TPR * p + tr), d, h[p]);
    }
  }
  float s = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += h[p][e];
  const float mean = row_sum<WPR>(s, red[0]) / (float)d;
  s = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[p][e] -= mean;
      if (8 * (TPR * p + tr) + e < d) s = fmaf(h[p][e], h[p][e], s);
    }
  const float rstd = rsqrtf(row_sum<WPR>(s, red[1]) / (float)d + a.eps);
  if (a.mean && tr == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T *y = (T *)a.y + row * d;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = 8 * (TPR * p + tr);
    float g[8], b[8];
    if (a.gamma) {
      load_cols<T, W>((const T *)a.gamma, c, d, g);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = 1.f;
    }
    if (a.beta) {
      load_cols<T, W>((const T *)a.beta, c, d, b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[p][e] = fmaf(h[p][e] * rstd, g[e], b[e]);
    store_cols<T, W>(y, c, d, h[p]);
  }
}

// 8 columns as they are stored, from column c of a row of d; zero at and past d.
template <typename T, bool W>
__device__ __forceinline__ Pack<T, 8> raw_cols(const T *row, int c, int d) {
  if constexpr (W) {
    Pack<T, 8> p = *(const Pack<T, 8> *)(row + (c < d ? c : 0));
    if (c >= d) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p.v[e] = (T)0.f;
    }
    return p;
  } else {
    if (c + 8 <= d) return *(const Pack<T, 8> *)(row + c);
    Pack<T, 8> p;
#pragma unroll
    for (int e = 0; e < 8; ++e) p.v[e] = c + e < d ? row[c + e] : (T)0.f;
    return p;
  }
}

// One row of the backward as it is stored.
template <typename T, int NP>
struct BwdRow {
  Pack<T, 8> h[NP], dy[NP], dh[NP];
  float mean, rstd;
};
template <typename T, int TPR, int NP, bool W>
__device__ __forceinline__ void load_row(const NormArgs &a, int64_t row, int tr, BwdRow<T, NP> &r) {
  const T *h = (const T *)a.x + row * a.x_stride, *dy = (const T *)a.dy + row * a.dy_stride;
  const T *dh = (const T *)a.r + row * a.r_stride;
  r.mean = a.mean[row];
  r.rstd = a.rstd[row];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    r.h[p] = raw_cols<T, W>(h, 8 * (TPR * p + tr), a.d);
    r.dy[p] = raw_cols<T, W>(dy, 8 * (TPR * p + tr), a.d);
  }
  if (a.r) {
#pragma unroll
    for (int p = 0; p < NP; ++p) r.dh[p] = raw_cols<T, W>(dh, 8 * (TPR * p + tr), a.d);
  }
}

// A block walks rows blockIdx, blockIdx + gridDim, ... (RB at a time) and keeps
// its columns' sums of dy xh and dy in registers; its waves' sums meet in LDS
// once at the end and go to part[block], which k_norm_sums adds in a fixed order.
// All of a row's loads are issued together, dh's too, which is used last: 131072
// x 2048 bf16 in 412 us, 5.2 TB/s (686 us with dh loaded where it is used).
template <typename T, int WPR, int NP, bool W>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void k_norm_bwd(NormArgs a) {
  constexpr int RB = WPR > 4 ? 1 : 4 / WPR;
  constexpr int TPR = 64 * WPR;
  __shared__ float red[2][WPR][2];
  __shared__ float comb[RB > 1 ? (RB - 1) * TPR * 8 : 1];
  const int tr = threadIdx.x % TPR;
  const int rb = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const int d = a.d;
  float dg[NP][8], db[NP][8];
  Pack<T, 8> gamma[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (a.gamma) gamma[p] = raw_cols<T, W>((const T *)a.gamma, 8 * (TPR * p + tr), d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dg[p][e] = db[p][e] = 0.f;
      if (!a.gamma) gamma[p].v[e] = (T)1.f;
    }
  }
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * RB + rb; row < a.n; row += (int64_t)gridDim.x * RB) {
    BwdRow<T, NP> cur;
    load_row<T, TPR, NP, W>(a, row, tr, cur);
    const float mean = cur.mean, rstd = cur.rstd;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // past the row dy is zero (xh is not)
        const float y = (float)cur.dy[p].v[e], xh = ((float)cur.h[p].v[e] - mean) * rstd;
        dg[p][e] = fmaf(y, xh, dg[p][e]);
        db[p][e] += y;
        const float q = y * (float)gamma[p].v[e];
        s0 += q;
        s1 = fmaf(q, xh, s1);
      }
    row_sum2<WPR>(s0, s1, red[par]);
    const float c0 = s0 / (float)d, c1 = s1 / (float)d;
    par ^= 1;
    T *dx = (T *)a.y + row * d;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = (float)cur.dy[p].v[e] * (float)gamma[p].v[e];
        const float xh = ((float)cur.h[p].v[e] - mean) * rstd;
        o[e] = fmaf(q - c0 - xh * c1, rstd, a.r ? (float)cur.dh[p].v[e] : 0.f);
      }
      store_cols<T, W>(dx, 8 * (TPR * p + tr), d, o);
    }
  }
  if (!a.part) return;
  float *part = a.part + (int64_t)blockIdx.x * 2 * d;
  const auto put = [&](float (&v)[NP][8], float *out) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      if constexpr (RB > 1) {
        __syncthreads();
        if (rb > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) comb[((rb - 1) * 8 + e) * TPR + tr] = v[p][e];
        }
        __syncthreads();
        if (rb == 0) {
#pragma unroll
          for (int w = 0; w < RB - 1; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[p][e] += comb[(w * 8 + e) * TPR + tr];
        }
      }
      if (rb == 0) {
        const int c = 8 * (TPR * p + tr);
        store_cols<float, W>(out, c, d, v[p]);
      }
    }
  };
  put(dg, part);
  put(db, part + d);
}

// dgamma and dbeta: column sums of the nb partial rows [nb][2][d]. A block owns
// 64 columns; its 16 waves take interleaved rows and meet in LDS.
__global__ __launch_bounds__(1024) void k_norm_sums(const float *__restrict__ part, int nb, int d,
                                                    float *__restrict__ dgamma,
                                                    float *__restrict__ dbeta) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float *out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int c = blockIdx.x * 64 + lane;
  const float *src = part + blockIdx.y * d + min(c, d - 1);
  float s = 0.f;
#pragma unroll 8
  for (int b = wave; b < nb; b += 16) s += src[(int64_t)b * 2 * d];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += red[w][lane];
    out[c] = t;
  }
}

// Waves a row is spread over. Forward: one wave to 4096 columns, four beyond;
// with too few rows to fill the GPU a row takes four waves from 1024 columns on.
int fwd_waves(int d, int64_t n) { return d > 4096 || (d >= 1024 && n <= 2048) ? 4 : 1; }
// Backward: a lane also holds its columns' sums, so a wave takes 2560 columns at
// most, and each wave should walk several rows per sum it writes (one wave a row
// against four: 131072 x 2048 412 and 419 us, 65536 x 2560 276 and 318, 4096 x
// 2560 44 and 27). Rows of odd width, whose tails take branches, run better on
// four (32768 x 2047: 177 and 146 us).
int bwd_waves(int d, int64_t n) {
  if (d > 8192) return 8;
  return d > 2560 || (d > 512 && (n < 16384 || d % 8)) ? 4 : 1;
}

template <typename T, int WPR, int NP>
hipError_t fwd_launch(const NormArgs &a, hipStream_t st) {
  constexpr int RB = 4 / WPR;
  const unsigned grid = (unsigned)((a.n + RB - 1) / RB);
  const dim3 block(256);
  if (a.d % 8 == 0)
    hipLaunchKernelGGL((k_norm_fwd<T, WPR, NP, true>), dim3(grid), block, 0, st, a);
  else
    hipLaunchKernelGGL((k_norm_fwd<T, WPR, NP, false>), dim3(grid), block, 0, st, a);
  return hipGetLastError();
}
template <typename T, int WPR, int NP>
hipError_t bwd_launch(const NormArgs &a, hipStream_t st) {
  const unsigned grid = (unsigned)norm_bwd_blocks(a.d, a.n);
  const dim3 block(WPR > 4 ? 64 * WPR : 256);
  if (a.d % 8 == 0)
    hipLaunchKernelGGL((k_norm_bwd<T, WPR, NP, true>), dim3(grid), block, 0, st, a);
  else
    hipLaunchKernelGGL((k_norm_bwd<T, WPR, NP, false>), dim3(grid), block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

int norm_bwd_blocks(int d, int64_t n) {
  const int w = bwd_waves(d, n), rb = w == 1 ? 4 : 1, most = w == 8 ? 512 : 1024;
  return (int)std::max<int64_t>(1, std::min<int64_t>((n + rb - 1) / rb, most));
}

#define PIECES(WPR, F)                                   \
  switch (np) {                                          \
    case 1: return F<T, WPR, 1>(a, st);                  \
    case 2: return F<T, WPR, 2>(a, st);                  \
    case 3: return F<T, WPR, 3>(a, st);                  \
    case 4: return F<T, WPR, 4>(a, st);

template <typename T>
hipError_t norm_forward(const NormArgs &a, hipStream_t st) {
  const int wpr = fwd_waves(a.d, a.n), np = (a.d + 512 * wpr - 1) / (512 * wpr);
  if (wpr == 1) {
    PIECES(1, fwd_launch)
      case 5: return fwd_launch<T, 1, 5>(a, st);
      case 6: return fwd_launch<T, 1, 6>(a, st);
      case 7: return fwd_launch<T, 1, 7>(a, st);
      default: return fwd_launch<T, 1, 8>(a, st);
    }
  }
  PIECES(4, fwd_launch)
    case 5: return fwd_launch<T, 4, 5>(a, st);
    case 6: return fwd_launch<T, 4, 6>(a, st);
    case 7: return fwd_launch<T, 4, 7>(a, st);
    default: return fwd_launch<T, 4, 8>(a, st);
  }
}

template <typename T>
hipError_t norm_backward(const NormArgs &a, hipStream_t st) {
  const int wpr = bwd_waves(a.d, a.n), np = (a.d + 512 * wpr - 1) / (512 * wpr);
  const auto main_pass = [&]() -> hipError_t {
    if (wpr == 1) {
      PIECES(1, bwd_launch)
        default: return bwd_launch<T, 1, 5>(a, st);
      }
    }
    if (wpr == 4) {
      PIECES(4, bwd_launch)
        default: return hipErrorInvalidValue;
      }
    }
    return np <= 3 ? bwd_launch<T, 8, 3>(a, st) : bwd_launch<T, 8, 4>(a, st);
  };
  hipError_t e = main_pass();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(k_norm_sums, dim3((a.d + 63) / 64, 2), dim3(1024), 0, st, a.part,
                     norm_bwd_blocks(a.d, a.n), a.d, a.dgamma, a.dbeta);
  return hipGetLastError();
}
#undef PIECES

template hipError_t norm_forward<float>(const NormArgs &, hipStream_t);
template hipError_t norm_forward<__bf16>(const NormArgs &, hipStream_t);
template hipError_t norm_backward<float>(const NormArgs &, hipStream_t);
template hipError_t norm_backward<__bf16>(const NormArgs &, hipStream_t);

}  // namespace ipttt
