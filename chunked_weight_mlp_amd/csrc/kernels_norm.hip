// Layer norm, forward (with the residual add) and backward.
//
// Both are bound by HBM: a row is read once, held in registers as fp32, and
// written once. A row of d elements is shared by WPR waves, each lane holding
// NP pieces of 8 consecutive elements. The variance is the mean of the squared
// deviations of the values held, not a difference of moments, so a large mean
// costs no accuracy. Forward with the residual add, 32768 x 2560 bf16: 124 us, 5.4 TB/s
// (a large copy reaches 4.8); 8 rows of 2560: 4.7 us, latency.
#include <algorithm>

#include "block_internal.h"

namespace ipttt {
namespace {

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

// Where a lane's NP pieces of a row of d columns are: piece p starts at column
// 8 (TPR p + lane). All but the last are whole; the last may lie past the row's
// end, or (W false: d is no multiple of 8) reach over it. A piece that would reach
// over is taken back to the row's last 8 columns, so that every access stays one
// wide one; the columns it then shares with its neighbour are computed twice, with
// the same results, and counted once (own). Rows of fewer than 8 columns go
// element by element.
template <int TPR, int NP, bool W>
struct Cols {
  int first, d;
  int at, off;  // last piece: its column, the first of its values that is its own
  bool in;      // last piece: whether it has any
  __device__ __forceinline__ Cols(int lane, int d_) : first(8 * lane), d(d_) {
    const int c = 8 * TPR * (NP - 1) + first;
    in = c < d;
    at = W ? (in ? c : 0) : max(min(c, d - 8), 0);
    off = in ? c - at : 8;
  }
  __device__ __forceinline__ int col(int p) const { return p < NP - 1 ? 8 * TPR * p + first : at; }
  __device__ __forceinline__ bool own(int p, int e) const {
    if (p < NP - 1) return true;
    return W ? in : e >= off && at + e < d;
  }
  template <typename T>
  __device__ __forceinline__ Pack<T, 8> load(const T *row, int p) const {
    if (W || p < NP - 1 || d >= 8) return *(const Pack<T, 8> *)(row + col(p));
    Pack<T, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] = e < d ? row[e] : (T)0.f;
    return v;
  }
  template <typename T>
  __device__ __forceinline__ void store(T *row, int p, const float (&v)[8]) const {
    if (p == NP - 1 && !in) return;
    if (W || p < NP - 1 || d >= 8) {
      store_pack<T, 8>(row + col(p), v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < d) row[e] = (T)v[e];
    }
  }
};

template <typename T, int WPR, int NP, bool W>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs a) {
  __shared__ float red[2][WPR];
  constexpr int RB = 4 / WPR;  // rows per block
  constexpr int TPR = 64 * WPR;
  const int tr = threadIdx.x % TPR;
  const int64_t row = blk::block_id() * RB + threadIdx.x / TPR;
  if (row >= a.n) return;  // whole rows: with WPR > 1 the block is one row
  const int d = a.d;
  const Cols<TPR, NP, W> cols(tr, d);
  const T *x = (const T *)a.x + row * a.x_stride;
  float h[NP][8];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const Pack<T, 8> v = cols.load(x, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[p][e] = (float)v.v[e];
  }
  if (a.r) {
    const T *r = (const T *)a.r + row * a.r_stride;
    T *ho = (T *)a.h + row * d;
    Pack<T, 8> q[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) q[p] = cols.load(r, p);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[p][e] += (float)q[p].v[e];
      cols.store(ho, p, h[p]);
    }
  }
  float s = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += cols.own(p, e) ? h[p][e] : 0.f;
  const float mean = row_sum<WPR>(s, red[0]) / (float)d;
  s = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[p][e] -= mean;
      s = cols.own(p, e) ? fmaf(h[p][e], h[p][e], s) : s;
    }
  const float rstd = rsqrtf(row_sum<WPR>(s, red[1]) / (float)d + a.eps);
  if (a.mean && tr == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T *y = (T *)a.y + row * d;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    Pack<T, 8> g, b;
    if (a.gamma) g = cols.load((const T *)a.gamma, p);
    if (a.beta) b = cols.load((const T *)a.beta, p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      h[p][e] = fmaf(h[p][e] * rstd, a.gamma ? (float)g.v[e] : 1.f, a.beta ? (float)b.v[e] : 0.f);
    cols.store(y, p, h[p]);
  }
}

// One row of the backward as it is stored.
template <typename T, int NP>
struct BwdRow {
  Pack<T, 8> h[NP], dy[NP], dh[NP];
  float mean, rstd;
};
template <typename T, class C, int NP>
__device__ __forceinline__ void load_row(const NormArgs &a, int64_t row, const C &cols, BwdRow<T, NP> &r) {
  const T *h = (const T *)a.x + row * a.x_stride, *dy = (const T *)a.dy + row * a.dy_stride;
  const T *dh = (const T *)a.r + row * a.r_stride;
  r.mean = a.mean[row];
  r.rstd = a.rstd[row];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    r.h[p] = cols.load(h, p);
    r.dy[p] = cols.load(dy, p);
  }
  if (a.r) {
#pragma unroll
    for (int p = 0; p < NP; ++p) r.dh[p] = cols.load(dh, p);
  }
}

// A block walks rows blockIdx, blockIdx + gridDim, ... (RB at a time) and keeps
// its columns' sums of dy xh and dy in registers; its waves' sums meet in LDS
// once at the end and go to part[block], which k_norm_sums adds in a fixed order.
// All of a row's loads are issued together, dh's too, which is used last: 131072
// x 2048 bf16 in 401 us, 5.3 TB/s (686 us with dh loaded where it is used).
template <typename T, int WPR, int NP, bool W>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void k_norm_bwd(NormArgs a) {
  constexpr int RB = WPR > 4 ? 1 : 4 / WPR;
  constexpr int TPR = 64 * WPR;
  __shared__ float red[2][WPR][2];
  __shared__ float comb[RB > 1 ? (RB - 1) * TPR * 8 : 1];
  const int tr = threadIdx.x % TPR;
  const int rb = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const int d = a.d;
  const Cols<TPR, NP, W> cols(tr, d);
  float dg[NP][8], db[NP][8];
  Pack<T, 8> gamma[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (a.gamma) gamma[p] = cols.load((const T *)a.gamma, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dg[p][e] = db[p][e] = 0.f;
      if (!a.gamma) gamma[p].v[e] = (T)1.f;
    }
  }
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * RB + rb; row < a.n; row += (int64_t)gridDim.x * RB) {
    BwdRow<T, NP> cur;
    load_row(a, row, cols, cur);
    const float mean = cur.mean, rstd = cur.rstd;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // a value that is not the lane's own counts as dy = 0 (and xh of one that
        // is past the row's end is still finite or meets that zero in no sum)
        const bool own = cols.own(p, e);
        const float y = own ? (float)cur.dy[p].v[e] : 0.f;
        const float xh = own ? ((float)cur.h[p].v[e] - mean) * rstd : 0.f;
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
      cols.store(dx, p, o);
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
        if (W || p < NP - 1) {
          cols.store(out, p, v[p]);
        } else {  // the columns shared with a neighbour hold its sums, not these
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (cols.own(p, e)) out[cols.col(p) + e] = v[p][e];
        }
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
// with too few rows to fill the GPU a row takes four waves from 1024 columns on (us, one
// wave a row / four, with the residual add, inputs and outputs not in cache: 8 x 2560 4.8 /
// 4.4, 256 x 2560 5.9 / 4.9, 1024 x 1024 5.0 / 5.2, 2048 x 2560 13.0 / 13.0, 32768 x 2560 122 /
// 125, 32768 x 512 27 / 64).
int fwd_waves(int d, int64_t n) { return d > 4096 || (d >= 1024 && n <= 1024) ? 4 : 1; }
// Backward: a lane also holds its columns' sums, so a wave takes 2560 columns at
// most, and each wave should walk several rows per sum it writes (one wave a row
// against four: 131072 x 2048 390 and 416 us, 65536 x 2560 267 and 249, 262144 x 639 484
// and 1262, but 4096 x 2560 39 and 22).
int bwd_waves(int d, int64_t n) {
  if (d > 8192) return 8;
  return d > 2560 || (d > 512 && n < 16384) ? 4 : 1;
}

template <typename T, int WPR, int NP>
hipError_t fwd_launch(const NormArgs &a, hipStream_t st) {
  constexpr int RB = 4 / WPR;
  const dim3 grid = blk::grid_of((a.n + RB - 1) / RB), block(256);
  if (a.d % 8 == 0)
    hipLaunchKernelGGL((k_norm_fwd<T, WPR, NP, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_norm_fwd<T, WPR, NP, false>), grid, block, 0, st, a);
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
  // two blocks a CU of the wide rows' kernels, whose registers leave room for no more
  // (13590 x 4672: 109 us, with 1024 blocks 120), four of the others
  const int w = bwd_waves(d, n), rb = w == 1 ? 4 : 1, most = w == 1 ? 1024 : 512;
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
