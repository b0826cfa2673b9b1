// Norms of queries and keys for each head with the rotation by position (gfx950).
//
// A head's channels are held as pairs (a, b): the rotated pairs first, then the
// others two by two, which only the norm concerns:
//   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),  n = x r gamma.
// A lane's run of pairs is all rotated or not at all (run_of), so it is told by one number.
// (The angle 0 for the others would serve finite values: 0 x infinity is NaN.)
// A wave takes one token: its 64 lanes compute the token's (at most 64) sines and
// cosines once, pass them on through LDS, and then go over the token's heads, some
// lanes a head and several heads at a time; each lane holds W consecutive pairs, two
// loads of W elements (one of 2 W where the pairs are neighbours). Every element is
// read once and written once: HBM bounds the large sizes, one kernel's latency the
// small ones, where a token's heads are spread over several waves. Measured: 32768 tokens
// of 32 + 8 heads of 128 bf16 128 us forward (5.25 TB/s), 131072 of 16 + 8 529 us backward
// (4.57 TB/s, 1 % of it for telling the rotated from the others), 32 tokens with their append 5.2 us of kernel.
#include <type_traits>

#include "attention_internal.h"
#include "block_internal.h"

namespace ipttt {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// How a head's channels fall to lanes.
struct Split {
  int r2;     // rotated pairs
  int pairs;  // all pairs
  int half;   // distance of a and b in the channels that are not rotated
  int lanes;  // lanes a head: a power of 2, of which pairs / W hold something
};

// The largest run of pairs that neither crosses the end of the rotated ones nor that
// of the head, up to 16 bytes a load.
int run_of(int dh, int rotary, int most) {
  if (dh % 2) return 1;
  for (int w = most; w > 1; w /= 2)
    if ((rotary / 2) % w == 0 && ((dh - rotary) / 2) % w == 0) return w;
  return 1;
}
Split split_of(const HeadArgs &a, int w) {
  Split s;
  s.r2 = a.rotary / 2;
  s.half = (a.dh - a.rotary + 1) / 2;
  s.pairs = s.r2 + s.half;
  s.lanes = 1;
  while (s.lanes * w < s.pairs) s.lanes *= 2;
  return s;
}

// A lane's place in a head: the first of its W pairs, and where their channels are.
template <int W, bool IL>
struct Place {
  int pair, ca, cb;
  bool on, has_b;  // anything here; the b of a lone last channel is missing (W = 1)
  bool turned;     // rotated
  __device__ __forceinline__ Place(const Split &s, int dh, int lane) {
    pair = (lane & (s.lanes - 1)) * W;
    on = pair < s.pairs;
    turned = pair < s.r2;
    const int r = 2 * s.r2;
    if (IL) {
      ca = 2 * pair;
      cb = ca + 1;
    } else if (pair < s.r2) {
      ca = pair;
      cb = pair + s.r2;
    } else {
      ca = r + pair - s.r2;
      cb = ca + s.half;
    }
    has_b = cb < dh;
  }
};

template <typename T, int W, bool IL>
__device__ __forceinline__ void load_pairs(const T *row, const Place<W, IL> &p, float (&a)[W],
                                           float (&b)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) a[e] = b[e] = 0.f;
  if (!p.on) return;
  if constexpr (W == 1) {
    a[0] = (float)row[p.ca];
    if (p.has_b) b[0] = (float)row[p.cb];
  } else if constexpr (IL) {
    float v[2 * W];
    blk::load_pack<T, 2 * W>(row + p.ca, v);
#pragma unroll
    for (int e = 0; e < W; ++e) a[e] = v[2 * e], b[e] = v[2 * e + 1];
  } else {
    blk::load_pack<T, W>(row + p.ca, a);
    blk::load_pack<T, W>(row + p.cb, b);
  }
}
template <typename T, int W, bool IL>
__device__ __forceinline__ void store_pairs(T *row, const Place<W, IL> &p, const float (&a)[W],
                                            const float (&b)[W]) {
  if (!p.on) return;
  if constexpr (W == 1) {
    row[p.ca] = (T)a[0];
    if (p.has_b) row[p.cb] = (T)b[0];
  } else if constexpr (IL) {
    float v[2 * W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[2 * e] = a[e], v[2 * e + 1] = b[e];
    blk::store_pack<T, 2 * W>(row + p.ca, v);
  } else {
    blk::store_pack<T, W>(row + p.ca, a);
    blk::store_pack<T, W>(row + p.cb, b);
  }
}

// Sum over the lanes of one head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int m = lanes >> 1; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// cos and sin of a token's pairs for this lane. The angle pos inv_freq is reduced to a
// fraction of a turn in 64 bits: at position 2^20 it has 20 bits before the point,
// which 32 bits would take from the angle. cs: this wave's 64 places in LDS.
template <int W>
__device__ __forceinline__ void angles(const double *inv_freq, int r2, int pos, int lane, int pair,
                                       float2 *cs, float (&c)[W], float (&s)[W]) {
  float2 v = make_float2(1.f, 0.f);
  if (lane < r2) {
    const double turns = (double)pos * inv_freq[lane] * 0.15915494309189533577;
    sincospif(2.f * (float)(turns - rint(turns)), &v.y, &v.x);
  }
  // one wave's own places: its LDS operations keep their order
  __builtin_amdgcn_wave_barrier();
  cs[lane] = v;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const float2 u = cs[(pair + e) & 63];
    c[e] = u.x;
    s[e] = u.y;
  }
}

template <typename T, int W, bool IL>
__device__ __forceinline__ void load_gamma(const T *g, const Place<W, IL> &p, float (&a)[W],
                                           float (&b)[W]) {
  if (g) {
    load_pairs<T, W, IL>(g, p, a, b);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) a[e] = b[e] = 1.f;
  }
}

// The page's row of a new token, or null.
template <typename T>
__device__ __forceinline__ T *cache_row(const HeadArgs &a, void *base, int64_t t, int pos) {
  const int64_t seq = a.seqs ? a.seqs[t] : t;
  if (seq < 0 || seq >= a.table.batch || pos < 0) return nullptr;
  const int ps = a.cache.page_size, at = pos / ps;
  if (at >= a.table.width) return nullptr;
  const int page = a.table.p[seq * a.table.stride + at];
  if (page < 0 || page >= a.cache.pages) return nullptr;
  return (T *)base + ((int64_t)page * a.hk * ps + (pos - at * ps)) * a.dh;
}

// slices: waves a token, each taking every slices-th batch of heads.
template <typename T, int W, bool IL, bool APPEND>
__global__ __launch_bounds__(kThreads) void k_heads(HeadArgs a, Split s, int slices) {
  __shared__ float2 cs[kThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t unit = blk::block_id() * kWaves + wave;
  const int64_t t = unit / slices;
  const int slice = (int)(unit - t * slices);
  if (t >= a.n) return;
  const Place<W, IL> p(s, a.dh, lane);
  const int pos = a.pos[t];
  T *kc = nullptr, *vc = nullptr;
  const int64_t cache_head = APPEND ? (int64_t)a.cache.page_size * a.dh : 0;
  if constexpr (APPEND) {
    kc = cache_row<T>(a, a.cache.k, t, pos);
    vc = cache_row<T>(a, a.cache.v, t, pos);
  }
  float gq[2][W], gk[2][W];
  load_gamma<T, W, IL>((const T *)a.q_gamma, p, gq[0], gq[1]);
  load_gamma<T, W, IL>((const T *)a.k_gamma, p, gk[0], gk[1]);
  const int at_once = 64 / s.lanes, sub = lane / s.lanes;
  const int rows = a.hq + a.hk + (APPEND ? a.hk : 0);
  const float inv_d = 1.f / (float)a.dh;
  float c[W], sn[W];
  angles<W>(a.inv_freq, s.r2, pos, lane, p.pair, cs + 64 * wave, c, sn);
  for (int base = slice * at_once; base < rows; base += slices * at_once) {
    const int h = base + sub;
    const bool live = h < rows, is_q = h < a.hq, is_v = h >= a.hq + a.hk;
    const T *src = nullptr;
    T *dst = nullptr;
    if (is_q) {
      src = (const T *)a.q.p + t * a.q.tok_stride + h * a.q.head_stride;
      dst = (T *)a.q_out.p + t * a.q_out.tok_stride + h * a.q_out.head_stride;
    } else if (!is_v) {
      const int hh = h - a.hq;
      src = (const T *)a.k.p + t * a.k.tok_stride + hh * a.k.head_stride;
      if constexpr (APPEND)
        dst = kc ? kc + hh * cache_head : nullptr;
      else
        dst = (T *)a.k_out.p + t * a.k_out.tok_stride + hh * a.k_out.head_stride;
    } else if (APPEND && live) {
      const int hh = h - a.hq - a.hk;
      src = (const T *)a.v.p + t * a.v.tok_stride + hh * a.v.head_stride;
      dst = vc ? vc + hh * cache_head : nullptr;
    }
    float xa[W], xb[W];
    if (live) {
      load_pairs<T, W, IL>(src, p, xa, xb);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) xa[e] = xb[e] = 0.f;
    }
    if (!is_v) {
      const bool normed = is_q ? a.q_gamma != nullptr : a.k_gamma != nullptr;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < W; ++e) sum += xa[e] * xa[e] + xb[e] * xb[e];
      sum = head_sum(sum, s.lanes);
      const float r = normed ? 1.f / sqrtf(sum * inv_d + a.eps) : 1.f;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float na = xa[e] * r * (is_q ? gq[0][e] : gk[0][e]);
        const float nb = xb[e] * r * (is_q ? gq[1][e] : gk[1][e]);
        xa[e] = p.turned ? na * c[e] - nb * sn[e] : na;
        xb[e] = p.turned ? nb * c[e] + na * sn[e] : nb;
      }
    }
    if (live && dst) store_pairs<T, W, IL>(dst, p, xa, xb);
  }
}

// A block goes over tokens of the queries, or of the keys (from block `q_blocks` on): each
// wave keeps its lanes' part of the weight's gradient, and the block leaves one row of
// partial sums. The next heads' rows are loaded beside this one's arithmetic.
template <typename T, int W, bool IL>
__global__ __launch_bounds__(kThreads) void k_heads_bwd(HeadArgs a, Split s, int q_blocks) {
  __shared__ float2 cs[kThreads];
  __shared__ float sums[kWaves][kHeadMaxDim];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool keys = (int)blockIdx.x >= q_blocks;
  const int block = keys ? blockIdx.x - q_blocks : blockIdx.x;
  const int blocks = keys ? gridDim.x - q_blocks : q_blocks;
  const ipttt_heads x = keys ? a.k : a.q, dy = keys ? a.dk : a.dq, dx = keys ? a.k_out : a.q_out;
  const T *const gamma = (const T *)(keys ? a.k_gamma : a.q_gamma);
  const bool normed = gamma != nullptr;
  const Place<W, IL> p(s, a.dh, lane);
  float g[2][W], sum_g[2][W];
  load_gamma<T, W, IL>(gamma, p, g[0], g[1]);
#pragma unroll
  for (int e = 0; e < W; ++e) sum_g[0][e] = sum_g[1][e] = 0.f;
  const int at_once = 64 / s.lanes, sub = lane / s.lanes, rows = keys ? a.hk : a.hq;
  const float inv_d = 1.f / (float)a.dh;
  for (int64_t t = (int64_t)block * kWaves + wave; t < a.n; t += (int64_t)blocks * kWaves) {
    // x and dy of head h (zero behind the last)
    const auto load = [&](int h, float (&x0)[W], float (&x1)[W], float (&y0)[W], float (&y1)[W])
                          __attribute__((always_inline)) {
      if (h < rows) {
        load_pairs<T, W, IL>((const T *)x.p + t * x.tok_stride + h * x.head_stride, p, x0, x1);
        load_pairs<T, W, IL>((const T *)dy.p + t * dy.tok_stride + h * dy.head_stride, p, y0, y1);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) x0[e] = x1[e] = y0[e] = y1[e] = 0.f;
      }
    };
    float xa[W], xb[W], ya[W], yb[W], na[W], nb[W], ma[W], mb[W], c[W], sn[W];
    load(sub, na, nb, ma, mb);
    angles<W>(a.inv_freq, s.r2, a.pos[t], lane, p.pair, cs + 64 * wave, c, sn);
    for (int h = sub; h - sub < rows; h += at_once) {
#pragma unroll
      for (int e = 0; e < W; ++e) xa[e] = na[e], xb[e] = nb[e], ya[e] = ma[e], yb[e] = mb[e];
      load(h + at_once, na, nb, ma, mb);
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        sum += xa[e] * xa[e] + xb[e] * xb[e];
        const float ga = p.turned ? ya[e] * c[e] + yb[e] * sn[e] : ya[e];
        const float gb = p.turned ? yb[e] * c[e] - ya[e] * sn[e] : yb[e];
        ya[e] = ga;
        yb[e] = gb;
        dot += ga * g[0][e] * xa[e] + gb * g[1][e] * xb[e];
      }
      if (normed) {
        sum = head_sum(sum, s.lanes);
        dot = head_sum(dot, s.lanes);
      }
      if (h >= rows) continue;  // whole heads drop out: no sum is split
      if (normed) {
        const float r = 1.f / sqrtf(sum * inv_d + a.eps);
        const float k = dot * r * r * r * inv_d;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          sum_g[0][e] += ya[e] * xa[e] * r;
          sum_g[1][e] += yb[e] * xb[e] * r;
          ya[e] = ya[e] * g[0][e] * r - xa[e] * k;
          yb[e] = yb[e] * g[1][e] * r - xb[e] * k;
        }
      }
      store_pairs<T, W, IL>((T *)dx.p + t * dx.tok_stride + h * dx.head_stride, p, ya, yb);
    }
  }
  if (!a.part) return;
  // over the lanes that hold the same pairs, then over the waves
  for (int m = s.lanes; m < 64; m <<= 1)
#pragma unroll
    for (int e = 0; e < W; ++e) {
      sum_g[0][e] += __shfl_xor(sum_g[0][e], m, 64);
      sum_g[1][e] += __shfl_xor(sum_g[1][e], m, 64);
    }
  if (sub == 0) store_pairs<float, W, IL>(sums[wave], p, sum_g[0], sum_g[1]);
  __syncthreads();
  for (int i = threadIdx.x; i < a.dh; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sums[w][i];
    a.part[(int64_t)blockIdx.x * a.dh + i] = v;
  }
}

// Column sums of the blocks' partial rows, in a fixed order: 32 columns a block, 32
// threads a column. blockIdx.y: the queries' or the keys' rows.
__global__ __launch_bounds__(1024) void k_heads_gamma(const float *part, int q_blocks, int k_blocks, int dh,
                                                      float *dq_gamma, float *dk_gamma) {
  __shared__ float sums[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const float *const first = part + (blockIdx.y ? (int64_t)q_blocks * dh : 0);
  const int blocks = blockIdx.y ? k_blocks : q_blocks;
  float v = 0.f;
  if (col < dh) {
#pragma unroll 8
    for (int b = row; b < blocks; b += 32) v += first[(int64_t)b * dh + col];
  }
  sums[row][threadIdx.x & 31] = v;
  __syncthreads();
  if (row == 0 && col < dh) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x];
    float *out = blockIdx.y ? dk_gamma : dq_gamma;
    if (out) out[col] = v;
  }
}

// f(run of pairs, neighbouring pairs) as compile-time constants.
template <typename T, class F>
void by_layout(const HeadArgs &a, F f) {
  constexpr int most = sizeof(T) == 2 ? 8 : 4;
  const auto run = [&](auto il) {
    switch (run_of(a.dh, a.rotary, most)) {
      case 8:
        if constexpr (most == 8) f(std::integral_constant<int, 8>(), il);
        break;
      case 4: f(std::integral_constant<int, 4>(), il); break;
      case 2: f(std::integral_constant<int, 2>(), il); break;
      default: f(std::integral_constant<int, 1>(), il);
    }
  };
  if (a.interleaved) run(std::true_type()); else run(std::false_type());
}

template <typename T, bool APPEND>
hipError_t launch_heads(const HeadArgs &a, hipStream_t st) {
  by_layout<T>(a, [&](auto w, auto il) {
    constexpr int W = decltype(w)::value;
    const Split s = split_of(a, W);
    const int at_once = 64 / s.lanes, rows = a.hq + a.hk * (APPEND ? 2 : 1);
    const int batches = (rows + at_once - 1) / at_once;
    // a wave a token once there are 8192 tokens, more while there are fewer (40 heads of 128
    // bf16: 8192 tokens 34 us, 42 with four waves a token)
    int64_t slices = (8192 + a.n - 1) / a.n;
    if (slices > batches) slices = batches;
    k_heads<T, W, decltype(il)::value, APPEND>
        <<<blk::grid_of((a.n * slices + kWaves - 1) / kWaves), kThreads, 0, st>>>(a, s, (int)slices);
  });
  return hipGetLastError();
}

}  // namespace

// 2048 blocks for all heads, each with a partial sum of the scales' gradients. (8192 tokens,
// 24 heads of 128 bf16: 51 us, 54 with 1024, 56 with 4096.)
int heads_bwd_blocks(int heads, int all, int64_t n) {
  const int64_t b = (n + kWaves - 1) / kWaves, most = (int64_t)2048 * heads / all;
  return (int)(b < 1 ? 1 : b > most ? (most < 1 ? 1 : most) : b);
}

template <typename T>
hipError_t heads_forward(const HeadArgs &a, hipStream_t st) {
  return launch_heads<T, false>(a, st);
}
template <typename T>
hipError_t heads_append(const HeadArgs &a, hipStream_t st) {
  return launch_heads<T, true>(a, st);
}
template <typename T>
hipError_t heads_backward(const HeadArgs &a, hipStream_t st) {
  const int qb = heads_bwd_blocks(a.hq, a.hq + a.hk, a.n), kb = heads_bwd_blocks(a.hk, a.hq + a.hk, a.n);
  by_layout<T>(a, [&](auto w, auto il) {
    constexpr int W = decltype(w)::value;
    k_heads_bwd<T, W, decltype(il)::value><<<qb + kb, kThreads, 0, st>>>(a, split_of(a, W), qb);
  });
  if (a.part)
    k_heads_gamma<<<dim3((a.dh + 31) / 32, 2), 1024, 0, st>>>(a.part, qb, kb, a.dh, a.dq_gamma, a.dk_gamma);
  return hipGetLastError();
}

template hipError_t heads_forward<float>(const HeadArgs &, hipStream_t);
template hipError_t heads_forward<__bf16>(const HeadArgs &, hipStream_t);
template hipError_t heads_append<float>(const HeadArgs &, hipStream_t);
template hipError_t heads_append<__bf16>(const HeadArgs &, hipStream_t);
template hipError_t heads_backward<float>(const HeadArgs &, hipStream_t);
template hipError_t heads_backward<__bf16>(const HeadArgs &, hipStream_t);

}  // namespace ipttt
