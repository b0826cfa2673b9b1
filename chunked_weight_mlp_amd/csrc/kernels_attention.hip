// Attention over packed prompts (gfx950): forward and backward.
#include "attention_common.h"

namespace ipttt {
namespace {

using namespace attn;

constexpr int kRows = 32;  // queries (keys) a wave holds
constexpr int kWaves = 8, kThreads = 64 * kWaves, kBlock = kRows * kWaves;
constexpr int kStage = 64;  // rows of the other side a step

// What becomes of a value on its way into a tile. A product of a tile with weights that are
// zero where a row is not seen still takes a value there that is not finite into the sum
// (0 x infinity). A block whose results are not all finite is therefore computed again:
// once for how many values that are not finite each result sees (kCount), and once with
// those values left out (kFinite); where the count is not zero the result is NaN.
enum Fix { kAsIs, kCount, kFinite };
template <typename T>
__device__ __forceinline__ T fixed(T v, int fix) {
  if (fix == kAsIs) return v;
  const bool ok = __builtin_isfinite((float)v);
  return fix == kCount ? (T)(ok ? 0.f : 1.f) : ok ? v : (T)0.f;
}

// Copies kStage rows from `first` of a tensor's head into a tile; rows at or behind `end`
// repeat the last one before it.
template <typename T, int DP>
__device__ __forceinline__ void stage(T *tile, const T *base, int64_t stride, int first, int end,
                                      int dh, int tid, int fix) {
  using L = Tile<T, DP>;
  for (int i = tid; i < kStage * L::NP; i += kThreads) {
    const int r = i / L::NP, p = i % L::NP;
    const int row = first + r < end ? first + r : end - 1;
    T v[L::PE];
    load_some<T, L::PE>(base + row * stride, p * L::PE, dh, v);
#pragma unroll
    for (int e = 0; e < L::PE; ++e) tile[L::at(r, p) + e] = fixed(v[e], fix);
  }
}

// What a query sees of its sequence's keys: [lo, hi).
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen_by(const AttnArgs &a, int i, int lq, int lk) {
  if (!a.causal) return Seen{0, lk};
  const int last = i + lk - lq;  // inclusive
  return Seen{a.window > 0 ? max(0, last - a.window + 1) : 0, max(0, min(lk, last + 1))};
}

template <int N>
__device__ __forceinline__ bool all_finite(const f32x16 (&x)[N]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) ok &= __builtin_isfinite(x[i][e]);
  return ok;
}

// Results that are not zero, and NaN for them.
template <int N>
__device__ __forceinline__ uint64_t nonzero(const f32x16 (&x)[N]) {
  uint64_t bits = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) bits |= (uint64_t)(x[i][e] != 0.f) << (16 * i + e);
  return bits;
}
template <int N>
__device__ __forceinline__ void spoil(f32x16 (&x)[N], uint64_t bits) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (bits >> (16 * i + e) & 1) x[i][e] = NAN;
}

// Rows of a lane's results x scale to a row of dh channels in memory.
template <typename T, int DP>
__device__ __forceinline__ void store_row(T *row, const f32x16 (&x)[DP / 32], float scale, int h,
                                          int dh) {
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * d + 8 * g + 4 * h;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[d][4 * g + e] * scale;
      if (c + 4 <= dh) {
        blk::store_pack<T, 4>(row + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < dh) row[c + e] = (T)v[e];
      }
    }
}

// Block of a (tile, head): heads of one key head on one XCD (consecutive blocks go to the
// 8 XCDs in turn), tiles from the last, whose queries see the most keys, to the first.
struct Work {
  int64_t tile;
  int head, kv;
};
__device__ __forceinline__ Work work_of(const AttnArgs &a, int64_t tiles) {
  const int64_t id = blk::block_id();
  const int group = a.hq / a.hk;
  Work w;
  w.kv = (int)(id % a.hk);
  const int64_t x = id / a.hk;
  w.head = w.kv * group + (int)(x % group);
  w.tile = tiles - 1 - x / group;
  return w;
}

template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void k_fwd(AttnArgs a, int64_t tiles) {
  using L = Tile<T, DP>;
  extern __shared__ __align__(16) char smem[];
  T *const kt = (T *)smem, *const vt = kt + kStage * DP;
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, h = l >> 5;
  const Work w = work_of(a, tiles);
  if (w.tile < 0) return;
  const int s = sequence_of(a.q_off, a.batch, a.n_q, kBlock, w.tile, l);
  const Rows rq = rows_of(a.q_off, s, a.batch, a.n_q);
  const Rows rk = s < a.batch ? rows_of(a.k_off, s, a.batch, a.n_k) : Rows{0, 0};
  const int first = (int)(w.tile - (rq.start / kBlock + s)) * kBlock;  // the block's first query
  if (first >= rq.len) return;
  const int lq = rq.len, lk = rk.len;
  const int q0 = first + kRows * wave, qi = q0 + (l & 31);
  const int qr = min(qi, lq - 1);
  const T *qp = (const T *)a.q.p + (rq.start + qr) * a.q.tok_stride + w.head * a.q.head_stride;
  const T *kp = (const T *)a.k.p + rk.start * a.k.tok_stride + w.kv * a.k.head_stride;
  const T *vp = (const T *)a.v.p + rk.start * a.v.tok_stride + w.kv * a.v.head_stride;
  Frag<T> q[L::STEPS];
#pragma unroll
  for (int i = 0; i < L::STEPS; ++i) q[i] = with_sign<T>(load_frag<T>(qp, i, h, a.dh), a.scale);
  const Seen mine = seen_by(a, qi, lq, lk);
  const Seen head = seen_by(a, first, lq, lk), tail = seen_by(a, min(first + kBlock, lq) - 1, lq, lk);
  // of this wave's rows (those behind the last query are not stored)
  const Seen wf = seen_by(a, q0, lq, lk), wl = seen_by(a, q0 + kRows - 1, lq, lk);
  const float c = log2_scale(a.scale);
  f32x16 acc[DP / 32];
  float m, sum;
  uint64_t bad = 0;
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
    m = -INFINITY;
    sum = 0.f;
    for (int k0 = head.lo / kStage * kStage; k0 < tail.hi; k0 += kStage) {
      __syncthreads();
      stage<T, DP>(kt, kp, a.k.tok_stride, k0, lk, a.dh, tid, kAsIs);
      stage<T, DP>(vt, vp, a.v.tok_stride, k0, lk, a.dh, tid, fix);
      __syncthreads();
      if (k0 >= wl.hi || k0 + kStage <= wf.lo) continue;  // nothing here for this wave
      f32x16 x[kStage / 32];
#pragma unroll
      for (int t = 0; t < kStage / 32; ++t) {
        x[t] = f32x16{};
#pragma unroll
        for (int i = 0; i < L::STEPS; ++i)
          x[t] = mma(L::row_frag(kt, 32 * t + (l & 31), i, h), q[i], x[t]);
      }
      const bool whole = k0 + kStage <= wf.hi && k0 >= wl.lo;
      if (!whole) {
#pragma unroll
        for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = k0 + 32 * t + 8 * (i / 4) + 4 * h + i % 4;
            if (j < mine.lo || j >= mine.hi) x[t][i] = -INFINITY;
          }
      }
      // running maximum
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          top = fmaxf(top, x[t][i]);
        }
      top = fmaxf(top, other_half(top));
      const float next = fmaxf(m, top);
      const float base = next == -INFINITY ? 0.f : next;
      const float f = exp2_((m - base) * c);
      m = next;
      sum *= f;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] *= f;
#pragma unroll
      for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[t][i] = exp2_((x[t][i] - base) * c);
          sum += x[t][i];
        }
      if (fix == kCount) {
#pragma unroll
        for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = k0 + 32 * t + 8 * (i / 4) + 4 * h + i % 4;
            x[t][i] = j >= mine.lo && j < mine.hi ? 1.f : 0.f;
          }
      }
#pragma unroll
      for (int i = 0; i < kStage / 16; ++i) {
        const Frag<T> p = as_operand<T>(x[i / 2], i % 2);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          acc[d] = mma(L::col_frag(vt, 16 * i, 32 * d, l), p, acc[d]);
      }
    }
    if (fix == kFinite) spoil(acc, bad);
    if (fix == kCount) bad = nonzero(acc);
    if (fix == kFinite || (fix == kAsIs && __syncthreads_and(all_finite(acc)))) break;
  }
  sum += other_half(sum);
  if (qi >= lq) return;
  const bool none = mine.lo >= mine.hi;
  T *const op = (T *)a.o.p + (rq.start + qi) * a.o.tok_stride + w.head * a.o.head_stride;
  if (none) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
  }
  store_row<T, DP>(op, acc, none ? 0.f : 1.f / sum, h, a.dh);
  if (a.lse && h == 0)
    a.lse[w.head * a.n_q + rq.start + qi] = none ? -INFINITY : (m * c + log2f(sum)) * kLn2;
}

// The forward's lse in units of log2. A row with an infinite score has no softmax.
__device__ __forceinline__ float log2_sum(float lse) { return lse == INFINITY ? NAN : lse * kLog2e; }

// delta = sum(dy o) of each query and head: 16 lanes a row.
template <typename T>
__global__ __launch_bounds__(256) void k_delta(AttnArgs a) {
  const int64_t row = (blk::block_id() * 256 + threadIdx.x) / 16;  // token-major
  const int64_t t = row / a.hq;
  const int hd = (int)(row - t * a.hq);
  if (t >= a.n_q) return;
  const T *o = (const T *)a.o.p + t * a.o.tok_stride + hd * a.o.head_stride;
  const T *dy = (const T *)a.dy.p + t * a.dy.tok_stride + hd * a.dy.head_stride;
  float v = 0.f;
  T x[8], y[8];
  const int c = 8 * (threadIdx.x & 15);
  if (c < a.dh) {
    load_some<T, 8>(o, c, a.dh, x);
    load_some<T, 8>(dy, c, a.dh, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) v += (float)x[e] * (float)y[e];
  }
#pragma unroll
  for (int k = 8; k >= 1; k >>= 1) v += __shfl_xor(v, k, 64);
  if ((threadIdx.x & 15) == 0) a.delta[hd * a.n_q + t] = v;
}

// dq: a block's queries, over the keys that they see.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void k_dq(AttnArgs a, int64_t tiles) {
  using L = Tile<T, DP>;
  extern __shared__ __align__(16) char smem[];
  T *const kt = (T *)smem, *const vt = kt + kStage * DP;
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, h = l >> 5;
  const Work w = work_of(a, tiles);
  if (w.tile < 0) return;
  const int s = sequence_of(a.q_off, a.batch, a.n_q, kBlock, w.tile, l);
  const Rows rq = rows_of(a.q_off, s, a.batch, a.n_q);
  const Rows rk = s < a.batch ? rows_of(a.k_off, s, a.batch, a.n_k) : Rows{0, 0};
  const int first = (int)(w.tile - (rq.start / kBlock + s)) * kBlock;
  if (first >= rq.len) return;
  const int lq = rq.len, lk = rk.len;
  const int q0 = first + kRows * wave, qi = q0 + (l & 31);
  const int64_t qr = rq.start + min(qi, lq - 1);
  const T *qp = (const T *)a.q.p + qr * a.q.tok_stride + w.head * a.q.head_stride;
  const T *yp = (const T *)a.dy.p + qr * a.dy.tok_stride + w.head * a.dy.head_stride;
  const T *kp = (const T *)a.k.p + rk.start * a.k.tok_stride + w.kv * a.k.head_stride;
  const T *vp = (const T *)a.v.p + rk.start * a.v.tok_stride + w.kv * a.v.head_stride;
  Frag<T> q[L::STEPS], dy[L::STEPS];
#pragma unroll
  for (int i = 0; i < L::STEPS; ++i) {
    q[i] = with_sign<T>(load_frag<T>(qp, i, h, a.dh), a.scale);
    dy[i] = load_frag<T>(yp, i, h, a.dh);
  }
  const Seen mine = seen_by(a, qi, lq, lk);
  const Seen head = seen_by(a, first, lq, lk), tail = seen_by(a, min(first + kBlock, lq) - 1, lq, lk);
  const Seen wf = seen_by(a, q0, lq, lk), wl = seen_by(a, q0 + kRows - 1, lq, lk);
  const float c = log2_scale(a.scale);
  const float lse = log2_sum(a.lse[w.head * a.n_q + qr]), delta = a.delta[w.head * a.n_q + qr];
  f32x16 acc[DP / 32];
  uint64_t bad = 0;
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
    for (int k0 = head.lo / kStage * kStage; k0 < tail.hi; k0 += kStage) {
      __syncthreads();
      stage<T, DP>(kt, kp, a.k.tok_stride, k0, lk, a.dh, tid, fix);
      stage<T, DP>(vt, vp, a.v.tok_stride, k0, lk, a.dh, tid, kAsIs);
      __syncthreads();
      if (k0 >= wl.hi || k0 + kStage <= wf.lo) continue;
      f32x16 x[kStage / 32];
      const bool whole = k0 + kStage <= wf.hi && k0 >= wl.lo;
#pragma unroll
      for (int t = 0; t < kStage / 32; ++t) {
        f32x16 dp{};
        x[t] = f32x16{};
#pragma unroll
        for (int i = 0; i < L::STEPS; ++i) {
          x[t] = mma(L::row_frag(kt, 32 * t + (l & 31), i, h), q[i], x[t]);
          dp = mma(L::row_frag(vt, 32 * t + (l & 31), i, h), dy[i], dp);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = exp2_(x[t][i] * c - lse);
          x[t][i] = p * (dp[i] - delta);
          const int j = k0 + 32 * t + 8 * (i / 4) + 4 * h + i % 4;
          if (!whole && (j < mine.lo || j >= mine.hi)) x[t][i] = 0.f;
        }
      }
      if (fix == kCount) {
#pragma unroll
        for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = k0 + 32 * t + 8 * (i / 4) + 4 * h + i % 4;
            x[t][i] = j >= mine.lo && j < mine.hi ? 1.f : 0.f;
          }
      }
#pragma unroll
      for (int i = 0; i < kStage / 16; ++i) {
        const Frag<T> ds = as_operand<T>(x[i / 2], i % 2);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          acc[d] = mma(L::col_frag(kt, 16 * i, 32 * d, l), ds, acc[d]);
      }
    }
    if (fix == kFinite) spoil(acc, bad);
    if (fix == kCount) bad = nonzero(acc);
    if (fix == kFinite || (fix == kAsIs && __syncthreads_and(all_finite(acc)))) break;
  }
  if (qi >= lq) return;
  T *const out = (T *)a.dq.p + (rq.start + qi) * a.dq.tok_stride + w.head * a.dq.head_stride;
  store_row<T, DP>(out, acc, a.scale, h, a.dh);
}

// dk and dv: a block's keys, over the queries of the group's heads that see them.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void k_dkv(AttnArgs a, int64_t tiles) {
  using L = Tile<T, DP>;
  extern __shared__ __align__(16) char smem[];
  T *const qt = (T *)smem, *const yt = qt + kStage * DP;
  float *const row_lse = (float *)(yt + kStage * DP), *const row_delta = row_lse + kStage;
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, h = l >> 5;
  const int64_t id = blk::block_id();
  const int kv = (int)(id % a.hk);
  const int64_t tile = id / a.hk;
  if (tile >= tiles) return;
  const int s = sequence_of(a.k_off, a.batch, a.n_k, kBlock, tile, l);
  const Rows rk = rows_of(a.k_off, s, a.batch, a.n_k);
  const Rows rq = s < a.batch ? rows_of(a.q_off, s, a.batch, a.n_q) : Rows{0, 0};
  const int first = (int)(tile - (rk.start / kBlock + s)) * kBlock;
  if (first >= rk.len) return;
  const int lq = rq.len, lk = rk.len, group = a.hq / a.hk;
  const int k0 = first + kRows * wave, kj = k0 + (l & 31);
  const int64_t kr = rk.start + min(kj, lk - 1);
  const T *kp = (const T *)a.k.p + kr * a.k.tok_stride + kv * a.k.head_stride;
  const T *vp = (const T *)a.v.p + kr * a.v.tok_stride + kv * a.v.head_stride;
  Frag<T> k[L::STEPS], v[L::STEPS];
#pragma unroll
  for (int i = 0; i < L::STEPS; ++i) {
    k[i] = with_sign<T>(load_frag<T>(kp, i, h, a.dh), a.scale);
    v[i] = load_frag<T>(vp, i, h, a.dh);
  }
  // the queries that see key j: [from(j), to(j))
  const int off = lk - lq;
  const auto from = [&](int j) { return a.causal ? max(0, j - off) : 0; };
  const auto to = [&](int j) {
    return a.causal && a.window > 0 ? max(0, min((int64_t)lq, (int64_t)j + a.window - off)) : lq;
  };
  const int my_from = from(kj), my_to = kj < lk ? (int)to(kj) : 0;
  const int q_from = from(first), q_to = (int)to(min(first + kBlock, lk) - 1);
  const int w_from = from(k0), w_to = k0 < lk ? (int)to(min(k0 + kRows, lk) - 1) : 0;
  const int w_all_from = from(k0 + kRows - 1), w_all_to = k0 + kRows <= lk ? (int)to(k0) : 0;
  const float c = log2_scale(a.scale);
  f32x16 dk[DP / 32], dv[DP / 32];
  uint64_t bad = 0;
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) dk[d] = dv[d] = f32x16{};
    for (int g = 0; g < group; ++g) {
      const int head = kv * group + g;
      const T *qp = (const T *)a.q.p + rq.start * a.q.tok_stride + head * a.q.head_stride;
      const T *yp = (const T *)a.dy.p + rq.start * a.dy.tok_stride + head * a.dy.head_stride;
      const float *lse = a.lse + head * a.n_q + rq.start, *delta = a.delta + head * a.n_q + rq.start;
      for (int i0 = q_from / kStage * kStage; i0 < q_to; i0 += kStage) {
        __syncthreads();
        stage<T, DP>(qt, qp, a.q.tok_stride, i0, lq, a.dh, tid, fix);
        stage<T, DP>(yt, yp, a.dy.tok_stride, i0, lq, a.dh, tid, fix);
        if (tid < kStage) {
          const int i = min(i0 + tid, lq - 1);
          row_lse[tid] = log2_sum(lse[i]);
          row_delta[tid] = delta[i];
        }
        __syncthreads();
        if (i0 >= w_to || i0 + kStage <= w_from) continue;
        const bool whole = i0 >= w_all_from && i0 + kStage <= w_all_to;
        f32x16 x[kStage / 32], y[kStage / 32];
#pragma unroll
        for (int t = 0; t < kStage / 32; ++t) {
          x[t] = y[t] = f32x16{};
#pragma unroll
          for (int i = 0; i < L::STEPS; ++i) {
            x[t] = mma(L::row_frag(qt, 32 * t + (l & 31), i, h), k[i], x[t]);
            y[t] = mma(L::row_frag(yt, 32 * t + (l & 31), i, h), v[i], y[t]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 32 * t + 8 * (i / 4) + 4 * h + i % 4;
            float p = exp2_(x[t][i] * c - row_lse[r]);
            float ds = p * (y[t][i] - row_delta[r]);
            if (!whole && (i0 + r < my_from || i0 + r >= my_to)) p = ds = 0.f;
            x[t][i] = p;
            y[t][i] = ds;
          }
        }
        if (fix == kCount) {
#pragma unroll
          for (int t = 0; t < kStage / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = i0 + 32 * t + 8 * (i / 4) + 4 * h + i % 4;
              x[t][i] = r >= my_from && r < my_to ? 1.f : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kStage / 16; ++i) {
          const Frag<T> p = as_operand<T>(x[i / 2], i % 2), ds = as_operand<T>(y[i / 2], i % 2);
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) {
            dv[d] = mma(L::col_frag(yt, 16 * i, 32 * d, l), p, dv[d]);
            dk[d] = mma(L::col_frag(qt, 16 * i, 32 * d, l), ds, dk[d]);
          }
        }
      }
    }
    if (fix == kFinite) spoil(dv, bad);
    if (fix == kCount) bad = nonzero(dv);
    if (fix == kFinite || (fix == kAsIs && __syncthreads_and(all_finite(dk) && all_finite(dv)))) break;
  }
  if (kj >= lk) return;
  store_row<T, DP>((T *)a.dk.p + kr * a.dk.tok_stride + kv * a.dk.head_stride, dk, a.scale, h, a.dh);
  store_row<T, DP>((T *)a.dv.p + kr * a.dv.tok_stride + kv * a.dv.head_stride, dv, 1.f, h, a.dh);
}

template <typename T, class F>
void by_width(int dh, F f) {
  if (dh <= 64) f(std::integral_constant<int, 64>()); else f(std::integral_constant<int, 128>());
}

}  // namespace

bool attn_size_ok(int hq, int batch, int64_t n) {
  return tiles_of(n, kBlock, batch) * hq < ((int64_t)1 << 31);
}

template <typename T>
hipError_t attn_forward(const AttnArgs &a, hipStream_t st) {
  by_width<T>(a.dh, [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    const int64_t tiles = tiles_of(a.n_q, kBlock, a.batch);
    k_fwd<T, DP><<<blk::grid_of(tiles * a.hq), kThreads, 2 * kStage * DP * sizeof(T), st>>>(a, tiles);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t attn_backward(const AttnArgs &a, hipStream_t st) {
  if (a.n_q > 0) k_delta<T><<<blk::grid_of((a.n_q * a.hq + 15) / 16), 256, 0, st>>>(a);
  by_width<T>(a.dh, [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    const size_t lds = 2 * kStage * DP * sizeof(T);
    if (a.n_k > 0) {
      const int64_t tiles = tiles_of(a.n_k, kBlock, a.batch);
      k_dkv<T, DP><<<blk::grid_of(tiles * a.hk), kThreads, lds + 8 * kStage, st>>>(a, tiles);
    }
    if (a.n_q > 0) {
      const int64_t tiles = tiles_of(a.n_q, kBlock, a.batch);
      k_dq<T, DP><<<blk::grid_of(tiles * a.hq), kThreads, lds, st>>>(a, tiles);
    }
  });
  return hipGetLastError();
}

template hipError_t attn_forward<float>(const AttnArgs &, hipStream_t);
template hipError_t attn_forward<__bf16>(const AttnArgs &, hipStream_t);
template hipError_t attn_backward<float>(const AttnArgs &, hipStream_t);
template hipError_t attn_backward<__bf16>(const AttnArgs &, hipStream_t);

}  // namespace ipttt
