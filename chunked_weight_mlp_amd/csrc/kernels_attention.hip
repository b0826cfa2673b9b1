// Attention over packed prompts (gfx950): forward and backward.
//
// A block of four waves takes 128 queries of one head (the forward, dq) or 128 keys of one
// key head (dk, dv) and goes over the other side in tiles that are copied into LDS a step
// ahead. Two blocks share a CU, so that one's products run beside the other's softmax; the
// 256 registers that leaves a wave are what its sums, its own rows and the operands in
// flight need (128 channels bf16: forward 233, dq 255, dk and dv all), and none may go to
// memory in a loop: a reload waits for every copy in flight before it. (dk and dv keep 12 bytes
// a lane there, for behind the loop.) Products and the arithmetic that does not wait for them
// are interleaved in the source; sched_barrier keeps the order.
//
// What bounds it: of the forward's cycles the matrix cores are busy 52 % and the vector units
// issue in 49 % (32768 tokens of 32/8 heads of 128 bf16: 8.4 to 8.8 ms from one GPU to another,
// 1000 to 1045 TFLOP/s; 16384 of 16/8: 1.08 ms, 1020, and the backward 3.7 ms, 740).
#include "attention_common.h"

namespace ipttt {
namespace {

using namespace attn;

constexpr int kRows = 32;  // queries (keys) a wave holds
constexpr int kWaves = 4, kThreads = 64 * kWaves, kBlock = kRows * kWaves;

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
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) z = __builtin_fmaf(x[i][e], 0.f, z);
  return z == 0.f;
}

// Block of a (tile, head): heads of one key head on one XCD (consecutive blocks go to the
// 8 XCDs in turn), tiles from the last, whose queries see the most keys, to the first.
struct Work {
  int64_t rank;  // the tile's place in the order
  int head, kv;
};
__device__ __forceinline__ Work work_of(const AttnArgs &a) {
  const int64_t id = blk::block_id();
  const int group = a.hq / a.hk;
  Work w;
  w.kv = (int)(id % a.hk);
  const int64_t x = id / a.hk;
  w.head = w.kv * group + (int)(x % group);
  w.rank = x / group;
  return w;
}
// Tile number `tile` of queries (keys); first is behind the sequence's end where the tile
// is empty.
__device__ __forceinline__ TilePlace tile_place(const AttnArgs &a, bool keys, int64_t tile, int lane) {
  constexpr int M = kBlock;
  const int32_t *off = keys ? a.k_off : a.q_off;
  const int64_t n = keys ? a.n_k : a.n_q;
  const int s = __builtin_amdgcn_readfirstlane(sequence_of(off, a.batch, n, M, tile, lane));
  const Rows mine = rows_of(off, s, a.batch, n);
  const Rows other = s < a.batch ? rows_of(keys ? a.q_off : a.k_off, s, a.batch, keys ? a.n_q : a.n_k) : Rows{0, 0};
  const int first = (int)(tile - (mine.start / M + s)) * M;
  if (keys) return TilePlace{first, (int)other.start, other.len, (int)mine.start, mine.len, {}};
  return TilePlace{first, (int)mine.start, mine.len, (int)other.start, other.len, {}};
}

// ---- the order of tiles ----------------------------------------------------------------
// Blocks start in the order of their numbers as others end, so the longest have to come
// first. Within one sequence that is known; tiles of several are sorted by how much they
// see, at most kOrderTiles of kOrderBatch sequences (more are so many that their order
// matters little), and only if they do not all run at once. (16384 tokens in six documents,
// 16/8 heads of 128 bf16: forward 290 us as they come, 272 sorted; dq 388, 364. Sorting 4 to 7.)
constexpr int kOrderTiles = 2048, kOrderBatch = 1024;
inline bool ordered(int batch, int64_t tiles, int heads) {
  return batch > 1 && batch <= kOrderBatch && tiles <= kOrderTiles && tiles * heads > 512;
}

// order[rank] = a tile's place, by falling numbers of keys (of queries for tiles of keys)
// that its rows see (are seen by), empty tiles last.
__global__ __launch_bounds__(256) void k_order(AttnArgs a, bool keys, int tiles, TilePlace *order) {
  constexpr int M = kBlock;
  __shared__ int mine[kOrderBatch + 1], other[kOrderBatch + 1], work[kOrderTiles];
  const int32_t *off = keys ? a.k_off : a.q_off, *oth = keys ? a.q_off : a.k_off;
  const int64_t n = keys ? a.n_k : a.n_q, no = keys ? a.n_q : a.n_k;
  for (int i = threadIdx.x; i <= a.batch; i += 256) {
    mine[i] = (int)offset_of(off, i, n);
    other[i] = (int)offset_of(oth, i, no);
  }
  __syncthreads();
  TilePlace place{};  // of tile 256 blockIdx.x + threadIdx.x
  for (int t = threadIdx.x; t < tiles; t += 256) {
    int s = 0;
    for (int step = 1024; step; step >>= 1)
      if (s + step <= a.batch && mine[s + step] / M + s + step <= t) s += step;
    const int end = s < a.batch ? mine[s + 1] : (int)n, len = max(0, end - mine[s]);
    const int r0 = (t - (mine[s] / M + s)) * M, r1 = min(r0 + M, len) - 1;
    const int lo = s < a.batch ? max(0, other[s + 1] - other[s]) : 0;  // rows of the other side
    int w = 0;
    if (r0 < len) {
      const int d = keys ? len - lo : lo - len;  // keys less queries
      int from = 0, to = lo;
      if (a.causal && keys) {
        from = max(0, r0 - d);
        if (a.window > 0) to = (int)min((int64_t)lo, (int64_t)r1 + a.window - d);
      } else if (a.causal) {
        to = min(lo, r1 + d + 1);
        if (a.window > 0) from = max(0, r0 + d - a.window + 1);
      }
      w = 1 + max(0, to - from);
    }
    work[t] = w;
    if (t / 256 == (int)blockIdx.x) {
      const int other0 = s < a.batch ? other[s] : 0;
      place = keys ? TilePlace{r0, other0, lo, mine[s], len, {}} : TilePlace{r0, mine[s], len, other0, lo, {}};
    }
  }
  __syncthreads();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= tiles) return;
  const int w = work[t];
  int rank = 0;
  for (int u = 0; u < tiles; ++u) rank += work[u] > w || (work[u] == w && u < t);
  order[rank] = place;
}

// Rows of the other side a step: two steps' tiles of two blocks fit a CU's LDS.
template <typename T>
constexpr int step_rows() { return sizeof(T) == 2 ? 64 : 32; }
// Blocks a CU that the registers of the forward and of dq must allow: operands of 128 fp32
// channels take twice the registers, and their products eight times as long. (4096 tokens of 8
// heads of 128 fp32: 902 us with two blocks, whose registers go to memory, 663 with one.)
template <typename T, int DP>
constexpr int blocks_a_cu() { return sizeof(T) == 4 && DP > 64 ? 1 : 2; }
constexpr int kAhead = 4;  // operands read from LDS ahead of their products

template <typename T, int DP, int CH>
__global__ __launch_bounds__(kThreads, (blocks_a_cu<T, DP>())) void k_fwd(AttnArgs a, int64_t tiles) {
  constexpr int KS = step_rows<T>(), NT = KS / 32;
  using C = Copier<T, DP, KS, kWaves>;
  extern __shared__ __align__(1024) char smem[];
  T *const buf = (T *)smem;  // two tiles of keys, two of values
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, h = l >> 5;
  const Work w = work_of(a);
  if (w.rank >= tiles) return;
  const TilePlace at = a.q_order ? a.q_order[w.rank] : tile_place(a, false, tiles - 1 - w.rank, l);
  const Rows rq{at.q_start, at.lq}, rk{at.k_start, at.lk};
  const int first = at.first;
  if (first < 0 || first >= rq.len) return;  // (below 0: offsets that fall)
  const int lq = rq.len, lk = rk.len;
  const int q0 = first + kRows * wave, qi = q0 + (l & 31);
  const int qr = min(qi, lq - 1);
  const T *qp = (const T *)a.q.p + (rq.start + qr) * a.q.tok_stride + w.head * a.q.head_stride;
  const C kc((const T *)a.k.p + rk.start * a.k.tok_stride + w.kv * a.k.head_stride, a.k.tok_stride, a.dh, wave, l);
  const C vc((const T *)a.v.p + rk.start * a.v.tok_stride + w.kv * a.v.head_stride, a.v.tok_stride, a.dh, wave, l);
  Frag<T> q[CH / 16];
#pragma unroll
  for (int i = 0; i < CH / 16; ++i) q[i] = with_sign<T>(load_frag<T>(qp, i, h, a.dh), a.scale);
  const Seen mine = seen_by(a, qi, lq, lk);
  const Seen head = seen_by(a, first, lq, lk), tail = seen_by(a, min(first + kBlock, lq) - 1, lq, lk);
  // what all, and what some, of this wave's rows see (those behind the last are not stored)
  const Seen wf = seen_by(a, q0, lq, lk), wl = seen_by(a, q0 + kRows - 1, lq, lk);
  const float c = log2_scale(a.scale);
  if (a.dh != DP) {
    clear(buf, 4 * KS * DP, tid, kThreads);
    __syncthreads();
  }
  f32x16 acc[CH / 32], x[NT];
  Frag<T> p[KS / 16], v[kAhead];
  float m, sum, base = 0.f, mc = 0.f;  // base: m, or 0 before any key
  const int begin = head.lo / KS * KS;
  constexpr int N = KS / 16 * (CH / 32), E = 16 * NT;
  constexpr int TILE = KS * DP * (int)sizeof(T);
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < CH / 32; ++d) acc[d] = f32x16{};
#pragma unroll
    for (int i = 0; i < KS / 16; ++i) p[i] = zero_frag<T>();
    m = -INFINITY;
    sum = 0.f;
    int cur = 0;  // this tile's buffers; the other value buffer holds the tile before
    RowReader<T, DP> kr(buf, l);
    ColReader<T, DP> vr(buf + 3 * KS * DP, l);
    const auto key = [&](int n) __attribute__((always_inline)) { return kr.read(32 * (n % NT), n / NT); };
    const auto value = [&](int n) __attribute__((always_inline)) {
      return vr.read(16 * (n / (CH / 32)), n % (CH / 32));
    };
    if (begin < tail.hi) kc.issue(buf, begin, lk, a.dh, wave, l, kAsIs);
    clear(buf + 3 * KS * DP, KS * DP, tid, kThreads);  // no tile before the first
    for (int k0 = begin; k0 < tail.hi; k0 += KS) {
      // this tile's keys and the values of the one before have landed, and no wave reads
      // what is overwritten now: the keys and values of the tiles before those
      mfma::wait_vm<0>();
      mfma::lds_barrier();
      vc.issue(buf + (2 + cur) * KS * DP, k0, lk, a.dh, wave, l, fix);
      cur ^= 1;
      if (k0 + KS < tail.hi) kc.issue(buf + cur * KS * DP, k0 + KS, lk, a.dh, wave, l, kAsIs);
      // whether the lane's query sees its key j of the tile
      const int from = k0 + 4 * h - mine.lo;
      const unsigned keys = max(0, mine.hi - mine.lo);
      const auto sees = [&](int j) { return (unsigned)(from + j) < keys; };
      {
        constexpr int M = NT * CH / 16;
        Frag<T> k[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) k[n] = key(n);
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < M; ++n) {
          x[n % NT] = mma(k[n % kAhead], q[n / NT], x[n % NT]);
          if (n + kAhead < M) k[n % kAhead] = key(n + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int n = 0; n < kAhead; ++n) v[n] = value(n);
      if (k0 + KS > wf.hi || k0 < wl.lo) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (!sees(32 * t + 8 * (i / 4) + i % 4)) x[t][i] = -INFINITY;
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[t][i]);
      top = half_max(top);
      const bool rescale = __ballot((top - m) * c > kSlack) != 0;
      float f = 1.f;
      if (rescale) {
        const float next = fmaxf(m, top);
        f = next == -INFINITY ? 1.f : exp2_((m - next) * c);
        m = next;
        base = m == -INFINITY ? 0.f : m;
        mc = base * c;
        sum *= f;
      }
      // The tile before is added to the values while this one's scores become weights: the
      // matrix cores work on the one, the vector units on the other.
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        f32x16 &o = acc[n % (CH / 32)];
        o = mma(v[n % kAhead], p[n / (CH / 32)], o);
        if (n + kAhead < N) v[n % kAhead] = value(n + kAhead);
#pragma unroll
        for (int e = E * n / N; e < E * (n + 1) / N; ++e) {
          // (fp32 as written: a query's only key then has the weight 1 to the bit)
          float weight = exp2_(sizeof(T) == 4 ? (x[e / 16][e % 16] - base) * c
                                              : __builtin_fmaf(x[e / 16][e % 16], c, -mc));
          asm volatile("" : "+v"(weight));  // here, not behind the products
          x[e / 16][e % 16] = weight;
          part[e % 4] += weight;
          asm volatile("" : "+v"(part[e % 4]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      sum += (part[0] + part[1]) + (part[2] + part[3]);
      if (rescale && fix != kCount) {  // (counts are no weights)
#pragma unroll
        for (int d = 0; d < CH / 32; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[d][e] *= f;
      }
      if (fix == kCount) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[t][i] = sees(32 * t + 8 * (i / 4) + i % 4) ? 1.f : 0.f;
          }
      }
#pragma unroll
      for (int i = 0; i < KS / 16; ++i) p[i] = as_operand<T>(x[i / 2], i % 2);
      kr.move(cur ? TILE : -TILE);
      vr.move(cur ? -TILE : TILE);
    }
    mfma::wait_vm<0>();
    mfma::lds_barrier();
#pragma unroll
    for (int n = 0; n < N; ++n)
      acc[n % (CH / 32)] = mma(value(n), p[n / (CH / 32)], acc[n % (CH / 32)]);
    if (fix == kAsIs && !__syncthreads_and(all_finite(acc))) continue;
    const float total = half_sum(sum);
    if (qi < lq) {
      const bool none = mine.lo >= mine.hi;
      T *const op = (T *)a.o.p + (rq.start + qi) * a.o.tok_stride + w.head * a.o.head_stride;
      if (none) {
#pragma unroll
        for (int d = 0; d < CH / 32; ++d) acc[d] = f32x16{};
      }
      store_row<T, CH>(op, acc, none ? 0.f : 1.f / total, h, a.dh, fix);
      if (a.lse && h == 0)
        a.lse[w.head * a.n_q + rq.start + qi] = none ? -INFINITY : (m * c + log2f(total)) * kLn2;
    }
    if (fix != kCount) break;
    __syncthreads();  // the buffers are filled anew
  }
}

// delta = sum(dy o) of each query and head, and the forward's lse in units of log2. A row
// with an infinite lse, if it sees a key at all, has no softmax, and one whose delta is not
// finite has differences infinity - infinity: both are NaN here, since the products beside
// them leave out what is not finite in q and dy, and would make infinities of them. (A row
// that sees no key is masked where it is used.) The sums are the diagonal of
// a 32 x 32 product of o and dy, so that they are added in the order in which the backward's
// products add dP = dy V: a query that sees one key, whose o is that key's v, then has
// dP = delta to the bit, and gradients of zero. (o is the forward's result as it was rounded to
// its type; with the rounding of ds that gives dq and dk in bf16 an error of 2.6e-3 to 3.2e-3,
// where rounding the exact gradients makes 1.7e-3.) A wave takes 32 tokens of one head.
template <typename T, int DP, int CH>
__global__ __launch_bounds__(256) void k_delta(AttnArgs a) {
  extern __shared__ __align__(1024) char smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, h = l >> 5, q = l & 31;
  const int64_t unit = (int64_t)uniform64(blk::block_id()) * 4 + wave;
  const int64_t t0 = unit / a.hq * 32;
  const int hd = (int)(unit % a.hq);
  if (t0 >= a.n_q) return;
  T *const ot = (T *)smem + wave * 64 * DP, *const yt = ot + 32 * DP;
  if (a.dh != DP) {
    clear(ot, 64 * DP, l, 64);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  const int left = (int)(a.n_q - t0 < 32 ? a.n_q - t0 : 32);
  const Copier<T, DP, 32, 1> oc((const T *)a.o.p + t0 * a.o.tok_stride + hd * a.o.head_stride, a.o.tok_stride, a.dh,
                                0, l);
  const Copier<T, DP, 32, 1> yc((const T *)a.dy.p + t0 * a.dy.tok_stride + hd * a.dy.head_stride, a.dy.tok_stride,
                                a.dh, 0, l);
  oc.issue(ot, 0, left, a.dh, 0, l, kAsIs);
  yc.issue(yt, 0, left, a.dh, 0, l, kAsIs);
  mfma::wait_vm<0>();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // one wave's own tiles
  const RowReader<T, DP> rows(ot, l);
  f32x16 x{};
#pragma unroll
  for (int i = 0; i < CH / 16; ++i) x = mma(rows.read(0, i), rows.read(32, i), x);
  const int64_t t = t0 + q;
  // row q of column q
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (8 * (i / 4) + i % 4 == (q & ~4)) v = x[i];
  if ((q >> 2 & 1) == h && q < left) {
    const float lse = a.lse[hd * a.n_q + t];
    a.delta[hd * a.n_q + t] = __builtin_isfinite(v) ? v : NAN;
    a.lse2[hd * a.n_q + t] = __builtin_isinf(lse) ? NAN : lse * kLog2e;
  }
}

// dq: a block's queries, over the keys that they see.
template <typename T, int DP, int CH>
__global__ __launch_bounds__(kThreads, (blocks_a_cu<T, DP>())) void k_dq(AttnArgs a, int64_t tiles) {
  constexpr int KS = step_rows<T>(), NT = KS / 32, STAGE = 2 * KS * DP * (int)sizeof(T);
  using C = Copier<T, DP, KS, kWaves>;
  extern __shared__ __align__(1024) char smem[];
  T *const buf = (T *)smem;  // [2][K tile, V tile]
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, h = l >> 5;
  const Work w = work_of(a);
  if (w.rank >= tiles) return;
  const TilePlace at = a.q_order ? a.q_order[w.rank] : tile_place(a, false, tiles - 1 - w.rank, l);
  const Rows rq{at.q_start, at.lq}, rk{at.k_start, at.lk};
  const int first = at.first;
  if (first < 0 || first >= rq.len) return;  // (below 0: offsets that fall)
  const int lq = rq.len, lk = rk.len;
  const int q0 = first + kRows * wave, qi = q0 + (l & 31);
  const int64_t qr = rq.start + min(qi, lq - 1);
  const T *qp = (const T *)a.q.p + qr * a.q.tok_stride + w.head * a.q.head_stride;
  const T *yp = (const T *)a.dy.p + qr * a.dy.tok_stride + w.head * a.dy.head_stride;
  const C kc((const T *)a.k.p + rk.start * a.k.tok_stride + w.kv * a.k.head_stride, a.k.tok_stride, a.dh, wave, l);
  const C vc((const T *)a.v.p + rk.start * a.v.tok_stride + w.kv * a.v.head_stride, a.v.tok_stride, a.dh, wave, l);
  Frag<T> q[CH / 16], dy[CH / 16];
#pragma unroll
  for (int i = 0; i < CH / 16; ++i) {
    q[i] = with_sign<T>(load_frag<T>(qp, i, h, a.dh), a.scale);
    dy[i] = load_frag<T>(yp, i, h, a.dh);
  }
  const Seen mine = seen_by(a, qi, lq, lk);
  const Seen head = seen_by(a, first, lq, lk), tail = seen_by(a, min(first + kBlock, lq) - 1, lq, lk);
  const Seen wf = seen_by(a, q0, lq, lk), wl = seen_by(a, q0 + kRows - 1, lq, lk);
  const float c = log2_scale(a.scale);
  const float lse = a.lse2[w.head * a.n_q + qr], delta = a.delta[w.head * a.n_q + qr];
  if (a.dh != DP) {
    clear(buf, 4 * KS * DP, tid, kThreads);
    __syncthreads();
  }
  const int begin = head.lo / KS * KS;
  f32x16 acc[CH / 32];
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < CH / 32; ++d) acc[d] = f32x16{};
    int cur = 0;
    RowReader<T, DP> rows(buf, l);
    ColReader<T, DP> cols(buf, l);
    // Scores are those of the keys as they are, also where dS meets keys with something left out
    // (an infinite key may have the score -infinity, and no weight). The passes that fix keys,
    // which are rare, have the fixed ones in the second buffer and copy nothing ahead.
    if (fix != kAsIs) cols.move(STAGE);
    const auto issue = [&](int k0, int b) __attribute__((always_inline)) {
      T *const t = buf + b * 2 * KS * DP;
      kc.issue(t, k0, lk, a.dh, wave, l, kAsIs);
      vc.issue(t + KS * DP, k0, lk, a.dh, wave, l, kAsIs);
    };
    for (int k0 = begin; k0 < tail.hi; k0 += KS) {
      if (fix != kAsIs || k0 == begin) {
        mfma::lds_barrier();  // no wave reads the tiles before
        issue(k0, 0);
      }
      mfma::wait_vm<0>();
      mfma::lds_barrier();
      if (fix == kAsIs) {
        cur ^= 1;
        if (k0 + KS < tail.hi) issue(k0 + KS, cur);
      } else {
        for (int i = here(tid); i < KS * DP; i += kThreads) buf[2 * KS * DP + i] = fixed(buf[i], fix);
        mfma::lds_barrier();
      }
      const bool whole = k0 + KS <= wf.hi && k0 >= wl.lo;
      const auto each_seen = [&](int t, auto f) __attribute__((always_inline)) {
        const int rel = k0 + 32 * t + 4 * h - mine.lo;
        const unsigned keys = max(0, mine.hi - mine.lo);
#pragma unroll
        for (int i = 0; i < 16; ++i) f(i, (unsigned)(rel + 8 * (i / 4) + i % 4) < keys);
      };
      // For each 32 keys S and dP, then the sums for all of them; what the vector units do
      // goes beside the products that do not wait for it:
      //   S(t) beside dS(t - 1), dP(t) beside P(t), the first sums beside the last dS.
      constexpr int S = CH / 16, ND = CH / 32, LEN = NT * (2 * S + 2 * ND);
      const auto operand = [&](int m) __attribute__((always_inline)) {
        if (m >= 2 * S * NT) {
          const int e = m - 2 * S * NT;
          return cols.read(16 * (e / ND), e % ND);
        }
        const int t = m / (2 * S), o = m % (2 * S);
        return rows.read((o < S ? 0 : KS) + 32 * t, o % S);
      };
      Frag<T> f[kAhead];
#pragma unroll
      for (int m = 0; m < kAhead; ++m) f[m] = operand(m);
      const auto refill = [&](int m) __attribute__((always_inline)) {
        if (m + kAhead < LEN) f[m % kAhead] = operand(m + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      };
      f32x16 x[NT], y[NT];
      Frag<T> ds[NT][2];
      // elements e0 .. e1 - 1 of dS(t), in x
      const auto grad = [&](int t, int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
        for (int e = e0; e < e1; ++e) {
          float v = x[t][e] * (y[t][e] - delta);
          asm volatile("" : "+v"(v));  // here, not behind the products
          x[t][e] = v;
        }
      };
      const auto finish = [&](int t) __attribute__((always_inline)) {
        if (!whole)
          each_seen(t, [&](int i, bool ok) __attribute__((always_inline)) {
            if (!ok) x[t][i] = 0.f;
          });
        if (fix == kCount)
          each_seen(t, [&](int i, bool ok) __attribute__((always_inline)) { x[t][i] = ok ? 1.f : 0.f; });
        ds[t][0] = as_operand<T>(x[t], 0);
        ds[t][1] = as_operand<T>(x[t], 1);
      };
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        x[t] = y[t] = f32x16{};
#pragma unroll
        for (int o = 0; o < S; ++o) {
          const int m = 2 * S * t + o;
          x[t] = mma(f[m % kAhead], q[o], x[t]);
          if (t > 0) grad(t - 1, 16 * o / S, 16 * (o + 1) / S);
          refill(m);
        }
        if (t > 0) finish(t - 1);
#pragma unroll
        for (int o = 0; o < S; ++o) {
          const int m = 2 * S * t + S + o;
          y[t] = mma(f[m % kAhead], dy[o], y[t]);
#pragma unroll
          for (int e = 16 * o / S; e < 16 * (o + 1) / S; ++e) {
            float v = exp2_(__builtin_fmaf(x[t][e], c, -lse));
            asm volatile("" : "+v"(v));
            x[t][e] = v;
          }
          refill(m);
        }
      }
      if constexpr (NT == 1) {
        grad(0, 0, 16);
        finish(0);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int o = 0; o < 2 * ND; ++o) {
          const int m = 2 * S * NT + 2 * ND * t + o;
          acc[o % ND] = mma(f[m % kAhead], ds[t][o / ND], acc[o % ND]);
          if (NT > 1 && t == 0) {
            grad(NT - 1, 16 * o / (2 * ND), 16 * (o + 1) / (2 * ND));
          }
          refill(m);
          if (NT > 1 && t == 0 && o == 2 * ND - 1) finish(NT - 1);
        }
      if (fix == kAsIs) {
        rows.move(cur ? STAGE : -STAGE);
        cols.move(cur ? STAGE : -STAGE);
      }
    }
    if (fix == kAsIs && !__syncthreads_and(all_finite(acc))) continue;
    if (qi < lq)
      store_row<T, CH>((T *)a.dq.p + (rq.start + qi) * a.dq.tok_stride + w.head * a.dq.head_stride, acc, a.scale,
                       h, a.dh, fix);
    if (fix != kCount) break;
    __syncthreads();
  }
}

// dk and dv: a block's keys, over the queries of the group's heads that see them. A wave
// holds 32 keys: their sums and K rows in registers, their V rows in LDS, since both do not
// fit beside the sums. (64 keys a wave halve the LDS reads of a product, but leave a SIMD one
// wave, which does not cover its own waits: 1090 us for 16384 tokens in six documents of 16/8
// heads of 128 bf16, where 32 took 590 at the time, 500 now.)
// For 32 queries the products are, with what the vector units do beside them,
//   scores S = Q K^T;   dP = dY V^T beside P = exp(S - lse);
//   dV += dY^T P beside dS = P (dP - delta);   dK += Q^T dS.
// Where the key tiles are few, `parts` blocks share a tile's steps (part blockIdx.z) and
// leave partial sums, which k_dkv_join adds up.
template <typename T, int DP, int CH>
__global__ __launch_bounds__(kThreads, (sizeof(T) == 2 ? 2 : 1)) void k_dkv(AttnArgs a, int64_t tiles, int parts) {
  constexpr int QS = 32, NT = QS / 32, STAGE = 2 * QS * DP * (int)sizeof(T);
  constexpr int ND = CH / 32, S = CH / 16;
  constexpr int AHEAD = 3;  // operands read from LDS ahead of their products
  using C = Copier<T, DP, QS, kWaves>;
  extern __shared__ __align__(1024) char smem[];
  T *const buf = (T *)smem;                            // [2][q tile, dy tile]
  T *const vt = buf + 4 * QS * DP;                     // the block's V rows
  float *const stats = (float *)(vt + kBlock * DP);    // [2][lse, delta][64]
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, h = l >> 5;
  const int64_t id = blk::block_id();
  const int kv = (int)(id % a.hk);
  if (id / a.hk >= tiles) return;
  const TilePlace place = a.k_order ? a.k_order[id / a.hk] : tile_place(a, true, id / a.hk, l);
  const Rows rq{place.q_start, place.lq}, rk{place.k_start, place.lk};
  const int first = place.first;
  if (first < 0 || first >= rk.len) return;
  const int lq = rq.len, lk = rk.len, group = a.hq / a.hk;
  const int k0 = first + kRows * wave;
  // the queries that see key j: [from(j), to(j))
  const int off = lk - lq;
  const auto from = [&](int j) { return a.causal ? max(0, j - off) : 0; };
  const auto to = [&](int j) -> int {
    if (!a.causal || a.window <= 0) return lq;
    return (int)max((int64_t)0, min((int64_t)lq, (int64_t)j + a.window - off));
  };
  Frag<T> k[S];
  {
    const int kj = k0 + (l & 31);
    const T *kp = (const T *)a.k.p + (rk.start + min(kj, lk - 1)) * a.k.tok_stride + kv * a.k.head_stride;
#pragma unroll
    for (int i = 0; i < S; ++i) k[i] = with_sign<T>(load_frag<T>(kp, i, h, a.dh), a.scale);
  }
  const int q_from = from(first), q_to = to(min(first + kBlock, lk) - 1);
  const int all_from = from(k0 + kRows - 1), all_to = k0 + kRows <= lk ? to(k0) : 0;
  const int begin = q_from / QS * QS, steps = q_to > begin ? (q_to - begin + QS - 1) / QS : 0;
  const float c = log2_scale(a.scale);
  if (a.dh != DP) {
    clear(buf, (4 * QS + kBlock) * DP, tid, kThreads);
    __syncthreads();
  }
  const Copier<T, DP, kBlock, kWaves> vc((const T *)a.v.p + rk.start * a.v.tok_stride + kv * a.v.head_stride,
                                         a.v.tok_stride, a.dh, wave, l);
  vc.issue(vt, first, lk, a.dh, wave, l, kAsIs);
  const C qc((const T *)a.q.p + rq.start * a.q.tok_stride + (int64_t)kv * group * a.q.head_stride, a.q.tok_stride,
             a.dh, wave, l, a.q.head_stride);
  const C yc((const T *)a.dy.p + rq.start * a.dy.tok_stride + (int64_t)kv * group * a.dy.head_stride,
             a.dy.tok_stride, a.dh, wave, l, a.dy.head_stride);
  const auto issue = [&](int g, int i0, int b, int fix) __attribute__((always_inline)) {
    T *const t = buf + b * 2 * QS * DP;
    qc.issue(t, i0, lq, a.dh, wave, l, fix, g * a.q.head_stride);
    yc.issue(t + QS * DP, i0, lq, a.dh, wave, l, fix, g * a.dy.head_stride);
    if (wave < 2) {
      const float *src = (wave ? a.delta : a.lse2) + (kv * group + g) * a.n_q + rq.start;
      copy_to_lds<4>(uniform(src), 4 * (uint32_t)min(i0 + here(l), lq - 1), stats + (2 * b + wave) * 64);
    }
  };
  f32x16 dk[ND], dv[ND];
  for (int fix = kAsIs;; ++fix) {
#pragma unroll
    for (int d = 0; d < ND; ++d) dk[d] = dv[d] = f32x16{};
    int cur = 0;
    RowReader<T, DP> rows(buf, l);
    ColReader<T, DP> cols(buf, l);
    // Step n of head g, from the last queries to the first: the blocks of a key head that
    // run at once then read the same queries at about the same time, from L2.
    const auto queries_of = [&](int n) { return begin + (steps - 1 - n) * QS; };
    const int64_t all = (int64_t)group * steps;
    const int64_t stop = all * (blockIdx.z + 1) / parts;
    int64_t at = all * blockIdx.z / parts;
    int g = steps ? (int)(at / steps) : 0, n = steps ? (int)(at - (int64_t)g * steps) : 0;
    if (at < stop) issue(g, queries_of(n), 0, fix);
    for (; at < stop; ++at) {
      mfma::wait_vm<0>();
      mfma::lds_barrier();
      const float *const lse = stats + 2 * cur * 64 + 4 * h, *const delta = lse + 64;
      // from this step's tiles to the wave's V rows
      const int to_v = (2 - cur) * STAGE + kRows * wave * DP * (int)sizeof(T);
      cur ^= 1;
      const int i0 = queries_of(n);
      if (++n == steps) n = 0, ++g;
      if (at + 1 < stop) issue(g, queries_of(n), cur, fix);
      const bool whole = i0 >= all_from && i0 + QS <= all_to;
      // f(e, whether the lane's key is seen by the query of result e), for e < 16
      const auto each_seen = [&](int t, auto f) __attribute__((always_inline)) {
        const int ln = here(l);
        const int kj = k0 + (ln & 31), first = from(kj);
        const unsigned queries = kj < lk ? max(0, to(kj) - first) : 0;
        const int rel = i0 + 32 * t + 4 * (ln >> 5) - first;
#pragma unroll
        for (int i = 0; i < 16; ++i) f(i, (unsigned)(rel + 8 * (i / 4) + i % 4) < queries);
      };
      // the operands of the products in their order: S steps of S and dP, 2 ND of dV and dK
      constexpr int LEN = 2 * S + 4 * ND;
      const auto operand = [&](int m) __attribute__((always_inline)) {
        const int t = m / LEN, r = 32 * t, o = m % LEN;
        if (o < S) return rows.read(r, o);
        if (o < 2 * S) return rows.read(QS + r, o - S);
        const int e = (o - 2 * S) % (2 * ND), q = (o - 2 * S) / (2 * ND);
        return cols.read((q ? 0 : QS) + r + 16 * (e / ND), e % ND);
      };
      Frag<T> f[AHEAD], vb;
#pragma unroll
      for (int m = 0; m < AHEAD; ++m) f[m] = operand(m);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int m0 = t * LEN;
        // the next operand, in the place of the one just used
        const auto refill = [&](int m) __attribute__((always_inline)) {
          if (m + AHEAD < NT * LEN) f[m % AHEAD] = operand(m + AHEAD);
          __builtin_amdgcn_sched_barrier(0);
        };
        f32x16 x{}, y{};
        f32x4v st;
        // a statistic of the rows of results e .. e + 3
        const auto stat = [&](const float *p, int e) __attribute__((always_inline)) {
          return *(const f32x4v *)(p + 32 * t + 8 * (e / 4));
        };
        vb = rows.read_from(to_v, 0, 0);
#pragma unroll
        for (int o = 0; o < S; ++o) {
          x = mma(f[(m0 + o) % AHEAD], k[o], x);
          refill(m0 + o);
        }
#pragma unroll
        for (int o = 0; o < S; ++o) {
          y = mma(f[(m0 + S + o) % AHEAD], vb, y);
          if (o + 1 < S) vb = rows.read_from(to_v, 0, o + 1);
#pragma unroll
          for (int e = 16 * o / S; e < 16 * (o + 1) / S; ++e) {
            if (e % 4 == 0 || e == 16 * o / S) st = stat(lse, e);
            float p = exp2_(__builtin_fmaf(x[e], c, -st[e % 4]));
            asm volatile("" : "+v"(p));  // here, not behind the products
            x[e] = p;
          }
          refill(m0 + S + o);
        }
        if (!whole)
          each_seen(t, [&](int e, bool ok) __attribute__((always_inline)) {
            if (!ok) x[e] = 0.f;
          });
        if (fix == kCount)
          each_seen(t, [&](int e, bool ok) __attribute__((always_inline)) { x[e] = ok ? 1.f : 0.f; });
        Frag<T> w[2] = {as_operand<T>(x, 0), as_operand<T>(x, 1)};
#pragma unroll
        for (int o = 0; o < 2 * ND; ++o) {
          dv[o % ND] = mma(f[(m0 + 2 * S + o) % AHEAD], w[o / ND], dv[o % ND]);
#pragma unroll
          for (int e = 16 * o / (2 * ND); e < 16 * (o + 1) / (2 * ND); ++e) {
            if (e % 4 == 0 || e == 16 * o / (2 * ND)) st = stat(delta, e);
            float ds = x[e] * (y[e] - st[e % 4]);
            asm volatile("" : "+v"(ds));
            y[e] = ds;
          }
          refill(m0 + 2 * S + o);
        }
        if (!whole)
          each_seen(t, [&](int e, bool ok) __attribute__((always_inline)) {
            if (!ok) y[e] = 0.f;
          });
        w[0] = as_operand<T>(y, 0);
        w[1] = as_operand<T>(y, 1);
#pragma unroll
        for (int o = 0; o < 2 * ND; ++o) {
          dk[o % ND] = mma(f[(m0 + 2 * S + 2 * ND + o) % AHEAD], w[o / ND], dk[o % ND]);
          refill(m0 + 2 * S + 2 * ND + o);
        }
      }
      rows.move(cur ? STAGE : -STAGE);
      cols.move(cur ? STAGE : -STAGE);
    }
    if (fix == kAsIs && !__syncthreads_and(all_finite(dk) && all_finite(dv))) continue;
    const int kj = k0 + here(l & 31);
    if (kj < lk) {
      const int64_t kr = rk.start + kj;
      if (parts > 1) {
        float *const pk = a.part + ((((int64_t)blockIdx.z * a.n_k + kr) * a.hk + kv) * 2) * a.dh;
        store_row<float, CH>(pk, dk, a.scale, h, a.dh, kAsIs);
        store_row<float, CH>(pk + a.dh, dv, 1.f, h, a.dh, fix);
      } else {
        store_row<T, CH>((T *)a.dk.p + kr * a.dk.tok_stride + kv * a.dk.head_stride, dk, a.scale, h, a.dh, kAsIs);
        store_row<T, CH>((T *)a.dv.p + kr * a.dv.tok_stride + kv * a.dv.head_stride, dv, 1.f, h, a.dh, fix);
      }
    }
    if (fix != kCount) break;
    __syncthreads();
  }
}

// dk and dv from the parts' sums [parts][n_k][hk][dk, dv][dh], in their order.
template <typename T>
__global__ __launch_bounds__(256) void k_dkv_join(AttnArgs a, int parts) {
  const int64_t i = blk::block_id() * 256 + threadIdx.x, size = a.n_k * a.hk * 2 * a.dh;
  if (i >= size) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v += a.part[p * size + i];
  const int64_t row = i / a.dh, kr = row / (2 * a.hk);
  const int c = (int)(i - row * a.dh), x = (int)(row - kr * 2 * a.hk);
  const ipttt_heads &out = x % 2 ? a.dv : a.dk;
  ((T *)out.p)[kr * out.tok_stride + x / 2 * out.head_stride + c] = (T)v;
}

// f(channels a row has in LDS, channels that are computed): rows of 65 to 96 channels leave
// out a quarter of the products (16384 tokens of 16/8 heads of 96 bf16: 1.20 -> 0.93 ms).
template <typename T, class F>
void by_width(int dh, F f) {
  using std::integral_constant;
  if (dh <= 64) f(integral_constant<int, 64>(), integral_constant<int, 64>());
  else if (dh <= 96) f(integral_constant<int, 128>(), integral_constant<int, 96>());
  else f(integral_constant<int, 128>(), integral_constant<int, 128>());
}

// Blocks that share a tile of keys: as many as bring the grid to two blocks a CU, while each
// has four steps of 32 queries of one head or more. (512 tokens of 8/2 heads of 128 bf16, 12
// blocks of their own: backward 142 us, shared 58.)
int parts_of(int hq, int hk, int64_t n_q, int64_t n_k, int batch) {
  const int64_t blocks = tiles_of(n_k, kBlock, batch) * hk;
  if (blocks >= 384 || n_k == 0) return 1;
  const int64_t most = (int64_t)(hq / hk) * (n_q / 32) / 4;
  const int64_t p = 512 / blocks;
  return (int)(p < most ? (p < 1 ? 1 : p) : most < 1 ? 1 : most);
}

// Fills the order of tiles, or says that it is not used.
TilePlace *order_tiles(const AttnArgs &a, bool keys, TilePlace *order, hipStream_t st) {
  const int64_t tiles = tiles_of(keys ? a.n_k : a.n_q, kBlock, a.batch);
  if (!ordered(a.batch, tiles, keys ? a.hk : a.hq)) return nullptr;
  k_order<<<(int)(tiles + 255) / 256, 256, 0, st>>>(a, keys, (int)tiles, order);
  return order;
}

}  // namespace

bool attn_size_ok(int hq, int batch, int64_t n) {
  return tiles_of(n, kBlock, batch) * hq < ((int64_t)1 << 31);
}
size_t attn_q_order(const ipttt_attention &d) {
  const int64_t tiles = tiles_of(d.n_q, kBlock, d.batch);
  return ordered(d.batch, tiles, d.q_heads) ? round_up(tiles * sizeof(TilePlace), 256) : 256;
}
size_t attn_parts(const ipttt_attention &d) {
  const int parts = parts_of(d.q_heads, d.k_heads, d.n_q, d.n_k, d.batch);
  return parts > 1 ? round_up(parts * d.n_k * d.k_heads * 2 * d.head_dim * 4, 256) : 0;
}
size_t attn_k_order(const ipttt_attention &d) {
  const int64_t tiles = tiles_of(d.n_k, kBlock, d.batch);
  return ordered(d.batch, tiles, d.k_heads) ? round_up(tiles * sizeof(TilePlace), 256) : 256;
}

template <typename T>
hipError_t attn_forward(const AttnArgs &args, hipStream_t st) {
  AttnArgs a = args;
  a.q_order = order_tiles(a, false, a.q_order, st);
  by_width<T>(a.dh, [&](auto dp, auto ch) {
    constexpr int DP = decltype(dp)::value, CH = decltype(ch)::value;
    const int64_t tiles = tiles_of(a.n_q, kBlock, a.batch);
    k_fwd<T, DP, CH><<<blk::grid_of(tiles * a.hq), kThreads, 4 * step_rows<T>() * DP * sizeof(T), st>>>(
        a, tiles);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t attn_backward(const AttnArgs &args, hipStream_t st) {
  AttnArgs a = args;
  a.q_order = order_tiles(a, false, a.q_order, st);
  a.k_order = order_tiles(a, true, a.k_order, st);
  const int parts = parts_of(a.hq, a.hk, a.n_q, a.n_k, a.batch);
  by_width<T>(a.dh, [&](auto dp, auto ch) {
    constexpr int DP = decltype(dp)::value, CH = decltype(ch)::value;
    const size_t lds = 4 * step_rows<T>() * DP * sizeof(T);
    if (a.n_q > 0)
      k_delta<T, DP, CH><<<blk::grid_of(((a.n_q + 31) / 32 * a.hq + 3) / 4), 256, 4 * 64 * DP * sizeof(T), st>>>(a);
    if (a.n_k > 0) {
      const int64_t tiles = tiles_of(a.n_k, kBlock, a.batch);
      dim3 grid = blk::grid_of(tiles * a.hk);
      grid.z = parts;
      constexpr size_t lds = (4 * 32 + kBlock) * DP * sizeof(T) + 4 * 64 * sizeof(float);
      k_dkv<T, DP, CH><<<grid, kThreads, lds, st>>>(a, tiles, parts);
      if (parts > 1) k_dkv_join<T><<<blk::grid_of((a.n_k * a.hk * 2 * a.dh + 255) / 256), 256, 0, st>>>(a, parts);
    }
    if (a.n_q > 0) {
      const int64_t tiles = tiles_of(a.n_q, kBlock, a.batch);
      k_dq<T, DP, CH><<<blk::grid_of(tiles * a.hq), kThreads, lds, st>>>(a, tiles);
    }
  });
  return hipGetLastError();
}

template hipError_t attn_forward<float>(const AttnArgs &, hipStream_t);
template hipError_t attn_forward<__bf16>(const AttnArgs &, hipStream_t);
template hipError_t attn_backward<float>(const AttnArgs &, hipStream_t);
template hipError_t attn_backward<__bf16>(const AttnArgs &, hipStream_t);

}  // namespace ipttt
