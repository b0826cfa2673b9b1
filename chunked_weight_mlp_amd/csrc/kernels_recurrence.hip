// The gated linear recurrence h_t = f_t h_{t-1} + (1 - f_t) v_t, f = sigmoid(g),
// forward and backward.
//
// Each step is an affine map of the state, s -> A s + B, and maps compose:
// (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2). So a sequence is cut into tiles
// of tokens that are read once and kept in registers: a tile reduces its tokens to
// one map per channel, learns the state before it from the maps of the tiles in
// front of it, and then runs its own tokens from that state. A document start
// makes a map that ignores the state (kept as a flag, not as A = 0, so that a
// state that is not finite does not leak through 0 x inf). The backward runs the
// same way from the last token to the first on the gradient of the state.
// Few tokens (SEQ_MAX) are walked by one thread per channel pair instead.
//
// A gate that remembers has f within a few 2^-24 of 1, and a rounded f is wrong in what it
// forgets, 1 - f, the same way at every token: at g = 12, 131072 tokens would leave a
// state off by 7e-3. So what is handed on, from tile to tile and from call to call,
// goes by 1 - f: a product of gates is kept as 1 minus itself while it is above a half
// (Factor). Rounded factors serve over 16 tokens, a wave's or a walk's, where they are off
// by 5e-7 at most.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "block_internal.h"

namespace ipttt {
namespace {

using blk::Pack;

// f = 1 / (1 + e^-x) and i = 1 - f = 1 / (1 + e^x): for x > 0 i is e^-x f (1 - f would
// cancel), else it is 1 - f (e^-x may overflow). e^-x is off by about |x| 2^-24 of
// itself, a rounding of x log2(e): so are i for x > 0 and f for x < 0 (8 ulp at |x| = 20,
// 31 at 80).
__device__ __forceinline__ void gate(float x, float &f, float &i) {
  const float e = __expf(-x);
  f = __builtin_amdgcn_rcpf(1.f + e);
  i = x > 0.f ? e * f : 1.f - f;
}

// s, or the largest value of its sign where it is infinite: what is then taken from an
// infinite state leaves it what it is.
__device__ __forceinline__ float finite(float s) {
  return __builtin_amdgcn_fmed3f(s, -FLT_MAX, FLT_MAX);
}

// A Factor is a product A of gates: A itself up to 1/2, and above that -(1 - A), told
// apart by the sign (-0 is 1). -1 stands for a document start between (kCut), past which
// the state before counts for nothing.
constexpr float kCut = -1.f;
__device__ __forceinline__ bool sign_set(float a) { return (int)__builtin_bit_cast(uint32_t, a) < 0; }
// A s + b (the factor no document start)
__device__ __forceinline__ float affine(float a, float s, float b) {
  const float x = fmaf(a, sign_set(a) ? finite(s) : s, b);
  return sign_set(a) ? s + x : x;
}
// The state s through the map (a, b).
__device__ __forceinline__ float through(float a, float b, float s) {
  const float x = affine(a, s, b);
  return a == kCut ? b : x;
}
// A product as it grows: itself, and the sum of what each gate took of it, which is 1
// minus it.
struct Product {
  float p = 1.f, n = 0.f;
  __device__ __forceinline__ void take(float f, float i) {
    n = fmaf(i, p, n);
    p *= f;
  }
  // the same for a Factor
  __device__ __forceinline__ void times(float a) {
    n = fmaf(sign_set(a) ? -a : 1.f - a, p, n);
    p *= sign_set(a) ? 1.f + a : a;
  }
  __device__ __forceinline__ float factor() const { return p > 0.5f ? -n : p; }
};

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

// One thread walks V channels of one sequence from its first token to its last, U tokens'
// loads in flight, and makes the map of them all for the state it hands on.
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
  float s0[SEQ_V], q[SEQ_V] = {};
  Product W[SEQ_V];
  bool any = false;  // a document start
#pragma unroll
  for (int e = 0; e < SEQ_V; ++e) s0[e] = s[e];
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
        q[e] = cut[u] ? b : fmaf(f, q[e], b);
        W[e].take(f, i);
      }
      any = any || cut[u];
      store_ch<T, SEQ_V>(h + (t0 + u) * a.h.tok_stride, c, a.d, s);
    }
  }
  if (a.h_last) {
#pragma unroll
    for (int e = 0; e < SEQ_V; ++e) s[e] = through(any ? kCut : W[e].factor(), q[e], s0[e]);
    store_ch<float, SEQ_V>(a.h_last + (int64_t)n * a.d, c, a.d, s);
  }
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
  float s0[SEQ_V], q[SEQ_V] = {};
  Product W[SEQ_V];
  bool any = false;  // a document start
#pragma unroll
  for (int e = 0; e < SEQ_V; ++e) s0[e] = s[e];
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
        q[e] = cut[u] ? 0.f : f * (dd[u][e] + q[e]);
        W[e].take(f, i);
      }
      any = any || cut[u];
      store_ch<T, SEQ_V>(dg + t * a.dg.tok_stride, c, a.d, og);
      store_ch<T, SEQ_V>(dv + t * a.dv.tok_stride, c, a.d, ov);
    }
  }
  if (a.dh0) {
#pragma unroll
    for (int e = 0; e < SEQ_V; ++e) s[e] = through(any ? kCut : W[e].factor(), q[e], s0[e]);
    store_ch<float, SEQ_V>(a.dh0 + (int64_t)n * a.d, c, a.d, s);
  }
}

// ---- tiles ---------------------------------------------------------------------------
// A block of NW waves takes TT = NW R tokens of 64 V channels of one sequence;
// a lane holds V channels, a wave R consecutive tokens.
//
// Tiles of one (sequence, channel block) form a chain in groups of G. They meet in
// slots of 8 bytes per channel: all ones (empty, written by k_rec_clear), then a map
// (A, B), A as a Factor, or (kCut, s) for one that ignores the state: a value that
// validates itself, so a slot needs no flag and no fence. A tile publishes its map. The
// last tile of a group composes the group's maps in order, publishes that map, and then,
// once it knows the state before the group, the state after it in the same slot. A tile's
// state is that of its group's start, the nearest published state behind it with the
// groups' maps in between applied in order, and the maps of the tiles before it in
// its group, in order: the same operations whichever slots already held states, so
// results do not depend on timing. Tiles are handed out by a counter in chain order,
// so every tile a block waits for is held by a block that already runs and, by
// induction from the first tile of each chain, ends.

constexpr uint64_t kEmpty = ~(uint64_t)0;
// Polls of a tile before it gives up and returns NaN (about a second; a chain in
// order never gets near it): a wait that cannot last for ever.
constexpr int kMaxPolls = 1 << 20;

__device__ __forceinline__ uint64_t slot_pack(float a, float b) {
  uint32_t ua = __builtin_bit_cast(uint32_t, a);
  const uint32_t ub = __builtin_bit_cast(uint32_t, b);
  if ((ua & ub) == ~0u) ua = 0x7fc00000u;  // a NaN pair that would read as empty
  return (uint64_t)ub << 32 | ua;
}
__device__ __forceinline__ void slot_put(uint64_t *p, float a, float b) {
  __hip_atomic_store(p, slot_pack(a, b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t slot_get(const uint64_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A chain's place in the workspace. Tile `ord` of the launch's order and group g of
// the chain have their channels' slots at tile(ord) and group(g).
constexpr int LB = 1;  // slots a wave reads of each kind: groups of NW LB tiles
struct Chain {
  uint64_t *tiles, *groups;
  int64_t step;  // slots between tiles, and between groups
  __device__ uint64_t *tile(int64_t ord) const { return tiles + ord * step; }
  __device__ uint64_t *group(int64_t g) const { return groups + g * step; }
};

// Slots t < count of a run, `stride` apart, into LDS as maps, LB of them per wave;
// w holds what was read ahead. With `state_last` the last one has to be a state.
template <int V, int NW>
__device__ __forceinline__ void take_slots(uint64_t (&w)[LB][V], const uint64_t *at, int64_t stride,
                                           int count, bool state_last, int &polls,
                                           float (&mapA)[NW * LB][64 * V], float (&mapB)[NW * LB][64 * V]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int k = 0; k < LB; ++k) {
    const int t = wave * LB + k;
    if (t < count) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const auto ready = [&]() {
          return w[k][e] != kEmpty && (!state_last || t < count - 1 ||
                                       __builtin_bit_cast(float, (uint32_t)w[k][e]) == kCut);
        };
        while (!ready() && polls < kMaxPolls) {
          __builtin_amdgcn_s_sleep(1);
          w[k][e] = slot_get(at + t * stride + e);
          ++polls;
        }
        const bool ok = ready();
        mapA[t][V * lane + e] = ok ? __builtin_bit_cast(float, (uint32_t)w[k][e]) : __builtin_nanf("");
        mapB[t][V * lane + e] =
            ok ? __builtin_bit_cast(float, (uint32_t)(w[k][e] >> 32)) : __builtin_nanf("");
      }
    }
  }
}

// The state before tile `ord`, the ci-th of its chain, whose own map is (A, B); state
// holds the chain's initial state (used in its first group). `more`: tiles follow.
// Called by the whole block with A, B valid in wave `pub`, which alone gets the state
// (the other waves' instructions are the other block's time).
template <int V, int NW>
__device__ __forceinline__ void chain_state(const Chain &c, int64_t ord, int ci, bool more, int pub,
                                            const float (&A)[V], const float (&B)[V],
                                            float (&mapA)[2][NW * LB][64 * V],
                                            float (&mapB)[2][NW * LB][64 * V], float (&state)[V]) {
  constexpr int G = NW * LB;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int idx = ci % G, g = ci / G, window = min(g, G);
  const bool last = more && idx == G - 1;  // the group's last: it publishes the group
  if (wave == pub && more && !last) {
#pragma unroll
    for (int e = 0; e < V; ++e) slot_put(c.tile(ord) + V * lane + e, A[e], B[e]);
  }
  // read ahead the tiles before this one in its group, first to last, and the
  // groups before it, nearest first
  const uint64_t *tiles = c.tile(ord - idx) + V * lane, *groups = c.group(max(g - 1, 0)) + V * lane;
  uint64_t wt[LB][V], wg[LB][V];
#pragma unroll
  for (int k = 0; k < LB; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int t = wave * LB + k;
      wt[k][e] = t < idx ? slot_get(tiles + t * c.step + e) : 0;
      wg[k][e] = t < window ? slot_get(groups - t * c.step + e) : 0;
    }
  int polls = 0;
  take_slots<V, NW>(wt, tiles, c.step, idx, false, polls, mapA[0], mapB[0]);
  __syncthreads();
  float p[V], q[V];
  if (wave == pub && last) {  // the group's map
#pragma unroll
    for (int e = 0; e < V; ++e) {
      Product P;
      bool cut = false;
      q[e] = 0.f;
      for (int t = 0; t < G; ++t) {
        const float x = t < G - 1 ? mapA[0][t][V * lane + e] : A[e];
        const float y = t < G - 1 ? mapB[0][t][V * lane + e] : B[e];
        q[e] = through(x, y, q[e]);
        P.times(x);
        cut = cut || x == kCut;
      }
      p[e] = cut ? kCut : P.factor();
      if (g > 0) slot_put(c.group(g) + V * lane + e, p[e], q[e]);
    }
  }
  if (g > 0) {
    take_slots<V, NW>(wg, groups, -c.step, window, true, polls, mapA[1], mapB[1]);
    __syncthreads();
  }
  if (wave != pub) return;
  if (g > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int ch = V * lane + e;
      int t = 0;
      while (t < window - 1 && mapA[1][t][ch] != kCut) ++t;
      float s = mapB[1][t][ch];
      for (--t; t >= 0; --t) s = affine(mapA[1][t][ch], s, mapB[1][t][ch]);
      state[e] = s;
    }
  }
  if (last) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (g == 0 || p[e] != kCut)
        slot_put(c.group(g) + V * lane + e, kCut, through(p[e], q[e], state[e]));
  }
#pragma unroll
  for (int e = 0; e < V; ++e)
    for (int t = 0; t < idx; ++t)
      state[e] = through(mapA[0][t][V * lane + e], mapB[0][t][V * lane + e], state[e]);
}

// Composes the maps (sA, sB; sCut: with a document start) of a tile's waves, first to last
// or, with `back`, last to first: (A, B) is all of them as one, and each wave's own is
// replaced by the one of the waves before it.
template <int V, int NW>
__device__ __forceinline__ void compose_waves(float (&sA)[NW][64 * V], float (&sB)[NW][64 * V],
                                              const int (&sCut)[NW], bool back, float (&A)[V],
                                              float (&B)[V]) {
  const int lane = threadIdx.x & 63;
  Product P[V];
  bool cut = false;
#pragma unroll
  for (int e = 0; e < V; ++e) B[e] = 0.f;
#pragma unroll 4
  for (int k = 0; k < NW; ++k) {
    const int w = back ? NW - 1 - k : k;
    const bool here = sCut[w] != 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float &a = sA[w][V * lane + e], &b = sB[w][V * lane + e];
      const float x = a, y = b;
      a = cut ? kCut : P[e].factor();
      b = B[e];
      const float z = affine(x, B[e], y);
      B[e] = here ? y : z;
      P[e].times(x);
    }
    cut = cut || here;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = cut ? kCut : P[e].factor();
}

// The state before each wave, from the tile's in wave `pub`, through the waves before it.
template <int V, int NW>
__device__ __forceinline__ void wave_state(const float (&sA)[NW][64 * V], const float (&sB)[NW][64 * V],
                                           float (&sS)[64 * V], int pub, float (&s)[V]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave == pub) {
#pragma unroll
    for (int e = 0; e < V; ++e) sS[V * lane + e] = s[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e)
    s[e] = through(sA[wave][V * lane + e], sB[wave][V * lane + e], sS[V * lane + e]);
}

// The first of the V channels of a lane whose own ones start at channel c: c, or,
// where those would reach over the row's end, the row's last V. The lane's
// neighbour then computes some of them too, with the same results; so packs are
// whole but for rows of fewer than V channels.
template <int V>
__device__ __forceinline__ int lane_channel(int c, int d) {
  return c < d && d >= V ? min(c, d - V) : c;
}

// A raw pack of V channels; channels at or past d are zero.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_raw(const T *row, int c, int d) {
  if (c + V <= d) return *(const Pack<T, V> *)(row + c);
  Pack<T, V> p;
#pragma unroll
  for (int e = 0; e < V; ++e) p.v[e] = c + e < d ? row[c + e] : (T)0.f;
  return p;
}

// The same for the byte offset of a channel that is known to hold a whole pack:
// one load from a wave-uniform row, with no branch around it.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_at(const T *row, uint32_t bytes) {
  return *(const Pack<T, V> *)((const char *)row + bytes);
}
template <typename T, int V>
__device__ __forceinline__ void store_at(T *row, uint32_t bytes, const float (&v)[V]) {
  Pack<T, V> p;
#pragma unroll
  for (int e = 0; e < V; ++e) p.v[e] = (T)v[e];
  *(Pack<T, V> *)((char *)row + bytes) = p;
}

// Where a block's tile is. `ord`: position in its chain (0 runs first; nt: none).
struct Tile {
  int n, cb;
  int64_t ord;
};
template <int V>
__device__ __forceinline__ Tile next_tile(const RecArgs &a, int nt) {
  __shared__ unsigned ticket;
  unsigned id = (unsigned)blk::block_id();
  if (nt > 1) {
    if (threadIdx.x == 0)
      ticket = __hip_atomic_fetch_add((unsigned *)a.ws, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    id = ticket;
  }
  const unsigned cbs = (a.d + 64 * V - 1) / (64 * V), per = cbs * a.n;
  id = __builtin_amdgcn_readfirstlane(id);
  return {(int)((id % per) / cbs), (int)(id % cbs), (int64_t)(id / per)};
}

// Bit r: a document starts at token t0 + r, for the R tokens from t0 below `end`.
template <int R>
__device__ __forceinline__ uint64_t start_bits(const RecArgs &a, int n, int64_t t0, int64_t end) {
  if (!a.starts) return 0;
  const int lane = threadIdx.x & 63;
  const int64_t t = t0 + lane;
  return __ballot(lane < R && t < end && a.starts[(int64_t)n * a.L + t] != 0);
}

constexpr int64_t kSlotBase = 256;  // bytes in front of the slots: the tile counter

template <int V>
__device__ __forceinline__ Chain chain_of(const RecArgs &a, const Tile &t, int64_t nt) {
  const int64_t cbs = (a.d + 64 * V - 1) / (64 * V), step = (int64_t)a.n * cbs * 64 * V;
  uint64_t *const at = (uint64_t *)((char *)a.ws + kSlotBase) + ((int64_t)t.n * cbs + t.cb) * 64 * V;
  return {at, at + nt * step, step};
}

template <typename T, int V, int R, int NW>
__global__ __launch_bounds__(64 * NW) void k_rec_fwd(RecArgs a, int nt) {
  constexpr int TT = NW * R, CH = 64 * V;
  __shared__ float sA[NW][CH], sB[NW][CH], lA[2][NW * LB][CH], lB[2][NW * LB][CH];
  __shared__ float sS[CH];
  __shared__ int sCut[NW];
  const Tile tl = next_tile<V>(a, nt);
  if (tl.ord >= nt) return;
  const int lane = threadIdx.x & 63, n = tl.n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t len = seq_length(a, n), t0 = tl.ord * TT;
  const int d = a.d, c = lane_channel<V>(CH * tl.cb + V * lane, d);
  const int64_t tb = t0 + wave * R;
  const int cnt = (int)min(max(len - tb, (int64_t)0), (int64_t)R);
  T *h = seq_of<T>(a.h, n);
  const float zero[V] = {};
  if (c < d)
    for (int r = cnt; r < R && tb + r < a.L; ++r) store_ch<T, V>(h + (tb + r) * a.h.tok_stride, c, d, zero);
  float s[V] = {};
  if (a.h0 && c < d) load_ch<float, V>(a.h0 + (int64_t)n * d, c, d, s);
  if (t0 >= len) {  // nothing of the sequence here, and nobody waits for it
    if (tl.ord == 0 && wave == 0 && a.h_last && c < d)
      store_ch<float, V>(a.h_last + (int64_t)n * d, c, d, s);
    return;
  }
  // the wave's tokens as local states hl (from a zero state) and products P.
  // FAST: all R tokens, whole packs and no document start, as most waves have it:
  // straight code.
  float P[R][V], hl[R][V];
  Product W[V];
  const uint64_t cuts = start_bits<R>(a, n, tb, tb + cnt);
  const bool fast = cnt == R && d >= V && cuts == 0;
  const uint32_t at = (c < d ? c : 0) * (uint32_t)sizeof(T);
  const auto local = [&](auto tag) __attribute__((always_inline)) {
    constexpr bool FAST = decltype(tag)::value;
    const T *g = seq_of<T>(a.g, n), *v = seq_of<T>(a.v, n);
    Pack<T, V> gr[R], vr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t t = FAST ? tb + r : min(tb + r, len - 1);
      if constexpr (FAST) {
        gr[r] = load_at<T, V>(g + t * a.g.tok_stride, at);
        vr[r] = load_at<T, V>(v + t * a.v.tok_stride, at);
      } else {
        gr[r] = load_raw<T, V>(g + t * a.g.tok_stride, c, d);
        vr[r] = load_raw<T, V>(v + t * a.v.tok_stride, c, d);
      }
    }
    float q[V] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) W[e] = Product();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (FAST || r < cnt) {
        const bool cut = !FAST && (cuts >> r & 1);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float f, i;
          gate((float)gr[r].v[e], f, i);
          const float b = i * (float)vr[r].v[e];
          q[e] = cut ? b : fmaf(f, q[e], b);
          W[e].take(f, i);
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        P[r][e] = W[e].p;
        hl[r][e] = q[e];
      }
    }
  };
  if (fast)
    local(std::true_type());
  else
    local(std::false_type());
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sA[wave][V * lane + e] = W[e].factor();
    sB[wave][V * lane + e] = hl[R - 1][e];
  }
  if (lane == 0) sCut[wave] = cuts != 0;
  __syncthreads();
  float A[V], B[V];
  if (wave == 0) compose_waves<V, NW>(sA, sB, sCut, false, A, B);
  if (nt > 1)
    chain_state<V, NW>(chain_of<V>(a, tl, nt), tl.ord, (int)tl.ord, t0 + TT < len, 0, A, B, lA, lB, s);
  wave_state<V, NW>(sA, sB, sS, 0, s);
  if (c >= d) return;
  float o[V] = {};
  if (fast) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(P[r][e], s[e], hl[r][e]);
      store_at<T, V>(h + (tb + r) * a.h.tok_stride, at, o);
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < cnt) {
        const bool k = (cuts & ((uint64_t)2 << r) - 1) != 0;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = k ? hl[r][e] : fmaf(P[r][e], s[e], hl[r][e]);
        store_ch<T, V>(h + (tb + r) * a.h.tok_stride, c, d, o);
      }
  }
  if (a.h_last && cnt > 0 && tb + cnt == len) {
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = through(cuts ? kCut : W[e].factor(), hl[R - 1][e], s[e]);
    store_ch<float, V>(a.h_last + (int64_t)n * d, c, d, s);
  }
}

// The gradient G of the state before token t: G_t = f_t (dh_t + G_{t+1}), 0 at a
// document start; chain order runs from the last tile of the longest sequence.
template <typename T, int V, int R, int NW>
__global__ __launch_bounds__(64 * NW) void k_rec_bwd(RecArgs a, int nt) {
  constexpr int TT = NW * R, CH = 64 * V;
  __shared__ float sA[NW][CH], sB[NW][CH], lA[2][NW * LB][CH], lB[2][NW * LB][CH];
  __shared__ float sS[CH];
  __shared__ int sCut[NW];
  const Tile tl = next_tile<V>(a, nt);
  if (tl.ord >= nt) return;
  const int lane = threadIdx.x & 63, n = tl.n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t len = seq_length(a, n), tile = nt - 1 - tl.ord, t0 = tile * TT;
  const int d = a.d, c = lane_channel<V>(CH * tl.cb + V * lane, d);
  const int64_t tb = t0 + wave * R;
  const int cnt = (int)min(max(len - tb, (int64_t)0), (int64_t)R);
  T *dg = seq_of<T>(a.dg, n), *dv = seq_of<T>(a.dv, n);
  const float zero[V] = {};
  if (c < d)
    for (int r = cnt; r < R && tb + r < a.L; ++r) {
      store_ch<T, V>(dg + (tb + r) * a.dg.tok_stride, c, d, zero);
      store_ch<T, V>(dv + (tb + r) * a.dv.tok_stride, c, d, zero);
    }
  float s[V] = {};
  if (a.dh_last && c < d) load_ch<float, V>(a.dh_last + (int64_t)n * d, c, d, s);
  if (t0 >= len) {
    if (tile == 0 && wave == 0 && a.dh0 && c < d)
      store_ch<float, V>(a.dh0 + (int64_t)n * d, c, d, s);
    return;
  }
  const uint64_t cuts = start_bits<R>(a, n, tb, tb + cnt);
  const bool fast = cnt == R && d >= V && cuts == 0 && tb > 0;
  const uint32_t at = (c < d ? c : 0) * (uint32_t)sizeof(T);
  Pack<T, V> gr[R], dr[R], vr[R], pr[R];
  float A[V], B[V] = {}, own[V];
  Product W[V];
  // FAST: all R tokens with a token before them, whole packs, no document start
  const auto local = [&](auto tag) __attribute__((always_inline)) {
    constexpr bool FAST = decltype(tag)::value;
    const T *g = seq_of<T>(a.g, n), *dh = seq_of<T>(a.dh, n);
    const T *v = seq_of<T>(a.v, n), *h = seq_of<T>(a.h, n);
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const int64_t t = FAST ? tb + r : min(tb + r, len - 1);
      if constexpr (FAST) {
        gr[r] = load_at<T, V>(g + t * a.g.tok_stride, at);
        dr[r] = load_at<T, V>(dh + t * a.dh.tok_stride, at);
      } else {
        gr[r] = load_raw<T, V>(g + t * a.g.tok_stride, c, d);
        dr[r] = load_raw<T, V>(dh + t * a.dh.tok_stride, c, d);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {  // used after the wait
      const int64_t t = FAST ? tb + r : min(tb + r, len - 1);
      if constexpr (FAST) {
        vr[r] = load_at<T, V>(v + t * a.v.tok_stride, at);
        pr[r] = load_at<T, V>(h + (t - 1) * a.h.tok_stride, at);
      } else {
        vr[r] = load_raw<T, V>(v + t * a.v.tok_stride, c, d);
        pr[r] = load_raw<T, V>(h + max(t - 1, (int64_t)0) * a.h.tok_stride, c, d);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (FAST || r < cnt) {
        const bool k = !FAST && (cuts >> r & 1);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float f, i;
          gate((float)gr[r].v[e], f, i);
          B[e] = k ? 0.f : f * ((float)dr[r].v[e] + B[e]);
          W[e].take(f, i);
        }
      }
  };
  if (fast)
    local(std::true_type());
  else
    local(std::false_type());
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sA[wave][V * lane + e] = W[e].factor();
    sB[wave][V * lane + e] = own[e] = B[e];
  }
  if (lane == 0) sCut[wave] = cuts != 0;
  __syncthreads();
  if (wave == NW - 1) compose_waves<V, NW>(sA, sB, sCut, true, A, B);
  if (nt > 1)
    chain_state<V, NW>(chain_of<V>(a, tl, nt), tl.ord, (int)((len - 1) / TT - tile), tile > 0, NW - 1, A,
                       B, lA, lB, s);
  wave_state<V, NW>(sA, sB, sS, NW - 1, s);
  if (c >= d) return;
  if (a.dh0 && tb == 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) own[e] = through(cuts ? kCut : W[e].factor(), own[e], s[e]);
    store_ch<float, V>(a.dh0 + (int64_t)n * d, c, d, own);
  }
  const auto finish = [&](auto tag) __attribute__((always_inline)) {
    constexpr bool FAST = decltype(tag)::value;
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
      if (FAST || r < cnt) {
        const bool k = !FAST && (cuts >> r & 1);
        float prev[V], og[V], ov[V];
#pragma unroll
        for (int e = 0; e < V; ++e) prev[e] = (float)pr[r].v[e];
        if constexpr (!FAST) {
          if (tb + r == 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) prev[e] = 0.f;
            if (a.h0) load_ch<float, V>(a.h0 + (int64_t)n * d, c, d, prev);
          }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float f, i;
          gate((float)gr[r].v[e], f, i);
          const float delta = (float)dr[r].v[e] + s[e];
          ov[e] = i * delta;
          og[e] = delta * ((k ? 0.f : prev[e]) - (float)vr[r].v[e]) * (f * i);
          s[e] = k ? 0.f : f * delta;
        }
        if constexpr (FAST) {
          store_at<T, V>(dg + (tb + r) * a.dg.tok_stride, at, og);
          store_at<T, V>(dv + (tb + r) * a.dv.tok_stride, at, ov);
        } else {
          store_ch<T, V>(dg + (tb + r) * a.dg.tok_stride, c, d, og);
          store_ch<T, V>(dv + (tb + r) * a.dv.tok_stride, c, d, ov);
        }
      }
  };
  if (fast)
    finish(std::true_type());
  else
    finish(std::false_type());
}

// Empties the slots and the tile counter.
__global__ __launch_bounds__(256) void k_rec_clear(uint64_t *ws, int64_t slots) {
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i0 == 0) *(unsigned *)ws = 0;
  uint64_t *s = ws + kSlotBase / 8;
  for (int64_t i = 2 * i0; i < slots; i += (int64_t)gridDim.x * 512) {
    s[i] = kEmpty;
    s[i + 1] = kEmpty;  // slots come in multiples of 64
  }
}

// Tokens to which a thread walks its sequence itself (us, walked / in tiles, forward and
// backward: 32 sequences of 16 x 2560 9.5 / 14.0 and 15.8 / 29.5, of 32 17.2 / 14.5 and 31.7 /
// 30.5; one of 16 8.8 / 7.8 and 14.4 / 14.4, of 32 14.8 / 7.8 and 25.9 / 14.4). The number of
// sequences is left out: where it would decide, at 16 tokens of one, it is 1 us. Not
// more than 16, by the rounded factors above.
constexpr int64_t SEQ_MAX = 16;

// Tokens per wave in the forward and the backward, waves, and channels per lane, all
// measured on 128k x 2560 forward / 8 x 16k x 2048 backward, bf16, where a copy of
// the same bytes takes 421 / 674 us. As here 497 / 602 us (with the measured cases'
// gates 460 / 633); before what is handed on went by 1 - f 483 / 601, and so the
// variants: 8 tokens a wave 688 / 686,
// 32 (forward) 476 but 28 us against 17 for 5 x 1237 x 331; 4 waves of 16 tokens 572 /
// 640, 16 waves of 8 (backward) 760; 4 channels a lane 725 / 899 and up (registers).
// Slots a wave reads (LB) 1, 2, 3: 483, 513, 530 (forward). Bound by HBM.
constexpr int kFwdTokens = 16, kBwdTokens = 16, kWaves = 8;
// Two channels a lane, one where 64 lanes hold them all: 15 x 8670 x 64 fp32 forward 32 us
// (two: 47), backward 45 (87); 5 x 33168 x 64 bf16 39 (46), 44 (77).
int lane_channels(int d) { return d <= 64 ? 1 : 2; }
constexpr int kFwdTile = kFwdTokens * kWaves, kBwdTile = kBwdTokens * kWaves;
constexpr int kMinTile = kFwdTile < kBwdTile ? kFwdTile : kBwdTile;  // what the workspace holds

int64_t channel_blocks(int d) {
  const int ch = 64 * lane_channels(d);
  return (d + ch - 1) / ch;
}
// the tiles' and the groups', for either width of a tile
int64_t tile_slots(int n, int d, int64_t nt) {
  return (nt + nt / (kWaves * LB) + 1) * n * round_up(d, 128);
}

hipError_t clear_slots(const RecArgs &a, int64_t nt, hipStream_t st) {
  if (nt <= 1) return hipSuccess;
  const int64_t slots = tile_slots(a.n, a.d, nt);
  hipLaunchKernelGGL(k_rec_clear, dim3((unsigned)std::min<int64_t>((slots + 511) / 512, 2048)),
                     dim3(256), 0, st, (uint64_t *)a.ws, slots);
  return hipGetLastError();
}

}  // namespace

bool rec_size_ok(int n, int d, int64_t L) {
  const int64_t nt = (L + kMinTile - 1) / kMinTile;
  return nt * n <= INT32_MAX && nt * n * channel_blocks(d) <= INT32_MAX;
}

size_t rec_workspace(int n, int d, int64_t L) {
  const int64_t nt = (L + kMinTile - 1) / kMinTile;
  return (size_t)kSlotBase + (L <= SEQ_MAX || nt <= 1 ? 0 : 8 * tile_slots(n, d, nt));
}

template <typename T>
hipError_t rec_step(const RecArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_rec_seq_fwd<T>, dim3((a.d + 64 * SEQ_V - 1) / (64 * SEQ_V), a.n), dim3(64), 0,
                     st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t rec_forward(const RecArgs &a, hipStream_t st) {
  if (a.L <= SEQ_MAX) return rec_step<T>(a, st);
  const int64_t nt = (a.L + kFwdTile - 1) / kFwdTile;
  const hipError_t e = clear_slots(a, nt, st);
  if (e != hipSuccess) return e;
  const dim3 grid = blk::grid_of(nt * a.n * channel_blocks(a.d)), block(64 * kWaves);
  if (lane_channels(a.d) == 1)
    hipLaunchKernelGGL((k_rec_fwd<T, 1, kFwdTokens, kWaves>), grid, block, 0, st, a, (int)nt);
  else
    hipLaunchKernelGGL((k_rec_fwd<T, 2, kFwdTokens, kWaves>), grid, block, 0, st, a, (int)nt);
  return hipGetLastError();
}

template <typename T>
hipError_t rec_backward(const RecArgs &a, hipStream_t st) {
  if (a.L <= SEQ_MAX) {
    hipLaunchKernelGGL(k_rec_seq_bwd<T>, dim3((a.d + 64 * SEQ_V - 1) / (64 * SEQ_V), a.n), dim3(64),
                       0, st, a);
    return hipGetLastError();
  }
  const int64_t nt = (a.L + kBwdTile - 1) / kBwdTile;
  const hipError_t e = clear_slots(a, nt, st);
  if (e != hipSuccess) return e;
  const dim3 grid = blk::grid_of(nt * a.n * channel_blocks(a.d)), block(64 * kWaves);
  if (lane_channels(a.d) == 1)
    hipLaunchKernelGGL((k_rec_bwd<T, 1, kBwdTokens, kWaves>), grid, block, 0, st, a, (int)nt);
  else
    hipLaunchKernelGGL((k_rec_bwd<T, 2, kBwdTokens, kWaves>), grid, block, 0, st, a, (int)nt);
  return hipGetLastError();
}

template hipError_t rec_step<float>(const RecArgs &, hipStream_t);
template hipError_t rec_step<__bf16>(const RecArgs &, hipStream_t);
template hipError_t rec_forward<float>(const RecArgs &, hipStream_t);
template hipError_t rec_forward<__bf16>(const RecArgs &, hipStream_t);
template hipError_t rec_backward<float>(const RecArgs &, hipStream_t);
template hipError_t rec_backward<__bf16>(const RecArgs &, hipStream_t);

}  // namespace ipttt
