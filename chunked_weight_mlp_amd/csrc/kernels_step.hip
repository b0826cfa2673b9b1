// Attention of one new token of each sequence over the paged cache (gfx950).
//
// HBM bounds it: every key and value is read once, by one wave, for all heads of its key
// head's group (columns of one 32-column tile). The steps (kKeys keys of a sequence and key
// head) of all sequences are numbered in a row and shared evenly among the blocks, however
// long each sequence is; a block that ends inside a sequence, or begins there, leaves a
// partial result, and a second kernel joins those. The host knows no lengths: blocks find
// their place from lens.
//
// A block is one wave, which copies a step's keys and values into its LDS while it computes
// with the ones before; four or more of them share a CU and wait for nobody.
#include <float.h>

#include "attention_common.h"

namespace ipttt {
namespace {

using namespace attn;

constexpr int kKeys = 32;  // keys of a step
// What a block spends on beginning and ending a sequence and key head, in steps: each has so
// many places before its steps in the row of steps. (64 sequences of 26 to 7875 tokens: 151
// us without it, the blocks of the short ones come last.)
constexpr int kBegin = 1;
// Steps in LDS: the next one's are copied beside this one's products, but where rows have
// 512 bytes (fp32), whose products take longer than the copies and leave LDS to twice the
// blocks. (131072 tokens, 4 key heads of 128 fp32: 252 us with two steps, 191 with one.)
template <typename T, int DP>
constexpr int stages_of() { return sizeof(T) * DP > 256 ? 1 : 2; }

// Heads of a key head's group are columns of a 32-column tile; wider groups take several.
__host__ __device__ inline int chunks_of(int hq, int hk) { return (hq / hk + 31) / 32; }

struct Plan {
  int blocks;    // blocks of the first kernel (for each chunk of heads)
  bool whole;    // a block for each sequence and key head: nothing to join
  int cols;      // heads a partial result has room for
};
Plan plan_of(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t) {
  Plan p;
  const int dp = c.head_dim <= 64 ? 64 : 128;
  const int64_t most = ((int64_t)t.width * c.page_size + kKeys - 1) / kKeys;  // steps a sequence may have
  const int64_t pairs = (int64_t)t.batch * c.k_heads;
  // 8 steps, once such blocks fill the GPU (heads of 128 bf16; 2048 blocks of 8 steps: 72.5
  // us joined, 62.5 whole; 512: 33.3, 27.8; but 128: 21.6, 26.5; ragged ones of up to 32 steps:
  // 43 joined, 68 whole.) 2 steps always (2048 blocks: 35.0, 26.5).
  p.whole = most <= 2 || (most <= 8 && pairs >= 512);
  const int64_t steps = (most + kBegin) * pairs;
  // as many as run at once, or nearly: four waves a CU, one a SIMD, which the registers of 128
  // channels leave (LDS would hold five), eight at 64 bf16 (131072 tokens, 32/8 heads of 128
  // bf16: 173 us with 512, 107 with 1024, 123 with 2048)
  const int blocks = (c.dtype == IPTTT_BF16 && dp == 64) ? 2048 : 1024;
  p.blocks = (int)(p.whole ? pairs : steps < blocks ? steps : blocks);
  p.cols = hq / c.k_heads < 32 ? hq / c.k_heads : 32;
  return p;
}
// A partial result: for each head the maximum (-infinity: no key), the sum, and dh sums of values.
__host__ __device__ inline int64_t part_size(int cols, int dh) { return (int64_t)cols * (dh + 2); }

// The workspace: for each sequence and key head the blocks where it begins and ends, then
// the partial results.
__host__ __device__ inline int64_t places_bytes(int batch, int hk) { return ((int64_t)batch * hk * 8 + 255) / 256 * 256; }
__device__ __forceinline__ float *parts_at(const StepArgs &a) {
  return (float *)((char *)a.ws + places_bytes(a.table.batch, a.cache.k_heads));
}

// The keys of a sequence: [lo, hi), read in steps first .. first + n - 1 of so many.
struct Span {
  int lo, hi, first, n;
};
__device__ __forceinline__ Span span_of(const StepArgs &a, int b) {
  Span s;
  const int most = a.table.width * a.cache.page_size;
  s.hi = min(max(a.lens[b], 0), most);
  s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
  s.first = s.lo / kKeys;
  s.n = s.hi == 0 ? 0 : (s.hi - 1) / kKeys + 1 - s.first;
  return s;
}

// Places in the row of steps of one key head of sequence b, and of all of those before
// sequence upto. Every wave for itself.
__device__ __forceinline__ int places(const StepArgs &a, int b) {
  const int n = span_of(a, b).n;
  return n ? n + kBegin : 0;
}
__device__ __forceinline__ int64_t steps_before(const StepArgs &a, int upto, int lane) {
  int64_t n = 0;
  for (int b = lane; b < upto; b += 64) n += places(a, b);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  return n * a.cache.k_heads;
}
// The sequence whose places hold `want`, and the number of places before it.
__device__ __forceinline__ int find_step(const StepArgs &a, int64_t want, int lane,
                                          int64_t &before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.table.batch; b0 += 64) {
    const int b = b0 + lane;
    int64_t n = b < a.table.batch ? (int64_t)places(a, b) * a.cache.k_heads : 0, run = n;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t up = __shfl_up(run, m, 64);
      if (lane >= m) run += up;
    }
    const uint64_t hit = __ballot(base + run > want);
    if (hit) {
      const int i = __ffsll((unsigned long long)hit) - 1;
      before = base + __shfl(run - n, i, 64);
      return b0 + i;
    }
    base += __shfl(run, 63, 64);
  }
  before = base;
  return a.table.batch;
}
// Blocks share the places evenly; where there are fewer than blocks, one each.
__device__ __forceinline__ int64_t first_step(int64_t total, int blocks, int block) {
  const int64_t used = total < blocks ? total : blocks;
  return block < used ? total * block / used : total;
}

__device__ const uint4 zero_row[kHeadMaxDim * 4 / 16] = {};

// A place in the row of steps: one step of a sequence and key head.
struct Cursor {
  int64_t at;      // the step's place
  int64_t from;    // that of the first step of this sequence and key head
  int b, kv;
  Span sp;
  __device__ __forceinline__ int64_t to() const { return from + sp.n; }
  // to the next sequence and key head that has keys
  __device__ __forceinline__ void next(const StepArgs &a) {
    at = from = to() + kBegin;
    if (++kv < a.cache.k_heads) return;
    kv = 0;
    do {
      if (++b >= a.table.batch) return;
      sp = span_of(a, b);
    } while (sp.n == 0);
  }
};

template <typename T, int DP>
__global__ __launch_bounds__(64) void k_step(StepArgs a, Plan plan) {
  using L = Tile<T, DP>;
  constexpr int STAGES = stages_of<T, DP>(), TILE = kKeys * DP, NEXT = 2 * TILE * (int)sizeof(T);
  constexpr int RPI = 64 / L::NP, NI = kKeys / RPI;  // rows an instruction copies, instructions a tile
  extern __shared__ __align__(1024) char smem[];
  T *const buf = (T *)smem;  // [STAGES][keys, values]
  const int l = threadIdx.x, h = l >> 5, col = l & 31;
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, ps = a.cache.page_size;
  const int group = a.hq / hk, chunks = chunks_of(a.hq, hk);
  const int block = blockIdx.x, chunk = blockIdx.y;
  const int cols = min(32, group - 32 * chunk);
  Cursor cc;  // what is computed
  int64_t end;
  if (plan.whole) {
    cc.b = block / hk;
    cc.kv = block % hk;
    cc.sp = span_of(a, cc.b);
    cc.at = cc.from = 0;
    end = cc.sp.n;
    if (end == 0) {  // no key
      const int head0 = cc.kv * group + 32 * chunk;
      for (int i = l; i < cols * dh; i += 64)
        ((T *)a.o.p)[cc.b * a.o.tok_stride + (head0 + i / dh) * a.o.head_stride + i % dh] = (T)0.f;
      if (a.lse && l < cols) a.lse[(int64_t)cc.b * a.hq + head0 + l] = -INFINITY;
      return;
    }
  } else {
    const int64_t total = (int64_t)uniform64((uint64_t)steps_before(a, a.table.batch, l));
    cc.at = first_step(total, plan.blocks, block);
    end = first_step(total, plan.blocks, block + 1);
    if (cc.at >= end) return;
    int64_t before;
    cc.b = __builtin_amdgcn_readfirstlane(find_step(a, cc.at, l, before));
    before = (int64_t)uniform64((uint64_t)before);
    cc.sp = span_of(a, cc.b);
    cc.kv = __builtin_amdgcn_readfirstlane((int)((cc.at - before) / (cc.sp.n + kBegin)));
    cc.from = before + (int64_t)cc.kv * (cc.sp.n + kBegin) + kBegin;
    if (cc.at < cc.from) cc.at = cc.from;
    if (cc.at >= end) return;
  }
  const bool direct = dh % L::PE == 0;  // the cache's rows are then on 16-byte boundaries
  if (dh != DP) clear(buf, STAGES * 2 * TILE, l, 64);
  const float c = log2_scale(a.scale);
  // The page of this lane's key (key col of the step, in both halves), or -1.
  const auto page_of = [&](const Cursor &u) __attribute__((always_inline)) {
    const int key = (u.sp.first + (int)(u.at - u.from)) * kKeys + col;
    if (key < u.sp.lo || key >= u.sp.hi) return -1;
    return a.table.p[u.b * a.table.stride + key / ps];
  };
  // Copies a step's keys and values; returns which of the 32 keys are there.
  const auto issue = [&](const Cursor &u, int page, int b) __attribute__((always_inline)) {
    const int key = (u.sp.first + (int)(u.at - u.from)) * kKeys + col;
    const bool ok = page >= 0 && page < a.cache.pages;
    const int64_t place = ok ? (((int64_t)page * hk + u.kv) * ps + key % ps) * dh : -1;
    const uint32_t there = (uint32_t)__ballot(ok);
    if (there == 0) return there;
    T *const kt = buf + b * 2 * TILE, *const vt = kt + TILE;
    if (direct) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + l / L::NP, piece = (l % L::NP) ^ L::swizzle(r);
        const int64_t row = __shfl(place, r, 64);
        if (DP == dh || piece * L::PE < dh) {
          const T *const ks = row < 0 ? (const T *)zero_row : (const T *)a.cache.k + row;
          const T *const vs = row < 0 ? (const T *)zero_row : (const T *)a.cache.v + row;
          copy_to_lds16(ks + piece * L::PE, kt + i * RPI * DP);
          copy_to_lds16(vs + piece * L::PE, vt + i * RPI * DP);
        }
      }
    } else {
      const int ln = here(l), width = here(dh);
#pragma unroll 1
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + ln / L::NP, p = ln % L::NP;
        const int64_t row = __shfl(place, r, 64);
        const T *const ks = row < 0 ? (const T *)zero_row : (const T *)a.cache.k + row;
        const T *const vs = row < 0 ? (const T *)zero_row : (const T *)a.cache.v + row;
        T x[L::PE];
        load_some<T, L::PE>(ks, p * L::PE, width, x);
#pragma unroll
        for (int e = 0; e < L::PE; ++e) kt[L::at(r, p) + e] = x[e];
        load_some<T, L::PE>(vs, p * L::PE, width, x);
#pragma unroll
        for (int e = 0; e < L::PE; ++e) vt[L::at(r, p) + e] = x[e];
      }
    }
    return there;
  };
  // The queries of a sequence and key head, loaded beside the copies of its first step.
  Frag<T> q[L::STEPS], q_next[L::STEPS];
  const auto load_queries = [&](const Cursor &u) __attribute__((always_inline)) {
    const T *qp = (const T *)a.q.p + u.b * a.q.tok_stride +
                  (u.kv * group + 32 * chunk + min(col, cols - 1)) * a.q.head_stride;
#pragma unroll
    for (int i = 0; i < L::STEPS; ++i) q_next[i] = load_frag<T>(qp, i, h, dh);
  };
  Cursor ic = cc, copied = cc;  // what is copied next, and what was last
  const auto ahead = [&]() __attribute__((always_inline)) {
    if (++ic.at == ic.to()) ic.next(a);
    return ic.at < end ? page_of(ic) : -1;
  };
  load_queries(ic);
  uint32_t there = issue(ic, page_of(ic), 0), next = 0;
  int page = ahead(), cur = 0;
  RowReader<T, DP> rows(buf, l);
  ColReader<T, DP> vals(buf + TILE, l);
  for (;;) {
    // one sequence and key head, to its last step or the block's
    const bool begins = cc.at == cc.from;
    const int64_t stop = min(end, cc.to());
    const bool whole = begins && stop == cc.to();
#pragma unroll
    for (int i = 0; i < L::STEPS; ++i) q[i] = with_sign<T>(q_next[i], a.scale);
    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
    float m = -INFINITY, sum = 0.f;
    uint32_t any = 0;  // keys that are there
    for (; cc.at < stop; ++cc.at) {
      // this step's tiles, and the next one's pages, have landed
      mfma::wait_vm<0>();
      next = 0;
      const auto copy_next = [&](int b) __attribute__((always_inline)) {
        if (ic.at < end) {
          copied = ic;
          if (ic.at == ic.from) load_queries(ic);
          next = issue(ic, page, b);
          page = ahead();
        }
      };
      if constexpr (STAGES == 2) copy_next(cur ^= 1);
      any |= there;
      if (there != 0) {
        f32x16 x{};
#pragma unroll
        for (int i = 0; i < L::STEPS; ++i)
          if (16 * i < dh) x = mma(rows.read(0, i), q[i], x);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = there >> (8 * (i / 4) + i % 4 + 4 * h) & 1 ? x[i] : -INFINITY;
          top = fmaxf(top, x[i]);
        }
        top = half_max(top);
        if (__ballot((top - m) * c > kSlack)) {
          const float best = fmaxf(m, top);
          const float f = best == -INFINITY ? 1.f : exp2_((m - best) * c);
          m = best;
          sum *= f;
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[d][e] *= f;
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = exp2_(__builtin_fmaf(x[i], c, -mc));
          sum += x[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Frag<T> p = as_operand<T>(x, i);
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
            if (32 * d < dh) acc[d] = mma(vals.read(16 * i, d), p, acc[d]);
        }
      }
      if constexpr (STAGES == 2) {
        rows.move(cur ? NEXT : -NEXT);
        vals.move(cur ? NEXT : -NEXT);
      } else {
        copy_next(0);  // the products have what they read
      }
      there = next;
    }
    sum = half_sum(sum);
    // Keys, but none with a score above -infinity: sum is 0, or NaN where a score is NaN, and m
    // becomes a number, so that -infinity says that no key was there.
    if (any && m == -INFINITY) m = -FLT_MAX;
    const int head0 = cc.kv * group + 32 * chunk;
    if (l == 0 && chunk == 0 && !plan.whole) {  // the blocks that k_join finds it in
      int *const in = (int *)a.ws + 2 * ((int64_t)cc.b * hk + cc.kv);
      if (begins) in[0] = block;
      if (stop == cc.to()) in[1] = block;
    }
    if (col < cols) {
      if (whole) {
        const bool none = !any;  // no page
        store_row<T, DP>((T *)a.o.p + cc.b * a.o.tok_stride + (head0 + col) * a.o.head_stride, acc,
                         none ? 0.f : 1.f / sum, h, dh, kAsIs);
        if (a.lse && h == 0)
          a.lse[(int64_t)cc.b * a.hq + head0 + col] = none ? -INFINITY : (m * c + log2f(sum)) * kLn2;
      } else {
        float *const part = parts_at(a) + ((int64_t)(block * chunks + chunk) * 2 + (begins ? 1 : 0)) *
                                              part_size(plan.cols, dh) + col * (dh + 2);
        if (h == 0) {
          part[0] = m;
          part[1] = sum;
        }
        store_row<float, DP>(part + 2, acc, 1.f, h, dh, kAsIs);
      }
    }
    if (copied.at < stop) break;  // nothing was copied behind the block's last step
    cc = copied;                  // the step after this one's last
  }
}

// Joins the partial results of a sequence's key head: the second of the block where it
// begins and the first of those up to the one where it ends.
constexpr int kJoin = 512;
template <typename T>
__global__ __launch_bounds__(kJoin) void k_join(StepArgs a, Plan plan) {
  constexpr int GROUPS = kJoin / 128;  // threads of a channel
  __shared__ float weight[2048], red[2][kJoin / 64], sums[GROUPS][kHeadMaxDim];
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, group = a.hq / hk;
  const int b = blockIdx.z, kv = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int *const in = (const int *)a.ws + 2 * ((int64_t)b * hk + kv);
  const int g0 = in[0], g1 = in[1];
  const bool none = span_of(a, b).n == 0;
  if (!none && g0 == g1) return;  // written already
  const int n = none ? 0 : g1 - g0 + 1;  // up to 2048
  const int64_t size = part_size(plan.cols, dh), step = 2 * chunks_of(a.hq, hk) * size;
  const float c = log2_scale(a.scale);
  for (int hh = blockIdx.y; hh < group; hh += gridDim.y) {
    // the part of block g0 + i is at first + i step; the first's is the second of its block
    const float *const first = parts_at(a) + (none ? 0 : g0) * step + (int64_t)(hh / 32) * 2 * size +
                               (hh % 32) * (dh + 2);
    const auto part = [&](int i) { return first + i * step + (i == 0 ? size : 0); };
    float top = -INFINITY;
    for (int i = tid; i < n; i += kJoin) {
      weight[i] = part(i)[0];
      top = fmaxf(top, weight[i]);
    }
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor(top, k, 64));
    if (lane == 0) red[0][wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoin / 64; ++i) top = fmaxf(top, red[0][i]);
    // (a part of weight 0 is added all the same: what is NaN in it stays NaN)
    float sum = 0.f;
    for (int i = tid; i < n; i += kJoin) {
      const float f = weight[i] == -INFINITY ? 0.f : exp2_((weight[i] - top) * c);
      weight[i] = f;
      sum += f * part(i)[1];
    }
    sum = blk::wave_sum(sum);
    if (lane == 0) red[1][wave] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoin / 64; ++i) sum += red[1][i];
    const int ch = tid & 127, mine = tid >> 7;
    float o = 0.f;
    if (ch < dh) {
      for (int i0 = mine; i0 < n; i0 += 8 * GROUPS) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = part(min(i0 + u * GROUPS, n - 1))[2 + ch];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = i0 + u * GROUPS;
          if (i < n) o += weight[i] * v[u];
        }
      }
      sums[mine][ch] = o;
    }
    __syncthreads();
    const int head = kv * group + hh;
    if (tid < dh) {
      o = 0.f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) o += sums[i][tid];
      ((T *)a.o.p)[b * a.o.tok_stride + head * a.o.head_stride + tid] =
          (T)(top == -INFINITY ? 0.f : o / sum);  // -infinity: no key
    }
    if (a.lse && tid == 0)
      a.lse[(int64_t)b * a.hq + head] = top == -INFINITY ? -INFINITY : (top * c + log2f(sum)) * kLn2;
    __syncthreads();
  }
}

}  // namespace

size_t step_workspace(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t) {
  const Plan p = plan_of(hq, c, t);
  if (p.whole) return 256;
  return (size_t)places_bytes(t.batch, c.k_heads) + (size_t)round_up(
      (int64_t)p.blocks * chunks_of(hq, c.k_heads) * 2 * part_size(p.cols, c.head_dim) * 4, 256);
}

template <typename T>
hipError_t step_forward(const StepArgs &a, hipStream_t st) {
  const Plan p = plan_of(a.hq, a.cache, a.table);
  const int chunks = chunks_of(a.hq, a.cache.k_heads);
  const auto go = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    k_step<T, DP><<<dim3(p.blocks, chunks), 64, stages_of<T, DP>() * 2 * kKeys * DP * sizeof(T), st>>>(a, p);
  };
  if (a.cache.head_dim <= 64) go(std::integral_constant<int, 64>());
  else go(std::integral_constant<int, 128>());
  if (!p.whole) {
    const int group = a.hq / a.cache.k_heads;
    // (fewer than 2^32 threads along x)
    k_join<T><<<dim3(a.cache.k_heads, group < 32 ? group : 32, a.table.batch), kJoin, 0, st>>>(a, p);
  }
  return hipGetLastError();
}

template hipError_t step_forward<float>(const StepArgs &, hipStream_t);
template hipError_t step_forward<__bf16>(const StepArgs &, hipStream_t);

}  // namespace ipttt
