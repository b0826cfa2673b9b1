// Attention of one new token of each sequence over the paged cache (gfx950).
//
// HBM bounds it: every key and value is read once, by one wave, for all heads of its key
// head's group (columns of one 32-column tile). The steps (kKeys keys of a sequence and key
// head) of all sequences are numbered in a row and shared evenly among the blocks, however
// long each sequence is; a block that ends inside a sequence, or begins there, leaves a
// partial result, and a second kernel joins those. The host knows no lengths: blocks find
// their place from lens.
//
// A wave reads 32 of a step's keys into LDS of its own, the next step's while it computes
// with this one's, and meets the block's other waves only at the end of a sequence.
#include "attention_common.h"

namespace ipttt {
namespace {

using namespace attn;

// Waves a block: two steps of each wave's keys and values, and the joining, fit LDS.
template <typename T, int DP>
constexpr int waves_of() { return sizeof(T) * DP > 256 ? 2 : 4; }
constexpr int kJoinCols = 8;  // heads joined at a time

// Heads of a key head's group are columns of a 32-column tile; wider groups take several.
__host__ __device__ inline int chunks_of(int hq, int hk) { return (hq / hk + 31) / 32; }

struct Plan {
  int keys;      // keys of a step
  int blocks;    // blocks of the first kernel (for each chunk of heads)
  bool whole;    // a block for each sequence and key head: nothing to join
  int cols;      // heads a partial result has room for
};
Plan plan_of(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t) {
  Plan p;
  const int dp = c.head_dim <= 64 ? 64 : 128;
  p.keys = 32 * ((c.dtype == IPTTT_BF16 ? 2 : 4) * dp > 256 ? 2 : 4);
  const int64_t most = ((int64_t)t.width * c.page_size + p.keys - 1) / p.keys;  // steps a sequence may have
  const int64_t pairs = (int64_t)t.batch * c.k_heads;
  p.whole = most <= 4;
  const int64_t steps = most * pairs;
  // a block a CU holds all of LDS; twice that for narrow heads
  const int blocks = (c.dtype == IPTTT_BF16 && dp == 64) ? 512 : 256;
  p.blocks = (int)(p.whole ? pairs : steps < blocks ? steps : blocks);
  p.cols = hq / c.k_heads < 32 ? hq / c.k_heads : 32;
  return p;
}
// A partial result: for each head the maximum, the sum, and dh sums of values.
__host__ __device__ inline int64_t part_size(int cols, int dh) { return (int64_t)cols * (dh + 2); }

// The keys of a sequence: [lo, hi), read in steps first .. first + n - 1 of so many.
struct Span {
  int lo, hi, first, n;
};
__device__ __forceinline__ Span span_of(const StepArgs &a, int keys, int b) {
  Span s;
  const int most = a.table.width * a.cache.page_size;
  s.hi = min(max(a.lens[b], 0), most);
  s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
  s.first = s.lo / keys;
  s.n = (s.hi + keys - 1) / keys - s.first;
  if (s.hi == 0) s.n = 0;
  return s;
}

// Steps of all sequences before sequence upto, times the key heads. Every wave for itself.
__device__ __forceinline__ int64_t steps_before(const StepArgs &a, int keys, int upto, int lane) {
  int64_t n = 0;
  for (int b = lane; b < upto; b += 64) n += span_of(a, keys, b).n;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  return n * a.cache.k_heads;
}
// The sequence whose steps hold `want`, and the number of steps before it.
__device__ __forceinline__ int find_step(const StepArgs &a, int keys, int64_t want, int lane,
                                          int64_t &before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.table.batch; b0 += 64) {
    const int b = b0 + lane;
    int64_t n = b < a.table.batch ? (int64_t)span_of(a, keys, b).n * a.cache.k_heads : 0, run = n;
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
// Blocks share the steps evenly; where there are fewer steps than blocks, a step each.
__device__ __forceinline__ int64_t first_step(int64_t total, int blocks, int block) {
  const int64_t used = total < blocks ? total : blocks;
  return block < used ? total * block / used : total;
}

__device__ const uint4 zero_row[kHeadMaxDim * 4 / 16] = {};

// A place in the row of steps: one step of a sequence and key head.
struct Cursor {
  int64_t at;      // the step
  int64_t from;    // the first step of this sequence and key head
  int b, kv;
  Span sp;
  __device__ __forceinline__ int64_t to() const { return from + sp.n; }
  // to the next sequence and key head that has keys
  __device__ __forceinline__ void next(const StepArgs &a, int keys) {
    from += sp.n;
    if (++kv < a.cache.k_heads) return;
    kv = 0;
    do {
      if (++b >= a.table.batch) return;
      sp = span_of(a, keys, b);
    } while (sp.n == 0);
  }
};

template <typename T, int DP>
__global__ __launch_bounds__((64 * waves_of<T, DP>())) void k_step(StepArgs a, Plan plan) {
  using L = Tile<T, DP>;
  constexpr int WAVES = waves_of<T, DP>(), KEYS = 32 * WAVES, TILE = 32 * DP;
  constexpr int RPI = 64 / L::NP, NI = 32 / RPI;  // rows an instruction copies, instructions a tile
  extern __shared__ __align__(1024) char smem[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, h = l >> 5,
            col = l & 31;
  T *const buf = (T *)smem + wave * 4 * TILE;  // this wave's [2][keys, values]
  float *const wm = (float *)((T *)smem + WAVES * 4 * TILE), *const wsum = wm + WAVES * 32;
  float *const wo = wsum + WAVES * 32;         // [WAVES][kJoinCols][DP]
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, ps = a.cache.page_size;
  const int group = a.hq / hk, chunks = chunks_of(a.hq, hk);
  const int block = blockIdx.x, chunk = blockIdx.y;
  const int cols = min(32, group - 32 * chunk);
  Cursor cc;  // what is computed
  int64_t end;
  if (plan.whole) {
    cc.b = block / hk;
    cc.kv = block % hk;
    cc.sp = span_of(a, KEYS, cc.b);
    cc.at = cc.from = 0;
    end = cc.sp.n;
    if (end == 0) {  // no key
      for (int i = tid; i < cols * dh; i += 64 * WAVES) {
        const int head = cc.kv * group + 32 * chunk + i / dh;
        ((T *)a.o.p)[cc.b * a.o.tok_stride + head * a.o.head_stride + i % dh] = (T)0.f;
      }
      if (a.lse && tid < cols) a.lse[(int64_t)cc.b * a.hq + cc.kv * group + 32 * chunk + tid] = -INFINITY;
      return;
    }
  } else {
    const int64_t total = (int64_t)uniform64((uint64_t)steps_before(a, KEYS, a.table.batch, l));
    cc.at = first_step(total, plan.blocks, block);
    end = first_step(total, plan.blocks, block + 1);
    if (cc.at >= end) return;
    int64_t before;
    cc.b = __builtin_amdgcn_readfirstlane(find_step(a, KEYS, cc.at, l, before));
    before = (int64_t)uniform64((uint64_t)before);
    cc.sp = span_of(a, KEYS, cc.b);
    cc.kv = __builtin_amdgcn_readfirstlane((int)((cc.at - before) / cc.sp.n));
    cc.from = before + (int64_t)cc.kv * cc.sp.n;
  }
  const bool direct = dh % L::PE == 0;  // the cache's rows are then on 16-byte boundaries
  if (dh != DP) {
    for (int i = l; i < 4 * TILE / L::PE; i += 64) ((uint4 *)buf)[i] = make_uint4(0, 0, 0, 0);
  }
  const float c = log2_scale(a.scale);
  // The page of this lane's key (lanes of both halves: key col) of a step, or -1.
  const auto page_of = [&](const Cursor &u) __attribute__((always_inline)) {
    const int key = (u.sp.first + (int)(u.at - u.from)) * KEYS + 32 * wave + col;
    if (key < u.sp.lo || key >= u.sp.hi) return -1;
    return a.table.p[u.b * a.table.stride + key / ps];
  };
  // Copies a step's keys and values; returns which of the 32 keys are there.
  const auto issue = [&](const Cursor &u, int page, int b) __attribute__((always_inline)) {
    const int key = (u.sp.first + (int)(u.at - u.from)) * KEYS + 32 * wave + col;
    const bool ok = page >= 0 && page < a.cache.pages;
    const int64_t place = ok ? (((int64_t)page * hk + u.kv) * ps + key % ps) * dh : -1;
    const uint32_t there = (uint32_t)__ballot(ok);
    if (there == 0) return there;
    T *const kt = buf + b * 2 * TILE, *const vt = kt + TILE;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + l / L::NP;
      const int64_t row = __shfl(place, r, 64);
      if (direct) {
        const int piece = (l % L::NP) ^ L::swizzle(r);
        if (DP == dh || piece * L::PE < dh) {
          const T *const ks = row < 0 ? (const T *)zero_row : (const T *)a.cache.k + row;
          const T *const vs = row < 0 ? (const T *)zero_row : (const T *)a.cache.v + row;
          copy_to_lds16(ks + piece * L::PE, kt + i * RPI * DP);
          copy_to_lds16(vs + piece * L::PE, vt + i * RPI * DP);
        }
      } else {
        const int ln = here(l), width = here(dh), p = ln % L::NP;
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
  Cursor ic = cc;  // what is copied: the step after the one computed
  uint32_t there = issue(ic, page_of(ic), 0), next = 0;
  const auto ahead = [&]() __attribute__((always_inline)) {
    if (++ic.at == ic.to() && ic.at < end) ic.next(a, KEYS);
    return ic.at < end ? page_of(ic) : -1;
  };
  int page = ahead();
  int cur = 0;
  RowReader<T, DP> rows(buf, l);
  ColReader<T, DP> vals(buf + TILE, l);
  while (cc.at < end) {
    // one sequence and key head, to its last step or the block's
    const bool begins = cc.at == cc.from;
    const int64_t stop = min(end, cc.to());
    const bool whole = begins && stop == cc.to();
    const T *qp = (const T *)a.q.p + cc.b * a.q.tok_stride +
                  (cc.kv * group + 32 * chunk + min(col, cols - 1)) * a.q.head_stride;
    Frag<T> q[L::STEPS];
#pragma unroll
    for (int i = 0; i < L::STEPS; ++i) q[i] = with_sign<T>(load_frag<T>(qp, i, h, dh), a.scale);
    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
    float m = -INFINITY, sum = 0.f;
    for (; cc.at < stop; ++cc.at) {
      // this step's tiles (and the next one's pages) have landed; all of this is one wave's
      mfma::wait_vm<0>();
      next = 0;
      if (ic.at < end) {
        next = issue(ic, page, cur ^ 1);
        page = ahead();
      }
      cur ^= 1;
      if (there != 0) {
        f32x16 x{};
#pragma unroll
        for (int i = 0; i < L::STEPS; ++i) x = mma(rows.read(0, i), q[i], x);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = there >> (8 * (i / 4) + i % 4 + 4 * h) & 1 ? x[i] : -INFINITY;
          top = fmaxf(top, x[i]);
        }
        top = half_max(top);
        if (__ballot((top - m) * c > 8.f)) {  // the maximum may fall behind by 2^8
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
          for (int d = 0; d < DP / 32; ++d) acc[d] = mma(vals.read(16 * i, d), p, acc[d]);
        }
      }
      there = next;
      rows.move(cur ? 2 * TILE * (int)sizeof(T) : -2 * TILE * (int)sizeof(T));
      vals.move(cur ? 2 * TILE * (int)sizeof(T) : -2 * TILE * (int)sizeof(T));
    }
    // the waves' results, joined through LDS
    sum = half_sum(sum);
    if (h == 0) {
      wm[wave * 32 + col] = m;
      wsum[wave * 32 + col] = sum;
    }
    __syncthreads();
    float top = -INFINITY, all = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, wm[i * 32 + col]);
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const float mi = wm[i * 32 + col];
      all += mi == -INFINITY ? 0.f : wsum[i * 32 + col] * exp2_((mi - top) * c);
    }
    const float f = m == -INFINITY ? 0.f : exp2_((m - top) * c) * (whole ? 1.f / all : 1.f);
    float *const part = (float *)a.ws + ((int64_t)(block * chunks + chunk) * 2 + (begins ? 1 : 0)) *
                                            part_size(plan.cols, dh);
    const int head0 = cc.kv * group + 32 * chunk;
    if (wave == 0 && h == 0 && col < cols) {
      if (!whole) {
        part[col * (dh + 2)] = top;
        part[col * (dh + 2) + 1] = all;
      } else if (a.lse) {
        a.lse[(int64_t)cc.b * a.hq + head0 + col] = top == -INFINITY ? -INFINITY : (top * c + log2f(all)) * kLn2;
      }
    }
    for (int c0 = 0; c0 < cols; c0 += kJoinCols) {
      if (col >= c0 && col < c0 + kJoinCols) {
        float *const mine = wo + (wave * kJoinCols + col - c0) * DP + 4 * h;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float4 v = make_float4(acc[d][4 * g] * f, acc[d][4 * g + 1] * f, acc[d][4 * g + 2] * f,
                                   acc[d][4 * g + 3] * f);
            if (m == -INFINITY) v = make_float4(0.f, 0.f, 0.f, 0.f);
            *(float4 *)(mine + 32 * d + 8 * g) = v;
          }
      }
      __syncthreads();
      const int n = min(kJoinCols, cols - c0) * dh;
      for (int i = tid; i < n; i += 64 * WAVES) {
        const int hh = i / dh, ch = i - hh * dh;
        float o = 0.f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) o += wo[(u * kJoinCols + hh) * DP + ch];
        if (whole) ((T *)a.o.p)[cc.b * a.o.tok_stride + (head0 + c0 + hh) * a.o.head_stride + ch] = (T)o;
        else part[(c0 + hh) * (dh + 2) + 2 + ch] = o;
      }
      __syncthreads();
    }
    if (cc.at < end) cc.next(a, KEYS);
  }
}

// Joins the partial results of a sequence's key head: the second of the block where it
// begins and the first of those up to the one where it ends.
template <typename T>
__global__ __launch_bounds__(256) void k_join(StepArgs a, Plan plan) {
  __shared__ float weight[512], red[8], half[kHeadMaxDim];
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, group = a.hq / hk;
  const int b = blockIdx.x / hk, kv = blockIdx.x % hk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunks = chunks_of(a.hq, hk);
  const Span sp = span_of(a, plan.keys, b);
  int g0 = 0, g1 = -1;  // the blocks whose steps hold the first and the last
  if (sp.n) {
    const int64_t from = steps_before(a, plan.keys, b, lane) + (int64_t)kv * sp.n;
    const int64_t total = steps_before(a, plan.keys, a.table.batch, lane);
    const int64_t used = total < plan.blocks ? total : plan.blocks;
    const auto block_of = [&](int64_t step) {
      int g = (int)(step * used / total);
      while (first_step(total, plan.blocks, g + 1) <= step) ++g;
      while (first_step(total, plan.blocks, g) > step) --g;
      return g;
    };
    g0 = block_of(from);
    g1 = block_of(from + sp.n - 1);
    if (g0 == g1) return;  // written already
  }
  const int n = g1 - g0 + 1;  // up to 512
  const int64_t size = part_size(plan.cols, dh);
  const float c = log2_scale(a.scale);
  for (int hh = blockIdx.y; hh < group; hh += gridDim.y) {
    const int64_t place = (int64_t)(hh / 32) * 2 * size + (hh % 32) * (dh + 2);
    const auto part = [&](int i) {
      return (const float *)a.ws + ((int64_t)(g0 + i) * chunks * 2 + (i == 0 ? 1 : 0)) * size + place;
    };
    float top = -INFINITY;
    for (int i = tid; i < n; i += 256) {
      weight[i] = part(i)[0];
      top = fmaxf(top, weight[i]);
    }
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor(top, k, 64));
    if (lane == 0) red[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float sum = 0.f;
    for (int i = tid; i < n; i += 256) {
      const float f = weight[i] == -INFINITY ? 0.f : exp2_((weight[i] - top) * c);
      weight[i] = f;
      sum += f * part(i)[1];
    }
    sum = blk::wave_sum(sum);
    if (lane == 0) red[4 + wave] = sum;
    __syncthreads();
    sum = (red[4] + red[5]) + (red[6] + red[7]);
    const int ch = tid & 127;
    float o = 0.f;
    if (ch < dh) {
#pragma unroll 8
      for (int i = tid >> 7; i < n; i += 2) {
        const float v = part(i)[2 + ch];
        o += weight[i] == 0.f ? 0.f : weight[i] * v;
      }
    }
    if (tid >= 128 && ch < dh) half[ch] = o;
    __syncthreads();
    const int head = kv * group + hh;
    if (tid < dh)
      ((T *)a.o.p)[b * a.o.tok_stride + head * a.o.head_stride + tid] =
          (T)(top == -INFINITY ? 0.f : (o + half[tid]) / sum);
    if (a.lse && tid == 0)
      a.lse[(int64_t)b * a.hq + head] = top == -INFINITY ? -INFINITY : (top * c + log2f(sum)) * kLn2;
    __syncthreads();
  }
}

}  // namespace

size_t step_workspace(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t) {
  const Plan p = plan_of(hq, c, t);
  if (p.whole) return 256;
  return (size_t)round_up(
      (int64_t)p.blocks * chunks_of(hq, c.k_heads) * 2 * part_size(p.cols, c.head_dim) * 4, 256);
}

template <typename T>
hipError_t step_forward(const StepArgs &a, hipStream_t st) {
  const Plan p = plan_of(a.hq, a.cache, a.table);
  const int chunks = chunks_of(a.hq, a.cache.k_heads);
  const auto go = [&](auto dp) {
    constexpr int DP = decltype(dp)::value, WAVES = waves_of<T, DP>();
    const size_t lds = WAVES * (4 * 32 * DP * sizeof(T) + (64 + kJoinCols * DP) * sizeof(float));
    k_step<T, DP><<<dim3(p.blocks, chunks), 64 * WAVES, lds, st>>>(a, p);
  };
  if (a.cache.head_dim <= 64) go(std::integral_constant<int, 64>());
  else go(std::integral_constant<int, 128>());
  if (!p.whole) {
    const int group = a.hq / a.cache.k_heads;
    k_join<T><<<dim3(a.table.batch * a.cache.k_heads, group < 32 ? group : 32), 256, 0, st>>>(a, p);
  }
  return hipGetLastError();
}

template hipError_t step_forward<float>(const StepArgs &, hipStream_t);
template hipError_t step_forward<__bf16>(const StepArgs &, hipStream_t);

}  // namespace ipttt
