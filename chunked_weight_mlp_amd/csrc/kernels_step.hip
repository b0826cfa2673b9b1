// Attention of one new token of each sequence over the paged cache (gfx950).
#include "attention_common.h"

namespace ipttt {
namespace {

using namespace attn;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kKeys = 32 * kWaves;   // keys a block reads a step, 32 a wave
constexpr int kMostBlocks = 1024;

// Heads of a key head's group are columns of a 32-column tile; wider groups take several.
__host__ __device__ inline int chunks_of(int hq, int hk) { return (hq / hk + 31) / 32; }

struct Plan {
  int blocks;    // blocks of the first kernel (for each chunk of heads)
  bool whole;    // a block for each sequence and key head: nothing to join
  int cols;      // heads a partial result has room for
};
Plan plan_of(int hq, const ipttt_kv_cache &c, const ipttt_page_table &t) {
  Plan p;
  const int64_t most = ((int64_t)t.width * c.page_size + kKeys - 1) / kKeys;  // steps a sequence may have
  const int64_t pairs = (int64_t)t.batch * c.k_heads;
  p.whole = most <= 4;
  const int64_t steps = most * pairs;
  p.blocks = (int)(p.whole ? pairs : steps < kMostBlocks ? steps : kMostBlocks);
  p.cols = hq / c.k_heads < 32 ? hq / c.k_heads : 32;
  return p;
}
// A partial result: for each head the maximum, the sum, and dh sums of values.
__host__ __device__ inline int64_t part_size(int cols, int dh) { return (int64_t)cols * (dh + 2); }

// The keys of a sequence: [lo, hi), read in steps first .. first + n - 1 of kKeys.
struct Span {
  int lo, hi, first, n;
};
__device__ __forceinline__ Span span_of(const StepArgs &a, int b) {
  Span s;
  const int most = a.table.width * a.cache.page_size;
  s.hi = min(max(a.lens[b], 0), most);
  s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
  s.first = s.lo / kKeys;
  s.n = (s.hi + kKeys - 1) / kKeys - s.first;
  if (s.hi == 0) s.n = 0;
  return s;
}

// Steps of all sequences before sequence b (of all for b = batch), times the key heads.
// The sequence that holds step `want`, if given. Every wave does this by itself.
__device__ __forceinline__ int64_t steps_before(const StepArgs &a, int upto, int lane) {
  int64_t n = 0;
  for (int b = lane; b < upto; b += 64) n += span_of(a, b).n;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  return n * a.cache.k_heads;
}
// The sequence whose steps hold `want`, and the number of steps before it.
__device__ __forceinline__ int find_step(const StepArgs &a, int64_t want, int lane, int64_t &before) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.table.batch; b0 += 64) {
    const int b = b0 + lane;
    int64_t n = b < a.table.batch ? (int64_t)span_of(a, b).n * a.cache.k_heads : 0, run = n;
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

template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void k_step(StepArgs a, Plan plan) {
  using L = Tile<T, DP>;
  extern __shared__ __align__(1024) char smem[];
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, h = l >> 5, col = l & 31;
  T *const kt = (T *)smem + wave * 64 * DP, *const vt = kt + 32 * DP;
  const RowReader<T, DP> rows(kt, l);
  const ColReader<T, DP> vals(vt, l);
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, ps = a.cache.page_size;
  const int group = a.hq / hk, chunks = chunks_of(a.hq, hk);
  const int block = blockIdx.x, chunk = blockIdx.y;
  const int cols = min(32, group - 32 * chunk);
  int64_t at, end;  // this block's steps
  int b;
  int64_t before;
  if (plan.whole) {
    b = block / hk;
    const int n = span_of(a, b).n;
    before = 0;
    at = (int64_t)(block % hk) * n;
    end = at + n;
    if (n == 0) {  // no key
      const int kv = block % hk;
      for (int i = tid; i < cols * dh; i += kThreads) {
        const int head = kv * group + 32 * chunk + i / dh;
        ((T *)a.o.p)[b * a.o.tok_stride + head * a.o.head_stride + i % dh] = (T)0.f;
      }
      if (a.lse && tid < cols) a.lse[(int64_t)b * a.hq + kv * group + 32 * chunk + tid] = -INFINITY;
      return;
    }
  } else {
    const int64_t total = steps_before(a, a.table.batch, l);
    at = first_step(total, plan.blocks, block);
    end = first_step(total, plan.blocks, block + 1);
    if (at >= end) return;
    b = find_step(a, at, l, before);
  }
  const float c = log2_scale(a.scale);
  while (at < end) {
    // one sequence and key head: steps [at, stop) of its [from, from + n)
    Span sp = span_of(a, b);
    const int kv = (int)((at - before) / sp.n);
    const int64_t from = before + (int64_t)kv * sp.n;
    const int64_t stop = min(end, from + sp.n);
    const T *qp = (const T *)a.q.p + b * a.q.tok_stride +
                  (kv * group + 32 * chunk + min(col, cols - 1)) * a.q.head_stride;
    Frag<T> q[L::STEPS];
#pragma unroll
    for (int i = 0; i < L::STEPS; ++i) q[i] = with_sign<T>(load_frag<T>(qp, i, h, dh), a.scale);
    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) acc[d] = f32x16{};
    float m = -INFINITY, sum = 0.f;
    const int32_t *pages = a.table.p + b * a.table.stride;
    for (int64_t st = at; st < stop; ++st) {
      const int k0 = (sp.first + (int)(st - from)) * kKeys + 32 * wave;
      // lane l < 32: the place of key k0 + l, or -1
      const int key = k0 + col;
      int64_t place = -1;
      if (key >= sp.lo && key < sp.hi) {
        const int pg = key / ps, page = pages[pg];
        if (page >= 0 && page < a.cache.pages)
          place = (((int64_t)page * hk + kv) * ps + (key - pg * ps)) * dh;
      }
      const uint32_t there = (uint32_t)__ballot(place >= 0);  // the lower half's 32 keys
      if (there == 0) continue;
      for (int i = l; i < 32 * L::NP; i += 64) {
        const int r = i / L::NP, p = i % L::NP;
        const int64_t row = __shfl(place, r, 64);
        const T *ks = row < 0 ? (const T *)zero_row : (const T *)a.cache.k + row;
        const T *vs = row < 0 ? (const T *)zero_row : (const T *)a.cache.v + row;
        T x[L::PE];
        load_some<T, L::PE>(ks, p * L::PE, dh, x);
#pragma unroll
        for (int e = 0; e < L::PE; ++e) kt[L::at(r, p) + e] = x[e];
        load_some<T, L::PE>(vs, p * L::PE, dh, x);
#pragma unroll
        for (int e = 0; e < L::PE; ++e) vt[L::at(r, p) + e] = x[e];
      }
      __builtin_amdgcn_wave_barrier();
      f32x16 x{};
#pragma unroll
      for (int i = 0; i < L::STEPS; ++i) x = mma(rows.read(0, i), q[i], x);
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i / 4) + 4 * h + i % 4;
        x[i] = there >> r & 1 ? x[i] : -INFINITY;
        top = fmaxf(top, x[i]);
      }
      top = half_max(top);
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
      for (int i = 0; i < 16; ++i) {
        x[i] = exp2_((x[i] - base) * c);
        sum += x[i];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Frag<T> p = as_operand<T>(x, i);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          acc[d] = mma(vals.read(16 * i, d), p, acc[d]);
      }
      __builtin_amdgcn_wave_barrier();
    }
    sum = half_sum(sum);
    // the waves' results, joined through LDS
    __syncthreads();
    float *const wm = (float *)smem, *const ws = wm + kWaves * 32, *const wo = ws + kWaves * 32;
    if (h == 0) {
      wm[wave * 32 + col] = m;
      ws[wave * 32 + col] = sum;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, wm[i * 32 + col]);
    const float f = m == -INFINITY ? 0.f : exp2_((m - top) * c);
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
      all += ws[i * 32 + col] * (wm[i * 32 + col] == -INFINITY ? 0.f : exp2_((wm[i * 32 + col] - top) * c));
    for (int i = 0; i < kWaves; ++i) {
      if (wave == i && col < cols) {
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int ch = 32 * d + 8 * (e / 4) + 4 * h + e % 4;
            float &o = wo[col * DP + ch];
            o = (i ? o : 0.f) + (m == -INFINITY ? 0.f : acc[d][e] * f);
          }
      }
      __syncthreads();
    }
    const bool begins = at == from, ends = stop == from + sp.n;
    float *const part = (float *)a.ws + ((int64_t)(block * chunks + chunk) * 2 + (begins ? 1 : 0)) *
                                            part_size(plan.cols, dh);
    if (wave == 0 && h == 0 && col < cols) {
      wm[col] = top;
      ws[col] = all;
      if (!(begins && ends)) {
        part[col * (dh + 2)] = top;
        part[col * (dh + 2) + 1] = all;
      } else if (a.lse) {
        a.lse[(int64_t)b * a.hq + kv * group + 32 * chunk + col] =
            top == -INFINITY ? -INFINITY : (top * c + log2f(all)) * kLn2;
      }
    }
    __syncthreads();
    for (int i = tid; i < cols * dh; i += kThreads) {
      const int hh = i / dh, ch = i - hh * dh;
      if (begins && ends) {
        const float o = wm[hh] == -INFINITY ? 0.f : wo[hh * DP + ch] / ws[hh];
        ((T *)a.o.p)[b * a.o.tok_stride + (kv * group + 32 * chunk + hh) * a.o.head_stride + ch] = (T)o;
      } else {
        part[hh * (dh + 2) + 2 + ch] = wo[hh * DP + ch];
      }
    }
    __syncthreads();
    at = stop;
    if (at < end && kv == hk - 1) {  // the next sequence that has a key
      before += (int64_t)sp.n * hk;
      do ++b; while (b < a.table.batch && span_of(a, b).n == 0);
    }
  }
}

// Joins the partial results of a sequence's key head: the second of the block where it
// begins and the first of those up to the one where it ends.
template <typename T>
__global__ __launch_bounds__(128) void k_join(StepArgs a, Plan plan) {
  const int hk = a.cache.k_heads, dh = a.cache.head_dim, group = a.hq / hk;
  const int b = blockIdx.x / hk, kv = blockIdx.x % hk, tid = threadIdx.x, lane = tid & 63;
  const int chunks = chunks_of(a.hq, hk);
  const Span sp = span_of(a, b);
  const int64_t from = sp.n ? steps_before(a, b, lane) + (int64_t)kv * sp.n : 0;
  const int64_t total = sp.n ? steps_before(a, a.table.batch, lane) : 1;
  // the blocks whose steps hold the first and the last
  const auto block_of = [&](int64_t step) {
    int g = (int)(step * (total < plan.blocks ? total : plan.blocks) / total);
    while (first_step(total, plan.blocks, g + 1) <= step) ++g;
    while (first_step(total, plan.blocks, g) > step) --g;
    return g;
  };
  const int g0 = block_of(from), g1 = sp.n ? block_of(from + sp.n - 1) : g0;
  if (sp.n && g0 == g1) return;  // written already
  const int64_t size = part_size(plan.cols, dh);
  const float c = log2_scale(a.scale);
  for (int hh = blockIdx.y; hh < group; hh += gridDim.y) {
    const int chunk = hh / 32, col = hh % 32;
    const auto part = [&](int g) {
      return (const float *)a.ws + ((int64_t)(g * chunks + chunk) * 2 + (g == g0 ? 1 : 0)) * size +
             col * (dh + 2);
    };
    float top = -INFINITY, sum = 0.f, o = 0.f;
    if (sp.n) {
      for (int g = g0; g <= g1; ++g) top = fmaxf(top, part(g)[0]);
      for (int g = g0; g <= g1; ++g) {
        const float *p = part(g);
        if (p[0] == -INFINITY) continue;
        const float f = exp2_((p[0] - top) * c);
        sum += f * p[1];
        if (tid < dh) o += f * p[2 + tid];
      }
    }
    const int head = kv * group + hh;
    if (tid < dh)
      ((T *)a.o.p)[b * a.o.tok_stride + head * a.o.head_stride + tid] =
          (T)(top == -INFINITY ? 0.f : o / sum);
    if (a.lse && tid == 0)
      a.lse[(int64_t)b * a.hq + head] = top == -INFINITY ? -INFINITY : (top * c + log2f(sum)) * kLn2;
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
    constexpr int DP = decltype(dp)::value;
    const size_t lds = kWaves * 64 * DP * sizeof(T), join = (kWaves * 64 + 32 * DP) * 4;
    k_step<T, DP><<<dim3(p.blocks, chunks), kThreads, lds > join ? lds : join, st>>>(a, p);
  };
  if (a.cache.head_dim <= 64) go(std::integral_constant<int, 64>());
  else go(std::integral_constant<int, 128>());
  if (!p.whole) {
    const int group = a.hq / a.cache.k_heads;
    k_join<T><<<dim3(a.table.batch * a.cache.k_heads, group < 32 ? group : 32), 128, 0, st>>>(a, p);
  }
  return hipGetLastError();
}

template hipError_t step_forward<float>(const StepArgs &, hipStream_t);
template hipError_t step_forward<__bf16>(const StepArgs &, hipStream_t);

}  // namespace ipttt
