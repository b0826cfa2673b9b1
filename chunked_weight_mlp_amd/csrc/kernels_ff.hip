// The gated feed-forward block y = (SiLU(x W_g) * (x W_u)) W_d, forward and
// backward.
//
// Every product of the block runs on one bf16 MFMA kernel (k_ff_gemm) over
// operands whose K values are contiguous and padded with zeros to whole steps of
// 64, with the output written contiguously along the first operand's rows:
//   a, u [n][F]  = W_g, W_u rows x x rows          K = d   (one launch, z fused)
//   y    [n][d]  = W_d rows x z rows               K = F
//   dz   [n][F]  = W_d^T rows x dy rows            K = d   (dA, dU, z fused)
//   dx   [n][d]  = [W_g^T W_u^T] rows x [dA dU] rows   K = 2F
//   dW_g, dW_u [F][d] = x^T rows x [dA dU]^T rows  K = n   (one launch)
//   dW_d [d][F]  = z^T rows x dy^T rows            K = n
// bf16 operands that already have that layout are used in place; the others are
// copied or transposed into the workspace first. An fp32 operand is split there
// into three bf16 planes (p0 + p1 + p2 is the value exactly: each plane takes the
// next 8 bits of its significand), and its products sum the six plane pairs
// p0 q2, p2 q0, p1 q1, p0 q1, p1 q0, p0 q0, which leaves out only terms below
// 2^-24 of a product: fp32 accuracy at six times the bf16 work, against
// 1/16 of the bf16 rate for the fp32 MFMA.
#include <algorithm>

#include "block_internal.h"
#include "mfma_common.h"

namespace ipttt {
namespace mfma {
namespace {

using blk::Pack;

constexpr int64_t kStep = 64;  // K values of one step
inline int64_t kpad(int64_t k) { return round_up(k, kStep); }

template <typename T>
constexpr int planes_of() {
  return sizeof(T) == 2 ? 1 : 3;
}

// Plane q of an fp32 value: its first, second and third 8 significand bits
// (truncated, so no plane overflows; a non-finite value is plane 0 alone).
__device__ __forceinline__ void split3(float v, __bf16 (&p)[3]) {
  const float a = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u);
  const bool fin = (__builtin_bit_cast(uint32_t, v) & 0x7f800000u) != 0x7f800000u;
  const float r = fin ? v - a : 0.f;
  const float b = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r) & 0xffff0000u);
  p[0] = fin ? (__bf16)a : (__bf16)v;
  p[1] = (__bf16)b;
  p[2] = (__bf16)(r - b);
}

// v as NP planes: one rounded bf16 value, or the exact split.
template <int NP>
__device__ __forceinline__ void store8_planes(__bf16 *p, int64_t plane, const float (&v)[8]) {
  bf16x8 o[NP];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (NP == 1) {
      o[0][e] = (__bf16)v[e];
    } else {
      __bf16 q[3];
      split3(v[e], q);
#pragma unroll
      for (int k = 0; k < NP; ++k) o[k][e] = q[k];
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) *(bf16x8 *)(p + k * plane) = o[k];
}

// ---- the product ---------------------------------------------------------------------

// out(m, n) = sum_k A[m][k] B[n][k]. A rows (and A2 rows, for a pair of products
// sharing B) at and past M, and B rows at and past N, repeat the last one; what
// they give is not written. nk: steps of 64 per plane pair.
struct FfProb {
  const __bf16 *a, *a2, *b;
  int64_t lda, ldb, pa, pb;  // row pitches and plane distances
  int M, N, nk;
  int splits;  // parts of K, each its own blocks (epilogue: partial sums)
};

template <class C, int NP, bool DUAL, class Epi>
__global__ __launch_bounds__(C::NTHR) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_ff_gemm(
    FfProb g, Epi epi) {
  static_assert(C::SMEM_ELEMS * 2 <= 160 * 1024, "LDS overflow");
  __shared__ __attribute__((aligned(1024))) __bf16 smem[C::SMEM_ELEMS];
  using M = typename C::M;
  static_assert(M::NG == 1 && C::MI % 4 == 0, "pairs of 16-row tiles");
  constexpr int MT = DUAL ? C::BM / 2 : C::BM;    // output rows per block
  constexpr int WT = DUAL ? C::WTM / 2 : C::WTM;  // and per wave
  constexpr int HI = DUAL ? C::MI / 2 : C::MI;
  const int nm = (g.M + MT - 1) / MT, nn = (g.N + C::BN - 1) / C::BN;
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int sp = id / (nm * nn);
  int tm, tn;
  tile_of<C::GM>(id % (nm * nn), nm, nn, tm, tn);
  const int m0 = tm * MT, n0 = tn * C::BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  DmaLoader<C, C::BM> la;
  DmaLoader<C, C::BN> lb;
  la.init(wave, lane, [&](int r) {
    if constexpr (DUAL)
      return (r < MT ? g.a : g.a2) + (int64_t)min(m0 + (r < MT ? r : r - MT), g.M - 1) * g.lda;
    else
      return g.a + (int64_t)min(m0 + r, g.M - 1) * g.lda;
  });
  lb.init(wave, lane, [&](int r) { return g.b + (int64_t)min(n0 + r, g.N - 1) * g.ldb; });
  int brow[C::NJ], arow[C::MI];
#pragma unroll
  for (int j = 0; j < C::NJ; ++j) brow[j] = wn * C::WTN + C::FM * j;
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
    arow[i] = (i < HI ? 0 : MT) + wm * WT + C::FM * (i < HI ? i : i - HI);
  typename C::acc_t acc[C::MI][C::NJ];
  zero_acc<C>(acc);
  // this block's steps of the (plane pair, K step) sequence
  constexpr int PAIRS = NP == 1 ? 1 : 6;
  const int total = PAIRS * g.nk, per = (total + g.splits - 1) / g.splits;
  const int first = sp * per, count = min(per, total - first);
  int pair = NP == 1 ? 0 : first / g.nk, ks = NP == 1 ? first : first % g.nk;
  kloop_dma_pl<C, 2, true, C::MI + C::NJ>(
      smem, la, lb, count, wave, acc,
      [&](const __bf16 *As, const __bf16 *Bs, int u, Frags<C> &f) __attribute__((always_inline)) {
        const int r = M::orow(lane), kq = M::okoff(lane);
#pragma unroll
        for (int j = 0; j < C::NJ; ++j)
          f.b[j] = *(const bf16x8 *)(Bs + (brow[j] + r) * C::PITCH +
                                     kslot<C>(brow[j] + r, M::K * u + kq));
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
          f.a[i] = *(const bf16x8 *)(As + (arow[i] + r) * C::PITCH +
                                     kslot<C>(arow[i] + r, M::K * u + kq));
      },
      [&](int, int64_t &ka, int64_t &kb) __attribute__((always_inline)) {  // called in order
        ka = kb = (int64_t)ks * kStep;
        if constexpr (NP == 3) {  // pairs (0,2) (2,0) (1,1) (0,1) (1,0) (0,0), small ones first
          ka += ((0x010120 >> (4 * pair)) & 15) * g.pa;
          kb += ((0x001102 >> (4 * pair)) & 15) * g.pb;
          if (++ks == g.nk) {
            ks = 0;
            ++pair;
          }
        } else {
          ++ks;
        }
      },
      [](int) {}, [](int) {});
  // Lane l holds rows 4 (l / 16) .. + 3 of a 16-row tile at column l % 16.
  // Swapping lane groups of tiles i and i + 1 leaves each lane 8 consecutive
  // rows: m .. m + 7 at column n.
  const int gq = lane >> 4;
  const auto rows8 = [](f32x4 a, f32x4 b, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = a[r], y = b[r];
      const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x),
                                                      __builtin_bit_cast(unsigned, y), false, false);
      v[r] = __builtin_bit_cast(float, (unsigned)s[0]);
      v[4 + r] = __builtin_bit_cast(float, (unsigned)s[1]);
    }
  };
#pragma unroll
  for (int i = 0; i < HI; i += 2) {
    const int m = m0 + wm * WT + C::FM * i + 8 * (gq >> 1) + C::FM * (gq & 1);
    typename Epi::In in[C::NJ];
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)  // all loads of these tiles before their stores
      in[j] = epi.load(m, min(n0 + brow[j] + M::rcol(lane), g.N - 1));
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) {
      const int n = n0 + brow[j] + M::rcol(lane);
      float v[8];
      rows8(acc[i][j], acc[i + 1][j], v);
      if constexpr (DUAL) {
        float w[8];
        rows8(acc[i + HI][j], acc[i + HI + 1][j], w);
        if (n < g.N) epi.store(m, n, v, w);
      } else {
        if (n < g.N) epi.store(m, n, v, in[j], sp);
      }
    }
  }
}

struct NoIn {};

// 8 outputs m .. m + 7 of a row of M
template <typename T>
__device__ __forceinline__ void store8(T *row, int m, int M, const float (&v)[8]) {
  if (m + 8 <= M) {
    blk::store_pack<T, 8>(row + m, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (m + e < M) row[m + e] = (T)v[e];
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T *row, int m, int M, float (&v)[8]) {
  if (m + 8 <= M) {
    blk::load_pack<T, 8>(row + m, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = m + e < M ? (float)row[m + e] : 0.f;
  }
}

// z = SiLU(a) u as the next product's operand (padded with zeros to Fp), and a,
// u themselves when saved.
template <typename T>
struct EpiZ {
  using In = NoIn;
  __bf16 *z;
  int64_t plane;
  int F, Fp;
  T *a, *u;
  __device__ In load(int, int) const { return {}; }
  __device__ void store(int m, int n, const float (&av)[8], const float (&uv)[8]) const {
    if (m >= Fp) return;
    float zv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      zv[e] = m + e < F ? av[e] * fast_sigmoid(av[e]) * uv[e] : 0.f;
    store8_planes<planes_of<T>()>(z + (int64_t)n * Fp + m, plane, zv);
    if (a) {
      store8<T>(a + (int64_t)n * F, m, F, av);
      store8<T>(u + (int64_t)n * F, m, F, uv);
    }
  }
};

// out[n][m], rows ld apart; columns n >= cut go to out2 (n - cut).
template <typename T>
struct EpiOut {
  using In = NoIn;
  T *out, *out2;
  int64_t ld;
  int M, N, cut;  // N: rows of each output
  __device__ In load(int, int) const { return {}; }
  __device__ void store(int m, int n, const float (&v)[8], In, int) const {
    const bool second = n >= cut;
    const int row = second ? n - cut : n;
    if (m < M && row < N) store8<T>((second ? out2 : out) + (int64_t)row * ld, m, M, v);
  }
};

// Partial sums of one part of K: fp32 [part][n][ld], ld a multiple of 8.
struct EpiPart {
  using In = NoIn;
  float *out;
  int64_t stride, ld;
  __device__ In load(int, int) const { return {}; }
  __device__ void store(int m, int n, const float (&v)[8], In, int sp) const {
    if (m < ld) blk::store_pack<float, 8>(out + sp * stride + (int64_t)n * ld + m, v);
  }
};

// dz -> dA = dz u SiLU'(a), dU = dz SiLU(a), z = SiLU(a) u, operands padded with
// zeros to Fp; a and u come from the forward in the block's type.
template <typename T>
struct EpiDz {
  struct In {
    float a[8], u[8];
  };
  const T *a, *u;
  __bf16 *dau, *z;  // [n][2 Fp]: dA then dU; [n][Fp]
  int64_t dau_plane, z_plane;
  int F, Fp;
  __device__ In load(int m, int n) const {
    In in;
    load8<T>(a + (int64_t)n * F, m, F, in.a);
    load8<T>(u + (int64_t)n * F, m, F, in.u);
    return in;
  }
  __device__ void store(int m, int n, const float (&v)[8], const In &in, int) const {
    if (m >= Fp) return;
    float da[8], du[8], zv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool real = m + e < F;
      const float s = fast_sigmoid(in.a[e]), h = in.a[e] * s;
      da[e] = real ? v[e] * in.u[e] * (s + h * (1.f - s)) : 0.f;
      du[e] = real ? v[e] * h : 0.f;
      zv[e] = real ? h * in.u[e] : 0.f;
    }
    constexpr int NP = planes_of<T>();
    __bf16 *row = dau + (int64_t)n * 2 * Fp + m;
    store8_planes<NP>(row, dau_plane, da);
    store8_planes<NP>(row + Fp, dau_plane, du);
    store8_planes<NP>(z + (int64_t)n * Fp + m, z_plane, zv);
  }
};

// out[n][m] = sum of the parts, in order
template <typename T>
__global__ __launch_bounds__(256) void k_ff_join(const float *__restrict__ part, int parts,
                                                 int64_t stride, int64_t ld, int64_t n, int M,
                                                 T *__restrict__ out, int64_t out_ld) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = ld / 8;
  if (i >= n * per) return;
  const int64_t row = i / per;
  const int m = 8 * (int)(i % per);
  float s[8] = {};
  for (int p = 0; p < parts; ++p) {
    float v[8];
    blk::load_pack<float, 8>(part + p * stride + row * ld + m, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[e];
  }
  store8<T>(out + row * out_ld, m, M, s);
}

// ---- operand layouts -------------------------------------------------------------------

// src [R][C] (rows src_ld apart) -> planes [R][ld], columns C .. ld zero; ld a multiple of 8
template <typename T>
__global__ __launch_bounds__(256) void k_ff_rows(const T *__restrict__ src, int64_t src_ld,
                                                 int64_t R, int C, __bf16 *__restrict__ out,
                                                 int64_t ld, int64_t plane) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = ld / 8;
  if (i >= R * per) return;
  const int64_t r = i / per;
  const int c = 8 * (int)(i % per);
  float v[8];
  load8<T>(src + r * src_ld, c, C, v);
  store8_planes<planes_of<T>()>(out + r * ld + c, plane, v);
}

// src [R][C] -> planes [C][ld], out[c][r] = src[r][c] for r < R, zero for R <= r <
// Rp (a multiple of 64). NP planes from an fp32 source; a bf16 source has NS
// planes of its own (gridDim.z), each transposed. 64 x 64 tiles through LDS.
template <typename T>
__global__ __launch_bounds__(256) void k_ff_trans(const T *__restrict__ src, int64_t src_ld,
                                                  int64_t src_plane, int64_t R, int C,
                                                  __bf16 *__restrict__ out, int64_t ld,
                                                  int64_t plane) {
  __shared__ float tile[64][65];
  constexpr int NP = planes_of<T>();
  src += blockIdx.z * src_plane;
  out += blockIdx.z * plane;
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int c0 = blockIdx.y * 64;
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (tid >> 3) + 32 * k, c = 8 * (tid & 7);
    float v[8] = {};
    if (r0 + r < R && c0 + c < C) load8<T>(src + (r0 + r) * src_ld, c0 + c, C, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[r][c + e] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = (tid >> 3) + 32 * k, r = 8 * (tid & 7);
    if (c0 + c < C) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[r + e][c];
      store8_planes<NP>(out + (int64_t)(c0 + c) * ld + r0 + r, plane, v);
    }
  }
}

__global__ __launch_bounds__(256) void k_ff_zero(uint16_t *__restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

// ---- few tokens -------------------------------------------------------------------------
// Up to 64 tokens every weight is read once and little else moves, so the weights
// go straight from memory into MFMA operands: a block owns 16 weight rows (of both
// W_g and W_u in the first product), its WV waves take interleaved pieces of K,
// and their sums meet in LDS. A lane's 16 bytes of row l % 16 are one operand
// register set: 8 bf16 values of one 16x16x32 MFMA, or 4 fp32 values of four
// 16x16x4 ones (any assignment of K values to lanes gives the same sum as long
// as both operands share it). NT: groups of 16 tokens.

template <typename T>
struct Quad;  // 16 bytes of one operand row
template <>
struct Quad<__bf16> {
  static constexpr int E = 8;
  bf16x8 v;
  __device__ __forceinline__ void set(int e, float x) { v[e] = (__bf16)x; }
  __device__ static __forceinline__ f32x4 mma(const Quad &a, const Quad &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
  }
};
template <>
struct Quad<float> {
  static constexpr int E = 4;
  f32x4 v;
  __device__ __forceinline__ void set(int e, float x) { v[e] = x; }
  __device__ static __forceinline__ f32x4 mma(const Quad &a, const Quad &b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
};

template <typename T>
__device__ __forceinline__ Quad<T> quad_at(const T *p) {
  const Pack<T, Quad<T>::E> k = *(const Pack<T, Quad<T>::E> *)p;
  return __builtin_bit_cast(Quad<T>, k);
}
// the same with zeros at and past the row's end
template <typename T>
__device__ __forceinline__ Quad<T> quad_end(const T *row, int k, int K) {
  if (k + Quad<T>::E <= K) return quad_at<T>(row + k);
  Quad<T> q;
#pragma unroll
  for (int e = 0; e < Quad<T>::E; ++e) q.set(e, k + e < K ? (float)row[k + e] : 0.f);
  return q;
}

// acc[t] (and acc2[t]) += the block's 16 weight rows times token group t over this
// wave's pieces of K. U MFMA steps per piece.
template <typename T, int NT, int WV, bool DUAL>
__device__ __forceinline__ void small_dot(const T *wrow, const T *w2row, const T *const (&xrow)[NT],
                                          int K, int wave, int lane, f32x4 (&acc)[NT],
                                          f32x4 (&acc2)[NT]) {
  constexpr int U = DUAL ? 4 : 8;
  constexpr int S = 4 * Quad<T>::E;  // K values of one step (64 bytes of a row)
  constexpr int P = U * S;
  const int kl = Quad<T>::E * (lane >> 4);
  int k0 = wave * P;
  for (; k0 + P <= K; k0 += WV * P) {
    Quad<T> w[U], w2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = quad_at<T>(wrow + k0 + S * u + kl);
      if constexpr (DUAL) w2[u] = quad_at<T>(w2row + k0 + S * u + kl);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Quad<T> x = quad_at<T>(xrow[t] + k0 + S * u + kl);
        acc[t] = Quad<T>::mma(w[u], x, acc[t]);
        if constexpr (DUAL) acc2[t] = Quad<T>::mma(w2[u], x, acc2[t]);
      }
  }
  if (k0 < K)  // the row's last, partial piece (one wave)
    for (int k = k0; k < K; k += S) {
      const Quad<T> w = quad_end<T>(wrow, k + kl, K);
      Quad<T> w2{};
      if constexpr (DUAL) w2 = quad_end<T>(w2row, k + kl, K);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Quad<T> x = quad_end<T>(xrow[t], k + kl, K);
        acc[t] = Quad<T>::mma(w, x, acc[t]);
        if constexpr (DUAL) acc2[t] = Quad<T>::mma(w2, x, acc2[t]);
      }
    }
}

// DUAL: out = SiLU(W x) (W2 x), with W x and W2 x saved to a, u when given.
// Otherwise out = W x. W [M][K] dense, x rows x_ld apart, out rows out_ld apart.
template <typename T, int NT, int WV, bool DUAL>
__global__ __launch_bounds__(64 * WV) void k_ff_small(const T *__restrict__ w,
                                                      const T *__restrict__ w2,
                                                      const T *__restrict__ x, int64_t x_ld, int n,
                                                      int M, int K, T *__restrict__ out,
                                                      int64_t out_ld, T *__restrict__ a,
                                                      T *__restrict__ u) {
  __shared__ f32x4 sum[WV][DUAL ? 2 : 1][NT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = 16 * blockIdx.x;
  const int64_t row = (int64_t)min(m0 + (lane & 15), M - 1) * K;
  const T *xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = x + (int64_t)min(16 * t + (lane & 15), n - 1) * x_ld;
  f32x4 acc[NT] = {}, acc2[NT] = {};
  small_dot<T, NT, WV, DUAL>(w + row, DUAL ? w2 + row : nullptr, xrow, K, wave, lane, acc, acc2);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    sum[wave][0][t][lane] = acc[t];
    if constexpr (DUAL) sum[wave][1][t][lane] = acc2[t];
  }
  __syncthreads();
  // lane holds rows 4 (l / 16) .. + 3 at token l % 16
  for (int t = wave; t < NT; t += WV) {
    const int tok = 16 * t + (lane & 15), m = m0 + 4 * (lane >> 4);
    f32x4 s{}, s2{};
#pragma unroll
    for (int q = 0; q < WV; ++q) {
      s += sum[q][0][t][lane];
      if constexpr (DUAL) s2 += sum[q][1][t][lane];
    }
    if (tok < n) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (m + r < M) {
          if constexpr (DUAL) {
            if (a) {
              a[(int64_t)tok * M + m + r] = (T)s[r];
              u[(int64_t)tok * M + m + r] = (T)s2[r];
            }
            out[tok * out_ld + m + r] = (T)(s[r] * fast_sigmoid(s[r]) * s2[r]);
          } else {
            out[tok * out_ld + m + r] = (T)s[r];
          }
        }
    }
  }
}

constexpr int kSmallTokens = 64;

template <typename T, int WV, bool DUAL>
hipError_t launch_small(const T *w, const T *w2, const T *x, int64_t x_ld, int n, int M, int K,
                        T *out, int64_t out_ld, T *a, T *u, hipStream_t st) {
  const dim3 grid((M + 15) / 16), block(64 * WV);
#define SMALL(NT) \
  hipLaunchKernelGGL((k_ff_small<T, NT, WV, DUAL>), grid, block, 0, st, w, w2, x, x_ld, n, M, K, \
                     out, out_ld, a, u)
  if (n <= 16)
    SMALL(1);
  else if (n <= 32)
    SMALL(2);
  else
    SMALL(4);
#undef SMALL
  return hipGetLastError();
}

// ---- launches ------------------------------------------------------------------------------

using FfBig = Cfg<2, 4, 64, 16, 0, 8>;    // 256 x 256 tiles, 8 waves
using FfMid = Cfg<1, 2, 64, 16, 0, 8>;    // 128 x 128 tiles, 2 waves

template <class C, int NP, bool DUAL, class Epi>
hipError_t launch_tiles(FfProb g, const Epi &epi, hipStream_t st) {
  constexpr int MT = DUAL ? C::BM / 2 : C::BM;
  const int64_t nb = (int64_t)((g.M + MT - 1) / MT) * ((g.N + C::BN - 1) / C::BN) * g.splits;
  hipLaunchKernelGGL((k_ff_gemm<C, NP, DUAL, Epi>), dim3((unsigned)nb), dim3(C::NTHR), 0, st, g, epi);
  return hipGetLastError();
}
int64_t big_tiles(int64_t M, int64_t N, bool dual) {
  return ((M + (dual ? 127 : 255)) / (dual ? 128 : 256)) * ((N + 255) / 256);
}
// Large tiles once they fill three quarters of the CUs, small ones below.
template <int NP, bool DUAL, class Epi>
hipError_t launch_product(const FfProb &g, const Epi &epi, hipStream_t st) {
  if (big_tiles(g.M, g.N, DUAL) >= 192) return launch_tiles<FfBig, NP, DUAL>(g, epi, st);
  return launch_tiles<FfMid, NP, DUAL>(g, epi, st);
}

// Parts of K of a product [M][N] with `steps` steps whose tiles do not fill the
// GPU: enough for two blocks per CU, each with at least 8 steps.
int split_parts(int64_t M, int64_t N, int64_t steps) {
  if (big_tiles(M, N, false) >= 192) return 1;
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  int64_t s = std::min<int64_t>({512 / std::max<int64_t>(tiles, 1), steps / 8, 16});
  if (s < 2) return 1;
  const int64_t per = (steps + s - 1) / s;
  return (int)((steps + per - 1) / per);  // no empty part
}

struct Area {
  char *base;
  size_t off = 0;
  void *take(int64_t bytes) {
    char *p = base ? base + off : nullptr;
    off += (size_t)round_up(bytes, 256);
    return p;
  }
  __bf16 *planes(int np, int64_t rows, int64_t ld) { return (__bf16 *)take(2 * np * rows * ld); }
};

// A matrix as an operand: planes `plane` elements apart, rows ld apart.
struct Opnd {
  const __bf16 *p;
  int64_t ld, plane;
};

bool in_place(const void *p, int64_t cols, int64_t ld) {
  return cols % kStep == 0 && ld % 8 == 0 && ((uintptr_t)p & 15) == 0;
}

// src's rows as an operand: in place, or laid out in buf.
template <typename T>
hipError_t rows_operand(const T *src, int64_t src_ld, int64_t R, int C, __bf16 *buf, Opnd &o,
                        hipStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (in_place(src, C, src_ld)) {
      o = Opnd{(const __bf16 *)src, src_ld, 0};
      return hipSuccess;
    }
  }
  const int64_t ld = kpad(C), plane = R * ld;
  o = Opnd{buf, ld, plane};
  hipLaunchKernelGGL(k_ff_rows<T>, dim3((unsigned)((R * (ld / 8) + 255) / 256)), dim3(256), 0, st, src,
                     src_ld, R, C, buf, ld, plane);
  return hipGetLastError();
}

// src's columns as an operand: out[c][r], rows ld apart, zero past R to a whole step.
template <typename T>
hipError_t trans_operand(const T *src, int64_t src_ld, int64_t src_plane, int planes, int64_t R, int C,
                         __bf16 *out, int64_t ld, int64_t plane, hipStream_t st) {
  hipLaunchKernelGGL(k_ff_trans<T>, dim3((unsigned)(kpad(R) / 64), (C + 63) / 64, planes), dim3(256),
                     0, st, src, src_ld, src_plane, R, C, out, ld, plane);
  return hipGetLastError();
}

#define TRYH(expr)                       \
  do {                                   \
    const hipError_t _e = (expr);        \
    if (_e != hipSuccess) return _e;     \
  } while (0)

struct FwdWs {
  __bf16 *x, *wg, *wu, *wd, *z;
  float *part;
  int parts;
  size_t bytes;
  FwdWs(void *base, int np, int d, int F, int64_t n) {
    Area w{(char *)base};
    const int64_t dp = kpad(d), Fp = kpad(F);
    const bool copy_d = np > 1 || d != dp, copy_f = np > 1 || F != Fp;
    x = w.planes(np, n, dp);
    wg = w.planes(np, copy_d ? F : 0, dp);
    wu = w.planes(np, copy_d ? F : 0, dp);
    wd = w.planes(np, copy_f ? d : 0, Fp);
    z = w.planes(np, n, Fp);
    parts = split_parts(d, n, (np == 1 ? 1 : 6) * (Fp / kStep));
    part = (float *)w.take(parts > 1 ? 4 * parts * n * round_up(d, 8) : 0);
    bytes = w.off;
  }
};

struct BwdWs {
  __bf16 *dy, *wdt, *dau, *z, *wgut, *xt, *dyt, *daut, *zt;
  float *part;
  int parts;
  size_t bytes;
  BwdWs(void *base, int np, int d, int F, int64_t n) {
    Area w{(char *)base};
    const int64_t dp = kpad(d), Fp = kpad(F), Tp = kpad(n);
    dy = w.planes(np, n, dp);
    wdt = w.planes(np, F, dp);
    dau = w.planes(np, n, 2 * Fp);
    z = w.planes(np, n, Fp);
    wgut = w.planes(np, d, 2 * Fp);
    xt = w.planes(np, d, Tp);
    dyt = w.planes(np, d, Tp);
    daut = w.planes(np, 2 * Fp, Tp);
    zt = w.planes(np, Fp, Tp);
    parts = split_parts(d, n, (np == 1 ? 1 : 6) * (2 * Fp / kStep));
    part = (float *)w.take(parts > 1 ? 4 * parts * n * round_up(d, 8) : 0);
    bytes = w.off;
  }
};

// out[n][m] = A rows times B rows with K split when the tiles are few.
template <typename T>
hipError_t product_out(FfProb g, int parts, float *part, T *out, int64_t out_ld, hipStream_t st) {
  constexpr int NP = planes_of<T>();
  if (parts == 1) {
    g.splits = 1;
    return launch_product<NP, false>(g, EpiOut<T>{out, nullptr, out_ld, g.M, g.N, 1 << 30}, st);
  }
  g.splits = parts;
  const int64_t ld = round_up(g.M, 8), stride = (int64_t)g.N * ld;
  TRYH((launch_product<NP, false>(g, EpiPart{part, stride, ld}, st)));
  hipLaunchKernelGGL(k_ff_join<T>, dim3((unsigned)((stride / 8 + 255) / 256)), dim3(256), 0, st, part,
                     parts, stride, ld, (int64_t)g.N, g.M, out, out_ld);
  return hipGetLastError();
}

}  // namespace
}  // namespace mfma

using namespace mfma;

size_t ff_forward_workspace(int elem, int d, int F, int64_t n) {
  if (n <= kSmallTokens) return (size_t)round_up(std::max<int64_t>(n, 1) * F * elem, 256);
  return FwdWs(nullptr, elem == 2 ? 1 : 3, d, F, n).bytes;
}
size_t ff_backward_workspace(int elem, int d, int F, int64_t n) {
  return std::max<size_t>(256, BwdWs(nullptr, elem == 2 ? 1 : 3, d, F, n).bytes);
}

template <typename T>
hipError_t ff_forward(const FfArgs &p, hipStream_t st) {
  const int d = p.d, F = p.F, n = (int)p.n;
  const T *wg = (const T *)p.w_gate, *wu = (const T *)p.w_up, *wd = (const T *)p.w_down;
  if (n <= kSmallTokens) {
    T *z = (T *)p.ws;
    TRYH((launch_small<T, 4, true>(wg, wu, (const T *)p.x, p.x_stride, n, F, d, z, F, (T *)p.a,
                                   (T *)p.u, st)));
    return launch_small<T, 16, false>(wd, nullptr, z, F, n, d, F, (T *)p.y, p.y_stride, nullptr,
                                      nullptr, st);
  }
  constexpr int NP = planes_of<T>();
  const FwdWs w(p.ws, NP, d, F, n);
  const int64_t Fp = kpad(F);
  Opnd x, g, u, o;
  TRYH(rows_operand((const T *)p.x, p.x_stride, n, d, w.x, x, st));
  TRYH(rows_operand(wg, (int64_t)d, F, d, w.wg, g, st));
  TRYH(rows_operand(wu, (int64_t)d, F, d, w.wu, u, st));
  TRYH(rows_operand(wd, (int64_t)F, d, F, w.wd, o, st));
  FfProb q{g.p, u.p, x.p, g.ld, x.ld, g.plane, x.plane, F, n, (int)(kpad(d) / kStep), 1};
  TRYH((launch_product<NP, true>(
      q, EpiZ<T>{w.z, n * Fp, F, (int)Fp, (T *)p.a, (T *)p.u}, st)));
  FfProb r{o.p, nullptr, w.z, o.ld, Fp, o.plane, n * Fp, d, n, (int)(Fp / kStep), 1};
  return product_out<T>(r, w.parts, w.part, (T *)p.y, p.y_stride, st);
}

template <typename T>
hipError_t ff_backward(const FfArgs &p, hipStream_t st) {
  const int d = p.d, F = p.F, n = (int)p.n;
  if (n == 0) {
    const int64_t halves = (int64_t)d * F * (int64_t)(sizeof(T) / 2);
    for (void *w : {p.dw_gate, p.dw_up, p.dw_down})
      hipLaunchKernelGGL(k_ff_zero, dim3((unsigned)std::min<int64_t>((halves + 255) / 256, 4096)),
                         dim3(256), 0, st, (uint16_t *)w, halves);
    return hipGetLastError();
  }
  constexpr int NP = planes_of<T>();
  const BwdWs w(p.ws, NP, d, F, n);
  const int64_t dp = kpad(d), Fp = kpad(F), Tp = kpad(n);
  Opnd dy;
  TRYH(rows_operand((const T *)p.dy, p.dy_stride, n, d, w.dy, dy, st));
  // W_d^T [F][dp]; W_g^T and W_u^T side by side [d][2 Fp]; x^T and dy^T [d][Tp]
  TRYH(trans_operand((const T *)p.w_down, (int64_t)F, 0, 1, d, F, w.wdt, dp, F * dp, st));
  TRYH(trans_operand((const T *)p.w_gate, (int64_t)d, 0, 1, F, d, w.wgut, 2 * Fp, d * 2 * Fp, st));
  TRYH(trans_operand((const T *)p.w_up, (int64_t)d, 0, 1, F, d, w.wgut + Fp, 2 * Fp, d * 2 * Fp, st));
  TRYH(trans_operand((const T *)p.x, p.x_stride, 0, 1, n, d, w.xt, Tp, d * Tp, st));
  TRYH(trans_operand((const T *)p.dy, p.dy_stride, 0, 1, n, d, w.dyt, Tp, d * Tp, st));
  // dz, and from it dA, dU and z
  FfProb q{w.wdt, nullptr, dy.p, dp, dy.ld, F * dp, dy.plane, F, n, (int)(dp / kStep), 1};
  TRYH((launch_product<NP, false>(q,
                                  EpiDz<T>{(const T *)p.a, (const T *)p.u, w.dau, w.z, n * 2 * Fp,
                                           n * Fp, F, (int)Fp},
                                  st)));
  TRYH(trans_operand(w.dau, 2 * Fp, n * 2 * Fp, NP, n, (int)(2 * Fp), w.daut, Tp, 2 * Fp * Tp, st));
  TRYH(trans_operand(w.z, Fp, n * Fp, NP, n, (int)Fp, w.zt, Tp, Fp * Tp, st));
  // dx = [dA dU] [W_g; W_u]
  FfProb r{w.wgut, nullptr, w.dau, 2 * Fp, 2 * Fp, d * 2 * Fp, n * 2 * Fp, d, n,
           (int)(2 * Fp / kStep), 1};
  TRYH(product_out<T>(r, w.parts, w.part, (T *)p.dx, p.dx_stride, st));
  // dW_g, dW_u (rows f < F of [dA dU]^T and from Fp on) and dW_d
  FfProb s{w.xt, nullptr, w.daut, Tp, Tp, d * Tp, 2 * Fp * Tp, d, (int)(2 * Fp), (int)(Tp / kStep), 1};
  TRYH((launch_product<NP, false>(
      s, EpiOut<T>{(T *)p.dw_gate, (T *)p.dw_up, (int64_t)d, d, F, (int)Fp}, st)));
  FfProb t{w.zt, nullptr, w.dyt, Tp, Tp, Fp * Tp, d * Tp, F, d, (int)(Tp / kStep), 1};
  return launch_product<NP, false>(
      t, EpiOut<T>{(T *)p.dw_down, nullptr, (int64_t)F, F, d, 1 << 30}, st);
}

template hipError_t ff_forward<float>(const FfArgs &, hipStream_t);
template hipError_t ff_forward<__bf16>(const FfArgs &, hipStream_t);
template hipError_t ff_backward<float>(const FfArgs &, hipStream_t);
template hipError_t ff_backward<__bf16>(const FfArgs &, hipStream_t);

}  // namespace ipttt
