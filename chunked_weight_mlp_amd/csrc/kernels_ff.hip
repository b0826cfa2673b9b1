// The gated feed-forward block y = (SiLU(x W_g) * (x W_u)) W_d, forward and
// backward.
//
// Three kernels, by the number of tokens: k_ff_small streams the weights past single
// tokens, k_ff_direct takes few tokens' operands as they lie, and with many tokens
// every product runs on one bf16 MFMA kernel (k_ff_gemm) over operands whose K values
// are contiguous and padded with zeros to whole steps of 64, with the output written
// contiguously along the first operand's rows:
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
//
// k_ff_gemm's large tiles keep the matrix cores busy for 58 to 68 % of the cycles, and LDS,
// which each MFMA's operands pass through, for as many: its reads take half of them and
// the copies into it a sixth, with no bank conflicts. Neither is full: one block fills a
// CU, so that one's barriers and epilogue pause both; and under this load the clock is
// 1.5 to 1.9 GHz of 2.4. 16384 tokens of 2560 x 9728 in bf16 take 1.9 ms, 1260 TFLOP/s,
// where a large library product reaches 1581. The epilogues' traffic comes on top: the dz
// product of 8192 tokens of 2048 x 8192 has 1.2 GB of it and takes 515 us, a quarter of
// them busy with MFMAs.
//
// In bf16 what goes from one product into the next (z, and dA and dU) is rounded to bf16,
// in every kernel alike, as the operand of an MFMA has to be: results are off by 2.35e-3
// where rounding the exact ones is 1.7e-3. Two bf16 planes of it would save that at
// twice the time of the products it enters; fp32 keeps it all, at six times the time.
#include <algorithm>
#include <type_traits>

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
// Independent products of one launch: problem p has the blocks start[p] ..
// start[p + 1], a multiple of 8, so that its tiles keep their XCDs.
template <class Epi, int G>
struct FfGroup {
  FfProb prob[G];
  Epi epi[G];
  int start[G + 1];
};

// Lane l holds rows 4 (l / 16) .. + 3 of a 16-row tile at column l % 16. Swapping
// lane groups of two tiles, one below the other, leaves each lane 8 consecutive
// rows of its column: 8 (l / 32) + 16 (l / 16 % 2) and on.
__device__ __forceinline__ void rows8(f32x4 a, f32x4 b, float (&v)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = a[r], y = b[r];
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x),
                                                    __builtin_bit_cast(unsigned, y), false, false);
    v[r] = __builtin_bit_cast(float, (unsigned)s[0]);
    v[4 + r] = __builtin_bit_cast(float, (unsigned)s[1]);
  }
}

template <class C, int NP, bool DUAL, class Epi, int G>
__global__ __launch_bounds__(C::NTHR) __attribute__((amdgpu_waves_per_eu(C::OCC))) void k_ff_gemm(
    FfGroup<Epi, G> grp) {
  static_assert(C::SMEM_ELEMS * 2 <= 160 * 1024, "LDS overflow");
  __shared__ __attribute__((aligned(1024))) __bf16 smem[C::SMEM_ELEMS];
  using M = typename C::M;
  static_assert(M::NG == 1 && C::MI % 4 == 0, "pairs of 16-row tiles");
  constexpr int MT = DUAL ? C::BM / 2 : C::BM;    // output rows per block
  constexpr int WT = DUAL ? C::WTM / 2 : C::WTM;  // and per wave
  constexpr int HI = DUAL ? C::MI / 2 : C::MI;
  int which = 0;
#pragma unroll
  for (int p = 1; p < G; ++p) which += (int)blockIdx.x >= grp.start[p];
  const FfProb g = grp.prob[which];
  const Epi epi = grp.epi[which];
  const int nm = (g.M + MT - 1) / MT, nn = (g.N + C::BN - 1) / C::BN;
  const int blocks = nm * nn * g.splits, bid = blockIdx.x - grp.start[which];
  if (bid >= blocks) return;
  const int id = xcd_remap(bid, blocks);
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
  const int first = sp * per;
  int pair = NP == 1 ? 0 : first / g.nk, ks = NP == 1 ? first : first % g.nk;
  kloop_dma_pl<C, 2, true, C::MI + C::NJ>(
      smem, la, lb, min(per, total - first), wave, acc,
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
  const int gq = lane >> 4;
  const auto write = [&](auto tag) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(tag)::value;
    constexpr int TURN = Epi::TURN, PT = 40;  // pitch of a turned tile's rows (32 values)
    static_assert(TURN * C::WM * C::WN * C::WTN * PT <= C::SMEM_ELEMS, "turned tiles fit the stages");
    // this wave's own part of the stages, which every wave has left
    __bf16 *const mine = smem + wave * (TURN * C::WTN * PT);
#pragma unroll
    for (int i = 0; i < HI; i += 2) {
      const int mw = m0 + wm * WT + C::FM * i, ml = 8 * (gq >> 1) + C::FM * (gq & 1), m = mw + ml;
      typename Epi::In in[C::NJ];
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {  // all loads of these tiles before their stores
        const int n = n0 + brow[j] + M::rcol(lane);
        in[j] = epi.template load<FULL>(m, FULL ? n : min(n, g.N - 1));
      }
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {
        const int n = n0 + brow[j] + M::rcol(lane);
        float v[8];
        rows8(acc[i][j], acc[i + 1][j], v);
        if constexpr (DUAL) {
          float w[8];
          rows8(acc[i + HI][j], acc[i + HI + 1][j], w);
          if (FULL || n < g.N) epi.template store<FULL>(m, n, v, w);
        } else if constexpr (TURN > 0) {
          bf16x8 t[TURN] = {};  // columns past the last are zero
          if (FULL || n < g.N) epi.template store<FULL>(m, n, v, in[j], sp, t);
#pragma unroll
          for (int k = 0; k < TURN; ++k)
            *(bf16x8 *)(mine + (k * C::WTN + C::FM * j + M::rcol(lane)) * PT + ml) = t[k];
        } else {
          if (FULL || n < g.N) epi.template store<FULL>(m, n, v, in[j], sp, nullptr);
        }
      }
      if constexpr (TURN > 0) {  // 32 rows x 64 columns, read back 8 columns of a row a lane
#pragma unroll
        for (int k = 0; k < TURN; ++k)
#pragma unroll
          for (int u = 0; u < C::WTN / 32; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const __bf16 *p = mine + (k * C::WTN + 32 * u + M::tr_row(lane)) * PT + C::FM * h +
                                M::tr_col(lane);
              const v4i16 lo = ds_read_tr16(p), hi = ds_read_tr16(p + 4 * PT);
              epi.template turned<FULL>(
                  k, mw + C::FM * h + (lane & 15), n0 + wn * C::WTN + 32 * u + 8 * gq,
                  __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
            }
      }
    }
  };
  // whole tiles store without predicates: each would make every later memory
  // operation of the wave wait (16384 tokens of the 4B-shaped forward 2.50 -> 2.02 ms)
  if (m0 + MT <= g.M && n0 + C::BN <= g.N && epi.whole())
    write(std::true_type());
  else
    write(std::false_type());
}

struct NoIn {};

// 8 outputs m .. m + 7 of a row of M
template <typename T, bool FULL = false>
__device__ __forceinline__ void store8(T *row, int m, int M, const float (&v)[8]) {
  if (FULL || m + 8 <= M) {
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

// 8 values m .. m + 7 of a row of M as they are stored, zero past it
template <typename T, bool FULL>
__device__ __forceinline__ Pack<T, 8> pack8(const T *row, int m, int M) {
  if (FULL || m + 8 <= M) return *(const Pack<T, 8> *)(row + m);
  Pack<T, 8> p;
#pragma unroll
  for (int e = 0; e < 8; ++e) p.v[e] = m + e < M ? row[m + e] : (T)0.f;
  return p;
}

// z = SiLU(a) u as the next product's operand (padded with zeros to Fp), and a,
// u themselves when saved: in fp32, so that the backward's only roundings are
// those of its products' operands (with a and u in bf16 its errors against 64 bits
// are 3.5e-3 instead of 2.3e-3, where rounding the exact result alone gives 1.7e-3).
template <typename T>
struct EpiZ {
  using In = NoIn;
  static constexpr int TURN = 0;
  __bf16 *z;
  int64_t plane;
  int F, Fp;
  float *a, *u;
  template <bool FULL>
  __device__ In load(int, int) const {
    return {};
  }
  __device__ bool whole() const { return true; }
  template <bool FULL>
  __device__ void store(int m, int n, const float (&av)[8], const float (&uv)[8]) const {
    if (!FULL && m >= Fp) return;
    float zv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      zv[e] = FULL || m + e < F ? av[e] * fast_sigmoid(av[e]) * uv[e] : 0.f;
    store8_planes<planes_of<T>()>(z + (int64_t)n * Fp + m, plane, zv);
    if (a) {
      store8<float, FULL>(a + (int64_t)n * F, m, F, av);
      store8<float, FULL>(u + (int64_t)n * F, m, F, uv);
    }
  }
};

// out[n][m], rows ld apart; columns n >= cut go to out2 (n - cut). With part: the
// sums of one part of K instead, fp32 [part][n][part_ld].
template <typename T>
struct EpiOut {
  using In = NoIn;
  static constexpr int TURN = 0;
  T *out, *out2;
  int64_t ld;
  int M, N, cut;  // N: rows of each output
  float *part;
  int64_t part_stride, part_ld;
  template <bool FULL>
  __device__ In load(int, int) const {
    return {};
  }
  // a tile may hold columns between the two outputs
  __device__ bool whole() const { return part || !out2 || cut == N; }
  template <bool FULL>
  __device__ void store(int m, int n, const float (&v)[8], In, int sp, bf16x8 *) const {
    if (part) {
      if (FULL || m < part_ld)
        blk::store_pack<float, 8>(part + sp * part_stride + (int64_t)n * part_ld + m, v);
      return;
    }
    const bool second = n >= cut;
    const int row = second ? n - cut : n;
    if (FULL || (m < M && row < N))
      store8<T, FULL>((second ? out2 : out) + (int64_t)row * ld, m, M, v);
  }
};

// dz -> dA = dz u SiLU'(a), dU = dz SiLU(a), z = SiLU(a) u as operands: dA and dU
// by token for dx, [n][2 Fp] padded with zeros to Fp; and all three by feature for
// the weights' gradients. In bf16 the block turns its tile in LDS for that (TURN
// results of store(), written by turned()); in fp32, three planes each, z is
// written by token too and k_ff_lay turns them afterwards.
template <typename T>
struct EpiDz {
  static constexpr int NP = planes_of<T>();
  static constexpr int TURN = NP == 1 ? 3 : 0;
  struct In {
    Pack<float, 8> a, u;
  };
  const float *a, *u;
  __bf16 *dau, *z;  // z: fp32 only
  int64_t dau_plane, z_plane;
  __bf16 *daut, *zt;  // bf16 only: [2 Fp][Tp], [Fp][Tp], zero past the last token
  int64_t Tp;
  int F, Fp;
  __device__ bool whole() const { return true; }
  template <bool FULL>
  __device__ In load(int m, int n) const {
    return {pack8<float, FULL>(a + (int64_t)n * F, m, F), pack8<float, FULL>(u + (int64_t)n * F, m, F)};
  }
  template <bool FULL>
  __device__ void store(int m, int n, const float (&v)[8], const In &in, int, bf16x8 *turn) const {
    if (!FULL && m >= Fp) return;
    float da[8], du[8], zv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool real = FULL || m + e < F;
      const float av = in.a.v[e], uv = in.u.v[e];
      const float s = fast_sigmoid(av), h = av * s;
      da[e] = real ? v[e] * uv * (s + h * (1.f - s)) : 0.f;
      du[e] = real ? v[e] * h : 0.f;
      zv[e] = real ? h * uv : 0.f;
    }
    __bf16 *row = dau + (int64_t)n * 2 * Fp + m;
    store8_planes<NP>(row, dau_plane, da);
    store8_planes<NP>(row + Fp, dau_plane, du);
    if constexpr (NP > 1) {
      store8_planes<NP>(z + (int64_t)n * Fp + m, z_plane, zv);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        turn[0][e] = (__bf16)da[e];
        turn[1][e] = (__bf16)du[e];
        turn[2][e] = (__bf16)zv[e];
      }
    }
  }
  // tokens n .. n + 7 of feature m of result k
  template <bool FULL>
  __device__ void turned(int k, int m, int n, bf16x8 v) const {
    if (FULL || (m < Fp && n < Tp))
      *(bf16x8 *)((k == 2 ? zt + (int64_t)m * Tp : daut + ((int64_t)k * Fp + m) * Tp) + n) = v;
  }
};

// out[n][m] = sum of the parts, in order, for up to G products (gridDim.y)
template <typename T>
struct FfJoin {
  EpiOut<T> e;
  int parts, n;  // n: columns of the product
};
template <typename T, int G>
struct FfJoins {
  FfJoin<T> j[G];
};
template <typename T, int G>
__global__ __launch_bounds__(256) void k_ff_join(FfJoins<T, G> js) {
  const FfJoin<T> j = js.j[blockIdx.y];
  const int64_t per = j.e.part_ld / 8, count = per * j.n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int n = (int)(i / per), m = 8 * (int)(i % per);
    float s[8] = {};
    for (int p = 0; p < j.parts; ++p) {
      float v[8];
      blk::load_pack<float, 8>(j.e.part + p * j.e.part_stride + (int64_t)n * j.e.part_ld + m, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    const bool second = n >= j.e.cut;
    const int row = second ? n - j.e.cut : n;
    if (row < j.e.N) store8<T>((second ? j.e.out2 : j.e.out) + (int64_t)row * j.e.ld, m, j.e.M, s);
  }
}

// ---- operand layouts -------------------------------------------------------------------

// One operand to lay out from src [R][C] (rows src_ld apart): its rows, planes
// [R][ld] with zeros from column C on, or its columns, planes [C][ld] with out[c][r]
// = src[r][c] and zeros from r = R to the next multiple of 64. An fp32 source is
// split into its planes; a bf16 source may have `planes` planes of its own.
struct FfLay {
  const void *src;
  int64_t src_ld, src_plane, R, ld, plane;
  __bf16 *out;
  int C, planes, cols;  // cols: lay out columns
  int start;            // first block
};
constexpr int kLays = 6;
struct FfLays {
  FfLay lay[kLays];
  int count;
};

// A block moves one 64 x 64 tile, columns through LDS (pitch 65: its reads and
// writes touch 64 different banks). Bound by HBM.
template <typename T>
__global__ __launch_bounds__(256) void k_ff_lay(FfLays ls) {
  __shared__ float tile[64][65];
  constexpr int NP = planes_of<T>();
  int which = 0;
#pragma unroll
  for (int k = 1; k < kLays; ++k) which += k < ls.count && (int)blockIdx.x >= ls.lay[k].start;
  const FfLay l = ls.lay[which];
  int id = blockIdx.x - l.start;
  // columns of tiles: of the source; a row operand also covers its padding
  const int across = l.cols ? (l.C + 63) / 64 : (int)(l.ld / 64);
  const int per = across * (int)((l.R + 63) / 64), p = id / per;
  id %= per;
  const int64_t r0 = (int64_t)(id / across) * 64;
  const int c0 = (id % across) * 64, tid = threadIdx.x;
  const T *src = (const T *)l.src + p * l.src_plane;
  __bf16 *out = l.out + p * l.plane;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (tid >> 3) + 32 * k, c = 8 * (tid & 7);
    float v[8] = {};
    if (r0 + r < l.R && c0 + c < l.C) load8<T>(src + (r0 + r) * l.src_ld, c0 + c, l.C, v);
    if (!l.cols) {
      if (r0 + r < l.R) store8_planes<NP>(out + (r0 + r) * l.ld + c0 + c, l.plane, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[r][c + e] = v[e];
    }
  }
  if (!l.cols) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = (tid >> 3) + 32 * k, r = 8 * (tid & 7);
    if (c0 + c < l.C) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[r + e][c];
      store8_planes<NP>(out + (int64_t)(c0 + c) * l.ld + r0 + r, l.plane, v);
    }
  }
}

__global__ __launch_bounds__(256) void k_ff_zero(uint16_t *__restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0;
}

// ---- single tokens ----------------------------------------------------------------------
// For up to 32 tokens every weight is read once and little else moves, so the weights
// go straight from memory into MFMA operands: 16 bytes of a weight row per lane
// are 8 bf16 values of one 16x16x32 MFMA, or 4 fp32 values of four 16x16x4 ones
// (any assignment of K values to lanes gives the same sum as long as both operands
// share it). The MFMA's 16 operand rows would be 16 weight rows, whose 16-byte
// pieces lie a row apart: 64 cache lines a load, and the loads' address work, not
// memory, sets the time (n = 16: 46 us so, 27 as here, 2048 x 8192 in bf16). So an
// operand row is a weight row i and one of KF neighbouring pieces of K, s: rows i KF + s,
// and columns j KF + s
// of the other operand for token j. Lanes next to each other then read pieces
// next to each other; of the products, those whose two s agree are summed.
// A block owns RG groups of 16 / KF weight rows (of both W_g and W_u in the first
// product), so that the tokens' operands serve several weight rows; its WV waves
// take interleaved steps of K and meet in LDS. NT: groups of 16 / KF tokens.

typedef unsigned U32x4 __attribute__((ext_vector_type(4)));
template <typename T>
struct Quad;  // 16 bytes of one operand row
template <>
struct Quad<__bf16> {
  static constexpr int E = 8;
  bf16x8 v;
  __device__ __forceinline__ void set(int e, float x) { v[e] = (__bf16)x; }
  __device__ __forceinline__ void keep(int e, bool k) {  // zero a value unless k
    U32x4 w = __builtin_bit_cast(U32x4, v);
    w[e >> 1] &= k ? 0xffffffff : e & 1 ? 0xffff : 0xffff0000;
    v = __builtin_bit_cast(bf16x8, w);
  }
  __device__ static __forceinline__ f32x4 mma(const Quad &a, const Quad &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
  }
};
template <>
struct Quad<float> {
  static constexpr int E = 4;
  f32x4 v;
  __device__ __forceinline__ void set(int e, float x) { v[e] = x; }
  __device__ __forceinline__ void keep(int e, bool k) { v[e] = k ? v[e] : 0.f; }
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
// the same with zeros at and past `end`
template <typename T>
__device__ __forceinline__ Quad<T> quad_end(const T *row, int k, int end) {
  if (k + Quad<T>::E <= end) return quad_at<T>(row + k);
  Quad<T> q;
#pragma unroll
  for (int e = 0; e < Quad<T>::E; ++e) q.set(e, k + e < end ? (float)row[k + e] : 0.f);
  return q;
}

// DUAL: out = SiLU(W x) (W2 x), with W x and W2 x saved to a, u when given.
// Otherwise out = W x. W [M][K] dense, x rows x_ld apart, out rows out_ld apart.
template <typename T, int NT, int RG, int WV, bool DUAL>
__global__ __launch_bounds__(64 * WV) void k_ff_small(const T *__restrict__ w,
                                                      const T *__restrict__ w2,
                                                      const T *__restrict__ x, int64_t x_ld, int n,
                                                      int M, int K, T *__restrict__ out,
                                                      int64_t out_ld, float *__restrict__ a,
                                                      float *__restrict__ u) {
  constexpr int KF = 4, RB = 16 / KF;  // weight rows, tokens of a group
  constexpr int D = DUAL ? 2 : 1;
  constexpr int E = Quad<T>::E, S = 4 * KF * E;  // K values of a lane, of a step
  // steps whose loads go together: about 8 KB of weights a wave, fewer where the
  // tokens' operands fill the registers
  constexpr int U = NT >= 8 || RG * D >= 8 ? 1 : RG * D >= 4 ? 2 : 4;
  constexpr int P = U * S;
  __shared__ float sum[WV][D][RG * NT][RB * RB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = RG * RB * blockIdx.x;
  const int r = lane & 15, kl = E * (r % KF + KF * (lane >> 4));
  const T *wrow[D][RG], *xrow[NT];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    const int64_t at = (int64_t)min(m0 + RB * g + r / KF, M - 1) * K;
    wrow[0][g] = w + at;
    if constexpr (DUAL) wrow[1][g] = w2 + at;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = x + (int64_t)min(RB * t + r / KF, n - 1) * x_ld;
  f32x4 acc[D][RG][NT] = {};
  Quad<T> cur[U][D][RG], next[U][D][RG];
  const auto load = [&](Quad<T> (&q)[U][D][RG], int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int i = 0; i < D; ++i)
#pragma unroll
        for (int g = 0; g < RG; ++g) q[s][i][g] = quad_at<T>(wrow[i][g] + kl + k0 + S * s);
  };
  int k0 = wave * P;
  if (k0 + P <= K) load(cur, k0);
  for (; k0 + P <= K; k0 += WV * P) {
    // this piece's tokens, then the next piece's weights: loads return in order,
    // so the MFMAs wait for the tokens (from L2) and not for memory
    Quad<T> xv[U][NT];
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) xv[s][t] = quad_at<T>(xrow[t] + kl + k0 + S * s);
    const bool more = k0 + WV * P + P <= K;
    if (more) load(next, k0 + WV * P);
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < D; ++i)
#pragma unroll
          for (int g = 0; g < RG; ++g)
            acc[i][g][t] = Quad<T>::mma(cur[s][i][g], xv[s][t], acc[i][g][t]);
    if (more) {
#pragma unroll
      for (int s = 0; s < U; ++s)
#pragma unroll
        for (int i = 0; i < D; ++i)
#pragma unroll
          for (int g = 0; g < RG; ++g) cur[s][i][g] = next[s][i][g];
    }
  }
  // the rows' last, partial piece, by the wave whose turn it is
  const int whole = K / P * P;
  if (wave == whole / P % WV)
    for (int k = whole; k < K; k += S) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Quad<T> xe = quad_end<T>(xrow[t], kl + k, K);
#pragma unroll
        for (int i = 0; i < D; ++i)
#pragma unroll
          for (int g = 0; g < RG; ++g)
            acc[i][g][t] = Quad<T>::mma(quad_end<T>(wrow[i][g], kl + k, K), xe, acc[i][g][t]);
      }
    }
  // Lane l holds operand rows 4 (l / 16) + q, q = 0 .. 3, of column l % 16: its
  // column's piece s = l % KF matches q = s, s + KF, ..: weight rows
  // (4 / KF) (l / 16) + q / KF. The KF lanes of a token then add up.
  const int s = r % KF, tok = r / KF;
#pragma unroll
  for (int i = 0; i < D; ++i)
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 4 / KF; ++h) {
          float v = 0.f;
#pragma unroll
          for (int q = 0; q < KF; ++q) {
            const float p = acc[i][g][t][h * KF + q];
            v = q == s ? p : v;
          }
#pragma unroll
          for (int q = 1; q < KF; q *= 2) v += __shfl_xor(v, q, 64);
          if (s == 0) sum[wave][i][g * NT + t][((4 / KF) * (lane >> 4) + h) * RB + tok] = v;
        }
  __syncthreads();
  for (int o = tid; o < RG * NT * RB * RB; o += 64 * WV) {
    // neighbouring threads take neighbouring weight rows of one token
    const int row = o % (RG * RB), col = o / (RG * RB), g = row / RB, t = col / RB;
    const int m = m0 + row;
    float v[D] = {};
#pragma unroll
    for (int q = 0; q < WV; ++q)
#pragma unroll
      for (int i = 0; i < D; ++i) v[i] += sum[q][i][g * NT + t][row % RB * RB + col % RB];
    if (m < M && col < n) {
      if constexpr (DUAL) {
        if (a) {
          a[(int64_t)col * M + m] = v[0];
          u[(int64_t)col * M + m] = v[1];
        }
        out[col * out_ld + m] = (T)(v[0] * fast_sigmoid(v[0]) * v[1]);
      } else {
        out[col * out_ld + m] = (T)v[0];
      }
    }
  }
}

// Row groups of a block of four waves: two where that makes two blocks a CU, else
// one (2560 x 9728, one token: 29 us with 2 groups in the first product and 1 in
// the second, 31 with 4 and 1, 32 with 4 and 2; with eight waves 34).
template <typename T, bool DUAL>
hipError_t launch_small(const T *w, const T *w2, const T *x, int64_t x_ld, int n, int M, int K, T *out,
                        int64_t out_ld, float *a, float *u, hipStream_t st) {
  constexpr int WV = 4;
#define SMALL(NT, RG)                                                                     \
  hipLaunchKernelGGL((k_ff_small<T, NT, RG, WV, DUAL>), dim3((M + RG * 4 - 1) / (RG * 4)), \
                     dim3(64 * WV), 0, st, w, w2, x, x_ld, n, M, K, out, out_ld, a, u)
#define SMALL_TOKENS(RG) \
  if (n <= 4)            \
    SMALL(1, RG);        \
  else if (n <= 8)       \
    SMALL(2, RG);        \
  else if (n <= 16)      \
    SMALL(4, RG);        \
  else                   \
    SMALL(8, RG)
  if (M >= 16 * 2 * 256) {
    SMALL_TOKENS(2);
  } else {
    SMALL_TOKENS(1);
  }
#undef SMALL_TOKENS
#undef SMALL
  return hipGetLastError();
}

// ---- few tokens ---------------------------------------------------------------------------
// With few tokens the operands' layout passes and the 64-wide padded steps cost more
// than the products. Here a product takes its operands as they lie, of either
// orientation and any type, stride and width, turns them on their way into LDS and
// uses the MFMA of their own type (fp32: no planes), in 64 x 64 tiles of which many
// fit a small matrix (or 64 x 32, direct_with). 128 bytes of K a step, two steps' loads in
// flight in registers while a third is in LDS (four steps': 2048 x 8192 bf16, 64 tokens 90
// us against 76). Bound by the weights' traffic with the fewest tokens (one token of 2048
// x 8192, backward: fp32 149 us, 2.7 TB/s, bf16 72), else by the fp32 MFMA (512 tokens
// forward 441 us, 117 of 154 TFLOP/s) or, in bf16, by its small tiles' LDS reads.

// One operand: element (row, k) is p[row ld + k], or, turned, p[k ld + row]; the second
// of two runs of K continues in p2.
template <typename T>
struct FfSide {
  const T *p, *p2;
  int64_t ld;
};
template <typename T>
struct FfDirect {  // out(m, n) = sum over the runs and k of a(m, k) b(n, k)
  FfSide<T> a, b;
  bool b_turned;
  int M, N, K, runs;
  int splits;
};
template <typename T, class Epi, int G>
struct FfDirects {
  FfDirect<T> prob[G];
  Epi epi[G];
  int start[G + 1];
};
constexpr int kDTile = 64;
template <typename T>
constexpr int kDStep = 128 / sizeof(T);  // K values of a step

// A side's 64 rows x 128 bytes of K in LDS: the 16-byte piece q of row r is stored at
// piece q ^ r ^ r / 8, so that neither 16 rows' reads of a piece nor the turned
// operand's writes, 8 rows apart, meet in a bank.
__device__ __forceinline__ int dslot(int r, int q) { return r * 8 + (q ^ ((r ^ (r >> 3)) & 7)); }

// A thread's part of a step of one side: two pieces, of E values of K of a row each, or
// turned, of E rows at a value of K each. No load branches or reaches over its row: a
// piece at the end moves back. Rows are then stored where they belong (a neighbour's,
// with the same values, once more); of K, the values the piece before holds are zeroed,
// on both sides of the product. A pair: 32 rows of p, then the same 32 of p2.
template <typename T, bool turned, bool pair, int ROWS>
struct DirectLoader {
  static constexpr int E = Quad<T>::E, S = kDStep<T>;
  static_assert(ROWS == 64 || (ROWS == 32 && !turned), "two pieces a thread, or one straight one");
  // pieces of a thread, and turned ones' distance in the step (bf16 takes pairs of values)
  static constexpr int NQ = ROWS / 32, KI = E == 8 ? 1 : 16;
  const T *p, *p2;
  int64_t at[NQ];  // of its rows
  int64_t ks;      // distance between values of K
  int row[NQ];     // in the tile
  int pos;         // its place in the step (the first of turned values)
  // the place in the step of piece i
  __device__ __forceinline__ int place(int i) const { return turned ? pos + KI * i : pos; }
  __device__ __forceinline__ DirectLoader(const FfSide<T> &s, int r0, int R) : p(s.p), p2(s.p2) {
    constexpr int GR = ROWS / E;  // groups of E rows
    const int tid = threadIdx.x;
    ks = turned ? s.ld : 1;
    pos = turned ? (E == 8 ? 2 : 1) * (tid / GR) : E * (tid & 7);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int r = turned ? min(r0 + E * (tid & (GR - 1)), R - E)
                           : min(r0 + (tid >> 3) + (pair ? 0 : 32 * i), R - 1);
      at[i] = turned ? r : r * s.ld;
      // (rows before the tile go to its end, past the matrix's last)
      row[i] = turned ? r - r0 : (tid >> 3) + 32 * i;
    }
  }
  // where piece i's value (turned) or first value of K is, of a step from k0 on
  __device__ __forceinline__ int first_k(int i, int k0, int K) const {
    const int p = place(i), in = p & (E - 1);
    return min(min(k0 + p - in, max(K - E, 0)) + in, K - 1);
  }
  __device__ __forceinline__ void load(Quad<T> (&q)[2], bool second, int k0, int K) const {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      q[i] = quad_at<T>(((pair ? i == 1 : second) ? p2 : p) + at[i] + first_k(i, k0, K) * ks);
  }
  __device__ __forceinline__ void store(Quad<T> (&q)[2], Quad<T> *lds, int k0, int K) const {
    if (k0 + S > K) {  // the last step
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int p = place(i), in = p & (E - 1), from = k0 + p - in, at0 = min(from, max(K - E, 0));
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int k = at0 + (turned ? in : e);
          q[i].keep(e, k >= from && k < K);
        }
      }
    }
    if constexpr (!turned) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) lds[dslot(row[i], pos / E)] = q[i];
    } else if constexpr (E == 8) {
      const U32x4 lo = __builtin_bit_cast(U32x4, q[0]), hi = __builtin_bit_cast(U32x4, q[1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // the e-th halves of both
        const unsigned h = hi[e >> 1], l = lo[e >> 1];
        ((unsigned *)(lds + dslot((row[0] + e) & (ROWS - 1), pos >> 3)))[(pos & 7) >> 1] =
            __builtin_amdgcn_perm(h, l, e & 1 ? 0x07060302 : 0x05040100);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ((float *)(lds + dslot((row[i] + e) & (ROWS - 1), place(i) >> 2)))[pos & 3] = q[i].v[e];
    }
  }
};

// TURNED: a is (b where its problem says so). DUAL: two products of 32 rows each, of a.p
// and a.p2, for one epilogue. TN: columns of a tile.
template <typename T, bool TURNED, bool DUAL, int TN, class Epi, int G>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void k_ff_direct(
    FfDirects<T, Epi, G> grp) {
  constexpr int S = kDStep<T>, AHEAD = 2, MT = DUAL ? kDTile / 2 : kDTile, NJ = TN / 32;
  __shared__ Quad<T> lds[2][2][kDTile * 8];
  int which = 0;
#pragma unroll
  for (int p = 1; p < G; ++p) which += (int)blockIdx.x >= grp.start[p];
  const FfDirect<T> g = grp.prob[which];
  const Epi epi = grp.epi[which];
  const int nm = (g.M + MT - 1) / MT, nn = (g.N + TN - 1) / TN;
  const int blocks = nm * nn * g.splits, bid = blockIdx.x - grp.start[which];
  if (bid >= blocks) return;
  const int id = xcd_remap(bid, blocks), sp = id / (nm * nn);
  int tm, tn;
  tile_of<8>(id % (nm * nn), nm, nn, tm, tn);
  const int m0 = tm * MT, n0 = tn * TN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = TN / 2 * (wave & 1), gq = lane >> 4, lr = lane & 15;
  const int wm = (DUAL ? 16 : 32) * (wave >> 1), wi = DUAL ? 32 : 16;  // its rows: 16 each from wm, wm + wi
  const int per_run = (g.K + S - 1) / S, steps = g.runs * per_run;
  const int per = (steps + g.splits - 1) / g.splits, first = sp * per, count = min(per, steps - first);
  f32x4 acc[2][NJ] = {};
  const auto run = [&](auto tag) __attribute__((always_inline)) {
    const DirectLoader<T, TURNED, DUAL, kDTile> la(g.a, m0, g.M);
    const DirectLoader<T, decltype(tag)::value, false, TN> lb(g.b, n0, g.N);
    Quad<T> qa[AHEAD][2], qb[AHEAD][2];
    const auto fetch = [&](int s, int j) __attribute__((always_inline)) {
      const bool second = first + s >= per_run;
      const int k0 = S * (first + s - (second ? per_run : 0));
      la.load(qa[j], second, k0, g.K);
      lb.load(qb[j], second, k0, g.K);
    };
    // Step s, whose loads are in set j. Of the two stages in LDS it fills the one whose
    // reads, two steps ago, every wave has behind it at the last step's barrier.
    const auto step = [&](int s, int j, bool more) __attribute__((always_inline)) {
      Quad<T> *const as = lds[j][0], *const bs = lds[j][1];
      const int k0 = S * (first + s - (first + s >= per_run ? per_run : 0));
      la.store(qa[j], as, k0, g.K);
      lb.store(qb[j], bs, k0, g.K);
      if (more) fetch(s + AHEAD, j);
      lds_barrier();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        Quad<T> a[2], b[NJ];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = as[dslot(wm + wi * i + lr, 4 * u + gq)];
#pragma unroll
        for (int k = 0; k < NJ; ++k) b[k] = bs[dslot(wn + 16 * k + lr, 4 * u + gq)];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < NJ; ++k) acc[i][k] = Quad<T>::mma(a[i], b[k], acc[i][k]);
      }
    };
    fetch(0, 0);
    fetch(min(1, count - 1), 1);
    int s = 0;
    for (; s + 2 * AHEAD <= count; s += AHEAD) {  // straight: waits count the loads in flight
      step(s, 0, true);
      step(s + 1, 1, true);
    }
    step(s, 0, s + 2 < count);
    if (s + 1 < count) step(s + 1, 1, false);
    if (s + 2 < count) step(s + 2, 0, false);
  };
  if constexpr (G > 1) {
    if (g.b_turned)
      run(std::true_type());
    else
      run(std::false_type());
  } else {
    run(std::false_type());
  }
  if constexpr (DUAL) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + wn + 16 * j + lr;
      if (n < g.N) epi.store(m0 + wm + 4 * gq, n, acc[0][j], acc[1][j]);
    }
  } else {
    const int m = m0 + wm + 8 * (gq >> 1) + 16 * (gq & 1);
    typename Epi::In in[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      in[j] = epi.template load<false>(m, min(n0 + wn + 16 * j + lr, g.N - 1));
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + wn + 16 * j + lr;
      float v[8];
      rows8(acc[0][j], acc[1][j], v);
      if (n < g.N) epi.template store<false>(m, n, v, in[j], sp, nullptr);
    }
  }
}

// z = SiLU(a) u, and a and u when saved, for 4 features m .. m + 3 of token n
template <typename T>
struct EpiZDirect {
  T *z;
  float *a, *u;
  int F;
  template <typename O>
  __device__ void put(O *row, int m, f32x4 v) const {
    if (m + 4 <= F) {
      const float w[4] = {v[0], v[1], v[2], v[3]};
      blk::store_pack<O, 4>(row + m, w);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < F) row[m + e] = (O)v[e];
    }
  }
  __device__ void store(int m, int n, f32x4 av, f32x4 uv) const {
    const int64_t row = (int64_t)n * F;
    f32x4 zv;
#pragma unroll
    for (int e = 0; e < 4; ++e) zv[e] = av[e] * fast_sigmoid(av[e]) * uv[e];
    put(z + row, m, zv);
    if (a) {
      put(a + row, m, av);
      put(u + row, m, uv);
    }
  }
};

// dz -> dA, dU and z by token, in T, as the products after it take them.
template <typename T>
struct EpiDzDirect {
  struct In {
    Pack<float, 8> a, u;
  };
  const float *a, *u;
  T *da, *du, *z;
  int F;
  template <bool FULL>
  __device__ In load(int m, int n) const {
    return {pack8<float, FULL>(a + (int64_t)n * F, m, F), pack8<float, FULL>(u + (int64_t)n * F, m, F)};
  }
  template <bool FULL>
  __device__ void store(int m, int n, const float (&v)[8], const In &in, int, bf16x8 *) const {
    float av[8], uv[8], zv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = in.a.v[e], y = in.u.v[e];
      const float s = fast_sigmoid(x), h = x * s;
      av[e] = v[e] * y * (s + h * (1.f - s));
      uv[e] = v[e] * h;
      zv[e] = h * y;
    }
    const int64_t row = (int64_t)n * F;
    store8<T, FULL>(da + row, m, F, av);
    store8<T, FULL>(du + row, m, F, uv);
    store8<T, FULL>(z + row, m, F, zv);
  }
};

// ---- launches ------------------------------------------------------------------------------

constexpr int kCUs = 256;
using FfBig = Cfg<2, 4, 64, 16, 0, 8>;  // 256 x 256 tiles, 8 waves, one block per CU
using FfMid = Cfg<2, 2, 64, 16, 0, 8, 1, 8, 64, 0, 64>;  // 128 x 128 tiles, 4 waves, two blocks per CU

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t tiles_of(const FfProb &g, int edge, bool dual) {
  return ceil_div(g.M, dual ? edge / 2 : edge) * ceil_div(g.N, edge);
}

template <class C, int NP, bool DUAL, class Epi, int G>
hipError_t launch_tiles(FfGroup<Epi, G> grp, hipStream_t st) {
  int at = 0;
  for (int p = 0; p < G; ++p) {
    grp.start[p] = at;
    at += (int)round_up(tiles_of(grp.prob[p], C::BM, DUAL) * grp.prob[p].splits, 8);
  }
  grp.start[G] = at;
  hipLaunchKernelGGL((k_ff_gemm<C, NP, DUAL, Epi, G>), dim3((unsigned)at), dim3(C::NTHR), 0, st,
                     grp);
  return hipGetLastError();
}

// 256 x 256 tiles once they fill three quarters of the CUs, 128 x 128 ones below
// (4B-shaped, 1024 tokens forward: 187 us so, 192 with small tiles up to the point
// where a model of whole rounds favours large ones; with four stages of copies
// in flight instead of two, hence one small block per CU, 267).
template <class Epi, int G>
bool use_big(const FfGroup<Epi, G> &grp, bool dual) {
  int64_t tiles = 0;
  for (int p = 0; p < G; ++p) tiles += tiles_of(grp.prob[p], 256, dual);
  return tiles >= kCUs * 3 / 4;
}

// Parts of K for a product whose small tiles do not fill the GPU: two blocks per
// CU in all, each with at least 8 steps (below that the copies' latency is most
// of a block's time).
int parts_of(const FfProb &g, int64_t steps) {
  const int64_t tiles = tiles_of(g, 128, false);
  const int64_t s = std::min<int64_t>({2 * kCUs / std::max<int64_t>(tiles, 1), steps / 8, 32});
  if (s < 2) return 1;
  return (int)ceil_div(steps, ceil_div(steps, s));  // no empty part
}
int64_t part_bytes(const FfProb &g, int parts) {
  return parts > 1 ? 4 * (int64_t)parts * g.N * round_up(g.M, 8) : 0;
}

// Adds up the parts of the products that were split.
template <typename T, int G, class Group>
hipError_t joins(const Group &grp, hipStream_t st) {
  FfJoins<T, G> js{};
  int used = 0;
  int64_t most = 0;
  for (int p = 0; p < G; ++p)
    if (grp.prob[p].splits > 1) {
      js.j[used++] = {grp.epi[p], grp.prob[p].splits, grp.prob[p].N};
      most = std::max(most, grp.epi[p].part_stride / 8);
    }
  if (used == 0) return hipSuccess;
  hipLaunchKernelGGL((k_ff_join<T, G>), dim3((unsigned)std::min<int64_t>(ceil_div(most, 256), 2048), used),
                     dim3(256), 0, st, js);
  return hipGetLastError();
}

// Up to G independent products written out, each split over K by its `splits`
// (its partial sums then in epi.part), and the joins.
template <typename T, int G>
hipError_t products_out(FfGroup<EpiOut<T>, G> grp, hipStream_t st) {
  constexpr int NP = planes_of<T>();
  bool split = false;
  for (int p = 0; p < G; ++p) {
    EpiOut<T> &e = grp.epi[p];
    e.part_ld = round_up(grp.prob[p].M, 8);
    e.part_stride = grp.prob[p].N * e.part_ld;
    if (grp.prob[p].splits == 1) e.part = nullptr;
    split = split || e.part;
  }
  if (!split && use_big(grp, false)) return launch_tiles<FfBig, NP, false>(grp, st);
  const hipError_t err = launch_tiles<FfMid, NP, false>(grp, st);
  return err != hipSuccess || !split ? err : joins<T, G>(grp, st);
}

// One product with an epilogue of its own.
template <int NP, bool DUAL, class Epi>
hipError_t product_with(const FfProb &g, const Epi &epi, hipStream_t st) {
  const FfGroup<Epi, 1> grp{{g}, {epi}, {}};
  if (use_big(grp, DUAL)) return launch_tiles<FfBig, NP, DUAL>(grp, st);
  return launch_tiles<FfMid, NP, DUAL>(grp, st);
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

// Collects the operands to lay out and launches them together.
template <typename T>
struct Layouts {
  FfLays ls{};
  int64_t blocks = 0;
  void add(const void *src, int64_t src_ld, int64_t src_plane, int planes, int64_t R, int C,
           __bf16 *out, int64_t ld, int64_t plane, bool cols) {
    FfLay &l = ls.lay[ls.count++];
    l = FfLay{src, src_ld, src_plane, R, ld, plane, out, C, planes, cols, (int)blocks};
    blocks += planes * ceil_div(R, 64) * (cols ? ceil_div(C, 64) : ld / 64);
  }
  // the rows of src: used in place if they are an operand already
  Opnd rows(const T *src, int64_t src_ld, int64_t R, int C, __bf16 *buf) {
    if (sizeof(T) == 2 && C % kStep == 0 && src_ld % 8 == 0 && ((uintptr_t)src & 15) == 0)
      return {(const __bf16 *)src, src_ld, 0};
    const int64_t ld = kpad(C);
    add(src, src_ld, 0, 1, R, C, buf, ld, R * ld, false);
    return {buf, ld, R * ld};
  }
  void cols(const T *src, int64_t src_ld, int64_t R, int C, __bf16 *out, int64_t ld, int64_t plane) {
    add(src, src_ld, 0, 1, R, C, out, ld, plane, true);
  }
  hipError_t launch(hipStream_t st) const {
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(k_ff_lay<T>, dim3((unsigned)blocks), dim3(256), 0, st, ls);
    return hipGetLastError();
  }
};

#define TRYH(expr)                       \
  do {                                   \
    const hipError_t _e = (expr);        \
    if (_e != hipSuccess) return _e;     \
  } while (0)

struct FwdPlan {
  __bf16 *x, *wg, *wu, *wd, *z;
  float *part;
  FfProb down;  // sizes and parts; operands are set by the call
  size_t bytes;
  FwdPlan(void *base, int np, int d, int F, int64_t n) {
    Area w{(char *)base};
    const int64_t dp = kpad(d), Fp = kpad(F);
    const bool copy_d = np > 1 || d != dp, copy_f = np > 1 || F != Fp;
    x = w.planes(np, n, dp);
    wg = w.planes(np, copy_d ? F : 0, dp);
    wu = w.planes(np, copy_d ? F : 0, dp);
    wd = w.planes(np, copy_f ? d : 0, Fp);
    z = w.planes(np, n, Fp);
    down = FfProb{};
    down.M = d;
    down.N = (int)n;
    down.nk = (int)(Fp / kStep);
    down.splits = parts_of(down, (np == 1 ? 1 : 6) * down.nk);
    part = (float *)w.take(part_bytes(down, down.splits));
    bytes = w.off;
  }
};

struct BwdPlan {
  __bf16 *dy, *wdt, *dau, *z, *wgut, *xt, *dyt, *daut, *zt;
  FfProb out[3];  // dx, [dW_g dW_u], dW_d: sizes and parts
  float *part[3];
  size_t bytes;
  BwdPlan(void *base, int np, int d, int F, int64_t n) {
    Area w{(char *)base};
    const int64_t dp = kpad(d), Fp = kpad(F), Tp = kpad(n);
    dy = w.planes(np, n, dp);
    wdt = w.planes(np, F, dp);
    dau = w.planes(np, n, 2 * Fp);
    z = w.planes(np, np > 1 ? n : 0, Fp);
    wgut = w.planes(np, d, 2 * Fp);
    xt = w.planes(np, d, Tp);
    dyt = w.planes(np, d, Tp);
    daut = w.planes(np, 2 * Fp, Tp);
    zt = w.planes(np, Fp, Tp);
    const int64_t M[3] = {d, d, F}, N[3] = {n, 2 * Fp, d}, K[3] = {2 * Fp, Tp, Tp};
    for (int p = 0; p < 3; ++p) {
      out[p] = FfProb{};
      out[p].M = (int)M[p];
      out[p].N = (int)N[p];
      out[p].nk = (int)(K[p] / kStep);
      out[p].splits = parts_of(out[p], (np == 1 ? 1 : 6) * out[p].nk);
      part[p] = (float *)w.take(part_bytes(out[p], out[p].splits));
    }
    bytes = w.off;
  }
};

// Whether a forward streams its weights (k_ff_small). Measured against the operands as
// they lie below (us, streaming / that), fp32: 512 x 2048 at 8 tokens 13 / 22, at 32 20 / 22;
// 1024 x 4096 at 16 26 / 36, at 24 50 / 36; 2048 x 8192 at 8 53 / 61, at 16 82 / 61. bf16:
// 1024 x 4096 at 32 17 / 20; 2048 x 8192 at 8 21 / 27, at 16 27 / 27, at 24 42 / 27; 1999 x
// 3001 at 8 17 / 27, at 16 33 / 27.
bool single_tokens(int elem, int d, int F, int64_t n) {
  return n <= 8 || (n <= 32 && n * d * F * elem <= 1 << 28);
}
// Whether it takes its operands as they lie (k_ff_direct), or has those that need it laid
// out for the large tiles' kernel: whose time that pass is with few tokens. Both sides
// measured (us, direct / laid out), fp32: 250 x 671 at 333 tokens 20 / 39, at 2048 39 / 43; 512
// x 2048 at 512 46 / 64, at 2048 130 / 112; 1024 x 4096 at 64 37 / 102, at 512 123 / 128, at
// 1024 228 / 194; 2048 x 8192 at 64 78 / 294, at 512 439 / 430. bf16: 1999 x 3001 at 64 28 /
// 55, at 512 60 / 66, at 1024 102 / 83; whole steps of K: 256 x 1024 at 1024 15 / 18, at 2048
// 20 / 20; 512 x 2048 at 333 19 / 21, at 1024 27 / 24; 1024 x 4096 at 128 23 / 27, at 333 31 /
// 29; 2048 x 8192 at 64 29 / 39, at 128 37 / 44, at 200 57 / 50.
bool few_forward(int elem, int d, int F, int64_t n) {
  if (d < 8 || F < 8) return false;  // pieces of 8 values along a row
  return n <= (elem == 4 || d % kStep || F % kStep ? 512 : 128) || n * d * F <= 1 << 29;
}
// The same for a backward, whose operands all need laying out. Laying out the weights
// takes their bytes' time whatever the tokens, so with large ones the two cross at one
// number of tokens; with small ones, where launches count, at one n d d_ff. Measured (us,
// direct / laid out), bf16: 2048 x 8192 at 64 tokens 72 / 131, at 200 128 / 151, at 320 156 /
// 165, at 512 226 / 194; 2560 x 9728 at 200 206 / 237, at 320 238 / 256, at 512 348 / 311; 1024
// x 4096 at 64 39 / 51, at 512 67 / 74, at 768 91 / 85; 512 x 2048 at 1024 51 / 56, at 3200 115 /
// 112; 256 x 1024 at 6000 69 / 77; 1999 x 3001, where 16 bytes start at any element, at 320
// 89 / 102, at 512 124 / 111; 1000 x 1500 at 2000 101 / 101. fp32: 2048 x 8192 at 64 167 / 421,
// at 320 610 / 642, at 512 904 / 822; 2560 x 9728 at 320 875 / 916; 1024 x 4096 at 640 310 / 307,
// at 1024 457 / 413; 512 x 2048 at 4100 512 / 527; 1000 x 1500 at 1400 279 / 275, at 2600 476 /
// 414.
bool few_backward(int elem, int d, int F, int64_t n) {
  if (d < 8 || F < 8) return false;  // pieces of 8 values along a row
  const int64_t unit = (int64_t)1 << 30;
  const int64_t most = elem == 4 ? 4 * unit - 1 : d % 8 || F % 8 ? 2 * unit : 3 * unit;
  return n <= 320 || n <= most / ((int64_t)d * F);
}
int direct_parts(int64_t tiles, int64_t steps) {
  const int64_t s = std::min<int64_t>({2 * kCUs / std::max<int64_t>(tiles, 1), steps / 4, 64});
  if (s < 2) return 1;
  return (int)ceil_div(steps, ceil_div(steps, s));  // no empty part
}
// A product out of the direct kernel: its sizes and parts, and where those go.
template <typename T>
FfDirect<T> direct_product(Area &w, int M, int N, int K, int runs, float *&part) {
  FfDirect<T> g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.runs = runs;
  g.splits = direct_parts(ceil_div(M, kDTile) * ceil_div(N, kDTile), runs * ceil_div(K, kDStep<T>));
  part = g.splits > 1 ? (float *)w.take(4 * (int64_t)g.splits * N * round_up(M, 8)) : nullptr;
  return g;
}
template <typename T>
EpiOut<T> direct_out(const FfDirect<T> &g, float *part, void *to, int64_t ld) {
  const int64_t pl = round_up(g.M, 8);
  return {(T *)to, nullptr, ld, g.M, g.N, 1 << 30, part, g.N * pl, pl};
}
template <typename T>
struct DirectFwd {
  T *z;
  FfDirect<T> out;
  float *part;
  size_t bytes;
  DirectFwd(void *base, int d, int F, int n) {
    Area w{(char *)base};
    z = (T *)w.take((int64_t)n * F * (int64_t)sizeof(T));
    out = direct_product<T>(w, d, n, F, 1, part);
    bytes = w.off;
  }
};
template <typename T>
struct DirectBwd {
  T *da, *du, *z;
  FfDirect<T> out[4];  // dx, dW_g, dW_u, dW_d
  float *part[4];
  size_t bytes;
  DirectBwd(void *base, int d, int F, int n) {
    Area w{(char *)base};
    for (T **p : {&da, &du, &z}) *p = (T *)w.take((int64_t)n * F * (int64_t)sizeof(T));
    out[0] = direct_product<T>(w, d, n, F, 2, part[0]);
    out[1] = direct_product<T>(w, d, F, n, 1, part[1]);
    out[2] = direct_product<T>(w, d, F, n, 1, part[2]);
    out[3] = direct_product<T>(w, F, d, n, 1, part[3]);
    bytes = w.off;
  }
};

template <typename T, bool TURNED, bool DUAL, int TN, class Epi, int G>
hipError_t launch_direct(FfDirects<T, Epi, G> grp, hipStream_t st) {
  int at = 0;
  for (int p = 0; p < G; ++p) {
    const FfDirect<T> &g = grp.prob[p];
    grp.start[p] = at;
    at += (int)round_up(ceil_div(g.M, DUAL ? kDTile / 2 : kDTile) * ceil_div(g.N, TN) * g.splits, 8);
  }
  grp.start[G] = at;
  hipLaunchKernelGGL((k_ff_direct<T, TURNED, DUAL, TN, Epi, G>), dim3((unsigned)at), dim3(256), 0, st, grp);
  return hipGetLastError();
}
// A product with an epilogue of its own, which cannot be split: in narrow tiles where wide
// ones leave CUs without any or are half empty (us, narrow / wide, fp32: 512 x 2048, 64 tokens
// forward 23 / 27, backward 36 / 41; 1216 x 1864, 64 tokens 33 / 42, 58 / 69; 2048 x 8192, 17
// tokens forward 60 / 77; with narrow tiles up to two a CU 1024 x 4096, 175 tokens 61 / 68, but
// 1216 x 1864, 333 tokens backward 130 / 127).
template <typename T, bool TURNED, bool DUAL, class Epi>
hipError_t direct_with(const FfDirect<T> &g, const Epi &epi, hipStream_t st) {
  const FfDirects<T, Epi, 1> grp{{g}, {epi}, {}};
  if (g.N <= 32 || ceil_div(g.M, DUAL ? kDTile / 2 : kDTile) * ceil_div(g.N, kDTile) < kCUs)
    return launch_direct<T, TURNED, DUAL, 32>(grp, st);
  return launch_direct<T, TURNED, DUAL, kDTile>(grp, st);
}

template <typename T>
hipError_t forward_direct(const FfArgs &p, hipStream_t st) {
  const int d = p.d, F = p.F, n = (int)p.n;
  const DirectFwd<T> w(p.ws, d, F, n);
  const FfDirect<T> q{{(const T *)p.w_gate, (const T *)p.w_up, d}, {(const T *)p.x, nullptr, p.x_stride},
                      false, F, n, d, 1, 1};
  TRYH((direct_with<T, false, true>(q, EpiZDirect<T>{w.z, p.a, p.u, F}, st)));
  FfDirects<T, EpiOut<T>, 1> g{{w.out}, {direct_out(w.out, w.part, p.y, p.y_stride)}, {}};
  g.prob[0].a = {(const T *)p.w_down, nullptr, F};
  g.prob[0].b = {w.z, nullptr, F};
  TRYH((launch_direct<T, false, false, kDTile>(g, st)));
  return joins<T, 1>(g, st);
}

template <typename T>
hipError_t backward_direct(const FfArgs &p, hipStream_t st) {
  const int d = p.d, F = p.F, n = (int)p.n;
  const DirectBwd<T> w(p.ws, d, F, n);
  const T *x = (const T *)p.x, *dy = (const T *)p.dy, *wd = (const T *)p.w_down;
  // dz(f, t) = sum_c W_d(c, f) dy(t, c), and from it dA, dU and z
  const FfDirect<T> dz{{wd, nullptr, F}, {dy, nullptr, p.dy_stride}, false, F, n, d, 1, 1};
  TRYH((direct_with<T, true, false>(dz, EpiDzDirect<T>{p.a, p.u, w.da, w.du, w.z, F}, st)));
  FfDirects<T, EpiOut<T>, 4> g{};
  const auto out = [&](int k, FfSide<T> a, FfSide<T> b, void *to, int64_t ld) {
    g.prob[k] = w.out[k];
    g.prob[k].a = a;
    g.prob[k].b = b;
    g.prob[k].b_turned = k > 0;
    g.epi[k] = direct_out(w.out[k], w.part[k], to, ld);
  };
  out(0, {(const T *)p.w_gate, (const T *)p.w_up, d}, {w.da, w.du, F}, p.dx, p.dx_stride);
  out(1, {x, nullptr, p.x_stride}, {w.da, nullptr, F}, p.dw_gate, d);
  out(2, {x, nullptr, p.x_stride}, {w.du, nullptr, F}, p.dw_up, d);
  out(3, {w.z, nullptr, F}, {dy, nullptr, p.dy_stride}, p.dw_down, F);
  TRYH((launch_direct<T, true, false, kDTile>(g, st)));
  return joins<T, 4>(g, st);
}

FfProb with_operands(FfProb g, const Opnd &a, const Opnd &b) {
  g.a = a.p;
  g.lda = a.ld;
  g.pa = a.plane;
  g.b = b.p;
  g.ldb = b.ld;
  g.pb = b.plane;
  return g;
}

}  // namespace
}  // namespace mfma

using namespace mfma;

size_t ff_forward_workspace(int elem, int d, int F, int64_t n) {
  if (single_tokens(elem, d, F, n)) return (size_t)round_up(std::max<int64_t>(n, 1) * F * elem, 256);
  if (few_forward(elem, d, F, n))
    return elem == 2 ? DirectFwd<__bf16>(nullptr, d, F, (int)n).bytes
                     : DirectFwd<float>(nullptr, d, F, (int)n).bytes;
  return FwdPlan(nullptr, elem == 2 ? 1 : 3, d, F, n).bytes;
}
size_t ff_backward_workspace(int elem, int d, int F, int64_t n) {
  if (few_backward(elem, d, F, n))
    return std::max<size_t>(256, elem == 2 ? DirectBwd<__bf16>(nullptr, d, F, (int)n).bytes
                                           : DirectBwd<float>(nullptr, d, F, (int)n).bytes);
  return std::max<size_t>(256, BwdPlan(nullptr, elem == 2 ? 1 : 3, d, F, n).bytes);
}

template <typename T>
hipError_t ff_forward(const FfArgs &p, hipStream_t st) {
  const int d = p.d, F = p.F, n = (int)p.n;
  const T *wg = (const T *)p.w_gate, *wu = (const T *)p.w_up, *wd = (const T *)p.w_down;
  if (single_tokens((int)sizeof(T), d, F, n)) {
    T *z = (T *)p.ws;
    TRYH((launch_small<T, true>(wg, wu, (const T *)p.x, p.x_stride, n, F, d, z, F, p.a, p.u, st)));
    return launch_small<T, false>(wd, nullptr, z, F, n, d, F, (T *)p.y, p.y_stride, nullptr, nullptr,
                                  st);
  }
  if (few_forward((int)sizeof(T), d, F, n)) return forward_direct<T>(p, st);
  constexpr int NP = planes_of<T>();
  const FwdPlan w(p.ws, NP, d, F, n);
  const int64_t Fp = kpad(F);
  Layouts<T> lay;
  const Opnd x = lay.rows((const T *)p.x, p.x_stride, n, d, w.x);
  const Opnd g = lay.rows(wg, d, F, d, w.wg);
  const Opnd u = lay.rows(wu, d, F, d, w.wu);
  const Opnd o = lay.rows(wd, F, d, F, w.wd);
  TRYH(lay.launch(st));
  const FfProb q{g.p, u.p, x.p, g.ld, x.ld, g.plane, x.plane, F, n, (int)(kpad(d) / kStep), 1};
  TRYH((product_with<NP, true>(q, EpiZ<T>{w.z, n * Fp, F, (int)Fp, p.a, p.u}, st)));
  const FfGroup<EpiOut<T>, 1> y{{with_operands(w.down, o, {w.z, Fp, n * Fp})},
                                {EpiOut<T>{(T *)p.y, nullptr, p.y_stride, d, n, 1 << 30, w.part, 0, 0}},
                                {}};
  return products_out<T, 1>(y, st);
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
  if (few_backward((int)sizeof(T), d, F, n)) return backward_direct<T>(p, st);
  constexpr int NP = planes_of<T>();
  const BwdPlan w(p.ws, NP, d, F, n);
  const int64_t dp = kpad(d), Fp = kpad(F), Tp = kpad(n);
  // W_d^T [F][dp]; W_g^T and W_u^T side by side [d][2 Fp]; x^T and dy^T [d][Tp]
  Layouts<T> lay;
  const Opnd dy = lay.rows((const T *)p.dy, p.dy_stride, n, d, w.dy);
  lay.cols((const T *)p.w_down, F, d, F, w.wdt, dp, F * dp);
  lay.cols((const T *)p.w_gate, d, F, d, w.wgut, 2 * Fp, d * 2 * Fp);
  lay.cols((const T *)p.w_up, d, F, d, w.wgut + Fp, 2 * Fp, d * 2 * Fp);
  lay.cols((const T *)p.x, p.x_stride, n, d, w.xt, Tp, d * Tp);
  lay.cols((const T *)p.dy, p.dy_stride, n, d, w.dyt, Tp, d * Tp);
  TRYH(lay.launch(st));
  // dz, and from it dA, dU and z
  const FfProb q{w.wdt, nullptr, dy.p, dp, dy.ld, F * dp, dy.plane, F, n, (int)(dp / kStep), 1};
  TRYH((product_with<NP, false>(q,
                                EpiDz<T>{p.a, p.u, w.dau, w.z, n * 2 * Fp, n * Fp, w.daut, w.zt, Tp, F,
                                         (int)Fp},
                                st)));
  if constexpr (NP > 1) {
    Layouts<__bf16> turn;
    turn.add(w.dau, 2 * Fp, n * 2 * Fp, NP, n, (int)(2 * Fp), w.daut, Tp, 2 * Fp * Tp, true);
    turn.add(w.z, Fp, n * Fp, NP, n, (int)Fp, w.zt, Tp, Fp * Tp, true);
    TRYH(turn.launch(st));
  }
  // dx = [dA dU] [W_g; W_u]; dW_g, dW_u (rows f < F of [dA dU]^T and from Fp on); dW_d
  const Opnd xt{w.xt, Tp, d * Tp}, dyt{w.dyt, Tp, d * Tp}, daut{w.daut, Tp, 2 * Fp * Tp};
  const FfGroup<EpiOut<T>, 3> out{
      {with_operands(w.out[0], {w.wgut, 2 * Fp, d * 2 * Fp}, {w.dau, 2 * Fp, n * 2 * Fp}),
       with_operands(w.out[1], xt, daut), with_operands(w.out[2], {w.zt, Tp, Fp * Tp}, dyt)},
      {EpiOut<T>{(T *)p.dx, nullptr, p.dx_stride, d, n, 1 << 30, w.part[0], 0, 0},
       EpiOut<T>{(T *)p.dw_gate, (T *)p.dw_up, (int64_t)d, d, F, (int)Fp, w.part[1], 0, 0},
       EpiOut<T>{(T *)p.dw_down, nullptr, (int64_t)F, F, d, 1 << 30, w.part[2], 0, 0}},
      {}};
  return products_out<T, 3>(out, st);
}

template hipError_t ff_forward<float>(const FfArgs &, hipStream_t);
template hipError_t ff_forward<__bf16>(const FfArgs &, hipStream_t);
template hipError_t ff_backward<float>(const FfArgs &, hipStream_t);
template hipError_t ff_backward<__bf16>(const FfArgs &, hipStream_t);

}  // namespace ipttt
