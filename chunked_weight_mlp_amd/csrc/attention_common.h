// Building blocks of the attention kernels (gfx950): LDS tiles of heads' rows, the MFMA
// operands read from them, and the sequences of a packed batch. Device code only.
//
// All products are 32x32 MFMA tiles with 16 values of the summed index a step. Lane l
// has half h = l / 32 and column l % 32:
//   operand        8 values of row (column) l % 32: 8 h .. 8 h + 7 of the step's 16
//   result         16 values of column l % 32: rows 8 (i / 4) + 4 h + i % 4, i < 16
// Scores are computed so that a result's column is the row of the next product's other
// operand: the 8 results i = 8 s .. 8 s + 7 of a lane are then its operand values of
// step s, for the summed index in the order 16 s + 8 (j / 4) + 4 h + j % 4, j < 8, and
// the partner operand is read from LDS in the same order (ColReader). Nothing moves
// between lanes. In fp32 a step is 8 products of 2 values each, of the same shape.
#pragma once

#include <type_traits>

#include "attention_internal.h"
#include "block_internal.h"
#include "mfma_common.h"

namespace ipttt {
namespace attn {

using mfma::bf16x8;
using mfma::f32x16;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// The running maximum may fall behind by this much (in log2): weights are then up to 2^8,
// which costs neither bf16 nor fp32 precision, and the sums are seldom rescaled.
constexpr float kSlack = 8.f;

struct f32x8 {
  float v[8];
};
typedef float f32x4v __attribute__((ext_vector_type(4)));
struct F4x2 {
  f32x4v x, y;
};
template <typename T>
struct FragOf;
template <>
struct FragOf<__bf16> {
  typedef bf16x8 type;
};
template <>
struct FragOf<float> {
  typedef f32x8 type;
};
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x16 mma(const bf16x8 &a, const bf16x8 &b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const f32x8 &a, const f32x8 &b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}
// Results 8 s .. 8 s + 7 as an operand (bf16: rounded to nearest even). These are the weights p
// before p v and dv, and ds before dq and dk: the products run at the bf16 rate for it (large
// ones reach 1481 TFLOP/s, fp32 154), and their sums stay fp32. Rounding p takes o's error from
// 1.7e-3, that of rounding the exact o, to 2.2e-3.
template <typename T>
__device__ __forceinline__ Frag<T> as_operand(const f32x16 &x, int s) {
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (std::is_same<T, float>::value) f.v[j] = x[8 * s + j];
    else f[j] = (__bf16)x[8 * s + j];
  }
  return f;
}
template <typename T>
__device__ __forceinline__ Frag<T> zero_frag() {
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (std::is_same<T, float>::value) f.v[j] = 0.f;
    else f[j] = (__bf16)0.f;
  }
  return f;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
// The lower and the upper half's value of this lane's column.
__device__ __forceinline__ float2 halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_max(float v) {
  const float2 r = halves(v);
  return fmaxf(r.x, r.y);
}
__device__ __forceinline__ float half_sum(float v) {
  const float2 r = halves(v);
  return r.x + r.y;
}

// A tile of rows of DP channels (64 or 128, at least head_dim; the rest zero) in LDS, in
// pieces of 16 bytes. Piece p of row r is at place p ^ swizzle(r): the 16 rows that one
// step of a RowReader reads at one piece, and the 4 rows x 4 pieces that one of a ColReader
// reads, then fall on distinct banks.
template <typename T, int DP>
struct Tile {
  static constexpr int PE = 16 / sizeof(T);  // elements a piece
  static constexpr int NP = DP / PE;         // pieces a row: 8, 16 or 32
  static constexpr int STEPS = DP / 16;
  static_assert(NP >= 8, "rows of at least 128 bytes");
  __device__ static __forceinline__ int swizzle(int r) {
    if constexpr (NP >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  }
  __device__ static __forceinline__ int at(int r, int p) { return r * DP + ((p ^ swizzle(r)) * PE); }

};

// Reads of operands from tiles at LDS addresses kept in registers, so that a read costs no
// arithmetic: an address for each place of the pattern in a row, the rest in the instruction.
// move() goes to another tile that far away.
typedef __attribute__((address_space(3))) const char *lds_ptr;
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at, int offset) {
  return *(__attribute__((address_space(3))) const V *)((lds_ptr)(uintptr_t)at + offset);
}

// Operand values: channels 16 s + 8 h .. + 7 of row r0 + l % 32 (r0 a multiple of 32).
template <typename T, int DP>
struct RowReader {
  using L = Tile<T, DP>;
  uint32_t a[L::STEPS];
  __device__ __forceinline__ RowReader(const T *tile, int l) {
    const uint32_t base = (uint32_t)(uintptr_t)(mfma::lds_void_t *)tile;
    const int r = l & 31, h = l >> 5;
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s)
      a[s] = base + L::at(r, sizeof(T) == 2 ? 2 * s + h : 4 * s + 2 * h) * sizeof(T);
  }
  __device__ __forceinline__ void move(int bytes) {
#pragma unroll
    for (int s = 0; s < L::STEPS; ++s) a[s] += bytes;
  }
  __device__ __forceinline__ Frag<T> read(int r0, int s) const { return read_from(0, r0, s); }
  // The same of a tile that many bytes behind this one.
  __device__ __forceinline__ Frag<T> read_from(int behind, int r0, int s) const {
    const int off = r0 * DP * (int)sizeof(T);
    const uint32_t at = a[s] + behind;
    if constexpr (std::is_same<T, float>::value) {
      // the next piece: the tile begins on a multiple of 32 bytes, so its place differs in a bit
      return __builtin_bit_cast(f32x8, F4x2{lds_read<f32x4v>(at, off), lds_read<f32x4v>(at ^ 16, off)});
    } else {
      return lds_read<bf16x8>(at, off);
    }
  }
};

// Operand values: channel 32 d + l % 32 of rows r0 + 8 (j / 4) + 4 h + j % 4, j < 8 (r0 a
// multiple of 16). In bf16 by two transposing reads: 16 lanes read 4 rows x 16 channels and
// each gets one channel of the 4 rows. Rows r + 8 have row r's swizzle but for 2 pieces, a bit of
// the address (tiles begin on multiples of 256 bytes).
template <typename T, int DP>
struct ColReader {
  using L = Tile<T, DP>;
  uint32_t lo[DP / 32];
  __device__ __forceinline__ ColReader(const T *tile, int l) {
    const uint32_t base = (uint32_t)(uintptr_t)(mfma::lds_void_t *)tile;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) {
      const int r = 4 * (l >> 5) + (sizeof(T) == 2 ? (l & 15) >> 2 : 0);
      const int c = 32 * d + (sizeof(T) == 2 ? 16 * ((l >> 4) & 1) + 4 * (l & 3) : l & 31);
      lo[d] = base + (L::at(r, c / L::PE) + c % L::PE) * sizeof(T);
    }
  }
  __device__ __forceinline__ void move(int bytes) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) lo[d] += bytes;
  }
  __device__ __forceinline__ Frag<T> read(int r0, int d) const {
    const int off = r0 * DP * (int)sizeof(T);
    if constexpr (std::is_same<T, float>::value) {
      // row r + j % 4: its swizzle differs from row r's in bits 2 and 3 of the piece
      f32x8 f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int upper = j < 4 ? 0 : 32;
        f.v[j] = lds_read<float>(lo[d] ^ (swizzle_step(j % 4) | upper), off + (j % 4 + upper / 4) * DP * 4);
      }
      return f;
    } else {
      typedef __attribute__((address_space(3))) mfma::v4i16 lds_v4;
      const mfma::v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4 *)((__attribute__((address_space(3))) char *)(uintptr_t)lo[d] + off));
      const mfma::v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4 *)((__attribute__((address_space(3))) char *)(uintptr_t)(lo[d] ^ 32) + off + 8 * DP * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // bytes by which the swizzles of rows r and r + j, r a multiple of 4, differ
  __device__ static constexpr int swizzle_step(int j) {
    return 16 * (L::NP >= 16 ? j << 2 : (j >> 1) << 2);
  }
};

// Elements c .. c + N - 1 of a row of dh, zero behind it. Rows start anywhere.
template <typename T, int N>
__device__ __forceinline__ void load_some(const T *row, int c, int dh, T (&v)[N]) {
  if (c + N <= dh) {
    const blk::Pack<T, N> k = *(const blk::Pack<T, N> *)(row + c);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = k.v[e];
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = c + e < dh ? row[c + e] : (T)0.f;
  }
}
// The operand of a row in global memory: channels 16 s + 8 h .. + 7.
template <typename T>
__device__ __forceinline__ Frag<T> load_frag(const T *row, int s, int h, int dh) {
  T v[8];
  load_some<T, 8>(row, 16 * s + 8 * h, dh, v);
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (std::is_same<T, float>::value) f.v[j] = v[j];
    else f[j] = v[j];
  }
  return f;
}

// Scores are kept without the scale, whose size enters with the exponent (log2_scale); its
// sign is that of the operand held in registers. A scale of 0 is that of zeros, or of NaN where
// the operand is not finite.
__device__ __forceinline__ float log2_scale(float scale) {
  return scale == 0.f ? 1.f : fabsf(scale) * kLog2e;
}
template <typename T>
__device__ __forceinline__ Frag<T> with_sign(Frag<T> f, float scale) {
  if (scale > 0.f) return f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (std::is_same<T, float>::value) f.v[j] = scale == 0.f ? 0.f * f.v[j] : -f.v[j];
    else f[j] = scale == 0.f ? (__bf16)(0.f * (float)f[j]) : -f[j];
  }
  return f;
}

// A value that the compiler takes to be another one each time: what is computed from it in a
// rare path inside a loop is not computed, and held in registers, ahead of the loop.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// ---- rows of global memory into a tile ------------------------------------------------
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

// 16 (or 4) bytes a lane from base + offset in global memory to LDS at dst + 16 (4) x lane,
// counted by vmcnt. base and dst are wave-uniform. In assembly because behind the builtin
// the compiler waits for all copies in flight before every transposing LDS read; the loops
// below wait for a tile where they begin it. No register is loaded, and M0 is set and
// restored in the same block.
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const void *base, uint32_t offset, const void *dst) {
  static_assert(BYTES == 16 || BYTES == 4, "");
  const uint32_t at = __builtin_amdgcn_readfirstlane((int)(uintptr_t)(mfma::lds_void_t *)dst);
  uint32_t m0;
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(at), "v"(offset), "s"(base) : "memory");
  else
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dword %2, %3\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(at), "v"(offset), "s"(base) : "memory");
}
// The same from an address of each lane's own.
__device__ __forceinline__ void copy_to_lds16(const void *src, const void *dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((int)(uintptr_t)(mfma::lds_void_t *)dst);
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
               "global_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0) : "s"(at), "v"(src) : "memory");
}
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
template <typename T>
__device__ __forceinline__ const T *uniform(const T *p) {
  return (const T *)uniform64((uint64_t)p);
}

// Copies ROWS rows of one head into tiles, WAVES waves together: directly (16 bytes a
// lane, no registers; the copies are counted by vmcnt and land later) where every piece
// is whole and on a 16-byte boundary and a tile spans less than 2^31 bytes, else through
// registers. Rows at or behind `end` repeat the last one before it. Pieces behind dh are
// left as they are: clear() first.
template <typename T, int DP, int ROWS, int WAVES>
struct Copier {
  using L = Tile<T, DP>;
  static constexpr int RPI = 64 / L::NP;              // rows an instruction fills
  static constexpr int NI = ROWS / (RPI * WAVES);     // instructions a wave
  static_assert(ROWS % (RPI * WAVES) == 0, "rows must split evenly over the waves");
  // Instructions' rows that lie a multiple of 16 apart have the same swizzle: one register
  // then holds the lane's offset for all of them.
  static constexpr int STEP = WAVES * RPI, NO = STEP % 16 == 0 ? 1 : NI;
  const T *base;
  int64_t stride;
  uint32_t offset[NO];  // of this lane's piece from the tile's first row
  bool direct;
  // shift: what issue()'s shift is a multiple of
  __device__ __forceinline__ Copier(const T *p, int64_t tok_stride, int dh, int wave, int lane, int64_t shift = 0)
      : base(uniform(p)), stride(tok_stride) {
    direct = dh % L::PE == 0 && (uintptr_t)p % 16 == 0 && tok_stride * sizeof(T) % 16 == 0 &&
             shift * sizeof(T) % 16 == 0 && tok_stride < (1 << 30) / ROWS / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < NO; ++i) {
      const int r = row(i, wave, lane);
      offset[i] = (r * (uint32_t)stride + piece(r, lane) * L::PE) * sizeof(T);
    }
  }
  __device__ static __forceinline__ int row(int i, int wave, int lane) {
    return (i * WAVES + wave) * RPI + lane / L::NP;
  }
  __device__ static __forceinline__ int piece(int r, int lane) { return (lane % L::NP) ^ L::swizzle(r); }
  // wave must be wave-uniform
  __device__ __forceinline__ void issue(T *tile, int first, int end, int dh, int wave, int lane,
                                        int fix, int64_t shift = 0) const {
    const T *const from_base = base + shift;
    if (direct && fix == kAsIs) {
      const T *const p0 = from_base + (int64_t)first * stride;
      const bool over = first + ROWS > end;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t at = NO == 1 ? offset[0] + i * (STEP * (uint32_t)stride * (uint32_t)sizeof(T)) : offset[i % NO];
        if (over) {
          const int r = row(i, wave, here(lane));
          at -= max(0, first + r - (end - 1)) * (uint32_t)stride * (uint32_t)sizeof(T);
        }
        if (DP == dh || piece(row(i, wave, lane), lane) * L::PE < dh)
          copy_to_lds<16>(p0, at, tile + (i * WAVES + wave) * RPI * DP);
      }
    } else {
      const int ln = here(lane), width = here(dh);
#pragma unroll 1
      for (int i = 0; i < NI; ++i) {
        const int r = row(i, wave, ln), p = ln % L::NP;
        const int from = first + r < end ? first + r : end - 1;
        T v[L::PE];
        load_some<T, L::PE>(from_base + from * stride, p * L::PE, width, v);
#pragma unroll
        for (int e = 0; e < L::PE; ++e) tile[L::at(r, p) + e] = fixed(v[e], fix);
      }
    }
  }
};
// All tiles zero, for those whose rows are narrower than DP. A barrier must follow.
template <typename T>
__device__ __forceinline__ void clear(T *tiles, int elems, int tid, int threads) {
  for (int i = tid; i < elems * (int)sizeof(T) / 16; i += threads)
    ((uint4 *)tiles)[i] = make_uint4(0, 0, 0, 0);
}

// A lane's results x scale to its row of dh channels in memory. kCount leaves NaN there where
// something was counted and zero elsewhere, and kFinite adds to that.
template <typename T, int DP>
__device__ __forceinline__ void store_row(T *row, const f32x16 (&x)[DP / 32], float scale, int half,
                                          int width, int fix) {
  const int h = here(half), dh = here(width);
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * d + 8 * g + 4 * h;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[d][4 * g + e] * scale;
      if (fix != kAsIs) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (fix == kCount) v[e] = x[d][4 * g + e] != 0.f ? NAN : 0.f;
          else if (c + e < dh) v[e] += (float)row[c + e];
        }
      }
      if (c + 4 <= dh) {
        blk::store_pack<T, 4>(row + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < dh) row[c + e] = (T)v[e];
      }
    }
}

// ---- the sequences of a packed batch -------------------------------------------------
// Offset i of a batch as the operators read it: the first is 0, all are within n (none
// given: one sequence).
__device__ __forceinline__ int64_t offset_of(const int32_t *off, int i, int64_t n) {
  if (i <= 0) return 0;
  if (!off) return n;
  const int64_t v = off[i];
  return v < 0 ? 0 : v > n ? n : v;
}
// One sequence's rows, of which sequence `batch` is what lies behind the last one.
struct Rows {
  int64_t start;
  int len;
};
__device__ __forceinline__ Rows rows_of(const int32_t *off, int s, int batch, int64_t n) {
  const int64_t b = batch ? offset_of(off, s, n) : 0;
  const int64_t e = s < batch ? offset_of(off, s + 1, n) : n;
  return Rows{b, (int)(e > b ? e - b : 0)};
}
// Tiles of at most M rows that lie in one sequence, without a table of them: sequence s
// has the numbers from start / M + s on, which is enough for any start and length, and
// n / M + batch + 1 in all. Some are empty. All 64 lanes take part.
inline int64_t tiles_of(int64_t n, int M, int batch) { return n / M + batch + 1; }
__device__ __forceinline__ int sequence_of(const int32_t *off, int batch, int64_t n, int M,
                                           int64_t tile, int lane) {
  int s = 0;
  for (int base = 1; base <= batch; base += 64) {
    const int i = base + lane;
    const bool before = i <= batch && offset_of(off, i, n) / M + i <= tile;
    const int k = __popcll(__ballot(before));
    s += k;
    if (k < 64) break;
  }
  return s;
}

}  // namespace attn
}  // namespace ipttt
