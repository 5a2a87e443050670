// Shared pieces of the decoding operators (norm, router, 4-bit products, expert
// layer for few tokens): element types, 64-lane reductions, and the streamed
// product of a few activation rows with long weight rows.
//
// The product. With T rows (tokens) of x and weight rows W[n][.], out[t][n] =
// sum_k x[t][k] W[n][k]. For the few rows of a decoding step every weight is
// read once and used T times, so the memory rate bounds it, and the arithmetic
// only has to stay out of the way: a wave multiplies 16 weight rows with 16
// token rows by a 16x16 matrix instruction (bf16, f16 or int8) even when T = 1 (the matrix unit is
// idle otherwise; products over 16 tokens cost it 16 clocks per 512 weights,
// while HBM delivers that many 4-bit weights to one SIMD in about 110).
// Tokens are the "A" operand and weights the "B" operand: lane l then holds, in
// every result register, column n = l % 16, so that a weight's group scale is
// one value per lane. Operand lane l holds row/column l % 16 and k = 8 (l / 16)
// + 0..7; result register i of lane l is D[token 4 (l / 16) + i][n = l % 16].
// The k order inside an MFMA is free as long as both operands agree, which lets
// every lane load 16 bytes of consecutive weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fg.h"

namespace fg {
namespace ops {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// vectors at addresses with only element alignment (the compiler picks a legal load)
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_f(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ uint16_t f_bf16(float f) {       // round to nearest even, NaN kept
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t f2_bf16(float lo, float hi) {
  bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// Reductions over L = 16 neighbouring lanes or all 64 of a wave; every lane gets
// the result. Within 16 lanes by rotations in the instruction itself, then by lane
// swaps: a tenth of the latency of going through LDS.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
  static_assert(L == 16 || L == 64, "lanes");
  auto turned = [](T x, auto ctrl) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v = op(v, turned(v, std::integral_constant<int, 0x128>()));      // row_ror:8
  v = op(v, turned(v, std::integral_constant<int, 0x124>()));
  v = op(v, turned(v, std::integral_constant<int, 0x122>()));
  v = op(v, turned(v, std::integral_constant<int, 0x121>()));
  if constexpr (L == 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)a[0]), __builtin_bit_cast(T, (uint32_t)a[1]));
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)b[0]), __builtin_bit_cast(T, (uint32_t)b[1]));
  }
  return v;
}
template <int L = 64>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L = 64>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L = 64>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// Sum over this lane and the lanes before it.
__device__ __forceinline__ int lanes_before_and_own(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);      // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);      // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);      // row_bcast:31 into rows 2 and 3
  return v;
}

// ------------------------------------------------------------- activations
// X_PACKED: bf16 in operand order (the expert layer's own intermediate, see
// PackedRows); X_LDS: one bf16 row that the workgroup has copied to LDS; X_I8G, X_E4M3G: 8-bit rows
// with one scale per 128 k, the others have one per row, which the caller
// applies to the finished sums.
enum { X_BF16 = FG_BF16, X_I8 = FG_I8, X_E4M3 = FG_E4M3, X_PACKED = 16, X_I8G = 17, X_E4M3G = 18, X_LDS = 19 };
constexpr bool x_is_i8(int xk) { return xk == X_I8 || xk == X_I8G; }
constexpr bool x_is_e4m3(int xk) { return xk == X_E4M3 || xk == X_E4M3G; }
constexpr bool x_is_8bit(int xk) { return x_is_i8(xk) || x_is_e4m3(xk); }
constexpr bool x_grouped(int xk) { return xk == X_I8G || xk == X_E4M3G; }
constexpr bool x_row_scaled(int xk) { return xk == X_I8 || xk == X_E4M3; }

// 4-bit weights come out of a word as k pairs (0,4) (1,5) (2,6) (3,7) in 16 bits,
// or as k (0,2,4,6) and (1,3,5,7) in 8 bits (see frag16, half16, bytes8); activations
// are brought into that order once for all the weight rows of a wave.
__device__ __forceinline__ u32x4 paired(u32x4 w) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(w[2], w[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(w[2], w[0], 0x07060302u);
  r[2] = __builtin_amdgcn_perm(w[3], w[1], 0x05040100u);
  r[3] = __builtin_amdgcn_perm(w[3], w[1], 0x07060302u);
  return r;
}
// place of element k in that order of eight
__device__ __forceinline__ int paired_place(int k) { return (k & ~7) | (2 * (k & 3)) | ((k >> 2) & 1); }
__device__ __forceinline__ u32x2 even_odd(uint32_t a, uint32_t b) {
  return u32x2{__builtin_amdgcn_perm(b, a, 0x06040200u), __builtin_amdgcn_perm(b, a, 0x07050301u)};
}

// Eight 8-bit activations as bf16 (both kinds are exact there).
template <bool I8>
__device__ __forceinline__ bf16x8 widen8(u32x2 v) {
  u32x4 r;
  if constexpr (I8) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)(int)(int8_t)(v[i / 4] >> (8 * (i % 4)));
    // integers up to 128: the upper half of their fp32 pattern
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_amdgcn_perm(__float_as_uint(f[2 * i + 1]), __float_as_uint(f[2 * i]), 0x07060302u);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
    }
  }
  return __builtin_bit_cast(bf16x8, r);
}

// Eight e4m3 activations as f16, exactly, in paired() order.
__device__ __forceinline__ f16x8 half8(u32x2 v) {
  const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u), b = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
  return __builtin_bit_cast(f16x8, r);
}

constexpr int kStep = 128;                      // k of a step of the products

// Loads and operands. A matrix instruction wants row l % 16 and k 8 (l / 16) + 0..7
// in lane l; four lanes next to each other would then read from four rows, and
// the address unit takes one row's piece per clock, 64 clocks for a load of 1 KB.
// So lane l loads 16 bytes at 16 (l % 4) of row l / 4, 64 contiguous bytes by four
// lanes (16 clocks), and ds_bpermute carries every word to the lane that needs it.
struct Lanes {
  int lane, quarter;
  int to_operand;                               // ds_bpermute index: lane 4 (l % 16) + l / 16
  int to_pairs;                                 // the same with the pieces in the order 0, 2, 1, 3
  __device__ __forceinline__ Lanes() {
    lane = threadIdx.x & 63;
    quarter = lane >> 4;
    to_operand = 16 * (lane & 15) + 4 * quarter;
    to_pairs = 16 * (lane & 15) + 4 * (2 * (quarter & 1) + (quarter >> 1));
  }
  __device__ __forceinline__ int load_row() const { return lane >> 2; }
  __device__ __forceinline__ int piece() const { return lane & 3; }
};
__device__ __forceinline__ uint32_t from_lane(int index, uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(index, (int)v); }
__device__ __forceinline__ u32x4 from_lane(int index, u32x4 v) {
  return u32x4{from_lane(index, v[0]), from_lane(index, v[1]), from_lane(index, v[2]), from_lane(index, v[3])};
}
__device__ __forceinline__ u32x2 from_lane(int index, u32x2 v) { return u32x2{from_lane(index, v[0]), from_lane(index, v[1])}; }

// Activations of a tile: base + row[m] is the row that this lane loads from (16 m +
// l / 4) and its piece of it. Where the tile has no such row, which a decoding step's
// few rows leave most lanes to, it is kNoRow and buffer loads return zeros without
// asking for memory (MASKED; 64 tokens over 64 4-bit experts take 398 us a layer with
// it, 399 without), or one that exists (16-bit weights, whose first product it made
// slower, 79 -> 81 us). The base is uniform and the rest of an address 32 bits, as for
// the weights. Scales per 128 k: those of the row start at scale + at[m].
constexpr uint32_t kNoRow = 0xfffff000u;
template <int MT>
struct XPtr {
  const char* base;
  uint32_t row[MT];
  const float* scale;
  uint32_t at[MT];
  uint32_t plane;                               // X_PACKED: bytes of 8 elements of all rows
};
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const char* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, (int)kNoRow, 0x00020000);
}

// X_PACKED rows: for every 8 elements those of all rows, 16 bytes each. Rows that
// are used together lie side by side, so lanes load straight into the operand's
// places: row[m] is row 16 m + l % 16 at 8 (l / 16). Elements in paired() order for
// 4-bit weights.
struct PackedRows {
  static __device__ __forceinline__ int64_t at(int64_t row, int k, uint32_t plane) {
    return (int64_t)(k >> 3) * plane + 16 * row + 2 * (k & 7);
  }
};

// X_LDS: every row of the operand is that one, 128 k after 128 k in paired() order.
// A read takes four pieces of 16 bytes whatever the lanes, so nothing is loaded 16
// times from L2 and no lanes change places.
__device__ __forceinline__ char* lds_row() {
  extern __shared__ __attribute__((aligned(16))) char row[];
  return row;
}
__device__ __forceinline__ void copy_row_to_lds(const char* x, int k, int threads) {
  for (int c = threadIdx.x; c < k / 8; c += threads) ((u32x4*)lds_row())[c] = paired(((const u32x4*)x)[c]);
  __syncthreads();
}

template <int XK, int MT, bool PAIRS, bool MASKED>
struct XRows {
  static constexpr bool k8 = x_is_8bit(XK);
  typedef typename std::conditional<k8, u32x2, u32x4>::type V;      // eight elements
  V v[MT][4];
  // Elements 64 (j / 2) + 32 (q % 2) + 16 (q / 2) + 8 (j % 2) of the step (PAIRS; one load for two j) or 32 j + 8 q
  // into v[..][j]; those at or past lim: any.
  template <bool TAIL>
  __device__ __forceinline__ void load(int j, const XPtr<MT>& xp, int step, int lim) {
    const int jj = TAIL && (PAIRS ? 64 * (j / 2) : 32 * j) >= lim ? 0 : j;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (XK == X_LDS) {
        v[m][j] = *(const u32x4*)(lds_row() + 2 * kStep * step + 64 * jj + xp.row[m]);
      } else if constexpr (XK == X_PACKED) {
        const auto r = rows_at(xp.base + (uint64_t)(16 * (uint32_t)step + 4 * jj) * xp.plane);
        v[m][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)xp.row[m], 0, 0));
      } else if constexpr (PAIRS) {
        const auto r = rows_at(xp.base + (int64_t)step * kStep);
        const u32x4 t = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(xp.row[m] + 32 * (jj & ~1)), 0, 0));
        v[m][j & ~1] = u32x2{t[0], t[1]};
        v[m][j | 1] = u32x2{t[2], t[3]};
      } else {
        const char* base = xp.base + (k8 ? 1 : 2) * (int64_t)step * kStep;
        const auto r = rows_at(base);
        const int at = (int)(xp.row[m] + (k8 ? 32 : 64) * jj);
        if constexpr (!MASKED) v[m][j] = *(const V*)(base + (k8 ? 32 : 64) * jj + xp.row[m]);
        else if constexpr (k8) v[m][j] = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
        else v[m][j] = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
      }
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void load_all(const XPtr<MT>& xp, int step, int lim) {
#pragma unroll
    for (int j = 0; j < 4; j += PAIRS ? 2 : 1) load<TAIL>(j, xp, step, lim);
  }
  __device__ __forceinline__ V get(const Lanes& ln, int m, int j) const {
    return XK == X_PACKED || XK == X_LDS ? v[m][j] : from_lane(PAIRS ? ln.to_pairs : ln.to_operand, v[m][j]);
  }
};

// ----------------------------------------------------------------- products
// The scale of step t that the lanes of row 4 (l / 16) + i hold.
__device__ __forceinline__ float row_scale(float v, const Lanes& ln, int t, int i) {
  return __uint_as_float(from_lane(64 * ln.quarter + 16 * i + 4 * t, __float_as_uint(v)));
}

// One step of a wave is kStep = 128 k of 16 R weight rows. A weight matrix is a
// uniform base (Mat) and 32-bit distances per lane (Row), so that an address costs
// no vector arithmetic. What a step needs besides weights and activations, the
// scales (Aux), comes for four steps at once: lane l loads those of row l / 4 for the
// l % 4-th of them, which lie close together (with a row a lane side by side they took
// as many of the address unit's clocks as the weights).
//
// Loads in flight. What a step has taken out of its registers is loaded for a later
// step at once: activations of the next one, weights of the P-th next. Loads return
// in order, so activations are asked for before the weights of the same step.

// 16-bit weights [rows][K]: four 16-byte loads, each 64 contiguous bytes of a
// row. 8-bit activations are widened to bf16 (the weights' bytes bound this
// form, the conversion hides behind them).
template <int XK, int MT, int R, int P>
struct Dense {
  static constexpr int kR = R, kMT = MT, kP = P;
  static constexpr bool kGrouped = x_grouped(XK);
  static constexpr bool k8 = x_is_8bit(XK);
  struct Mat {
    const char* w;                              // bf16 [rows][K]
    int64_t stride;                             // bytes per row
    __device__ __forceinline__ Mat at(int64_t row) const { return Mat{w + row * stride, stride}; }
  };
  struct Row {
    uint32_t w;
    __device__ __forceinline__ void set(const Mat& m, int row, const Lanes& ln) {
      w = (uint32_t)row * (uint32_t)m.stride + 16 * ln.piece();
    }
  };
  struct Weights {
    u32x4 w[R][4];
  };
  static constexpr bool kMasked = XK == X_PACKED;
  typedef XRows<XK, MT, false, kMasked> X;
  struct Aux {
    float xs[MT];
  };

  static __device__ __forceinline__ void load_aux(Aux& a, const Mat&, const Row (&)[R], const XPtr<MT>& xp, int step, int) {
    if constexpr (kGrouped) {
#pragma unroll
      for (int m = 0; m < MT; ++m) a.xs[m] = *(const float*)((const char*)xp.scale + 4 * (xp.at[m] + (uint32_t)step));
    }
  }
  static __device__ __forceinline__ void finish_aux(Aux&, const Mat&) {}
  template <bool TAIL>
  static __device__ __forceinline__ void load(Weights& w, const Mat& mat, const Row (&rows)[R], const Lanes&, int step, int lim) {
    const char* base = mat.w + 256 * (int64_t)step;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) w.w[r][j] = *(const u32x4*)(base + rows[r].w + 64 * (TAIL && 32 * j >= lim ? 0 : j));
  }

  // acc += the products of a step; x and then w are loaded for the steps nx and nw (MAYBE: unless negative).
  template <bool TAIL, bool MAYBE>
  static __device__ __forceinline__ void consume(Weights& wt, X& x, const Aux& aux, int t, f32x4 (&acc)[R][MT], const Mat& mat,
                                                 const Row (&rows)[R], const XPtr<MT>& xp, const Lanes& ln, int lim, int nx, int nw) {
    f32x4 part[R][MT];
    if constexpr (kGrouped) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    u32x4 w[R][4];
    typename X::V xv[MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TAIL && 32 * j >= lim) break;
#pragma unroll
      for (int r = 0; r < R; ++r) w[r][j] = from_lane(ln.to_operand, wt.w[r][j]);
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[m][j] = x.get(ln, m, j);
    }
    if (!MAYBE || nx >= 0) x.template load_all<false>(xp, nx, kStep);
    if (!MAYBE || nw >= 0) load<false>(wt, mat, rows, ln, nw, kStep);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TAIL && 32 * j >= lim) break;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        bf16x8 xo;
        if constexpr (k8) xo = widen8<x_is_i8(XK)>(xv[m][j]);
        else xo = __builtin_bit_cast(bf16x8, xv[m][j]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          f32x4& d = kGrouped ? part[r][m] : acc[r][m];
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, __builtin_bit_cast(bf16x8, w[r][j]), d, 0, 0, 0);
        }
      }
    }
    if constexpr (kGrouped) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xs = row_scale(aux.xs[m], ln, t, i);
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r][m][i] = __builtin_fmaf(part[r][m][i], xs, acc[r][m][i]);
        }
    }
  }
};

// 4-bit weights [rows][K / 2] (low nibble of a byte first) with one bf16 scale
// and optionally one zero point per G consecutive k of a row.
//
// Layout. Four lanes load 64 bytes, 128 consecutive weights of a row. When every
// word is in its row's lanes, lane quarter q holds 32 k, a group or less, but a
// matrix instruction sums over the quarters and must stay inside one group, for
// the scale to be applied to its fp32 result: so words change places between
// lanes l, l + 16, l + 32, l + 48 (v_permlane*_swap) until word j of quarter q
// holds k = 32 j + 8 q + 0..7, or for 8-bit rows and groups of 64 and 128, where
// one activation load serves two words, 64 (j / 2) + 32 (q % 2) + 16 (q / 2) + 8 (j % 2).
//
// Arithmetic, exact up to the sums, by the activations' type:
//   bf16: a nibble q becomes the bf16 number 128 + q by one and-or (0x4300 | q),
//     two at a time, 7 instructions per 8 weights. sum (q - z) x is then
//     sum (128 + q) x - (128 + z) sum x, sum x from one more matrix instruction
//     against ones, shared by all weight rows of the wave. The subtraction costs
//     about 5 bits of the fp32 sums, which leaves them 10 bits finer than the bf16
//     result; an infinity in x gives NaN in its row of the result.
//   e4m3: x and q - z are f16 numbers. A nibble is made 1024 + q by one and-or
//     (0x6400 | q), or 1024 + 16 q where it lies four bits higher, and one packed
//     subtraction or multiply-add takes it to q - z: 9 instructions per 8 weights, 6
//     per 8 activations. The 8-bit float matrix instruction would save 10 of them,
//     but it drops what lies 13 bits and more below the largest of a lane's eight
//     products, so that one large activation wipes out its neighbours; the 16-bit
//     one keeps 23 bits and more of normal numbers (of f16 subnormals 13, so q 2^-24
//     does not serve either).
//   int8: the byte (q + 128 - z) ^ 128 is q - z in two's complement (no carry or
//     borrow leaves a byte for z up to 128, and a 4-bit code needs 16 at most); int32
//     sums are exact and below 2^24. Larger zero points make their weight row NaN.
//     (z by the sum of x would take them all, for 2 to 9 % more time at 64 rows.)
template <int G, int XK, int MT, int R, int P>
struct Quant4 {
  static constexpr int kR = R, kMT = MT, kP = P;
  static constexpr bool kGrouped = x_grouped(XK);
  static constexpr bool k8 = x_is_8bit(XK);
  static constexpr bool kPairs = k8 && G >= 64;
  static constexpr int kGroups = kStep / G;     // groups of a step
  static constexpr int kWords = G / 32;         // words of a lane in a group
  struct Mat {
    const char* w;                              // uint8 [rows][K / 2]
    const uint16_t* s;                          // bf16 [rows][K / G]
    const uint8_t* z;                           // uint8 [rows][K / G] or NULL (8)
    int64_t stride, gstride;
    __device__ __forceinline__ Mat at(int64_t row) const {
      return Mat{w + row * stride, s + row * gstride, z ? z + row * gstride : nullptr, stride, gstride};
    }
  };
  struct Row {
    uint32_t w, s;
    __device__ __forceinline__ void set(const Mat& m, int row, const Lanes& ln) {
      w = (uint32_t)row * (uint32_t)m.stride + 16 * ln.piece();
      s = (uint32_t)row * (uint32_t)m.gstride;
    }
  };
  struct Weights {
    u32x4 w[R];
  };
  static constexpr bool kMasked = true;
  typedef XRows<XK, MT, kPairs, kMasked> X;
  struct Aux {
    uint32_t s[R][(kGroups + 1) / 2], z[R];     // bf16 pairs, bytes
    float xs[MT];
  };

  // lim: k of the step that exist; scales of the others are not read
  static __device__ __forceinline__ void load_aux(Aux& a, const Mat& mat, const Row (&rows)[R], const XPtr<MT>& xp, int step, int lim) {
    const char* const sb = (const char*)mat.s;
    const char* const zb = (const char*)mat.z;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t at = rows[r].s + (uint32_t)step * kGroups;
      if (lim < kStep) {
#pragma unroll
        for (int i = 0; i < (kGroups + 1) / 2; ++i) a.s[r][i] = 0;
#pragma unroll
        for (int h = 0; h < kGroups; ++h) {
          if (G * h >= lim) break;
          a.s[r][h / 2] |= (uint32_t)*(const uint16_t*)(sb + 2 * (at + h)) << (16 * (h % 2));
        }
      } else if constexpr (kGroups == 4) {
        const u32x2 v = *(const u32x2_a1*)(sb + 2 * at);
        a.s[r][0] = v[0]; a.s[r][1] = v[1];
      } else if constexpr (kGroups == 2) {
        a.s[r][0] = *(const u32_a1*)(sb + 2 * at);
      } else {
        a.s[r][0] = *(const uint16_t*)(sb + 2 * at);
      }
      a.z[r] = 0;
      if (mat.z) {
        if (lim < kStep) {
#pragma unroll
          for (int h = 0; h < kGroups; ++h) {
            if (G * h >= lim) break;
            a.z[r] |= (uint32_t)*(const uint8_t*)(zb + (at + h)) << (8 * h);
          }
        } else {
          if constexpr (kGroups == 4) a.z[r] = *(const u32_a1*)(zb + at);
          else if constexpr (kGroups == 2) a.z[r] = *(const u16_a1*)(zb + at);
          else a.z[r] = *(const uint8_t*)(zb + at);
        }
      }
    }
    if constexpr (kGrouped) {
#pragma unroll
      for (int m = 0; m < MT; ++m) a.xs[m] = *(const float*)((const char*)xp.scale + 4 * (xp.at[m] + (uint32_t)step));
    }
  }
  // What was loaded, ready for use; one word carries a group's scale and zero point where a step has one group.
  static __device__ __forceinline__ void finish_aux(Aux& a, const Mat& mat) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      a.z[r] = mat.z ? a.z[r] : 0x08080808u;
      if constexpr (x_is_i8(XK)) {
        const bool over = ((a.z[r] & 0x7f7f7f7fu) + 0x7f7f7f7fu) & a.z[r] & 0x80808080u;      // a byte above 128
#pragma unroll
        for (int i = 0; i < (kGroups + 1) / 2; ++i) a.s[r][i] = over ? 0x7fc07fc0u : a.s[r][i];
      }
      if constexpr (kGroups == 1) a.s[r][0] = a.s[r][0] << 16 | (a.z[r] & 0xffu);
    }
  }

  template <bool TAIL>
  static __device__ __forceinline__ void load(Weights& w, const Mat& mat, const Row (&rows)[R], const Lanes& ln, int step, int lim) {
    const char* base = mat.w + 64 * (int64_t)step;
    // past the end of a row: its last 32 weights again, in groups that are not used
    const int piece = ln.piece();
    const uint32_t back = TAIL && 32 * piece >= lim ? 16 * (piece + 1) - lim / 2 : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) w.w[r] = *(const u32x4*)(base + (rows[r].w - back));
  }

  static __device__ __forceinline__ u32x4 gather(u32x4 v, const Lanes& ln) {
    const u32x4 w = from_lane(ln.to_operand, v);
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    if constexpr (kPairs) return u32x4{a[0], b[0], a[1], b[1]};
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
  }
  static __device__ __forceinline__ bf16x8 frag16(uint32_t v) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((v >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    return __builtin_bit_cast(bf16x8, r);
  }
  // near: 1024 + z, far: -(64 + z), both twice
  static __device__ __forceinline__ f16x8 half16(uint32_t v, f16x2 near, f16x2 far) {
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t u = v >> (4 * i);
      const f16x2 a = __builtin_bit_cast(f16x2, (u & 0x000f000fu) | 0x64006400u);
      const f16x2 b = __builtin_bit_cast(f16x2, (u & 0x00f000f0u) | 0x64006400u);
      r[i] = __builtin_bit_cast(uint32_t, a - near);
      r[i + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, sixteenth, far));
    }
    return __builtin_bit_cast(f16x8, r);
  }
  static __device__ __forceinline__ u32x2 bytes8(uint32_t v) { return u32x2{v & 0x0f0f0f0fu, (v >> 4) & 0x0f0f0f0fu}; }
  static __device__ __forceinline__ long as_long(u32x2 v) { return __builtin_bit_cast(long, v); }
  static __device__ __forceinline__ i32x4 as_i32x4(u32x2 a, u32x2 b) { return i32x4{(int)a[0], (int)a[1], (int)b[0], (int)b[1]}; }

  // acc += the products of a step; x and then w are loaded for the steps nx and nw (MAYBE: unless negative).
  template <bool TAIL, bool MAYBE>
  static __device__ __forceinline__ void consume(Weights& wt, X& x, const Aux& aux, int t, f32x4 (&acc)[R][MT], const Mat& mat,
                                                 const Row (&rows)[R], const XPtr<MT>& xp, const Lanes& ln, int lim, int nx, int nw) {
    typedef typename std::conditional<x_is_i8(XK), i32x4, f32x4>::type Sum;
    constexpr int kBlock = x_is_i8(XK) && kWords > 1 ? 2 : 1;      // words a matrix instruction takes
    u32x4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = gather(wt.w[r], ln);
    const int row = 16 * (ln.lane & 15) + 4 * t;          // the lane with step t's of this lane's weight row
    uint32_t sw[R][(kGroups + 1) / 2], zw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < (kGroups + 1) / 2; ++i) sw[r][i] = from_lane(row, aux.s[r][i]);
      zw[r] = kGroups == 1 ? sw[r][0] : from_lane(row, aux.z[r]);
    }
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
      if (TAIL && G * h >= lim) break;
      Sum part[R][MT], sum[MT];                 // of the group: products, and x alone
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = Sum{0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < R; ++r) part[r][m] = Sum{0, 0, 0, 0};
      }
      f16x2 near[R], far[R];
      if constexpr (x_is_e4m3(XK)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const _Float16 z = (_Float16)(uint16_t)((zw[r] >> (8 * h)) & 0xffu), a = z + (_Float16)1024.0f, b = -z - (_Float16)64.0f;
          near[r] = f16x2{a, a};
          far[r] = f16x2{b, b};
        }
      }
#pragma unroll
      for (int f = 0; f < kWords; f += kBlock) {
        const int j = h * kWords + f;
        typename X::V xv[MT][kBlock];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < kBlock; ++i) {
            xv[m][i] = x.get(ln, m, j + i);
            if constexpr (x_is_i8(XK)) xv[m][i] = even_odd(xv[m][i][0], xv[m][i][1]);
            else if constexpr (!k8 && XK != X_PACKED && XK != X_LDS) xv[m][i] = paired(xv[m][i]);
          }
        // both words of a load have been taken
        if ((!kPairs || kBlock == 2 || j % 2 == 1) && (!MAYBE || nx >= 0)) x.template load<false>(j, xp, nx, kStep);
        if constexpr (x_is_i8(XK)) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t up = 0x80808080u - ((zw[r] >> (8 * h)) & 0xffu) * 0x01010101u;
            u32x2 d[kBlock];
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
              const u32x2 b = bytes8(w[r][j + i]);
              d[i] = u32x2{(b[0] + up) ^ 0x80808080u, (b[1] + up) ^ 0x80808080u};
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if constexpr (kBlock == 1)
                part[r][m] = __builtin_amdgcn_mfma_i32_16x16x32_i8(as_long(xv[m][0]), as_long(d[0]), part[r][m], 0, 0, 0);
              else
                part[r][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(as_i32x4(xv[m][0], xv[m][kBlock - 1]),
                                                                   as_i32x4(d[0], d[kBlock - 1]), part[r][m], 0, 0, 0);
            }
          }
        } else if constexpr (x_is_e4m3(XK)) {
          f16x8 xo[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) xo[m] = half8(xv[m][0]);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const f16x8 b = half16(w[r][j], near[r], far[r]);
#pragma unroll
            for (int m = 0; m < MT; ++m) part[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xo[m], b, part[r][m], 0, 0, 0);
          }
        } else {
          const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
          for (int m = 0; m < MT; ++m)
            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[m][0]), __builtin_bit_cast(bf16x8, one),
                                                             sum[m], 0, 0, 0);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bf16x8 b = frag16(w[r][j]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              part[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[m][0]), b, part[r][m], 0, 0, 0);
          }
        }
        // a word at a time: all of a step at once would not fit in the registers
        if constexpr (MT > 1) __builtin_amdgcn_sched_barrier(0);
      }
      if (h == kGroups - 1 && (!MAYBE || nw >= 0)) load<false>(wt, mat, rows, ln, nw, kStep);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < (XK == X_LDS ? 1 : 4); ++i) {
          const float xs = kGrouped ? row_scale(aux.xs[m], ln, t, i) : 1.0f;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float z = (float)((zw[r] >> (8 * h)) & 0xffu);
            const float s = kGroups == 1 || h % 2 ? bf16_hi(sw[r][h / 2]) : bf16_lo(sw[r][h / 2]);
            float v;
            if constexpr (k8) v = (float)part[r][m][i];
            else v = __builtin_fmaf(sum[m][i], -128.0f - z, part[r][m][i]);
            acc[r][m][i] = __builtin_fmaf(v, kGrouped ? s * xs : s, acc[r][m][i]);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// acc[r][m] += products over the n steps first, first + by, ... of 128 k.
template <class Prod>
__device__ __forceinline__ void run_steps(f32x4 (&acc)[Prod::kR][Prod::kMT], const typename Prod::Mat& mat,
                                          const typename Prod::Row (&rows)[Prod::kR], const XPtr<Prod::kMT>& xp, const Lanes& ln,
                                          int first, int by, int n) {
  constexpr int P = Prod::kP;
  static_assert(P == 1 || P == 2 || P == 4, "weights in flight");
  if (n <= 0) return;
  typename Prod::Weights w[P];
  typename Prod::X x;
  typename Prod::Aux cur, nxt;
  auto aux = [&](typename Prod::Aux& a, int i) { Prod::load_aux(a, mat, rows, xp, first + by * min(i + ln.piece(), n - 1), kStep); };
  aux(cur, 0);
  x.template load_all<false>(xp, first, kStep);
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (p < n) Prod::template load<false>(w[p], mat, rows, ln, first + by * p, kStep);
  Prod::finish_aux(cur, mat);
  int i = 0;
  for (; i + 4 + P <= n; i += 4) {      // no branches in here: the compiler's waits count the loads in flight
    aux(nxt, i + 4);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      Prod::template consume<false, false>(w[t % P], x, cur, t, acc, mat, rows, xp, ln, kStep, first + by * (i + t + 1),
                                           first + by * (i + t + P));
    __builtin_amdgcn_sched_barrier(0);
    cur = nxt;
    Prod::finish_aux(cur, mat);
  }
  for (; i < n; i += 4) {
    if (i + 4 < n) aux(nxt, i + 4);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (i + t >= n) break;
      Prod::template consume<false, true>(w[t % P], x, cur, t, acc, mat, rows, xp, ln, kStep, i + t + 1 < n ? first + by * (i + t + 1) : -1,
                                    i + t + P < n ? first + by * (i + t + P) : -1);
    }
    cur = nxt;
    Prod::finish_aux(cur, mat);
  }
}
// The same for the last `lim` < 128 k of the rows, which are those of `step`.
template <class Prod>
__device__ __forceinline__ void run_tail(f32x4 (&acc)[Prod::kR][Prod::kMT], const typename Prod::Mat& mat,
                                         const typename Prod::Row (&rows)[Prod::kR], const XPtr<Prod::kMT>& xp, const Lanes& ln,
                                         int step, int lim) {
  typename Prod::Weights w;
  typename Prod::X x;
  typename Prod::Aux aux;
  Prod::load_aux(aux, mat, rows, xp, step, lim);
  Prod::finish_aux(aux, mat);
  x.template load_all<true>(xp, step, lim);
  Prod::template load<true>(w, mat, rows, ln, step, lim);
  Prod::template consume<true, true>(w, x, aux, 0, acc, mat, rows, xp, ln, lim, -1, -1);
}

template <class Prod>
__device__ __forceinline__ void clear(f32x4 (&acc)[Prod::kR][Prod::kMT]) {
#pragma unroll
  for (int r = 0; r < Prod::kR; ++r)
#pragma unroll
    for (int m = 0; m < Prod::kMT; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Bytes to the piece of an activation row that a lane loads.
template <int G, int XK>
__device__ __forceinline__ int x_piece(const Lanes& ln) {
  return !x_is_8bit(XK) || G >= 64 ? 16 * ln.piece() : 8 * ln.piece();
}

// Which product serves weights of group size G (0: 16-bit).
template <int G, int XK, int MT, int R, int P>
struct ProductOf { typedef Quant4<G, XK, MT, R, P> T; };
template <int XK, int MT, int R, int P>
struct ProductOf<0, XK, MT, R, P> { typedef Dense<XK, MT, R, P> T; };

}  // namespace ops
}  // namespace fg
