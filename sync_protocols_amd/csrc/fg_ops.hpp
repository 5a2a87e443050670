// Shared pieces of the decoding operators (norm, router, 4-bit products, expert
// layer for few tokens): element types, 64-lane reductions, and the streamed
// product of a few activation rows with long weight rows.
//
// The product. With T rows (tokens) of x and weight rows W[n][.], out[t][n] =
// sum_k x[t][k] W[n][k]. For the few rows of a decoding step every weight is
// read once and used T times, so the memory rate bounds it, and the arithmetic
// only has to stay out of the way: a wave multiplies 16 weight rows with 16
// token rows by v_mfma_f32_16x16x32_bf16 even when T = 1 (the matrix unit is
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

// Reductions over the 64 lanes of a wave; every lane gets the result.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}

// ------------------------------------------------------------- activations
// X_SPLIT: two bf16 rows whose sum is the activation (the expert layer's own
// intermediate, in the element order of paired()); X_I8G, X_E4M3G: 8-bit rows
// with one scale per 128 k, the others have one per row, which the caller
// applies to the finished sums.
enum { X_BF16 = FG_BF16, X_I8 = FG_I8, X_E4M3 = FG_E4M3, X_SPLIT = 16, X_I8G = 17, X_E4M3G = 18 };
constexpr bool x_is_i8(int xk) { return xk == X_I8 || xk == X_I8G; }
constexpr bool x_is_e4m3(int xk) { return xk == X_E4M3 || xk == X_E4M3G; }
constexpr bool x_is_8bit(int xk) { return x_is_i8(xk) || x_is_e4m3(xk); }
constexpr bool x_grouped(int xk) { return xk == X_I8G || xk == X_E4M3G; }
constexpr bool x_row_scaled(int xk) { return xk == X_I8 || xk == X_E4M3; }

// 4-bit weights come out of a word as k pairs (0,4) (1,5) (2,6) (3,7) in 16 bits,
// or as k (0,2,4,6) and (1,3,5,7) in 8 bits (see frag16, bytes8); activations are
// brought into that order once for all the weight rows of a wave.
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

// Where a lane finds its activations: lane l's pointer is that of token
// 16 m + l % 16 (clamped by the caller to a token that exists; rows of D that
// belong to no token are never stored). Scales per 128 k: lane l needs those of
// tokens 4 (l / 16) + 0..3 of each tile, because that is what its sums are.
template <int KXR, int MT>
struct XPtr {
  const char* p[KXR][MT];
};
template <int MT>
struct XScale {
  const float* base;
  uint32_t at[MT][4];
};

// ----------------------------------------------------------------- products
// One step of a wave is kStep = 128 k of 16 R weight rows; lane l holds row
// l % 16 of each 16. A weight matrix is a uniform base (Mat) and a 32-bit
// distance per lane (Row), so that an address costs no vector arithmetic.
constexpr int kStep = 128;

// 16-bit weights [rows][K]: four 16-byte loads, each 64 contiguous bytes of a
// row. 8-bit activations are widened to bf16 (the weights' bytes bound this
// form, the conversion hides behind them).
template <int XK, int MT, int R, int P>
struct Dense {
  static constexpr int kR = R, kMT = MT, kP = P, kUnit = 32;
  static constexpr bool kGrouped = x_grouped(XK);
  static constexpr int kXR = XK == X_SPLIT ? 2 : 1;
  static constexpr bool k8 = x_is_8bit(XK);
  struct Mat {
    const char* w;                              // bf16 [rows][K]
    int64_t stride;                             // bytes per row
    __device__ __forceinline__ Mat at(int64_t row) const { return Mat{w + row * stride, stride}; }
  };
  struct Row {
    uint32_t w;
    __device__ __forceinline__ void set(const Mat& m, int row, int q) { w = (uint32_t)row * (uint32_t)m.stride + 16 * q; }
  };
  typedef typename std::conditional<k8, u32x2, u32x4>::type XV;
  struct Stage {
    u32x4 w[R][4];
    XV x[kXR][MT][4];
    float xs[MT][4];
  };

  template <bool TAIL>
  static __device__ __forceinline__ void load(Stage& st, const Mat& mat, const Row (&rows)[R], const XPtr<kXR, MT>& xp,
                                              const XScale<MT>& sc, int q, int step, int lim) {
    const char* base = mat.w + 256 * (int64_t)step;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.w[r][j] = *(const u32x4*)(base + rows[r].w + 64 * (TAIL && 32 * j >= lim ? 0 : j));
#pragma unroll
    for (int v = 0; v < kXR; ++v)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t k = (int64_t)step * kStep + 32 * (TAIL && 32 * j >= lim ? 0 : j) + 8 * q;
          st.x[v][m][j] = *(const XV*)(xp.p[v][m] + (k8 ? 1 : 2) * k);
        }
    if constexpr (kGrouped) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.xs[m][i] = (sc.base + step)[sc.at[m][i]];
    }
  }

  template <bool TAIL>
  static __device__ __forceinline__ void consume(const Stage& st, f32x4 (&acc)[R][MT], int lim) {
    f32x4 part[R][MT];
    if constexpr (kGrouped) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TAIL && 32 * j >= lim) break;
#pragma unroll
      for (int v = 0; v < kXR; ++v)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          bf16x8 x;
          if constexpr (k8) x = widen8<x_is_i8(XK)>(st.x[v][m][j]);
          else x = __builtin_bit_cast(bf16x8, st.x[v][m][j]);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4& d = kGrouped ? part[r][m] : acc[r][m];
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, __builtin_bit_cast(bf16x8, st.w[r][j]), d, 0, 0, 0);
          }
        }
    }
    if constexpr (kGrouped) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][m][i] = __builtin_fmaf(part[r][m][i], st.xs[m][i], acc[r][m][i]);
    }
  }
};

// 4-bit weights [rows][K / 2] (low nibble of a byte first) with one bf16 scale
// and optionally one zero point per G consecutive k of a row.
//
// Layout. A lane loads 16 bytes, 32 consecutive weights, so that a wave's load
// covers 64 contiguous bytes of 16 rows. A matrix instruction sums over lanes
// l, l + 16, l + 32, l + 48 and must stay inside one group, for the scale to be
// applied to its fp32 result: for G = 32 and 64 the words change places between
// those lanes (two v_permlane*_swap per two words). Word j of lane quarter q then
// holds k = koff(j, q) + 0..7.
//
// Arithmetic, exact up to the sums, by the activations' type:
//   bf16: a nibble q becomes the bf16 number 128 + q by one and-or (0x4300 | q),
//     two at a time, 7 instructions per 8 weights. sum (q - z) x is then
//     sum (128 + q) x - (128 + z) sum x, sum x from one more matrix instruction
//     against ones, shared by all weight rows of the wave. The subtraction costs
//     about 5 bits of the fp32 sums, which leaves them 10 bits finer than the bf16
//     result; an infinity in x gives NaN in its row of the result.
//   e4m3: the byte q is the 8-bit float q * 2^-9 (0..7 are its subnormals, 8..15
//     its first binade), so a nibble moved into a byte is a number already (3
//     instructions per 8 weights); z by the sum of x as above.
//   int8: the byte (q + 128 - z) ^ 128 is q - z in two's complement (no carry
//     leaves a byte); int32 sums are exact and below 2^24.
template <int G, int XK, int MT, int R, int P>
struct Quant4 {
  static constexpr int kR = R, kMT = MT, kP = P, kUnit = G;
  static constexpr bool kGrouped = x_grouped(XK);
  static constexpr int kXR = XK == X_SPLIT ? 2 : 1;
  static constexpr bool k8 = x_is_8bit(XK);
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
    __device__ __forceinline__ void set(const Mat& m, int row, int q) {
      w = (uint32_t)row * (uint32_t)m.stride + 16 * q;
      s = (uint32_t)row * (uint32_t)m.gstride;
    }
  };
  struct Stage {
    u32x4 w[R];
    uint32_t s[R][(kGroups + 1) / 2], z[R];     // bf16 pairs, bytes
    u32x4 x[kXR][MT][k8 ? 2 : 4];
    float xs[MT][4];
  };
  static __device__ __forceinline__ int koff(int j, int q) {
    return G == 128 ? 32 * q + 8 * j : G == 64 ? 64 * (j / 2) + 8 * (j % 2) + 32 * (q % 2) + 16 * (q / 2) : 32 * j + 8 * q;
  }

  template <bool TAIL>
  static __device__ __forceinline__ void load(Stage& st, const Mat& mat, const Row (&rows)[R], const XPtr<kXR, MT>& xp,
                                              const XScale<MT>& sc, int q, int step, int lim) {
    const char* base = mat.w + 64 * (int64_t)step;
    const int64_t g0 = (int64_t)step * kGroups;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // past the end of a row: the last 32 weights again, in groups that are not used
      const uint32_t back = TAIL && 32 * q >= lim ? 16 * (q + 1) - lim / 2 : 0;
      st.w[r] = *(const u32x4*)(base + (rows[r].w - back));
      const char* sp = (const char*)(mat.s + g0) + 2 * (uint64_t)rows[r].s;
      if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < (kGroups + 1) / 2; ++i) st.s[r][i] = 0;
        st.z[r] = 0;
#pragma unroll
        for (int h = 0; h < kGroups; ++h) {
          if (G * h >= lim) break;
          st.s[r][h / 2] |= (uint32_t)((const uint16_t*)sp)[h] << (16 * (h % 2));
          st.z[r] |= (mat.z ? (uint32_t)mat.z[g0 + h + rows[r].s] : 8u) << (8 * h);
        }
      } else {
        if constexpr (kGroups == 4) {
          const u32x2 v = *(const u32x2_a1*)sp;
          st.s[r][0] = v[0]; st.s[r][1] = v[1];
        } else if constexpr (kGroups == 2) {
          st.s[r][0] = *(const u32_a1*)sp;
        } else {
          st.s[r][0] = *(const uint16_t*)sp;
        }
        st.z[r] = 0x08080808u;
        if (mat.z) {
          const uint8_t* zp = mat.z + g0 + rows[r].s;
          if constexpr (kGroups == 4) st.z[r] = *(const u32_a1*)zp;
          else if constexpr (kGroups == 2) st.z[r] = *(const u16_a1*)zp;
          else st.z[r] = *zp;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < kXR; ++v)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int jj = TAIL && (j / kWords) * G >= lim ? j % kWords : j;
          const char* p = xp.p[v][m] + (k8 ? 1 : 2) * ((int64_t)step * kStep + koff(jj, q));
          if constexpr (!k8) {
            st.x[v][m][j] = *(const u32x4*)p;
          } else if (G == 32) {                // eight bytes a word; else two words are neighbours
            const u32x2 t = *(const u32x2*)p;
            st.x[v][m][j / 2][2 * (j % 2)] = t[0];
            st.x[v][m][j / 2][2 * (j % 2) + 1] = t[1];
          } else if (j % 2 == 0) {
            st.x[v][m][j / 2] = *(const u32x4_a8*)p;
          }
        }
    if constexpr (kGrouped) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.xs[m][i] = (sc.base + step)[sc.at[m][i]];
    }
  }

  // The words of a lane, group by group.
  static __device__ __forceinline__ u32x4 gather(u32x4 w) {
    if constexpr (G == 128) return w;
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    if constexpr (G == 64) return u32x4{a[0], b[0], a[1], b[1]};
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
  static __device__ __forceinline__ u32x2 bytes8(uint32_t v) { return u32x2{v & 0x0f0f0f0fu, (v >> 4) & 0x0f0f0f0fu}; }
  static __device__ __forceinline__ long as_long(u32x2 v) { return __builtin_bit_cast(long, v); }

  template <bool TAIL>
  static __device__ __forceinline__ void consume(const Stage& st, f32x4 (&acc)[R][MT], int lim) {
    u32x4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = gather(st.w[r]);
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
      if (TAIL && G * h >= lim) break;
      f32x4 sum[MT];                            // of x over the group
      u32x4 x16[kXR][MT][kWords];
      u32x2 x8[MT][kWords];
      if constexpr (!x_is_i8(XK)) {
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int f = 0; f < kWords; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int j = h * kWords + f;
          if constexpr (k8) {
            x8[m][f] = even_odd(st.x[0][m][j / 2][2 * (j % 2)], st.x[0][m][j / 2][2 * (j % 2) + 1]);
            if constexpr (x_is_e4m3(XK))
              sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(as_long(x8[m][f]), 0x3838383838383838l, sum[m], 0, 0, 0);
          } else {
            const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
            for (int v = 0; v < kXR; ++v) {
              x16[v][m][f] = XK == X_SPLIT ? st.x[v][m][j] : paired(st.x[v][m][j]);
              sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x16[v][m][f]),
                                                               __builtin_bit_cast(bf16x8, one), sum[m], 0, 0, 0);
            }
          }
        }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t sw = st.s[r][h / 2], z = (st.z[r] >> (8 * h)) & 0xffu;
        float s = h % 2 ? bf16_hi(sw) : bf16_lo(sw);
        f32x4 part[MT];
        if constexpr (x_is_i8(XK)) {
          const uint32_t up = 0x80808080u - z * 0x01010101u;
          i32x4 ip[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) ip[m] = i32x4{0, 0, 0, 0};
          u32x2 d[kWords];
#pragma unroll
          for (int f = 0; f < kWords; ++f) {
            const u32x2 b = bytes8(w[r][h * kWords + f]);
            d[f] = u32x2{(b[0] + up) ^ 0x80808080u, (b[1] + up) ^ 0x80808080u};
          }
          if constexpr (kWords == 1) {
#pragma unroll
            for (int m = 0; m < MT; ++m) ip[m] = __builtin_amdgcn_mfma_i32_16x16x32_i8(as_long(x8[m][0]), as_long(d[0]), ip[m], 0, 0, 0);
          } else {
#pragma unroll
            for (int f = 0; f < kWords; f += 2)
#pragma unroll
              for (int m = 0; m < MT; ++m)
                ip[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    i32x4{(int)x8[m][f][0], (int)x8[m][f][1], (int)x8[m][f + 1][0], (int)x8[m][f + 1][1]},
                    i32x4{(int)d[f][0], (int)d[f][1], (int)d[f + 1][0], (int)d[f + 1][1]}, ip[m], 0, 0, 0);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[m][i] = (float)ip[m][i];
        } else if constexpr (x_is_e4m3(XK)) {
          const float nz = (float)z * -0x1p-9f;
          s *= 512.0f;
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = sum[m] * nz;
#pragma unroll
          for (int f = 0; f < kWords; ++f) {
            const long b = as_long(bytes8(w[r][h * kWords + f]));
#pragma unroll
            for (int m = 0; m < MT; ++m) part[m] = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(as_long(x8[m][f]), b, part[m], 0, 0, 0);
          }
        } else {
          const float nz = -128.0f - (float)z;
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = sum[m] * nz;
#pragma unroll
          for (int f = 0; f < kWords; ++f) {
            const bf16x8 b = frag16(w[r][h * kWords + f]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int v = 0; v < kXR; ++v)
                part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x16[v][m][f]), b, part[m], 0, 0, 0);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r][m][i] = __builtin_fmaf(part[m][i], kGrouped ? s * st.xs[m][i] : s, acc[r][m][i]);
        // one row tile and group at a time: all of them at once would not fit in the registers
        if constexpr (MT > 1) __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// acc[r][m] += products over the steps first, first + by, ... < n_steps of 128 k
// and, if `tail` (0..127, a multiple of the weights' unit) is not 0 and this wave
// owns the step after the last full one, over the tail.
// P steps are kept in flight in registers.
template <class Prod>
__device__ __forceinline__ void run_steps(f32x4 (&acc)[Prod::kR][Prod::kMT], const typename Prod::Mat& mat,
                                          const typename Prod::Row (&rows)[Prod::kR], const XPtr<Prod::kXR, Prod::kMT>& xp,
                                          const XScale<Prod::kMT>& sc, int q, int first, int by, int n_steps, int tail) {
  constexpr int P = Prod::kP;
  const int n = first < n_steps ? (n_steps - first + by - 1) / by : 0;
  if (n > 0) {
    typename Prod::Stage st[P];
#pragma unroll
    for (int p = 0; p < P; ++p) Prod::template load<false>(st[p], mat, rows, xp, sc, q, first + by * (p < n ? p : n - 1), kStep);
    int i = 0;
    for (; i + P < n; i += P) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        Prod::template consume<false>(st[p], acc, kStep);
        const int nx = i + P + p;
        Prod::template load<false>(st[p], mat, rows, xp, sc, q, first + by * (nx < n ? nx : n - 1), kStep);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (i + p < n) Prod::template consume<false>(st[p], acc, kStep);
  }
  if (tail && n_steps % by == first) {
    typename Prod::Stage st;
    Prod::template load<true>(st, mat, rows, xp, sc, q, n_steps, tail);
    Prod::template consume<true>(st, acc, tail);
  }
}

template <class Prod>
__device__ __forceinline__ void clear(f32x4 (&acc)[Prod::kR][Prod::kMT]) {
#pragma unroll
  for (int r = 0; r < Prod::kR; ++r)
#pragma unroll
    for (int m = 0; m < Prod::kMT; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Which product serves weights of group size G (0: 16-bit).
template <int G, int XK, int MT, int R, int P>
struct ProductOf { typedef Quant4<G, XK, MT, R, P> T; };
template <int XK, int MT, int R, int P>
struct ProductOf<0, XK, MT, R, P> { typedef Dense<XK, MT, R, P> T; };

}  // namespace ops
}  // namespace fg
