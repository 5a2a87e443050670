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
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

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
// Eight consecutive activations of one token as loaded (raw) and as the MFMA
// operand. The 4-bit weights of a word come out as k pairs (0,4) (1,5) (2,6)
// (3,7) (see W4::frag), so `PAIRED` operands carry x in that order. X_SPLIT: two
// bf16 rows whose sum is the activation.
enum { X_BF16 = FG_BF16, X_I8 = FG_I8, X_E4M3 = FG_E4M3, X_SPLIT = 16 };

__device__ __forceinline__ u32x4 pair_order(u32x4 w) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(w[2], w[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(w[2], w[0], 0x07060302u);
  r[2] = __builtin_amdgcn_perm(w[3], w[1], 0x05040100u);
  r[3] = __builtin_amdgcn_perm(w[3], w[1], 0x07060302u);
  return r;
}

template <int XK>
struct XRaw;

template <>
struct XRaw<X_BF16> {
  u32x4 v;
  static constexpr int kBytes = 2;
  __device__ __forceinline__ void load(const char* p, int64_t k) { v = *(const u32x4*)(p + 2 * k); }
  template <bool PAIRED>
  __device__ __forceinline__ bf16x8 get() const {
    return __builtin_bit_cast(bf16x8, PAIRED ? pair_order(v) : v);
  }
};

template <>
struct XRaw<X_I8> {
  u32x2 v;
  static constexpr int kBytes = 1;
  __device__ __forceinline__ void load(const char* p, int64_t k) { v = *(const u32x2*)(p + k); }
  // integers up to 128 are exact in bf16: the upper half of their fp32 pattern
  template <bool PAIRED>
  __device__ __forceinline__ bf16x8 get() const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)(int)(int8_t)(v[i / 4] >> (8 * (i % 4)));
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = PAIRED ? f[i] : f[2 * i], b = PAIRED ? f[i + 4] : f[2 * i + 1];
      r[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x8, r);
  }
};

template <>
struct XRaw<X_E4M3> {
  u32x2 v;
  static constexpr int kBytes = 1;
  __device__ __forceinline__ void load(const char* p, int64_t k) { v = *(const u32x2*)(p + k); }
  // e4m3 is exact in bf16
  template <bool PAIRED>
  __device__ __forceinline__ bf16x8 get() const {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
    }
    return __builtin_bit_cast(bf16x8, PAIRED ? pair_order(r) : r);
  }
};

// ----------------------------------------------------------------- weights
// One step of a wave is kStep = 128 k of 16 weight rows; lane l holds row l % 16.
// Fragment j (0..3) of a step covers k = koff(j, l / 16) + 0..7 in lane l.
constexpr int kStep = 128;

// 16-bit weights [rows][K]: four 16-byte loads, each 64 contiguous bytes of a row.
struct W16 {
  static constexpr bool kQuant = false;
  static constexpr int kGroups = 4;             // units a step's tail is cut into (32 k)
  static constexpr int kFragsPerGroup = 1;
  struct Mat {
    const char* w;                              // bf16 [rows][K]
    int64_t stride;                             // bytes per row
    __device__ __forceinline__ Mat expert(int64_t e, int64_t rows, int K) const {
      return Mat{w + e * rows * stride, stride};
    }
  };
  struct Row {                                  // one lane's row
    const char* w;
    __device__ __forceinline__ void at(const Mat& m, int64_t row, int q) { w = m.w + row * m.stride + 16 * q; }
  };
  u32x4 w[4];
  static __device__ __forceinline__ int koff(int j, int q) { return 32 * j + 8 * q; }
  template <bool TAIL>
  __device__ __forceinline__ void load(const Row& r, int step, int lim) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int jj = TAIL && 32 * j >= lim ? 0 : j;
      w[j] = __builtin_nontemporal_load((const u32x4*)(r.w + 256 * (int64_t)step + 64 * jj));
    }
  }
  __device__ __forceinline__ bf16x8 frag(int j) const { return __builtin_bit_cast(bf16x8, w[j]); }
};

// 4-bit weights [rows][K / 2] (low nibble of a byte first) with one bf16 scale
// and optionally one zero point per G consecutive k of a row.
// A lane loads G / 8 bytes of every group, so that each MFMA stays inside one
// group and the scale can be applied to its fp32 result. A nibble q becomes the
// bf16 number 128 + q by one and-or (0x4300 | q, exact), two weights at a time
// and 7 instructions per 8 weights; the sum over k of (q - z) x is then
// sum (128 + q) x - (128 + z) sum x, with sum x from one more MFMA against ones,
// shared by all weight rows of the wave. The subtraction costs about 5 bits of
// the fp32 sums, which leaves them 10 bits finer than the bf16 result; an
// infinity in x gives NaN in its row of the result.
template <int G>
struct W4 {
  static constexpr bool kQuant = true;
  static constexpr int kGroups = kStep / G;
  static constexpr int kFragsPerGroup = G / 32;
  struct Mat {
    const char* w;                              // uint8 [rows][K / 2]
    const uint16_t* s;                          // bf16 [rows][K / G]
    const uint8_t* z;                           // uint8 [rows][K / G] or NULL (8)
    int64_t stride, gstride;
    __device__ __forceinline__ Mat expert(int64_t e, int64_t rows, int K) const {
      return Mat{w + e * rows * stride, s + e * rows * gstride, z ? z + e * rows * gstride : nullptr, stride, gstride};
    }
  };
  struct Row {
    const char* w;
    const uint16_t* s;
    const uint8_t* z;
    __device__ __forceinline__ void at(const Mat& m, int64_t row, int q) {
      w = m.w + row * m.stride + (G / 8) * q;
      s = m.s + row * m.gstride;
      z = m.z ? m.z + row * m.gstride : nullptr;
    }
  };
  uint32_t w[4];
  uint16_t s[kGroups];
  uint8_t z[kGroups];
  static __device__ __forceinline__ int koff(int j, int q) {
    return G * (j / kFragsPerGroup) + (G / 4) * q + 8 * (j % kFragsPerGroup);
  }
  template <bool TAIL>
  __device__ __forceinline__ void load(const Row& r, int step, int lim) {
#pragma unroll
    for (int h = 0; h < kGroups; ++h) {
      const int hh = TAIL && G * h >= lim ? 0 : h;
      const char* p = r.w + (kStep / 2) * (int64_t)step + (G / 2) * hh;
      if constexpr (G == 128) {
        const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
      } else if constexpr (G == 64) {
        const u32x2 v = __builtin_nontemporal_load((const u32x2*)p);
        w[2 * h] = v[0]; w[2 * h + 1] = v[1];
      } else {
        w[h] = __builtin_nontemporal_load((const uint32_t*)p);
      }
      s[h] = r.s[(int64_t)step * kGroups + hh];
      z[h] = r.z ? r.z[(int64_t)step * kGroups + hh] : 8;
    }
  }
  __device__ __forceinline__ bf16x8 frag(int j) const {
    const uint32_t v = w[j];
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((v >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    return __builtin_bit_cast(bf16x8, r);
  }
};

// ------------------------------------------------------------ the product
// Activations of MT tiles of 16 tokens: lane l's pointer is that of token
// 16 mt + l % 16 (clamped by the caller to a token that exists; rows of D that
// belong to no token are never stored).
// 8-bit activations carry fp32 scales, one per token (step 0) or one per 128 k
// (step 1): xs[token * stride + k / 128 * step], applied to the fp32 sums of a
// group. Lane l needs those of tokens 4 (l / 16) + 0..3 of each tile.
template <int MT>
struct XScale {
  const float* p[MT][4];
  int step;
};

// acc[r][mt] += products over the steps first, first + by, ... < n_steps of 128 k
// and, if `tail` (0..127, a multiple of the weights' unit) is not 0 and this wave
// owns the step after the last full one, over the tail.
// P steps are kept in flight in registers.
template <class WT, int XK, int MT, int R, int P>
struct Product {
  static constexpr bool kScaled = XK == X_I8 || XK == X_E4M3;
  static constexpr int kXR = XK == X_SPLIT ? 2 : 1;
  typedef XRaw<XK == X_SPLIT ? X_BF16 : XK> XR;

  struct Stage {
    WT w[R];
    XR x[kXR][MT][4];
    float xs[MT][4];
  };

  template <bool TAIL, class XP>
  static __device__ __forceinline__ void load(Stage& st, const typename WT::Row (&rows)[R], const XP& xp, const XScale<MT>& sc,
                                              int q, int step, int lim) {
#pragma unroll
    for (int r = 0; r < R; ++r) st.w[r].template load<TAIL>(rows[r], step, lim);
#pragma unroll
    for (int v = 0; v < kXR; ++v)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int jj = TAIL && (j / WT::kFragsPerGroup) * (kStep / WT::kGroups) >= lim ? j % WT::kFragsPerGroup : j;
          st.x[v][m][j].load(xp.p[v][m], (int64_t)step * kStep + WT::koff(jj, q));
        }
    if constexpr (kScaled) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.xs[m][i] = sc.p[m][i][(int64_t)step * sc.step];
    }
  }

  template <bool TAIL>
  static __device__ __forceinline__ void consume(const Stage& st, f32x4 (&acc)[R][MT], int lim) {
    const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    f32x4 step_sum[R][MT];                      // scaled activations, 16-bit weights: sums of this step
    if constexpr (kScaled && !WT::kQuant) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) step_sum[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int h = 0; h < WT::kGroups; ++h) {
      if (TAIL && (kStep / WT::kGroups) * h >= lim) break;
      bf16x8 x[kXR][MT][WT::kFragsPerGroup];
#pragma unroll
      for (int v = 0; v < kXR; ++v)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int f = 0; f < WT::kFragsPerGroup; ++f)
            x[v][m][f] = st.x[v][m][h * WT::kFragsPerGroup + f].template get<WT::kQuant>();
      if constexpr (WT::kQuant) {
        f32x4 sum[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          sum[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int v = 0; v < kXR; ++v)
#pragma unroll
            for (int f = 0; f < WT::kFragsPerGroup; ++f)
              sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[v][m][f], __builtin_bit_cast(bf16x8, one), sum[m], 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float s = bf16_f(st.w[r].s[h]);
          const float nz = -128.0f - (float)st.w[r].z[h];
          f32x4 part[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) part[m] = sum[m] * nz;
#pragma unroll
          for (int f = 0; f < WT::kFragsPerGroup; ++f) {
            const bf16x8 w = st.w[r].frag(h * WT::kFragsPerGroup + f);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int v = 0; v < kXR; ++v)
                part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[v][m][f], w, part[m], 0, 0, 0);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[r][m][i] = __builtin_fmaf(part[m][i], kScaled ? s * st.xs[m][i] : s, acc[r][m][i]);
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bf16x8 w = st.w[r].frag(h);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4& d = kScaled ? step_sum[r][m] : acc[r][m];
#pragma unroll
            for (int v = 0; v < kXR; ++v) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[v][m][0], w, d, 0, 0, 0);
          }
        }
      }
    }
    if constexpr (kScaled && !WT::kQuant) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][m][i] = __builtin_fmaf(step_sum[r][m][i], st.xs[m][i], acc[r][m][i]);
    }
  }

  // n = number of this wave's full steps, step(i) = first + i * by
  template <class XP>
  static __device__ __forceinline__ void run(f32x4 (&acc)[R][MT], const typename WT::Row (&rows)[R], const XP& xp,
                                             const XScale<MT>& sc, int q, int first, int by, int n_steps, int tail) {
    const int n = first < n_steps ? (n_steps - first + by - 1) / by : 0;
    if (n > 0) {
      Stage st[P];
#pragma unroll
      for (int p = 0; p < P; ++p) load<false>(st[p], rows, xp, sc, q, first + by * (p < n ? p : n - 1), kStep);
      int i = 0;
      for (; i + P < n; i += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          consume<false>(st[p], acc, kStep);
          const int nx = i + P + p;
          load<false>(st[p], rows, xp, sc, q, first + by * (nx < n ? nx : n - 1), kStep);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (i + p < n) consume<false>(st[p], acc, kStep);
    }
    if (tail && n_steps % by == first) {
      Stage st;
      load<true>(st, rows, xp, sc, q, n_steps, tail);
      consume<true>(st, acc, tail);
    }
  }
};

template <int KXR, int MT>
struct XPtr {
  const char* p[KXR][MT];
};

}  // namespace ops
}  // namespace fg
