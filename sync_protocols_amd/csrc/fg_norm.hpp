// Residual addition and RMS norm with bf16 and 8-bit outputs:
//   h = x + r,  y = h * (mean_n h^2 + eps)^(-1/2) * gamma   (fp32),
//   8 bits: a = max |y| over the row or over 128 columns, scale = a / Q,
//   q = rne(y Q / a), Q = 127 (int8) or 448 (e4m3), q = 0 where a = 0.
// One pass: a row lives in the registers of the threads that share it, so that
// x and r are read once and everything is written once; the memory rate bounds
// it: 8192 x 7168 with residual to e4m3 per 128 columns takes 79 us, 5.3 TB/s (a
// device copy reaches 4.9). One row takes 3.4 us, the latency of its steps.
// y is formed from the unrounded h: only what is stored is rounded.
#pragma once

#include "fg_ops.hpp"

namespace fg {
namespace ops {

struct NormArgs {
  const uint16_t* x; const uint16_t* res; const uint16_t* gamma;
  uint16_t* sum; uint16_t* y; uint8_t* q; float* scale;
  int64_t ldx, ldr, lds, ldy, ldq, rows;
  int32_t n, group;             // group: 0 (row) or 128
  int32_t q_type;
  float eps;
};

// Eight elements at p, `left` of them valid.
__device__ __forceinline__ void load8(const uint16_t* p, int left, float (&f)[8]) {
  if (left >= 8) {
    const u32x4 v = *(const u32x4_a2*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(v[i]); f[2 * i + 1] = bf16_hi(v[i]); }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < left ? bf16_f(p[i]) : 0.0f;
  }
}
// PAST: past the caches, for outputs larger than them.
template <bool PAST>
__device__ __forceinline__ void store8(uint16_t* p, int left, const float (&f)[8]) {
  if (left >= 8) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_bf16(f[2 * i], f[2 * i + 1]);
    if constexpr (PAST) __builtin_nontemporal_store(v, (u32x4_a2*)p);
    else *(u32x4_a2*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = f_bf16(f[i]);
  }
}

// Sum / maximum over the W waves that share a row. `buf` has W words; a buffer
// is used once per row, so one barrier per reduction is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = lanes_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += buf[i];
  }
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf) {
  v = lanes_max(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) v = buf[i] > v ? buf[i] : v;
  }
  return v;
}

// Q / a would leave fp32 for a below 2^-119, and make zeros NaN: numbers that small
// are taken by 2^100 first, exactly.
struct Inverse {
  float up, inv;
  __device__ __forceinline__ Inverse(float m, float top) {
    up = m < 0x1p-100f ? 0x1p100f : 1.0f;
    inv = m > 0.0f ? top / (m * up) : 0.0f;
  }
};

// Eight codes of one row from element e on. Q / a keeps |v| within a
// rounding of Q and the clamp takes that rounding off; a row (group) with a NaN or an
// infinity has a scale that says so, and its codes mean nothing.
template <bool PAST>
__device__ __forceinline__ void quantise8(const NormArgs& a, int64_t row, int e, int left, Inverse by, const float (&y)[8]) {
  u32x2 v = {0u, 0u};
  if (a.q_type == FG_I8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = __builtin_rintf(y[j] * by.up * by.inv);
      v[j / 4] |= ((uint32_t)(int)fminf(fmaxf(f, -127.0f), 127.0f) & 0xffu) << (8 * (j % 4));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = y[j + k] * by.up * by.inv;
        f[k] = f[k] > 448.0f ? 448.0f : f[k] < -448.0f ? -448.0f : f[k];
      }
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
      v[j / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
    }
  }
  uint8_t* p = a.q + row * a.ldq + e;
  if (left >= 8) {
    if constexpr (PAST) __builtin_nontemporal_store(v, (u32x2_a1*)p);
    else *(u32x2_a1*)p = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = (uint8_t)(v[j / 4] >> (8 * (j % 4)));
  }
}

// W waves per row; thread t of them holds elements 8 (t + 64 W i) + 0..7. Workgroups
// of one row, or of four where a wave has one to itself.
// The maximum is taken over the bit patterns of |y| as integers: their order is
// that of the numbers, and a NaN counts as larger than infinity, so that it
// reaches the scale instead of being dropped.
template <int W>
struct NormShape {
  static constexpr int kRows = W == 1 ? 4 : 1;
  static constexpr int kThreads = 64 * W * kRows;
};
template <int W, int V, bool PAST>
__global__ __launch_bounds__(NormShape<W>::kThreads) void add_rmsnorm_kernel(NormArgs a) {
  __shared__ float sbuf[W];
  __shared__ uint32_t mbuf[W];
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = W == 1 ? 4 * block + (threadIdx.x >> 6) : block;
  if (row >= a.rows) return;               // the same for all waves of a row
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 8 * (t + 64 * W * i);
    const int left = a.n - e;
    if (left > 0) {
      load8(a.x + row * a.ldx + e, left, h[i]);
      if (a.res) {
        float r[8];
        load8(a.res + row * a.ldr + e, left, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[i][j], h[i][j], ss);
  }
  ss = row_sum<W>(ss, sbuf);
  const float rstd = 1.0f / sqrtf(ss / (float)a.n + a.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 8 * (t + 64 * W * i);
    const int left = a.n - e;
    if (left > 0) {
      if (a.sum) store8<PAST>(a.sum + row * a.lds + e, left, h[i]);
      float g[8];
      load8(a.gamma + e, left, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rstd * g[j];
      if (a.y) store8<PAST>(a.y + row * a.ldy + e, left, h[i]);
      if (!a.q) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= left) continue;          // padding: 0 * rstd may be NaN
        const uint32_t b = __float_as_uint(h[i][j]) & 0x7fffffffu;
        amax = b > amax ? b : amax;
      }
    }
    if (a.q && a.group) {
      // 16 lanes hold one group of 128 columns (n is a multiple of 128)
      amax = lanes_max<16>(amax);
    }
    if (a.q && a.group && left > 0) {
      const float m = __uint_as_float(amax), top = a.q_type == FG_I8 ? 127.0f : 448.0f;
      if ((t & 15) == 0) a.scale[row * (a.n / 128) + e / 128] = m / top;
      quantise8<PAST>(a, row, e, left, Inverse(m, top), h[i]);
    }
    if (a.group) amax = 0;
  }
  if (a.q && !a.group) {
    const float m = __uint_as_float(row_max<W>(amax, mbuf)), top = a.q_type == FG_I8 ? 127.0f : 448.0f;
    if (t == 0) a.scale[row] = m / top;
    const Inverse by(m, top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 8 * (t + 64 * W * i);
      if (a.n - e > 0) quantise8<PAST>(a, row, e, a.n - e, by, h[i]);
    }
  }
}

}  // namespace ops
}  // namespace fg
