// Products of few activation rows with 4-bit weights:
//   out[t][n] = sum_k x[t][k] xs[t][k / 128 or 0] (q[n][k] - z[n][k / G]) s[n][k / G] + bias[n].
// A workgroup owns 16 R weight rows over the whole K: its waves take the steps
// of 128 k in turn, so that together they stream whole lines of every row, and
// their fp32 sums are joined through LDS in wave order (the result does not
// depend on timing). No workspace, one launch.
// The weights' bytes are the floor, and with 4 bits a weight the arithmetic is near
// it: 64 rows x 8192 x 8192, groups of 64, int8 rows take 19 us (38 MB, 5.4 us at
// the rate of streaming reads; loads alone 17, arithmetic alone 14), 5 x 8199 x 7200,
// groups of 32 with zero points, 16.5 us (loads alone 14, arithmetic alone 12), one
// row x 2048 x 7168 5.6 us, the latency of a few dependent steps.
#pragma once

#include "fg_ops.hpp"

namespace fg {
namespace ops {

struct W4Args {
  const char* x; const float* xs; const char* w; const uint16_t* s; const uint8_t* z; const uint16_t* bias;
  uint16_t* out;
  int64_t ldx, xs_stride, ldo;      // ldx in bytes
  int32_t rows, n, k;
};

// Joins the sums that W waves have of one tile of 16 tokens x 16 R columns and
// hands each element to `put(token, column, value)`; red: W * 16 * (16 R + 1) floats.
template <int R, int MT, int W, class Put>
__device__ __forceinline__ void join_tile(const f32x4 (&acc)[R][MT], int m, float* red, Put put) {
  constexpr int LD = 16 * R + 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(wave * 16 + 4 * (lane >> 4) + i) * LD + 16 * r + (lane & 15)] = acc[r][m][i];
  __syncthreads();
  for (int e = threadIdx.x; e < 256 * R; e += 64 * W) {
    const int tok = e / (16 * R), col = e % (16 * R);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[(w * 16 + tok) * LD + col];
    put(tok, col, v);
  }
  __syncthreads();
}

template <int G, int XK, int MT, int R, int P, int W, int MIN_WAVES = (W > 8 ? W / 4 : 2)>
__global__ __launch_bounds__(64 * W, MIN_WAVES) void w4_linear_kernel(W4Args a) {
  __shared__ float red[W * 16 * (16 * R + 1)];
  typedef Quant4<G, XK, MT, R, P> Prod;
  const Lanes ln;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * R, t0 = blockIdx.y * 16 * MT;
  const typename Prod::Mat mat = typename Prod::Mat{a.w, a.s, a.z, a.k / 2, a.k / G}.at(n0);
  typename Prod::Row rows[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int last = a.n - 1 - n0;
    rows[r].set(mat, min(16 * r + ln.load_row(), last), ln);
  }
  XPtr<MT> xp;
  xp.base = a.x + t0 * a.ldx;
  xp.scale = a.xs + t0 * a.xs_stride;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const uint32_t row = (uint32_t)min(16 * m + ln.load_row(), a.rows - 1 - t0);
    if constexpr (XK == X_LDS) xp.row[m] = 16 * ln.quarter;
    else xp.row[m] = 16 * m + ln.load_row() < a.rows - t0 ? row * (uint32_t)a.ldx + x_piece<G, XK>(ln) : kNoRow;
    xp.at[m] = row * (uint32_t)a.xs_stride;
  }
  if constexpr (XK == X_LDS) copy_row_to_lds(a.x, a.k, 64 * W);
  f32x4 acc[R][MT];
  clear<Prod>(acc);
  const int steps = a.k / kStep;
  run_steps<Prod>(acc, mat, rows, xp, ln, wave, W, (steps - wave + W - 1) / W);
  if (a.k % kStep && steps % W == wave) run_tail<Prod>(acc, mat, rows, xp, ln, steps, a.k % kStep);
#pragma unroll
  for (int m = 0; m < MT; ++m)
    join_tile<R, MT, W>(acc, m, red, [&](int tok, int col, float v) {
      const int t = t0 + 16 * m + tok, n = n0 + col;
      if (t < a.rows && n < a.n) {
        if constexpr (x_row_scaled(XK)) v *= a.xs[t];
        a.out[t * a.ldo + n] = f_bf16(a.bias ? v + bf16_f(a.bias[n]) : v);
      }
    });
}

}  // namespace ops
}  // namespace fg
