// Router: the k largest of a token's E logits (equal ones: lowest index first)
// and their gate weights, in the form that TOPK routes, the combine and the
// expert layer for few tokens take:
//   p = softmax(l) over all E, or sigmoid(l);  w_j = p[i_j] * scale,
//   divided by sum_j p[i_j] if asked.
// The choice is made on the logits themselves (both scores are monotonic), so it
// does not depend on the rounding of an exponential.
#pragma once

#include "fg_ops.hpp"

namespace fg {
namespace ops {

struct RouteArgs {
  const void* logits;
  int32_t* topk;
  float* weights;
  int64_t ld, rows;
  int32_t experts, k, score, renorm;
  float scale;
};

// Order-preserving key: larger number, larger key; NaN below -inf, 0 left for
// "taken". x + 0 makes -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return x != x ? 1u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 1u ? -__builtin_inff() : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// The same of a bf16 number in the upper half, and below it `last`, which tells equal
// numbers apart; NaN has 1 in the upper half.
__device__ __forceinline__ uint32_t order_key(float x, uint32_t last) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (x != x ? 0x10000u : (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) & 0xffff0000u) | last;
}
__device__ __forceinline__ float key_value_bf16(uint32_t k) {
  return k >> 16 == 1u ? -__builtin_inff() : __uint_as_float((k & 0x80000000u ? k & 0x7fffffffu : ~k) & 0xffff0000u);
}

// N consecutive logits of which `left` exist, in one load where they all do (rows
// need no more than element alignment).
template <int N, bool BF16>
__device__ __forceinline__ void load_logits(const char* p, int left, float (&x)[N]) {
  constexpr int kBytes = BF16 ? 2 : 4, kWords = N * kBytes / 4 ? N * kBytes / 4 : 1;
  if (N * kBytes >= 4 && left >= N) {
    uint32_t w[kWords];
    __builtin_memcpy(w, p, sizeof w);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = BF16 ? (j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) : __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j >= left ? 0.0f : BF16 ? bf16_f(((const uint16_t*)p)[j]) : ((const float*)p)[j];
  }
}

// L lanes per token; lane l of them holds logits l * N + 0..N-1. A pick is the
// largest key of the lanes' largest and then the lowest index among those equal to
// it; a bf16 logit's key leaves 16 bits free, so there the key itself ends in the
// index, lowest largest, and one maximum finds both. 16 lanes with up to 16 logits
// each need the fewest instructions, which bound it (8192 tokens, 256 experts, 8 picks:
// 4.5 us bf16, 5.8 us fp32, of which a launch with its loads and one pick is 3.7; with
// 64 lanes of 4 logits 11.8 us); more experts take 64 lanes.
// Lane j % 16 keeps the j-th pick, so that scores are computed once, side by side.
template <int L, int N, bool BF16>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  const int l = threadIdx.x % L, l16 = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
  if (row >= a.rows) return;               // whole groups of lanes: reductions stay among those that are left
  const int e0 = l * N;
  uint32_t key[N];
  float v[N];
  load_logits<N, BF16>((const char*)a.logits + (row * a.ld + e0) * (BF16 ? 2 : 4), a.experts - e0, v);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (BF16) key[i] = order_key(v[i], 0xffffu - (uint32_t)(e0 + i));
    else key[i] = order_key(v[i]);
    v[i] = v[i] == v[i] ? v[i] : -__builtin_inff();
  }
  if (a.experts - e0 < N) {                // the logits that do not exist count as taken
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i >= a.experts - e0) {
        key[i] = 0;
        v[i] = -__builtin_inff();
      }
  }
  uint32_t best, at;
  auto find_best = [&]() {
    best = key[0];
    at = e0;
#pragma unroll
    for (int i = 1; i < N; ++i) {
      if constexpr (!BF16) at = key[i] > best ? e0 + i : at;
      best = key[i] > best ? key[i] : best;
    }
  };
  find_best();
  uint32_t top = lanes_max<L>(best);
  auto value = [](uint32_t t) { return BF16 ? key_value_bf16(t) : key_value(t); };
  float m = 0.0f, denom = 1.0f;
  if (a.score == FG_SCORE_SOFTMAX) {
    m = value(top);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) s += v[j] == -__builtin_inff() ? 0.0f : expf(v[j] - m);
    denom = lanes_sum<L>(s);
  }
  constexpr int kKept = 4;                 // 64 picks over 16 lanes
  uint32_t kept[kKept], kept_e[kKept];
#pragma unroll
  for (int g = 0; g < kKept; ++g) {
    kept[g] = BF16 ? 0x10000u : 1u;
    for (int j = 16 * g; j < min(a.k, 16 * g + 16); ++j) {
      const uint32_t e = BF16 ? 0xffffu - (top & 0xffffu) : lanes_min<L>(best == top ? at : 0xffffffffu);
      if (l16 == j % 16) {
        kept[g] = top;
        kept_e[g] = e;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = (BF16 ? key[i] == top : e == (uint32_t)(e0 + i)) ? 0 : key[i];
      find_best();
      top = lanes_max<L>(best);
    }
  }
  float p[kKept], total = 0.0f;
#pragma unroll
  for (int g = 0; g < kKept; ++g) {
    const float x = value(kept[g]);
    p[g] = 0.0f;
    if (16 * g < a.k && x != -__builtin_inff())
      p[g] = a.score == FG_SCORE_SOFTMAX ? expf(x - m) / denom : 1.0f / (1.0f + expf(-x));
    total += p[g];
  }
  total = lanes_sum<16>(total);
  if (l >= 16) return;
#pragma unroll
  for (int g = 0; g < kKept; ++g) {
    const int j = 16 * g + l;
    if (j >= a.k) break;
    a.topk[row * a.k + j] = (int32_t)kept_e[g];
    a.weights[row * a.k + j] = a.renorm ? (total == 0.0f ? 0.0f : p[g] / total * a.scale) : p[g] * a.scale;
  }
}

}  // namespace ops
}  // namespace fg
