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
  if (x != x) return 1u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 1u ? -__builtin_inff() : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// N consecutive logits of which `left` exist, in one load where they all do (rows
// need no more than element alignment); the others count as taken.
template <int N, bool BF16>
__device__ __forceinline__ void load_logits(const char* p, int left, uint32_t (&key)[N], float (&v)[N]) {
  constexpr int kBytes = BF16 ? 2 : 4, kWords = N * kBytes / 4 ? N * kBytes / 4 : 1;
  float x[N];
  if (N * kBytes >= 4 && left >= N) {
    uint32_t w[kWords];
    __builtin_memcpy(w, p, sizeof w);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = BF16 ? (j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2])) : __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j >= left ? 0.0f : BF16 ? bf16_f(((const uint16_t*)p)[j]) : ((const float*)p)[j];
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    key[j] = j < left ? order_key(x[j]) : 0;
    v[j] = j < left && x[j] == x[j] ? x[j] : -__builtin_inff();
  }
}

// L lanes per token; lane l of them holds logits l * N + 0..N-1. A pick is the
// largest key of the lanes' largest and then the lowest index among those equal to
// it. 16 lanes with up to 16 logits each need the fewest instructions (8192 tokens,
// 256 experts, 8 picks: 6.4 us; with 64 lanes of 4 logits 11.8 us); more experts take 64 lanes.
// Lane j % 16 keeps the j-th pick, so that scores are computed once, side by side.
template <int L, int N, bool BF16>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  const int l = threadIdx.x % L, l16 = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 / L) + threadIdx.x / L;
  if (row >= a.rows) return;               // whole groups of lanes: reductions stay among those that are left
  const int e0 = l * N;
  uint32_t key[N];
  float v[N];
  load_logits<N, BF16>((const char*)a.logits + (row * a.ld + e0) * (BF16 ? 2 : 4), a.experts - e0, key, v);
  uint32_t best, at;
  auto find_best = [&]() {
    best = key[0];
    at = e0;
#pragma unroll
    for (int i = 1; i < N; ++i) {
      at = key[i] > best ? e0 + i : at;
      best = key[i] > best ? key[i] : best;
    }
  };
  find_best();
  uint32_t top = lanes_max<L>(best);
  float m = 0.0f, denom = 1.0f;
  if (a.score == FG_SCORE_SOFTMAX) {
    m = key_value(top);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) s += v[j] == -__builtin_inff() ? 0.0f : expf(v[j] - m);
    denom = lanes_sum<L>(s);
  }
  constexpr int kKept = 4;                 // 64 picks over 16 lanes
  uint32_t kept[kKept], kept_e[kKept];
#pragma unroll
  for (int g = 0; g < kKept; ++g) {
    kept[g] = 1;
    for (int j = 16 * g; j < min(a.k, 16 * g + 16); ++j) {
      const uint32_t e = lanes_min<L>(best == top ? at : 0xffffffffu);
      if (l16 == j % 16) {
        kept[g] = top;
        kept_e[g] = e;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = e == (uint32_t)(e0 + i) ? 0 : key[i];
      find_best();
      top = lanes_max<L>(best);
    }
  }
  float p[kKept], total = 0.0f;
#pragma unroll
  for (int g = 0; g < kKept; ++g) {
    const float x = key_value(kept[g]);
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
