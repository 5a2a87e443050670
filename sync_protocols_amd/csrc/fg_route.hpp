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

// One wave per token; lane l holds logits l * EPL + 0..EPL-1, so that the lowest
// lane with the maximum and the lowest of its elements are the lowest index.
template <int EPL, bool BF16>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  uint32_t key[EPL];
  float v[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane * EPL + j;
    key[j] = 0;
    v[j] = -__builtin_inff();
    if (e < a.experts) {
      const float x = BF16 ? bf16_f(((const uint16_t*)a.logits)[row * a.ld + e]) : ((const float*)a.logits)[row * a.ld + e];
      key[j] = order_key(x);
      v[j] = x == x ? x : -__builtin_inff();
    }
  }
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) best = key[j] > best ? key[j] : best;
  uint32_t top = wave_max(best);
  float m = 0.0f, denom = 1.0f;
  if (a.score == FG_SCORE_SOFTMAX) {
    m = key_value(top);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) s += v[j] == -__builtin_inff() ? 0.0f : expf(v[j] - m);
    denom = wave_sum(s);
  }
  float mine = 0.0f;        // lane j: score of the j-th pick
  int32_t mine_e = 0;
  float total = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int owner = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    int at = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) at = key[i] == top ? i : at;
    const int e = __shfl(lane * EPL + at, owner);
    const float l = key_value(top);
    float p = 0.0f;
    if (l != -__builtin_inff()) p = a.score == FG_SCORE_SOFTMAX ? expf(l - m) / denom : 1.0f / (1.0f + expf(-l));
    total += p;
    if (lane == j) { mine = p; mine_e = e; }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == at) key[i] = 0;
      best = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) best = key[i] > best ? key[i] : best;
    }
    top = wave_max(best);
  }
  if (lane < a.k) {
    a.topk[row * a.k + lane] = mine_e;
    a.weights[row * a.k + lane] = a.renorm ? (total == 0.0f ? 0.0f : mine / total * a.scale) : mine * a.scale;
  }
}

}  // namespace ops
}  // namespace fg
