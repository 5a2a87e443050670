// Work of attention over a paged cache, split over the cache's length.
//
// The lengths are on the GPU, so the split is made there: the requests' tokens, in
// units of U, stand one after the other, and every workgroup takes an equal number of
// consecutive ones, be they part of one request or of many. All workgroups then have the same work whatever the lengths (pieces of one request each,
// cut as evenly as 64 uneven lengths allow, left a latent cache's workgroups 30 %
// of the time without any). Every workgroup finds its own units from the lengths by sums
// over them, which takes less than a launch. A request without tokens counts as one unit, so
// that its outputs are written too. Pieces of one request that has several leave their
// sums (running maximum, sum of weights, weighted sum) in the workspace at place w + request, which no other
// piece has and which is consecutive for a request; join_kernel adds them up in order.
#pragma once

#include "fg_entry.hpp"
#include "fg_ops.hpp"

namespace fg {
namespace ops {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kNone = -__builtin_inff();
// The running maximum is only raised when a score exceeds it by more than this (in powers of two): a weight is then up to
// 2^8, which costs no accuracy, and the weighted sums are rescaled a few times a request instead of every tile.
constexpr float kSlack = 8.0f;

struct SplitArgs {
  const int32_t* lens;
  const int32_t* table;
  int64_t ldt;                       // entries
  int32_t batch, width, n_pages, page;
  int32_t window;                    // 0: all tokens
  int32_t target;                    // workgroups, at most one a unit
  int32_t* pieces;                   // workspace: {first place, number of pieces} of every request
};

struct SplitShared {
  int32_t sum[16], found[2];
};

__device__ __forceinline__ int seen_tokens(const SplitArgs& a, int b, int& first) {
  const int64_t most = (int64_t)a.width * a.page;
  int len = a.lens[b];
  len = len < 0 ? 0 : len > most ? (int)most : len;
  first = a.window > 0 && len > a.window ? len - a.window : 0;
  return len;
}
// Up to 2^31 - 1 tokens in steps of N.
template <int N>
__device__ __forceinline__ int steps_of(int tokens) { return (int)(((uint32_t)tokens + (N - 1)) / N); }
template <int U>
__device__ __forceinline__ int units_of(const SplitArgs& a, int b) {
  int first;
  const int len = seen_tokens(a, b, first);
  return max(1, steps_of<U>(len - (first & ~15)));
}

// The pieces of one workgroup, one after the other.
template <int U>
struct Pieces {
  int b;                             // request
  int begin, end;                    // tokens, begin a multiple of 16 (of U without a window)
  int first, len;                    // first token that is seen, tokens of the request
  int place, count;                  // of this piece's sums; pieces of this request
  int w, share, more;                // workgroup; its units, one more for the first `more` workgroups
  int at, left, skip;                // units: before this request, still to do, of this request before this piece

  __device__ __forceinline__ int owner(int unit) const {
    const uint32_t u = unit, big = (uint32_t)more * (uint32_t)(share + 1);
    return (int)(u < big ? u / (uint32_t)(share + 1) : more + (u - big) / (uint32_t)share);
  }

  // T threads, all of them call it; false: nothing to do. `w`: this workgroup's number.
  template <int T>
  __device__ __forceinline__ bool find(const SplitArgs& a, int w_, SplitShared& sh) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.batch + T - 1) / T, from = min(tid * per, a.batch), to = min(from + per, a.batch);
    int mine = 0;
    for (int i = from; i < to; ++i) mine += units_of<U>(a, i);
    int upto = lanes_before_and_own(mine);
    if (lane == 63) sh.sum[wave] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      if (i < wave) upto += sh.sum[i];
      total += sh.sum[i];
    }
    total = __builtin_amdgcn_readfirstlane(total);
    w = w_;
    const int n = min(a.target, total);
    if (w >= n) return false;
    share = total / n;
    more = total - n * share;
    const int start = w * share + min(w, more);
    if (start < upto && start >= upto - mine) {
      int before = upto - mine;
      for (int i = from; i < to; ++i) {
        const int u = units_of<U>(a, i);
        if (start < before + u) {
          sh.found[0] = i;
          sh.found[1] = before;
          break;
        }
        before += u;
      }
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(sh.found[0]);
    at = __builtin_amdgcn_readfirstlane(sh.found[1]);
    left = share + (w < more ? 1 : 0);
    skip = start - at;
    take(a, tid);
    return true;
  }
  __device__ __forceinline__ void take(const SplitArgs& a, int tid) {
    len = __builtin_amdgcn_readfirstlane(seen_tokens(a, b, first));
    first = __builtin_amdgcn_readfirstlane(first);
    const int origin = first & ~15, u = max(1, steps_of<U>(len - origin)), mine = min(left, u - skip);
    begin = origin + U * skip;
    end = mine == u - skip ? len : begin + U * mine;
    const int w0 = owner(at), w1 = owner(at + u - 1);
    place = w + b;
    count = w1 - w0 + 1;
    if (skip == 0 && tid == 0) {
      a.pieces[2 * b] = place;
      a.pieces[2 * b + 1] = count;
    }
    left -= mine;
    at += u;
    skip = 0;
  }
  __device__ __forceinline__ bool next(const SplitArgs& a, int tid) {
    if (left == 0) return false;
    ++b;
    take(a, tid);
    return true;
  }
};

// v as the sum of two bf16 numbers, within 2^-16 of it: the first is v rounded, this the rest (none beside an infinity).
__device__ __forceinline__ float bf16_rest(float v) {
  const float hi = bf16_f(f_bf16(v));
  return fabsf(hi) < __builtin_inff() ? v - hi : 0.0f;
}

// Sum of a head's pieces: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, in order. A wave has C columns of one request and head and
// asks for 16 pieces at once. Where a request may have more pieces than that, K waves share them and other columns are other
// workgroups', since one compute unit takes long for a row's megabyte (16 heads of 256 pieces and 512 columns: 16 workgroups 19.7 us, 128 of
// them 5.6). A request of one piece has been written by it.
struct JoinArgs {
  const int32_t* pieces;
  const float* part;                 // [places][heads][D]
  const float* ml;                   // [places][heads][2]: maximum (base 2), sum of weights
  uint16_t* out;
  float* lse;                        // or null
  int64_t out_b, out_h, lse_b;       // elements
  int32_t heads;
};

template <int D, bool MANY>
struct JoinShape {
  static constexpr int K = MANY ? 8 : 1, C = MANY || D < 128 ? 64 : 128;
  static constexpr int PARTS = D / C;                          // of a row's columns: workgroups, or waves of one
  static constexpr int WAVES = MANY ? K : PARTS, Z = MANY ? PARTS : 1;
};
template <int D, bool MANY>
__global__ __launch_bounds__((64 * JoinShape<D, MANY>::WAVES)) void join_kernel(JoinArgs a) {
  typedef JoinShape<D, MANY> Sh;
  constexpr int K = Sh::K, C = Sh::C, N = C / 64, B = 16;
  __shared__ float red[K][C], top[K], sum[K];
  const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = MANY ? wave : 0, col = C * (MANY ? blockIdx.z : wave) + N * lane;
  const int first = a.pieces[2 * b], n = a.pieces[2 * b + 1];
  if (n < 2) return;
  float m = kNone, l = 0.0f, o[N] = {};
  for (int i = k; i < n; i += K * B) {
    float pm[B], pl[B], po[B][N];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int at = i + j * K;
      const int64_t row = (int64_t)(first + (at < n ? at : i)) * a.heads + h;
      const float2 v = *(const float2*)(a.ml + 2 * row);
      pm[j] = at < n ? v.x : kNone;
      pl[j] = v.y;
#pragma unroll
      for (int e = 0; e < N; ++e) po[j][e] = a.part[row * D + col + e];
    }
    float t = m;
#pragma unroll
    for (int j = 0; j < B; ++j) t = pm[j] > t || pm[j] != pm[j] ? pm[j] : t;
    if (t == kNone) continue;
    const float f = exp2f(m - t);
    l *= f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= f;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (pm[j] == kNone) continue;
      const float g = exp2f(pm[j] - t);
      l = __builtin_fmaf(g, pl[j], l);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = __builtin_fmaf(g, po[j][e], o[e]);
    }
    m = t;
  }
  if constexpr (K > 1) {
    if (lane == 0) {
      top[k] = m;
      sum[k] = l;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) red[k][N * lane + e] = o[e];
    __syncthreads();
    if (k != 0) return;
    float t = kNone;
#pragma unroll
    for (int w = 0; w < K; ++w) t = top[w] > t || top[w] != top[w] ? top[w] : t;
    m = t;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < K; ++w) {
      if (top[w] == kNone) continue;
      const float g = exp2f(top[w] - t);
      l = __builtin_fmaf(g, sum[w], l);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = __builtin_fmaf(g, red[w][N * lane + e], o[e]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* to = a.out + b * a.out_b + h * a.out_h + col;
#pragma unroll
  for (int e = 0; e < N; ++e) to[e] = f_bf16(o[e] * inv);
  if (a.lse && col == 0) a.lse[b * a.lse_b + h] = l == 0.0f ? kNone : (m + log2f(l)) / kLog2E;
}

// MANY where requests have more than 16 pieces if their lengths are even.
template <int D, bool MANY>
void launch_join_as(const JoinArgs& a, int64_t batch, Launches& go) {
  typedef JoinShape<D, MANY> Sh;
  go(join_kernel<D, MANY>, dim3((unsigned)a.heads, (unsigned)batch, Sh::Z), dim3(64 * Sh::WAVES), 0, a);
}
template <int D>
void launch_join(const JoinArgs& a, int64_t batch, int target, Launches& go) {
  target > 16 * batch ? launch_join_as<D, true>(a, batch, go) : launch_join_as<D, false>(a, batch, go);
}

}  // namespace ops
}  // namespace fg
