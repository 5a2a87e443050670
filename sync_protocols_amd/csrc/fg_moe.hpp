// The expert layer for few tokens, in two kernels:
//   y[t] = sum_j c[t][j] W2[e] (silu(W1[e][0:F] x[t]) * (W1[e][F:2F] x[t])),  e = topk[t][j] - expert_base,
// over the picks with 0 <= e < n_local (this GPU's experts); a token with none
// gets zeros. The weights of every picked expert are read once, which bounds it.
//
// Every workgroup finds the picked experts and their tokens from topk by itself
// (at most 1024 picks, in LDS): that costs it a few hundred clocks, less than a
// launch of its own would. Kernel 1 forms c * silu(gate) * up per pick; it is
// kept as the sum of two bf16 numbers (16 mantissa bits), so that the second
// product takes it on the matrix unit without the rounding of one bf16, which
// would be as large as that of the result. Kernel 2 sums all picks of a token in
// a fixed order.
#pragma once

#include "fg_w4.hpp"

namespace fg {
namespace ops {

constexpr int kMaxPicks = FG_MOE_FEW_TOKENS * FG_MOE_FEW_TOPK;

template <class WT>
struct MoeArgs {
  const char* x; const float* xs; const int32_t* topk; const float* weights;
  typename WT::Mat w1, w2;
  uint16_t* hi; uint16_t* lo;        // [tokens * k][F]
  uint16_t* y;
  int64_t ldx, xs_stride, ldy;       // ldx in bytes
  int32_t tokens, k, base, n_local, K, F, xs_step;
};

// This GPU's expert of a pick, >= n_local for one that is not here (unsigned: no
// value of topk can overflow into range, n_local being at most 1024).
__device__ __forceinline__ uint32_t local_expert(int32_t pick, int32_t base) { return (uint32_t)pick - (uint32_t)base; }

// ---- kernel 1: workgroup (a, f) = 16 columns of the a-th picked expert
template <class WT, int XK, int MT, int P>
__device__ __forceinline__ void moe_up_pass(const MoeArgs<WT>& a, int e, int f0, const uint16_t* list, int s0, int cnt, float* red) {
  typedef Product<WT, XK, MT, 2, P> Prod;
  const int lane = threadIdx.x & 63, q = lane >> 4, wave = threadIdx.x >> 6;
  const typename WT::Mat mat = a.w1.expert(e, 2 * (int64_t)a.F, a.K);
  const int f = min(f0 + (lane & 15), a.F - 1);
  typename WT::Row rows[2];
  rows[0].at(mat, f, q);
  rows[1].at(mat, a.F + f, q);
  XPtr<1, MT> xp;
  XScale<MT> sc;
  sc.step = a.xs_step;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    xp.p[0][m] = a.x + (int64_t)(list[min(s0 + 16 * m + (lane & 15), cnt - 1)] / a.k) * a.ldx;
    if constexpr (Prod::kScaled) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc.p[m][i] = a.xs + (int64_t)(list[min(s0 + 16 * m + 4 * q + i, cnt - 1)] / a.k) * a.xs_stride;
    }
  }
  f32x4 acc[2][MT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  Prod::run(acc, rows, xp, sc, q, wave, kProdWaves, a.K / kStep, a.K % kStep);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (s0 + 16 * m >= cnt) break;
    constexpr int LD = 33;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(wave * 16 + 4 * q + i) * LD + 16 * r + (lane & 15)] = acc[r][m][i];
    __syncthreads();
    const int tok = threadIdx.x >> 4, col = threadIdx.x & 15, slot = s0 + 16 * m + tok;
    if (threadIdx.x < 256 && slot < cnt && f0 + col < a.F) {
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int w = 0; w < kProdWaves; ++w) {
        g += red[(w * 16 + tok) * LD + col];
        u += red[(w * 16 + tok) * LD + 16 + col];
      }
      const int p = list[slot];
      const float h = g / (1.0f + __expf(-g)) * u * a.weights[p];
      const uint16_t hi = f_bf16(h);
      a.hi[(int64_t)p * a.F + f0 + col] = hi;
      // an infinite hi has no remainder
      a.lo[(int64_t)p * a.F + f0 + col] = fabsf(bf16_f(hi)) < __builtin_inff() ? f_bf16(h - bf16_f(hi)) : 0;
    }
    __syncthreads();
  }
}

template <class WT, int XK, int MT, int P>
__global__ __launch_bounds__(64 * kProdWaves) void moe_up_kernel(MoeArgs<WT> a) {
  __shared__ uint32_t bits[FG_MOE_FEW_EXPERTS / 32];
  __shared__ uint16_t list[kMaxPicks];
  __shared__ int count;
  __shared__ float red[kProdWaves * 16 * 33];
  const int tid = threadIdx.x, lane = tid & 63;
  const int picks = a.tokens * a.k, ft = (a.F + 15) / 16;
  const int nth = blockIdx.x / ft, f0 = (blockIdx.x % ft) * 16;
  if (tid < FG_MOE_FEW_EXPERTS / 32) bits[tid] = 0;
  if (tid == 0) count = 0;
  __syncthreads();
  for (int p = tid; p < picks; p += 64 * kProdWaves) {
    const uint32_t e = local_expert(a.topk[p], a.base);
    if (e < (uint32_t)a.n_local) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  // the nth set bit, in every wave
  const uint32_t word = lane < FG_MOE_FEW_EXPERTS / 32 ? bits[lane] : 0;
  int upto = __popc(word);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  const unsigned long long past = __ballot(upto > nth);
  if (!past) return;                       // fewer experts are picked; the same in every wave
  const int at = __ffsll(past) - 1;
  uint32_t rest = __shfl(word, at);
  for (int i = nth - (__shfl(upto, at) - __popc(rest)); i > 0; --i) rest &= rest - 1;
  const int e = __builtin_amdgcn_readfirstlane(32 * at + __ffs(rest) - 1);
  // its picks, in no particular order: each is a row of its own in the products
  for (int p = tid; p < picks; p += 64 * kProdWaves)
    if (local_expert(a.topk[p], a.base) == (uint32_t)e) list[atomicAdd(&count, 1)] = (uint16_t)p;
  __syncthreads();
  const int cnt = count;
  if (cnt <= 16 || MT == 1) {
    for (int s0 = 0; s0 < cnt; s0 += 16) moe_up_pass<WT, XK, 1, P>(a, e, f0, list, s0, cnt, red);
  } else if constexpr (MT > 1) {
    for (int s0 = 0; s0 < cnt; s0 += 16 * MT) moe_up_pass<WT, XK, MT, 2>(a, e, f0, list, s0, cnt, red);
  }
}

// ---- kernel 2: workgroup = 16 R columns of y over every picked expert
template <class WT, int MT, int R, int P, bool TAIL>
__global__ __launch_bounds__(64 * kProdWaves) void moe_down_kernel(MoeArgs<WT> a) {
  typedef Product<WT, X_SPLIT, MT, R, P> Prod;
  __shared__ int cnt[FG_MOE_FEW_EXPERTS];          // picks of an expert; then where its next pick goes
  __shared__ uint16_t order[kMaxPicks];            // picks sorted by expert
  __shared__ uint16_t ent_e[kMaxPicks], ent_s[kMaxPicks];   // entries: up to 16 MT picks of one expert
  __shared__ uint8_t ent_c[kMaxPicks];
  __shared__ int entries;
  extern __shared__ float sums[];                  // [wave][token][16 R]
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, wave = tid >> 6, col = lane & 15;
  const int picks = a.tokens * a.k, n0 = blockIdx.x * 16 * R;
  for (int i = tid; i < a.n_local; i += 64 * kProdWaves) cnt[i] = 0;
  for (int i = tid; i < kProdWaves * a.tokens * 16 * R; i += 64 * kProdWaves) sums[i] = 0.0f;
  __syncthreads();
  for (int p = tid; p < picks; p += 64 * kProdWaves) {
    const uint32_t e = local_expert(a.topk[p], a.base);
    if (e < (uint32_t)a.n_local) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int at = 0, ent = 0;                           // picks and entries before this block of 64 experts
    for (int e0 = 0; e0 < a.n_local; e0 += 64) {
      const int e = e0 + lane, c = e < a.n_local ? cnt[e] : 0, n = (c + 16 * MT - 1) / (16 * MT);
      int cs = c, ns = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(cs, d), w = __shfl_up(ns, d);
        if (lane >= d) { cs += o; ns += w; }
      }
      const int start = at + cs - c, first = ent + ns - n;
      for (int i = 0; i < n; ++i) {
        ent_e[first + i] = (uint16_t)e;
        ent_s[first + i] = (uint16_t)(start + 16 * MT * i);
        ent_c[first + i] = (uint8_t)min(c - 16 * MT * i, 16 * MT);
      }
      if (e < a.n_local) cnt[e] = start;
      at += __shfl(cs, 63);
      ent += __shfl(ns, 63);
    }
    if (lane == 0) entries = ent;
  }
  __syncthreads();
  for (int p = tid; p < picks; p += 64 * kProdWaves) {
    const uint32_t e = local_expert(a.topk[p], a.base);
    if (e < (uint32_t)a.n_local) order[atomicAdd(&cnt[e], 1)] = (uint16_t)p;
  }
  __syncthreads();

  // The waves take the steps of all entries in turn, one list end to end, so
  // that they stay level whatever the number of experts, with P steps in flight
  // across the borders between experts.
  const int n_ent = __builtin_amdgcn_readfirstlane(entries);
  const int steps = (a.F + kStep - 1) / kStep;
  const int units = n_ent * steps;
  const int mine = wave < units ? (units - wave + kProdWaves - 1) / kProdWaves : 0;
  f32x4 acc[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  XScale<MT> sc;
  sc.step = 0;
  auto load = [&](typename Prod::Stage& st, int ent, int step) {
    const int e = __builtin_amdgcn_readfirstlane(ent_e[ent]), s = ent_s[ent], c = ent_c[ent];
    const typename WT::Mat mat = a.w2.expert(e, a.K, a.F);
    typename WT::Row rows[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rows[r].at(mat, min(n0 + 16 * r + col, a.K - 1), q);
    XPtr<2, MT> xp;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t p = order[s + min(16 * m + col, c - 1)];
      xp.p[0][m] = (const char*)(a.hi + p * a.F);
      xp.p[1][m] = (const char*)(a.lo + p * a.F);
    }
    Prod::template load<TAIL>(st, rows, xp, sc, q, step, TAIL ? a.F - step * kStep : kStep);
  };
  auto flush = [&](int ent) {
    const int s = ent_s[ent], c = ent_c[ent];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = 16 * m + 4 * q + i;
        if (slot < c) {
          const int t = order[s + slot] / a.k;
#pragma unroll
          for (int r = 0; r < R; ++r)
            unsafeAtomicAdd(&sums[(wave * a.tokens + t) * 16 * R + 16 * r + col], acc[r][m][i]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][m][i] = 0.0f;
      }
  };
  if (mine > 0) {
    int le = wave / steps, ls = wave % steps;      // next unit to load
    int ce = le, cs = ls, loaded = 0;              // next unit to consume
    typename Prod::Stage st[P];
    auto next = [&](typename Prod::Stage& to) {    // past the end: the last unit again, unused
      load(to, le, ls);
      if (++loaded < mine) {
        ls += kProdWaves;
        while (ls >= steps) { ls -= steps; ++le; }
      }
    };
    auto use = [&](const typename Prod::Stage& from) {
      Prod::template consume<TAIL>(from, acc, TAIL ? a.F - cs * kStep : kStep);
      const int was = ce;
      cs += kProdWaves;
      while (cs >= steps) { cs -= steps; ++ce; }
      if (ce != was) flush(was);
    };
#pragma unroll
    for (int p = 0; p < P; ++p) next(st[p]);
    int i = 0;
    for (; i + P < mine; i += P) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        use(st[p]);
        next(st[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (i + p < mine) use(st[p]);
    // entries a wave leaves between its last step and the end are flushed by use();
    // the last one is flushed there too, since the next unit lies past it
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * 16 * R; i += 64 * kProdWaves) {
    const int t = i / (16 * R), n = n0 + i % (16 * R);
    if (n < a.K) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kProdWaves; ++w) v += sums[(w * a.tokens) * 16 * R + i];
      a.y[t * a.ldy + n] = f_bf16(v);
    }
  }
}

}  // namespace ops
}  // namespace fg
