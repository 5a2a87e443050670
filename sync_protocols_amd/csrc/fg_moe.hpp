// The expert layer for few tokens, in two kernels:
//   y[t] = sum_j c[t][j] W2[e] (silu(W1[e][0:F] x[t]) * (W1[e][F:2F] x[t])),  e = topk[t][j] - expert_base,
// over the picks with 0 <= e < n_local (this GPU's experts); a token with none
// gets zeros. The weights of every picked expert are read once, which bounds it:
// one token over 8 bf16 experts of 7168 x 2048 takes 78 and 41 us, 5.9 TB/s; 64
// e4m3 tokens over 64 4-bit experts 388 us a pass (250 and 176 us under a tracer), of
// which the weight loads alone are 182 and 88.
//
// Every workgroup finds the picked experts and their tokens from topk by itself
// (at most 1024 picks, in LDS): that costs it a few hundred clocks, less than a
// launch of its own would. Kernel 1 forms c * silu(gate) * up per pick; it is
// kept as the sum of two bf16 numbers, so that the second product takes it on the
// matrix unit without the rounding of one bf16, which would be as large as that of
// the result. The two are within 2^-16 of it, which puts an rms error of 2.5e-6 into
// y, whose own rounding is 1.6e-3 (a third would make half as many bytes again of the
// reads that bound the second product). They are rows of their own in that product,
// next to each other, and their results are added: few picks, as a decoding step has
// per expert, leave half of the 16 rows of a matrix instruction
// free anyway. Kernel 2 sums all picks of a token in a fixed order.
#pragma once

#include "fg_w4.hpp"

namespace fg {
namespace ops {

constexpr int kMaxPicks = FG_MOE_FEW_TOKENS * FG_MOE_FEW_TOPK;

struct MoeArgs {
  const char* x; const float* xs; const int32_t* topk; const float* weights;
  const char* w1; const uint16_t* s1; const uint8_t* z1;
  const char* w2; const uint16_t* s2; const uint8_t* z2;
  char* h;                           // PackedRows: two rows a pick, by expert, by pick within an expert
  uint16_t* y;
  int64_t ldx, xs_stride, ldy;       // ldx in bytes
  int32_t tokens, k, base, n_local, K, F;
  uint32_t plane;                    // of h
};

// This GPU's expert of a pick, >= n_local for one that is not here (unsigned: no
// value of topk can overflow into range, n_local being at most 1024).
__device__ __forceinline__ uint32_t local_expert(int32_t pick, int32_t base) { return (uint32_t)pick - (uint32_t)base; }

template <int G, class Mat>
__device__ __forceinline__ Mat matrix(const char* w, const uint16_t* s, const uint8_t* z, int K) {
  if constexpr (G == 0) return Mat{w, 2 * (int64_t)K};
  else return Mat{w, s, z, K / 2, K / G};
}

// ---- kernel 1: workgroup (a, f) = 16 C columns of the a-th picked expert
template <int G, int XK, int MT, int C, int P, int W>
__device__ __forceinline__ void moe_up_pass(const MoeArgs& a, int e, int f0, const uint16_t* list, int start, int s0, int cnt, float* red) {
  typedef typename ProductOf<G, XK, MT, 2 * C, P>::T Prod;
  const Lanes ln;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const typename Prod::Mat mat = matrix<G, typename Prod::Mat>(a.w1, a.s1, a.z1, a.K).at((int64_t)e * 2 * a.F + f0);
  typename Prod::Row rows[2 * C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int f = min(16 * c + ln.load_row(), a.F - 1 - f0);
    rows[c].set(mat, f, ln);
    rows[C + c].set(mat, a.F + f, ln);
  }
  XPtr<MT> xp;
  xp.base = a.x;
  xp.scale = a.xs;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int slot = s0 + 16 * m + ln.load_row();
    const uint32_t token = list[min(slot, cnt - 1)] / a.k;
    xp.row[m] = !Prod::kMasked || slot < cnt ? token * (uint32_t)a.ldx + x_piece<G, XK>(ln) : kNoRow;
    xp.at[m] = token * (uint32_t)a.xs_stride;
  }
  f32x4 acc[2 * C][MT];
  clear<Prod>(acc);
  const int steps = a.K / kStep;
  run_steps<Prod>(acc, mat, rows, xp, ln, wave, W, (steps - wave + W - 1) / W);
  if (a.K % kStep && steps % W == wave) run_tail<Prod>(acc, mat, rows, xp, ln, steps, a.K % kStep);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (s0 + 16 * m >= cnt) break;
    constexpr int LD = 32 * C + 1;
#pragma unroll
    for (int r = 0; r < 2 * C; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(wave * 16 + 4 * ln.quarter + i) * LD + 16 * r + (ln.lane & 15)] = acc[r][m][i];
    __syncthreads();
    for (int o = threadIdx.x; o < 256 * C; o += 64 * W) {
      const int tok = o / (16 * C), col = o % (16 * C), slot = s0 + 16 * m + tok;
      if (slot >= cnt || f0 + col >= a.F) continue;
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        g += red[(w * 16 + tok) * LD + col];
        u += red[(w * 16 + tok) * LD + 16 * C + col];
      }
      const int p = list[slot];
      if constexpr (x_row_scaled(XK)) {
        const float s = a.xs[p / a.k];
        g *= s;
        u *= s;
      }
      const float h = g / (1.0f + expf(-g)) * u * a.weights[p];
      const uint16_t hi = f_bf16(h);
      char* to = a.h + PackedRows::at(2 * (start + slot), G == 0 ? f0 + col : paired_place(f0 + col), a.plane);
      *(uint16_t*)to = hi;
      // an infinite hi has no remainder
      *(uint16_t*)(to + 16) = fabsf(bf16_f(hi)) < __builtin_inff() ? f_bf16(h - bf16_f(hi)) : 0;
    }
    __syncthreads();
  }
}

template <int G, int XK, int MT, int C, int P, int W, int MIN_WAVES = (W > 8 ? W / 4 : 2)>
__global__ __launch_bounds__(64 * W, MIN_WAVES) void moe_up_kernel(MoeArgs a) {
  __shared__ uint32_t bits[FG_MOE_FEW_EXPERTS / 32];
  __shared__ uint16_t expert[kMaxPicks];   // of a pick; kElsewhere: not here
  __shared__ uint16_t list[kMaxPicks];
  __shared__ float red[W * 16 * (32 * C + 1)];
  constexpr uint32_t kElsewhere = 0xffffu;
  const int tid = threadIdx.x, lane = tid & 63;
  const int picks = a.tokens * a.k, ft = (a.F + 16 * C - 1) / (16 * C);
  const int nth = blockIdx.x / ft, f0 = (blockIdx.x % ft) * 16 * C;
  if (tid < FG_MOE_FEW_EXPERTS / 32) bits[tid] = 0;
  __syncthreads();
  for (int p = tid; p < picks; p += 64 * W) {
    const uint32_t e = local_expert(a.topk[p], a.base);
    const bool here = e < (uint32_t)a.n_local;
    expert[p] = (uint16_t)(here ? e : kElsewhere);
    if (here) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  // the nth set bit, in every wave
  const uint32_t word = lane < FG_MOE_FEW_EXPERTS / 32 ? bits[lane] : 0;
  int e = -1;
  for (int w = 0, left = nth; w < (a.n_local + 31) / 32; ++w) {
    uint32_t rest = (uint32_t)__builtin_amdgcn_readlane((int)word, w);
    if (left >= __popc(rest)) {
      left -= __popc(rest);
      continue;
    }
    for (; left > 0; --left) rest &= rest - 1;
    e = 32 * w + __ffs(rest) - 1;
    break;
  }
  if (e < 0) return;                       // fewer experts are picked; the same in every wave
  // its picks in order, and how many belong to experts before it: its place among h's rows
  int cnt = 0, start = 0;
  for (int p0 = 0; p0 < picks; p0 += 64) {
    const uint32_t l = p0 + lane < picks ? expert[p0 + lane] : kElsewhere;
    const unsigned long long here = __ballot(l == (uint32_t)e);
    if (tid < 64 && l == (uint32_t)e) list[cnt + __popcll(here & ((1ull << lane) - 1))] = (uint16_t)(p0 + lane);
    cnt += __popcll(here);
    start += __popcll(__ballot(l < (uint32_t)e));
  }
  __syncthreads();
  if (cnt <= 16 || MT == 1) {
    for (int s0 = 0; s0 < cnt; s0 += 16) moe_up_pass<G, XK, 1, C, P, W>(a, e, f0, list, start, s0, cnt, red);
  } else if constexpr (MT > 1) {
    for (int s0 = 0; s0 < cnt; s0 += 16 * MT) moe_up_pass<G, XK, MT, C, P, W>(a, e, f0, list, start, s0, cnt, red);
  }
}

// ---- kernel 2: workgroup = 16 R columns of y over every picked expert.
// Its work is a list of entries, each up to 8 MT picks (16 MT rows) of one expert,
// sorted by expert and within it by pick, as the rows of h are; the waves take
// equal, contiguous shares of the list's steps, so that they stay level whatever the
// number of experts. The rows of an entry's tile start at a multiple of four, the
// one before its first pick if that is odd: the 64 bytes that four lanes load are
// then one piece for the address unit (unaligned, the loads of h took twice as long).
struct DownPlan {
  unsigned long long mask[FG_MOE_FEW_EXPERTS];     // tokens that picked an expert
  uint16_t start[FG_MOE_FEW_EXPERTS];
  uint16_t ent_e[kMaxPicks], ent_s[kMaxPicks];     // entry: expert, first pick, picks
  uint8_t ent_c[kMaxPicks];
  uint8_t token[kMaxPicks];                        // of a pick
  int entries, again;
};

template <int MT, int W>
__device__ __forceinline__ void down_plan(const MoeArgs& a, DownPlan& pl) {
  constexpr int kMine = (kMaxPicks + 64 * W - 1) / (64 * W);
  const int tid = threadIdx.x, lane = tid & 63;
  const int picks = a.tokens * a.k;
  uint32_t mine[kMine];                            // experts of picks tid + 64 W i, n_local or more: not here
#pragma unroll
  for (int i = 0; i < kMine; ++i) mine[i] = tid + 64 * W * i < picks ? local_expert(a.topk[tid + 64 * W * i], a.base) : 0xffffffffu;
  for (int i = tid; i < a.n_local; i += 64 * W) pl.mask[i] = 0;
  if (tid == 0) pl.again = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const unsigned long long bit = 1ull << (((tid + 64 * W * i) / a.k) & 63);
    if (mine[i] < (uint32_t)a.n_local && (atomicOr(&pl.mask[mine[i]], bit) & bit)) pl.again = 1;
  }
  __syncthreads();
  const bool again = pl.again;     // some token picked an expert twice: the masks do not count it, so count here
  auto same_before = [&](uint32_t e, int end) {
    int n = 0;
    for (int p = 0; p < end; ++p) n += local_expert(a.topk[p], a.base) == e;
    return n;
  };
  if (tid < 64) {
    int at = 0, ent = 0;           // picks and entries before this block of 64 experts
    for (int e0 = 0; e0 < a.n_local; e0 += 64) {
      const int e = e0 + lane;
      const int c = e >= a.n_local ? 0 : again ? same_before(e, picks) : __popcll(pl.mask[e]);
      const int c_upto = lanes_before_and_own(c);
      const int start = at + c_upto - c, tile = start & ~1;
      const int n = c ? (start + c - tile + 8 * MT - 1) / (8 * MT) : 0;
      const int n_upto = lanes_before_and_own(n), first = ent + n_upto - n;
      for (int i = 0; i < n; ++i) {
        const int s = max(start, tile + 8 * MT * i);
        pl.ent_e[first + i] = (uint16_t)e;
        pl.ent_s[first + i] = (uint16_t)s;
        pl.ent_c[first + i] = (uint8_t)(min(start + c, tile + 8 * MT * (i + 1)) - s);
      }
      if (e < a.n_local) pl.start[e] = (uint16_t)start;
      at += __builtin_amdgcn_readlane(c_upto, 63);
      ent += __builtin_amdgcn_readlane(n_upto, 63);
    }
    if (lane == 0) pl.entries = ent;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (mine[i] >= (uint32_t)a.n_local) continue;
    const int p = tid + 64 * W * i, t = p / a.k;
    pl.token[pl.start[mine[i]] + (again ? same_before(mine[i], p) : __popcll(pl.mask[mine[i]] & ((1ull << t) - 1)))] = (uint8_t)t;
  }
  __syncthreads();
}

// Steps `step`..`end` - 1 of an entry with picks s..s + c - 1, into sums [token][16 R].
template <int G, int MT, int R, int P>
__device__ __forceinline__ void moe_down_pass(const MoeArgs& a, int e, int s, int c, int n0, int step, int end, const uint8_t* token,
                                              float* sums) {
  typedef typename ProductOf<G, X_PACKED, MT, R, P>::T Prod;
  const Lanes ln;
  const int col = ln.lane & 15, tile = s & ~1, full = a.F / kStep;
  const typename Prod::Mat mat = matrix<G, typename Prod::Mat>(a.w2, a.s2, a.z2, a.F).at((int64_t)e * a.K + n0);
  typename Prod::Row rows[R];
#pragma unroll
  for (int r = 0; r < R; ++r) rows[r].set(mat, min(16 * r + ln.load_row(), a.K - 1 - n0), ln);
  XPtr<MT> xp;
  xp.base = a.h;
  xp.plane = a.plane;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = 2 * tile + 16 * m + col;
    xp.row[m] = row >= 2 * s && row < 2 * (s + c) ? (uint32_t)PackedRows::at(row, 8 * ln.quarter, a.plane) : kNoRow;
  }
  f32x4 acc[R][MT];
  clear<Prod>(acc);
  run_steps<Prod>(acc, mat, rows, xp, ln, step, 1, min(end, full) - step);
  if (end > full) run_tail<Prod>(acc, mat, rows, xp, ln, full, a.F % kStep);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int pick = tile + (16 * m + 4 * ln.quarter + i) / 2;
      if (pick >= s && pick < s + c) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          unsafeAtomicAdd(&sums[token[pick] * 16 * R + 16 * r + col], acc[r][m][i] + acc[r][m][i + 1]);
      }
    }
}

template <int G, int MT, int R, int P, int W, int MIN_WAVES = (W > 8 ? W / 4 : 2)>
__global__ __launch_bounds__(64 * W, MIN_WAVES) void moe_down_kernel(MoeArgs a) {
  __shared__ DownPlan pl;
  extern __shared__ float sums[];                  // [wave][token][16 R]
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * R;
  for (int i = tid; i < W * a.tokens * 16 * R; i += 64 * W) sums[i] = 0.0f;
  down_plan<MT, W>(a, pl);
  const int steps = (a.F + kStep - 1) / kStep;
  const int64_t units = (int64_t)__builtin_amdgcn_readfirstlane(pl.entries) * steps;
  const int64_t from = units * wave / W, to = units * (wave + 1) / W;
  int ent = (int)(from / steps), step = (int)(from % steps);
  for (int64_t left = to - from; left > 0; ++ent, step = 0) {
    const int e = __builtin_amdgcn_readfirstlane(pl.ent_e[ent]), s = __builtin_amdgcn_readfirstlane(pl.ent_s[ent]);
    const int c = __builtin_amdgcn_readfirstlane(pl.ent_c[ent]);
    const int end = steps - step < left ? steps : step + (int)left;
    left -= end - step;
    float* to_sums = sums + wave * a.tokens * 16 * R;
    if (MT == 1 || (s & 1) + c <= 8) moe_down_pass<G, 1, R, P>(a, e, s, c, n0, step, end, pl.token, to_sums);
    else moe_down_pass<G, MT, R, P>(a, e, s, c, n0, step, end, pl.token, to_sums);
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * 16 * R; i += 64 * W) {
    const int t = i / (16 * R), n = n0 + i % (16 * R);
    if (n < a.K) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += sums[w * a.tokens * 16 * R + i];
      a.y[t * a.ldy + n] = f_bf16(v);
    }
  }
}

}  // namespace ops
}  // namespace fg
