// Attention of one new token over a paged cache:
//   out[b][h] = sum_t w_t v_t / sum_t w_t,  w_t = 2^(c s_t - m),  s_t = q[b][h] . k_t,  c = scale log2(e),
// m a running maximum of c s_t. Every key and value is read once for the `group`
// heads that share it, 4 group flops a value and 2 bytes, so memory bounds it up
// to about 128 heads a key.
//
// A wave takes 32 tokens at a time with 16 HT heads, and both products are
// 16x16x32 matrix instructions whose result has the head in the lane:
//   S^T[token][head] = K Q^T     K: lane l holds 8 dims of token l % 16, straight from memory
//   O^T[dim][head] += V^T P^T    P: what lane l has of S^T is tokens 4 (l / 16) + 0..3 of both blocks of 16,
//                                which is a legal k order of the second product if V^T has the same
// so weights never leave their lane, the maximum and the sum of a head stay in the
// lanes of that head, and nothing goes through LDS but the join of the waves. V^T
// needs 8 tokens of one dim in a lane: a lane loads D / 16 consecutive dims of its 8 tokens (16
// lanes a whole row) and one byte permutation per pair of tokens and dim turns them.
// The lane's i-th dim goes to the i-th matrix instruction. Loads of the next
// keys and of the values are in flight while a tile is computed.
// Weights are rounded to bf16 for the second product (2^-8 relative at most, random over tokens; the sum of weights takes the unrounded ones).
#pragma once

#include "fg_split.hpp"

namespace fg {
namespace ops {

struct PagedArgs {
  SplitArgs split;
  const char* q;
  const char* k;
  const char* v;
  const float* ks;                   // [n_pages][kv][page] or null
  const float* vs;
  uint16_t* out;
  float* lse;
  float* part;
  float* ml;
  int64_t q_b, q_h, out_b, out_h, lse_b;        // q in bytes, outputs in elements
  int64_t k_page, v_page, k_head, v_head;       // bytes
  int32_t k_tok, v_tok;                         // bytes
  int32_t kv, group, heads;
  float c;                                      // scale log2(e)
};

constexpr int kPagedWaves = 4, kPagedUnit = 32 * kPagedWaves;

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&to)[W], const char* p) {
  if constexpr (W == 1) {
    to[0] = *(const uint32_t*)p;
  } else if constexpr (W == 2) {
    const u32x2 v = *(const u32x2*)p;
    to[0] = v[0];
    to[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const u32x4 v = *(const u32x4*)(p + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) to[i + j] = v[j];
    }
  }
}

// Two blocks of 16 tokens: where they lie, and which of their tokens count.
struct Blocks {
  int64_t page[2];
  int32_t at[2];                     // token within its page
  int32_t lo[2], hi[2];
  __device__ __forceinline__ bool full() const { return lo[0] <= 0 && lo[1] <= 0 && hi[0] >= 16 && hi[1] >= 16; }
};

template <int D, bool E4M3, int HT>
struct PagedTile {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int KS = D / 32;             // matrix instructions of a score
  static constexpr int KL = D * ES / 64;        // 16-byte loads of a lane's share of a key
  static constexpr int NV = D / 16;             // dims of a value that a lane loads
  static constexpr int VW = NV * ES / 4;
  u32x4 k[2][KL];
  uint32_t v[8][VW];
  f32x4 ks[2], vs[2];

  // 32 ks + 8 (l / 16), or with 16 codes a load 64 (ks / 2) + 16 (l / 16) + 8 (ks % 2)
  static __device__ __forceinline__ int q_dim(int ks_, int quarter) {
    return E4M3 ? 64 * (ks_ / 2) + 16 * quarter + 8 * (ks_ % 2) : 32 * ks_ + 8 * quarter;
  }
  __device__ __forceinline__ void load_k(const PagedArgs& a, const Blocks& x, int h, int m, int quarter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* base = a.k + x.page[i] * a.k_page + (int64_t)x.at[i] * a.k_tok + h * a.k_head;
      const uint32_t off = (uint32_t)(m * a.k_tok + 16 * quarter);
#pragma unroll
      for (int j = 0; j < KL; ++j) k[i][j] = *(const u32x4*)(base + off + 64 * j);
      if constexpr (E4M3) ks[i] = *(const f32x4*)(a.ks + (x.page[i] * a.kv + h) * a.split.page + x.at[i] + 4 * quarter);
    }
  }
  __device__ __forceinline__ void load_v(const PagedArgs& a, const Blocks& x, int h, int m, int quarter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char* base = a.v + x.page[i] * a.v_page + (int64_t)x.at[i] * a.v_tok + h * a.v_head;
#pragma unroll
      for (int t = 0; t < 4; ++t) load_words<VW>(v[4 * i + t], base + (uint32_t)((4 * quarter + t) * a.v_tok + m * NV * ES));
      if constexpr (E4M3) vs[i] = *(const f32x4*)(a.vs + (x.page[i] * a.kv + h) * a.split.page + x.at[i] + 4 * quarter);
    }
  }
  __device__ __forceinline__ bf16x8 key(int i, int ks_) const {
    if constexpr (E4M3) {
      const u32x4 w = k[i][ks_ / 2];
      return widen8<false>(ks_ % 2 ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]});
    } else {
      return __builtin_bit_cast(bf16x8, k[i][ks_]);
    }
  }
  // dims j and j + 1 (j even) of the lane's eight tokens
  __device__ __forceinline__ void values(int j, bf16x8& a, bf16x8& b) const {
    u32x4 x, y;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (E4M3) {
        const uint32_t w = __builtin_amdgcn_perm(v[2 * t + 1][j / 4], v[2 * t][j / 4], j % 4 ? 0x07030602u : 0x05010400u);
        x[t] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
        y[t] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
      } else {
        x[t] = __builtin_amdgcn_perm(v[2 * t + 1][j / 2], v[2 * t][j / 2], 0x05040100u);
        y[t] = __builtin_amdgcn_perm(v[2 * t + 1][j / 2], v[2 * t][j / 2], 0x07060302u);
      }
    }
    a = __builtin_bit_cast(bf16x8, x);
    b = __builtin_bit_cast(bf16x8, y);
  }
};

// A page that is not the cache's, or none, has no tokens. Lane l holds page and place of the l-th block from `block0` on; the table is read up to the
// request's last token (which lies within its width).
struct BlockList {
  int32_t page, at, block0;
  __device__ __forceinline__ void fetch(const SplitArgs& s, int b, int len, int block, int lane) {
    block0 = block;
    const int64_t t = 16 * (int64_t)(block + lane);
    const int64_t i = t / s.page;
    at = (int32_t)(t - i * s.page);
    page = t < len ? s.table[b * s.ldt + i] : -1;
  }
  template <class P>
  __device__ __forceinline__ Blocks get(const SplitArgs& s, const P& p, int block) const {
    Blocks x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t id = __builtin_amdgcn_readlane(page, block - block0 + i);
      const bool there = id >= 0 && id < s.n_pages;
      x.page[i] = there ? id : 0;
      x.at[i] = there ? __builtin_amdgcn_readlane(at, block - block0 + i) : 0;
      x.lo[i] = max(p.first - 16 * (block + i), 0);
      x.hi[i] = there ? min(p.len - 16 * (block + i), 16) : 0;
    }
    return x;
  }
};

// Largest of the four lanes that share l % 16.
__device__ __forceinline__ float quarters_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quarters_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int D, bool E4M3, int HT>
__global__ __launch_bounds__(64 * kPagedWaves) void paged_kernel(PagedArgs a) {
  typedef PagedTile<D, E4M3, HT> Tile;
  constexpr int NV = Tile::NV, KS = Tile::KS, W = kPagedWaves;
  constexpr int DP = D < 128 ? D : 128;         // columns of the waves' join at a time
  __shared__ SplitShared sh;
  __shared__ float top[W][16 * HT], sum[W][16 * HT];
  __shared__ float red[W][16][DP + 4];
  Pieces<kPagedUnit> p;
  // workgroups go round the 8 dies: those that share rows, with other heads, are neighbours on one die, and the second one's rows come from its L2
  // (2 of them, 16 requests of 65536 tokens: 197 us with neighbours on different dies, 143)
  const int tiles = (a.group + 16 * HT - 1) / (16 * HT), turn = blockIdx.x >> 3, shares = (a.split.target + 7) >> 3, h = turn / tiles / shares, tile = turn % tiles;
  if (!p.template find<64 * W>(a.split, (turn / tiles - h * shares) * 8 + (blockIdx.x & 7), sh)) return;
  const int lane = threadIdx.x & 63, m = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head0 = 16 * HT * tile;
  do {
    bf16x8 q[HT][KS];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      const int i = head0 + 16 * t + m;
      const char* row = a.q + p.b * a.q_b + (h * a.group + min(i, a.group - 1)) * a.q_h;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        u32x4 w = *(const u32x4*)(row + 2 * Tile::q_dim(s, quarter));
        if (i >= a.group) w = u32x4{0u, 0u, 0u, 0u};
        q[t][s] = __builtin_bit_cast(bf16x8, w);
      }
    }
    f32x4 o[HT][NV];
    float top_m[HT], l[HT];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      top_m[t] = kNone;
      l[t] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) o[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // this wave's tiles of 32 tokens
    const int block0 = p.begin / 16, n = steps_of<32>(p.end - p.begin), t0 = n * wave / W, t1 = n * (wave + 1) / W;
    Tile x;
    BlockList list;
    Blocks now, next;
    auto place = [&](int t) {
      const int block = block0 + 2 * t;
      if (t == t0 || block - list.block0 >= 64) list.fetch(a.split, p.b, p.len, block, lane);
      return list.get(a.split, p, block);
    };
    if (t0 < t1) {
      now = place(t0);
      x.load_k(a, now, h, m, quarter);
    }
    for (int t = t0; t < t1; ++t) {
      x.load_v(a, now, h, m, quarter);
      f32x4 s[HT][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) s[ht][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const bf16x8 key = x.key(i, ks);
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) s[ht][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key, q[ht][ks], s[ht][i], 0, 0, 0);
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[ht][i][r] *= E4M3 ? a.c * x.ks[i][r] : a.c;
      }
      const bool full = now.full();
      if (t + 1 < t1) {
        next = place(t + 1);
        x.load_k(a, next, h, m, quarter);
      }
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = 4 * quarter + r;
            const bool seen = at >= now.lo[i] && at < now.hi[i];
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) s[ht][i][r] = seen ? s[ht][i][r] : kNone;
            // a weight of zero does not take out a NaN or an infinity
#pragma unroll
            for (int w = 0; w < Tile::VW; ++w) x.v[4 * i + r][w] = seen ? x.v[4 * i + r][w] : 0u;
            if constexpr (E4M3) x.vs[i][r] = seen ? x.vs[i][r] : 0.0f;
          }
      }
      bf16x8 w[HT];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        float high = s[ht][0][0];
#pragma unroll
        for (int r = 1; r < 8; ++r) high = fmaxf(high, s[ht][r / 4][r % 4]);
        if (__any(high > top_m[ht] + kSlack)) {
          const float up = fmaxf(top_m[ht], quarters_max(high));
          const float f = top_m[ht] == kNone ? 0.0f : exp2f(top_m[ht] - up);
          top_m[ht] = up;
          l[ht] *= f;
#pragma unroll
          for (int j = 0; j < NV; ++j) o[ht][j] *= f;
        }
        const float at = top_m[ht] == kNone ? 0.0f : top_m[ht];
        u32x4 pk;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float e[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            e[r] = __builtin_amdgcn_exp2f(s[ht][i][r] - at);
            l[ht] += e[r];
            if constexpr (E4M3) e[r] *= x.vs[i][r];
          }
          pk[2 * i] = f2_bf16(e[0], e[1]);
          pk[2 * i + 1] = f2_bf16(e[2], e[3]);
        }
        w[ht] = __builtin_bit_cast(bf16x8, pk);
      }
#pragma unroll
      for (int j = 0; j < NV; j += 2) {
        bf16x8 va, vb;
        x.values(j, va, vb);
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          o[ht][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, w[ht], o[ht][j], 0, 0, 0);
          o[ht][j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, w[ht], o[ht][j + 1], 0, 0, 0);
        }
      }
      now = next;
    }
    // the waves' sums, in wave order
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      const float all = quarters_sum(l[ht]);
      if (quarter == 0) {
        // scores of NaN alone: not "nothing seen"
        top[wave][16 * ht + m] = top_m[ht] == kNone && all != 0.0f ? 0.0f : top_m[ht];
        sum[wave][16 * ht + m] = all;
      }
    }
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += DP) {
        // D / DP lanes' columns at a time: lane rows of the result hold dims NV row + j
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 4 * quarter + r;
          if (NV * row < d0 || NV * row >= d0 + DP) continue;
#pragma unroll
          for (int j = 0; j < NV; ++j) red[wave][m][NV * row - d0 + j] = o[ht][j][r];
        }
        __syncthreads();
        const int hd = threadIdx.x >> 4, i = head0 + 16 * ht + hd;           // 16 threads a head
        if (i < a.group) {
          float t = kNone;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float u = top[w][16 * ht + hd];
            t = u > t || u != u ? u : t;
          }
          float f[W], all = 0.0f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float u = top[w][16 * ht + hd];
            f[w] = u == kNone ? 0.0f : exp2f(u - t);
            all = __builtin_fmaf(f[w], sum[w][16 * ht + hd], all);
          }
          constexpr int C = DP / 16;
          const int c0 = C * (threadIdx.x & 15), hh = h * a.group + i;
          const bool last = p.count == 1;
          const float inv = !last ? 1.0f : all == 0.0f ? 0.0f : 1.0f / all;
#pragma unroll
          for (int j = 0; j < C; j += 2) {
            float y[2] = {0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
              for (int k = 0; k < 2; ++k) y[k] = __builtin_fmaf(f[w], red[w][hd][c0 + j + k], y[k]);
            if (last) {
              uint16_t* to = a.out + p.b * a.out_b + hh * a.out_h + d0 + c0 + j;
              to[0] = f_bf16(y[0] * inv);
              to[1] = f_bf16(y[1] * inv);
            } else {
              float* to = a.part + ((int64_t)p.place * a.heads + hh) * D + d0 + c0 + j;
              to[0] = y[0];
              to[1] = y[1];
            }
          }
          if ((threadIdx.x & 15) == 0 && d0 == 0) {
            if (last) {
              if (a.lse) a.lse[p.b * a.lse_b + hh] = all == 0.0f ? kNone : (t + log2f(all)) / kLog2E;
            } else {
              float* to = a.ml + 2 * ((int64_t)p.place * a.heads + hh);
              to[0] = t;
              to[1] = all;
            }
          }
        }
      }
    }
    __syncthreads();                   // top, sum and red have been read
  } while (p.next(a.split, threadIdx.x));
}

}  // namespace ops
}  // namespace fg
