// Pages of a paged cache: a step's page tables and slots, and rows written to
// their slots (formulas and limits at fg_page_step and fg_kv_append in
// include/fg_attention.h).
//
// page_step is prefix sums over the requests: pages wanted, tokens given, pages
// brought back. One workgroup does them, T requests at a time with the sums
// carried on, and then hands out pages and tokens by their place in the sums, a
// binary search in LDS each, so that one request's thousand pages are no slower than
// a thousand requests' one. It is latency: load, sums, page, slot. Tokens beyond a few
// for each thread are left to a second kernel over the whole chip, which reads
// only what the first one wrote.
#pragma once

#include "fg_ops.hpp"

namespace fg {
namespace ops {

struct PageStepArgs {
  const int32_t* lens;
  const int32_t* add;
  int32_t* table;
  int32_t* ring;
  const int64_t* ends;
  int32_t* lens_out;
  int64_t* ends_out;
  int32_t* starts;
  int64_t* slots;
  int32_t* positions;
  int64_t ldt;
  int32_t batch, width, n_pages, page, tokens, fill;       // fill: this kernel writes slots and positions
};

// Sums that stop at the largest number: what they are compared with is below 2^31.
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive prefix sums of N numbers over a workgroup of T threads, and their totals; buf has no reader left.
template <int T, int N>
__device__ __forceinline__ void sums_upto(uint32_t (&v)[N], uint32_t (&total)[N], uint32_t (&buf)[N][T / 64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    auto moved = [&](auto ctrl, auto rows) {
      return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[i], decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
    };
    typedef std::integral_constant<int, 0xf> all;
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x111>(), all()));      // row_shr:1, 2, 4, 8
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x112>(), all()));
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x114>(), all()));
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x118>(), all()));
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>()));      // row_bcast:15 into rows 1 and 3
    v[i] = plus(v[i], moved(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>()));      // row_bcast:31 into rows 2 and 3
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 63) buf[i][wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t before = 0;
    total[i] = 0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) {
      const uint32_t u = buf[i][w];
      if (w < wave) before = plus(before, u);
      total[i] = plus(total[i], u);
    }
    v[i] = plus(v[i], before);
  }
}
// The largest of N numbers; buf has no reader left.
template <int T, int N>
__device__ __forceinline__ void max_of_all(uint32_t (&v)[N], uint32_t (&buf)[N][T / 64]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lanes_max<64>(v[i]);
    if ((threadIdx.x & 63) == 0) buf[i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v[i] = buf[i][w] > v[i] ? buf[i][w] : v[i];
}

// The last entry of at[0..n) that is not above i; at[0] <= i.
template <class At>
__device__ __forceinline__ int last_upto(const At* at, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (at[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void put_token(const PageStepArgs& a, int64_t t, int b, int pos) {
  const int32_t page = a.table[b * a.ldt + pos / a.page];
  a.slots[t] = page < 0 ? -1 : (int64_t)page * a.page + pos % a.page;
  a.positions[t] = pos;
}
__device__ __forceinline__ void put_none(const PageStepArgs& a, int64_t t) {
  a.slots[t] = -1;
  a.positions[t] = 0;
}

template <int T>
__global__ __launch_bounds__(T) void page_step_kernel(PageStepArgs a) {
  __shared__ uint32_t buf[2][T / 64], buf1[1][T / 64], buf2[2][T / 64];
  __shared__ int32_t fresh[T], back[T], given[T], held_at[T], len_at[T];
  const int tid = threadIdx.x;
  const int64_t head = a.ends[0], tail = a.ends[1], size = a.n_pages;
  const uint32_t free_pages = (uint32_t)(tail < head ? 0 : tail - head > size ? size : tail - head);
  const int64_t h0 = (head % size + size) % size, t0 = (tail % size + size) % size;
  uint32_t asked = 0, wanted = 0, taken = 0, served_tokens = 0, returned = 0;
  if (tid == 0) a.starts[0] = 0;
  for (int first = 0; first < a.batch; first += T) {
    const int b = first + tid;
    const bool in = b < a.batch;
    const uint32_t len = in && a.lens[b] > 0 ? a.lens[b] : 0, page = a.page;
    const int32_t add = in ? a.add[b] : 0;
    const uint32_t want = add > 0 ? add : 0;
    const uint32_t held = len / page + (len % page != 0), wants = (len + want) / page + ((len + want) % page != 0);     // len + want is below 2^32
    const bool fits = in && wants <= (uint32_t)a.width;
    const uint32_t need = fits ? wants - held : 0;
    const uint32_t ends = in && add < 0 ? (held < (uint32_t)a.width ? held : a.width) : 0;
    // Served: pages, then tokens, in request order; what does not come through asks for its share all the same. So those that
    // need pages and get them are the first that need any, and their places among the pages are those of all.
    uint32_t sums[2] = {need, ends}, all[2];
    sums_upto<T>(sums, all, buf);
    const uint32_t pages_upto = plus(asked, sums[0]);
    const bool paged = fits && (need == 0 || pages_upto <= free_pages);
    uint32_t tokens[1] = {paged ? want : 0}, all_tokens[1];
    sums_upto<T>(tokens, all_tokens, buf1);
    const uint32_t tokens_upto = plus(wanted, tokens[0]);
    const bool ok = paged && tokens_upto <= (uint32_t)a.tokens;
    uint32_t last[2] = {ok && need ? pages_upto : 0, ok ? tokens_upto : 0};
    max_of_all<T>(last, buf2);
    const uint32_t pages_here = last[0] > taken ? last[0] - taken : 0, tokens_here = last[1] > served_tokens ? last[1] - served_tokens : 0;
    // pages of ended requests, as many as the ring has places for
    const uint32_t room = (uint32_t)size - free_pages - returned, back_here = all[1] < room ? all[1] : room;
    auto place = [](uint32_t v, uint32_t from) { return (int32_t)(v < from ? 0 : v - from > 0x7fffffffu ? 0x7fffffffu : v - from); };
    const uint32_t start = plus(wanted, tokens[0] - (paged ? want : 0)), total = served_tokens + tokens_here;
    if (in) {
      a.lens_out[b] = add < 0 ? 0 : (int32_t)(len + (ok ? want : 0));
      a.starts[b + 1] = (int32_t)(tokens_upto < total ? tokens_upto : total);
    }
    fresh[tid] = place(plus(asked, sums[0] - need), taken);
    given[tid] = place(start, served_tokens);
    back[tid] = place(sums[1] - ends, 0);
    held_at[tid] = (int32_t)held;
    len_at[tid] = (int32_t)len;
    __syncthreads();
    // four at a time, their searches and loads beside each other
    constexpr int B = 4;
    for (uint32_t i = tid; i < pages_here; i += B * T) {
      int r[B];
      int32_t v[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const uint32_t n = i + j * T < pages_here ? i + j * T : i;
        r[j] = last_upto(fresh, T, (int)n);
        int64_t at = h0 + taken + n;
        v[j] = a.ring[at >= size ? at - size : at];
      }
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (i + j * T < pages_here) a.table[(int64_t)(first + r[j]) * a.ldt + held_at[r[j]] + ((int)(i + j * T) - fresh[r[j]])] = v[j];
    }
    for (uint32_t i = tid; i < back_here; i += B * T) {
      int32_t v[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const uint32_t n = i + j * T < back_here ? i + j * T : i;
        const int r = last_upto(back, T, (int)n);
        v[j] = a.table[(int64_t)(first + r) * a.ldt + ((int)n - back[r])];
      }
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (i + j * T < back_here) a.ring[(t0 + returned + i + j * T) % size] = v[j];
    }
    __syncthreads();
    if (a.fill)
      for (uint32_t i = tid; i < tokens_here; i += T) {
        const int r = last_upto(given, T, (int)i);
        put_token(a, (int64_t)served_tokens + i, first + r, len_at[r] + ((int)i - given[r]));
      }
    asked = plus(asked, all[0]);
    wanted = plus(wanted, all_tokens[0]);
    taken += pages_here;
    served_tokens += tokens_here;
    returned += back_here;
  }
  if (tid == 0) {
    a.ends_out[0] = head + taken;
    a.ends_out[1] = tail + returned;
  }
  if (a.fill)
    for (int64_t t = (int64_t)served_tokens + tid; t < a.tokens; t += T) put_none(a, t);
}

// Tokens of a large step: starts in LDS where they fit.
constexpr int kStartsInLds = 4096;
__global__ __launch_bounds__(256) void page_slots_kernel(PageStepArgs a) {
  __shared__ int32_t lds[kStartsInLds];
  const int n = a.batch;                         // starts has n + 1
  const int32_t* at = a.starts;
  if (n < kStartsInLds) {
    for (int i = threadIdx.x; i <= n; i += 256) lds[i] = at[i];
    __syncthreads();
    at = lds;
  }
  const int32_t total = at[n];
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < a.tokens; t += step) {
    if (t >= total) {
      put_none(a, t);
      continue;
    }
    const int b = last_upto(at, n, (int)t), got = at[b + 1] - at[b];
    put_token(a, t, b, a.lens_out[b] - got + (int)t - at[b]);
  }
}

// ------------------------------------------------------------------- append
struct AppendArgs {
  const char* x[2];                  // new rows: keys, values
  char* cache[2];
  float* scale[2];                   // [n_pages][heads][page]
  const int64_t* slots;
  int64_t x_row[2], x_head[2], c_page[2], c_tok[2], c_head[2];     // bytes
  int64_t rows, n_slots;
  int32_t heads, dim, page;
};

// Slot of a row as page and place; false for none.
struct Place {
  int64_t page;
  int32_t at;
  __device__ __forceinline__ bool find(const AppendArgs& a, int64_t row) {
    const int64_t s = a.slots[row];
    if (s < 0 || s >= a.n_slots) return false;
    if (s >> 32 == 0) {                // one 32-bit division where that is enough
      page = (uint32_t)s / (uint32_t)a.page;
      at = (uint32_t)s % (uint32_t)a.page;
    } else {
      page = s / a.page;
      at = (int32_t)(s % a.page);
    }
    return true;
  }
};

// 16 bytes a thread; neighbouring threads have neighbouring pieces of a row.
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  const int w = blockIdx.z, per_row = a.heads * (a.dim / 8);
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.rows * per_row) return;
  const int64_t row = i >> 32 == 0 ? (uint32_t)i / (uint32_t)per_row : i / per_row;
  const int piece = (int)(i - row * per_row), h = piece / (a.dim / 8), e = piece % (a.dim / 8);
  Place p;
  if (!p.find(a, row)) return;
  const u32x4 v = *(const u32x4*)(a.x[w] + row * a.x_row[w] + h * a.x_head[w] + 16 * e);
  *(u32x4*)(a.cache[w] + p.page * a.c_page[w] + p.at * a.c_tok[w] + h * a.c_head[w] + 16 * e) = v;
}

// For codes that are those of the exact quotient 448 x / a (a the row's maximum): with 448 x of 11 bits and a of 8 it lies on a border between two codes (5 bits) or at least 2^-13
// of itself away from one, and the product x (448 / a) is within 2^-22 of it, so rounded to 17 bits first it falls on the right side, or on the border itself, and none is above 448.
__device__ __forceinline__ float bits17(float v) { return __uint_as_float((__float_as_uint(v) + 0x40u) & ~0x7fu); }      // NaN stays: its low bits come from bf16

// 16 lanes a row and head, 8 V elements each. The maximum is taken over bit patterns,
// whose order is that of the numbers, so that a NaN reaches the scale. A row whose
// maximum is below 2^-100 is taken by 2^100 first, as 448 / a would leave fp32.
template <int V>
__global__ __launch_bounds__(256) void append8_kernel(AppendArgs a) {
  const int w = blockIdx.z, lane = threadIdx.x & 15;
  const int64_t i = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x) >> 4;
  if (i >= a.rows * a.heads) return;               // 16 lanes together
  const int64_t row = i >> 32 == 0 ? (uint32_t)i / (uint32_t)a.heads : i / a.heads;
  const int h = (int)(i - row * a.heads), pieces = a.dim / 8;
  Place p;
  if (!p.find(a, row)) return;
  const char* x = a.x[w] + row * a.x_row[w] + h * a.x_head[w];
  u32x4 v[V];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = u32x4{0u, 0u, 0u, 0u};
    if (lane + 16 * j < pieces) v[j] = *(const u32x4*)(x + 16 * (lane + 16 * j));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = v[j][k] & 0x7fffu, hi = (v[j][k] >> 16) & 0x7fffu, m = lo > hi ? lo : hi;
      top = m > top ? m : top;
    }
  }
  top = lanes_max<16>(top);
  const float m = bf16_f((uint16_t)top), up = m < 0x1p-100f ? 0x1p100f : 1.0f, inv = m > 0.0f ? 448.0f / (m * up) : m;
  char* c = a.cache[w] + p.page * a.c_page[w] + p.at * a.c_tok[w] + h * a.c_head[w];
  if (lane == 0) a.scale[w][(p.page * a.heads + h) * a.page + p.at] = m / 448.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (lane + 16 * j >= pieces) break;
    u32x2 q;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[4] = {bf16_lo(v[j][2 * k]), bf16_hi(v[j][2 * k]), bf16_lo(v[j][2 * k + 1]), bf16_hi(v[j][2 * k + 1])};
#pragma unroll
      for (int t = 0; t < 4; ++t) f[t] = bits17(f[t] * up * inv);
      const int word = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
      q[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], word, true);
    }
    *(u32x2*)(c + 8 * (lane + 16 * j)) = q;
  }
}

}  // namespace ops
}  // namespace fg
