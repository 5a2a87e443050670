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

// Inclusive prefix sum over a workgroup of T threads, and its total.
template <int T>
__device__ __forceinline__ int64_t sum_upto(int64_t v, int64_t& total, int64_t* buf) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();                       // buf's last readers
  if (lane == 63) buf[wave] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) {
    const int64_t u = buf[w];
    before += w < wave ? u : 0;
    total += u;
  }
  return v + before;
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
  __shared__ int64_t buf[T / 64];
  __shared__ int32_t fresh[T], back[T], given[T], held_at[T], len_at[T];
  const int tid = threadIdx.x;
  const int64_t head = a.ends[0], tail = a.ends[1], size = a.n_pages;
  const int64_t free_pages = tail < head ? 0 : tail - head > size ? size : tail - head;
  const int64_t h0 = (head % size + size) % size, t0 = (tail % size + size) % size;
  int64_t asked = 0, wanted = 0, taken = 0, served_tokens = 0, returned = 0;
  if (tid == 0) a.starts[0] = 0;
  for (int first = 0; first < a.batch; first += T) {
    const int b = first + tid;
    const bool in = b < a.batch;
    const int64_t len = in && a.lens[b] > 0 ? a.lens[b] : 0;
    const int64_t add = in ? a.add[b] : 0, want = add > 0 ? add : 0;
    const int64_t held = (len + a.page - 1) / a.page, wants = (len + want + a.page - 1) / a.page;
    const bool fits = in && wants <= a.width;
    const int64_t need = fits ? wants - held : 0;
    int64_t all;
    // served: pages, then tokens, in request order; what does not come through asks for its share all the same
    const int64_t upto = asked + sum_upto<T>(need, all, buf);
    asked += all;
    bool ok = fits && (need == 0 || upto <= free_pages);
    const int64_t tokens_upto = wanted + sum_upto<T>(ok ? want : 0, all, buf);
    wanted += all;
    ok = ok && tokens_upto <= a.tokens;
    const int64_t got = ok ? want : 0, got_upto = sum_upto<T>(got, all, buf);
    const int64_t tokens_here = all;
    const int64_t pages = ok ? need : 0, pages_upto = sum_upto<T>(pages, all, buf);
    const int64_t pages_here = all;
    // pages of ended requests, as many as the ring has places for
    const int64_t ends = in && add < 0 ? (held < a.width ? held : a.width) : 0;
    const int64_t room = size - free_pages - returned;
    const int64_t ends_upto = sum_upto<T>(ends, all, buf);
    const int64_t back_here = all < room ? all : room;
    if (in) {
      a.lens_out[b] = add < 0 ? 0 : (int32_t)(len + got);
      a.starts[b + 1] = (int32_t)(served_tokens + got_upto);
    }
    fresh[tid] = (int32_t)(pages_upto - pages);
    given[tid] = (int32_t)(got_upto - got);
    const int64_t from = ends_upto - ends;
    back[tid] = (int32_t)(from < 0x7fffffff ? from : 0x7fffffff);
    held_at[tid] = (int32_t)held;
    len_at[tid] = (int32_t)len;
    __syncthreads();
    for (int64_t i = tid; i < pages_here; i += T) {
      const int r = last_upto(fresh, T, (int)i);
      int64_t at = h0 + taken + i;
      if (at >= size) at -= size;
      a.table[(first + r) * a.ldt + held_at[r] + (i - fresh[r])] = a.ring[at];
    }
    for (int64_t i = tid; i < back_here; i += T) {
      const int r = last_upto(back, T, (int)i);
      a.ring[(t0 + returned + i) % size] = a.table[(first + r) * a.ldt + (i - back[r])];
    }
    __syncthreads();
    if (a.fill)
      for (int64_t i = tid; i < tokens_here; i += T) {
        const int r = last_upto(given, T, (int)i);
        put_token(a, served_tokens + i, first + r, len_at[r] + (int)(i - given[r]));
      }
    taken += pages_here;
    served_tokens += tokens_here;
    returned += back_here;
  }
  if (tid == 0) {
    a.ends_out[0] = head + taken;
    a.ends_out[1] = tail + returned;
  }
  if (a.fill)
    for (int64_t t = served_tokens + tid; t < a.tokens; t += T) put_none(a, t);
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
      for (int t = 0; t < 4; ++t) {
        f[t] = f[t] * up * inv;
        f[t] = f[t] > 448.0f ? 448.0f : f[t] < -448.0f ? -448.0f : f[t];
      }
      const int word = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
      q[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], word, true);
    }
    *(u32x2*)(c + 8 * (lane + 16 * j)) = q;
  }
}

}  // namespace ops
}  // namespace fg
