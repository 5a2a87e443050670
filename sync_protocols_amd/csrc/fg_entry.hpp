// What the C entries of the operators share: launches that report their own
// errors only, alignment and overlap of caller memory, wide grids.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "fg.h"

namespace fg {
namespace ops {

// Launches on one stream, with their own errors only (an error that an earlier call
// of the program left behind is not theirs); none after one that failed.
struct Launches {
  hipStream_t stream;
  hipError_t error = hipSuccess;
  template <class Args>
  void operator()(void (*kernel)(Args), dim3 grid, dim3 block, size_t lds, Args a) {
    void* args[1] = {&a};
    if (error == hipSuccess) error = hipLaunchKernel((const void*)kernel, grid, block, args, lds, stream);
  }
  fg_status status() const { return error == hipSuccess ? FG_OK : FG_EHIP; }
};

constexpr int kCUs = 256;          // compute units of the part

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool multiple(int64_t v, int64_t of) { return v >= 0 && v % of == 0; }

// Rows of `bytes` bytes, `pitch` apart (one row: any pitch). Pitch 0, as a broadcast dimension has: all of them are the one row.
struct Rows {
  const void* p;
  int64_t rows, bytes, pitch;
  uintptr_t begin() const { return (uintptr_t)p; }
  uintptr_t end() const { return begin() + (rows - 1) * pitch + bytes; }
};
inline Rows whole(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }
// Rows of a tensor [n][heads][dim] with consecutive columns.
inline Rows rows3(const void* p, int64_t element, int64_t n, int64_t ns, int64_t heads, int64_t hs, int64_t dim) {
  return {p, n, element * ((heads - 1) * hs + dim), element * ns};
}

// Do they share a byte? Rows that interleave, as columns of one buffer do, need not.
inline bool overlap(Rows a, Rows b) {
  if (a.pitch == 0) a.rows = 1;
  if (b.pitch == 0) b.rows = 1;
  if (!a.p || !b.p || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  if (a.rows > b.rows) return overlap(b, a);
  if (a.pitch == b.pitch && a.rows > 1) {
    const int64_t d = (int64_t)(b.begin() - a.begin()) % a.pitch, shift = d < 0 ? d + a.pitch : d;
    if (shift >= a.bytes && shift + b.bytes <= a.pitch) return false;
  }
  for (int64_t i = 0; i < a.rows; ++i) {         // the last row of b that starts before the end of a's
    const uintptr_t from = a.begin() + i * a.pitch, to = from + a.bytes;
    if (to <= b.begin()) continue;
    const int64_t j = b.rows == 1 ? 0 : (int64_t)((to - 1 - b.begin()) / b.pitch);
    if (b.begin() + (j < b.rows ? j : b.rows - 1) * b.pitch + b.bytes > from) return true;
  }
  return false;
}
template <class... Others>
bool overlaps(const Rows& a, const Others&... others) { return (overlap(a, others) || ...); }

// One dimension of a tensor: its size and the distance of two entries.
struct Dim {
  int64_t size, stride;
};
// Do different indices always mean different elements? True for every order of
// the dimensions in which each one steps over all of the smaller ones.
inline bool distinct(std::initializer_list<Dim> dims) {
  Dim d[4];
  int n = 0;
  for (const Dim& x : dims)
    if (x.size > 1) d[n++] = x;
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
      const Dim t = d[j];
      d[j] = d[j - 1];
      d[j - 1] = t;
    }
  int64_t reach = 1;                           // elements that the smaller dimensions span
  for (int i = 0; i < n; ++i) {
    if (d[i].stride < reach) return false;
    reach += (d[i].size - 1) * d[i].stride;
  }
  return true;
}

// Two tensors of the same sizes and strides, whose indices all mean different elements (distinct), the second `by` elements behind the first: do they
// share one? They do if `by` is a sum of strides, each up to size - 1 times, forwards or back. What the smaller dimensions reach is less than a stride,
// so only the two multiples of it around `by` come into question.
inline bool meet(std::initializer_list<Dim> dims, int64_t by) {
  const Dim* top = nullptr;
  for (const Dim& x : dims)
    if (x.size > 1 && (!top || x.stride > top->stride)) top = &x;
  if (!top) return by == 0;
  Dim rest[4];
  int n = 0;
  for (const Dim& x : dims)
    if (&x != top) rest[n++] = x;
  while (n < 4) rest[n++] = {1, 0};
  const int64_t q = by / top->stride;
  for (int64_t c = q - 1; c <= q + 1; ++c)
    if (c < top->size && -c < top->size && meet({rest[0], rest[1], rest[2], rest[3]}, by - c * top->stride)) return true;
  return false;
}

// A grid of n workgroups for any n below 2^31: more than 2^20 in two dimensions
// (a dimension holds fewer than 2^32 threads).
inline dim3 wide_grid(int64_t n) {
  const int64_t x = 1 << 20;
  return n <= x ? dim3((unsigned)n) : dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

}  // namespace ops
}  // namespace fg
