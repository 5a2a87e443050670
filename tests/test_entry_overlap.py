"""The overlap checks of the C entries, as a host program, against byte sets."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <random>
#include <set>
#include "fg_entry.hpp"
using namespace fg::ops;
static std::mt19937 rng(1);
static int64_t upto(int64_t n) { return (int64_t)(rng() % (n + 1)); }
static Rows some() { return {(const void*)(1000 + upto(60)), 1 + upto(5), 1 + upto(12), upto(3) ? upto(24) : 0}; }
static std::set<int64_t> bytes(const Rows& r) {
  std::set<int64_t> s;
  for (int64_t i = 0; i < r.rows; ++i)
    for (int64_t j = 0; j < r.bytes; ++j) s.insert((int64_t)r.p + i * r.pitch + j);
  return s;
}
int main() {
  int shared = 0, apart = 0, zero = 0;
  for (int n = 0; n < 200000; ++n) {
    const Rows a = some(), b = some();
    const std::set<int64_t> x = bytes(a);
    bool want = false;
    for (int64_t v : bytes(b)) want = want || x.count(v);
    if (overlap(a, b) != want || overlap(b, a) != want) {
      printf("%d: %ld %ld %ld %ld and %ld %ld %ld %ld: %d\n", n, (long)a.p, (long)a.rows, (long)a.bytes, (long)a.pitch, (long)b.p, (long)b.rows, (long)b.bytes, (long)b.pitch, want);
      return 1;
    }
    (want ? shared : apart) += 1;
    zero += (a.rows > 1 && a.pitch == 0) || (b.rows > 1 && b.pitch == 0);
  }
  printf("%d %d %d\n", shared, apart, zero);
  return 0;
}
"""


def run(tmp_path, source):
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "sync_protocols_amd", "csrc"),
                    "-I", "/opt/rocm/include", str(src), "-o", str(exe), "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_rows_that_overlap_and_interleave(tmp_path):
    """Any two sets of rows, broadcast ones (pitch 0) and rows that lie on each other among them."""
    r = run(tmp_path, SOURCE)
    assert r.returncode == 0, r.stdout
    assert all(int(n) > 10000 for n in r.stdout.split())


MEET = r"""
#include <cstdio>
#include <random>
#include <set>
#include "fg_entry.hpp"
using namespace fg::ops;
static std::mt19937 rng(2);
static int64_t upto(int64_t n) { return (int64_t)(rng() % (n + 1)); }
int main() {
  int shared = 0, apart = 0;
  while (shared + apart < 100000) {
    Dim d[4];
    for (Dim& x : d) x = {1 + upto(3), 1 + upto(20)};
    d[3].stride = 1;
    if (!distinct({d[0], d[1], d[2], d[3]})) continue;
    std::set<int64_t> s;
    for (int64_t n = 0; n < d[0].size * d[1].size * d[2].size * d[3].size; ++n) {
      int64_t at = 0, left = n;
      for (const Dim& x : d) at += left % x.size * x.stride, left /= x.size;
      s.insert(at);
    }
    const int64_t by = upto(120) - 60;
    bool want = false;
    for (int64_t v : s) want = want || s.count(v + by);
    if (meet({d[0], d[1], d[2], d[3]}, by) != want) {
      for (const Dim& x : d) printf("%ld x %ld, ", (long)x.size, (long)x.stride);
      printf("by %ld: %d\n", (long)by, want);
      return 1;
    }
    (want ? shared : apart) += 1;
  }
  printf("%d %d\n", shared, apart);
  return 0;
}
"""


def test_tensors_that_lie_within_each_other(tmp_path):
    """Any distance of two tensors of the same strides, against all their elements."""
    r = run(tmp_path, MEET)
    assert r.returncode == 0, r.stdout
    assert all(int(n) > 10000 for n in r.stdout.split())
