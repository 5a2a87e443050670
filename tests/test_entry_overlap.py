"""The overlap checks of the C entries, as a host program, against byte sets."""
import os
import subprocess

import pytest

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
