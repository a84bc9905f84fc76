"""The tile kernel's search for its rows and columns, run without a GPU over offsets of every kind: the
functions of csrc/ar_units.h as the kernel calls them, in a small library of their own."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "signed_gradient_rounding_b200", "csrc")

# cum as the kernel's warp scan gives it (32 experts at a time); units[t] = (e, m0, r1, n0)
SOURCE = r"""
#include "ar_units.h"
struct Args {
  int n, experts;
  const int32_t* offsets;
};
extern "C" long long walk(const int32_t* offsets, int n, int experts, int num_n, int bm, int bn, int* cum, int* units,
                          long long first, long long room) {
  const Args a = {n, experts, offsets};
  if (!offsets) {
    cum[0] = 0;
    cum[1] = (n + bm - 1) / bm;
  } else {
    const int limit = ar::most_row_blocks(a, bm);
    int carry = cum[0] = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      long long v = 0;
      for (int lane = 0; lane < 32; ++lane) {
        if (e0 + lane < experts) v += ar::row_blocks(a, e0 + lane, bm);
        if (carry + v > 2147483647ll) return -1;
        const int c = carry + v < limit ? static_cast<int>(carry + v) : limit;
        if (e0 + lane < experts) cum[e0 + lane + 1] = c;
        if (lane == 31) carry = c;
      }
    }
  }
  const long long total = static_cast<long long>(cum[experts]) * num_n;
  for (long long t = first; t < total && t < first + room; ++t, units += 4) {
    const ar::Unit u = ar::find_unit(a, cum, t, num_n, bm, bn);
    units[0] = u.e, units[1] = u.m0, units[2] = u.r1, units[3] = u.n0;
  }
  return total;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    assert cxx, "a C++ compiler"
    folder = tmp_path_factory.mktemp("units")
    src, lib = str(folder / "walk.cpp"), str(folder / "walk.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", src,
                    "-o", lib], check=True)
    fn = ctypes.CDLL(lib).walk
    fn.restype = ctypes.c_longlong

    def call(offsets, n, experts, num_n, bm, bn, first=0, room=None):
        most = (n // bm + experts + 1) * num_n
        room = most if room is None else room
        off = None if offsets is None else (ctypes.c_int32 * len(offsets))(*offsets)
        cum, units = (ctypes.c_int * (experts + 1))(), (ctypes.c_int * (4 * room))()
        total = fn(off, n, experts, num_n, bm, bn, cum, units, ctypes.c_longlong(first), ctypes.c_longlong(room))
        assert 0 <= total <= most
        return [tuple(units[4 * t:4 * t + 4]) for t in range(min(total - first, room))]
    return call


@pytest.mark.parametrize("bm,bn", [(128, 128), (128, 256), (256, 256)])
def test_offsets_that_keep_to_the_rules(walk, bm, bn):
    """Every block of rows of every expert with every block of columns, once; and no more than the launch allows for."""
    rng = random.Random(bm + bn)
    for _ in range(300):
        experts, n = rng.choice([1, 2, 5, 31, 32, 33, 70, 1024]), rng.choice([1, 7, 128, 500, 3000])
        num_n = rng.choice([1, 2, 5])
        offsets = sorted(rng.randint(0, n) for _ in range(experts + 1))
        units = walk(offsets, n, experts, num_n, bm, bn)
        want = {(e, r, offsets[e + 1], b * bn) for e in range(experts) for r in range(offsets[e], offsets[e + 1], bm)
                for b in range(num_n)}
        assert len(units) == len(want) and set(units) == want
        assert len(units) <= (-(-n // bm) + experts - 1) * num_n
    for n in (1, 128, 129, 5000):
        units = walk(None, n, 1, 3, bm, bn)
        assert sorted(units) == sorted((0, r, n, b * bn) for r in range(0, n, bm) for b in range(3))


@pytest.mark.parametrize("bm,bn", [(128, 128), (256, 256)])
def test_offsets_that_break_the_rules(walk, bm, bn):
    """Any 32-bit numbers: every unit's rows and columns stay inside the tensors."""
    rng = random.Random(bm)
    edge = [0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 30]
    for i in range(600):
        experts, n = rng.choice([1, 2, 5, 31, 32, 33, 70]), rng.choice([1, 7, 128, 500, 3000])
        num_n = rng.choice([1, 2, 5])
        offsets = [rng.choice(edge) if rng.random() < 0.2 else rng.randint(-(1 << 31), (1 << 31) - 1) if rng.random() < 0.2
                   else rng.randint(0, n) for _ in range(experts + 1)]
        for e, m0, r1, n0 in walk(offsets, n, experts, num_n, bm, bn):
            assert 0 <= e < experts and 0 <= m0 < r1 <= n and 0 <= n0 < num_n * bn and n0 % bn == 0


@pytest.mark.parametrize("bm", [128, 256])
@pytest.mark.parametrize("offsets", [[0, 1 << 30], [0, 1 << 30, 0, 1 << 30, 0, 1 << 30], [0, 1, (1 << 30) - 1, 1 << 30]])
def test_the_largest_tensors(walk, bm, offsets):
    """2^30 rows, or 2^30 columns over all experts: the last units are where they should be."""
    n, experts = 1 << 30, len(offsets) - 1
    rows = min(sum(-(-max(b - a, 0) // bm) for a, b in zip(offsets, offsets[1:])), n // bm + experts)
    for num_n in (1, (1 << 30) // experts // bm):
        total = rows * num_n
        for e, m0, r1, n0 in walk(offsets, n, experts, num_n, bm, bm, total - 50, 50):
            assert 0 <= e < experts and 0 <= m0 < r1 <= n and 0 <= n0 < num_n * bm
        assert len(walk(offsets, n, experts, num_n, bm, bm, total, 50)) <= 0
