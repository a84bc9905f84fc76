// Which rows and columns of a product a tile works on: the part of the tile kernel that depends on
// the experts' offsets, which are read on the device and may hold anything.  Plain C++, so that a
// test without a GPU can run it over any offsets.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define AR_HD __host__ __device__ __forceinline__
#else
#define AR_HD inline
#endif

namespace ar {

#ifndef __CUDACC__
inline int min(int a, int b) { return a < b ? a : b; }
inline int max(int a, int b) { return a > b ? a : b; }
#endif

// Args: n (rows of X), experts and offsets ([experts + 1], or null: one expert with all rows).

// Rows [r0, r1) of X that belong to expert e, clamped to the tensor: whatever the
// offsets hold, no access leaves it.
template <class Args>
AR_HD void expert_rows(const Args& a, int e, int& r0, int& r1) {
  if (!a.offsets) {
    r0 = 0;
    r1 = a.n;
    return;
  }
  r0 = min(max(a.offsets[e], 0), a.n);
  r1 = min(max(a.offsets[e + 1], r0), a.n);
}

// Blocks of bm rows.  cum[e] counts those of the experts before e, and is capped at what
// offsets that keep to the rules can give, so that none overflow the count.
template <class Args>
AR_HD int row_blocks(const Args& a, int e, int bm) {
  int r0, r1;
  expert_rows(a, e, r0, r1);
  return (r1 - r0 + bm - 1) / bm;
}
template <class Args>
AR_HD int most_row_blocks(const Args& a, int bm) {
  return a.n / bm + a.experts;
}

constexpr int kRasterM = 8;  // row blocks that share a sweep over the weight's columns

struct Unit {
  int e;       // expert
  int m0, r1;  // first row of X of the unit, end of the expert's rows
  int n0;      // first column of Y
};

// Unit t in order: experts in turn; inside an expert groups of kRasterM row blocks,
// each sweeping the weight's column blocks with the row blocks innermost (the
// group's rows of X stay in L2 while the weight passes by).  0 <= t < cum[experts] * num_n.
template <class Args>
AR_HD Unit find_unit(const Args& a, const int* cum, int64_t t, int num_n, int bm, int bn) {
  Unit u;
  const int mb = static_cast<int>(t / num_n);
  int e = 0;
  if (a.offsets) {
    int lo = 0, hi = a.experts;  // the last e with cum[e] <= mb
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= mb)
        lo = mid;
      else
        hi = mid;
    }
    e = lo;
  }
  int r0;
  expert_rows(a, e, r0, u.r1);
  const int64_t r = t - static_cast<int64_t>(cum[e]) * num_n;
  const int num_m = cum[e + 1] - cum[e];
  const int64_t per = static_cast<int64_t>(kRasterM) * num_n;
  const int grp = static_cast<int>(r / per);
  const int in_grp = static_cast<int>(r - grp * per);
  const int gm = min(kRasterM, num_m - grp * kRasterM);
  const int n_blk = in_grp / gm;
  u.e = e;
  u.m0 = r0 + (grp * kRasterM + in_grp - n_blk * gm) * bm;
  u.n0 = n_blk * bn;
  return u;
}

}  // namespace ar
