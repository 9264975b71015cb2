// Walking a launch's tiles: what the attention kernels share beside the
// partition (plan.cuh).
#pragma once

#include "oda_internal.cuh"

namespace oda {

// Bits [lo, hi) of a 16-bit tile mask whose bit 0 is slot `base`.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int base) {
  int l = min(max(lo - base, 0), 16);
  int h = min(max(hi - base, 0), 16);
  if (h <= l) return 0u;
  return ((1u << h) - 1u) & ~((1u << l) - 1u);
}

// Segment cursor over the CTA's tile range [lo, hi): segment (i, g) covers
// [s1 - nt, s1); rows with nt == 0 are skipped.
struct Cursor {
  int k;    // absolute tile index; == hi when exhausted
  int i;    // row slot
  int g;    // KV head
  int nt;   // tiles per segment of row i
  int s1;   // segment end
};

__device__ __forceinline__ void locate(const int* rowstart, int nrows, int hkv, int k, Cursor& c) {
  // largest i in [0, nrows) with rowstart[i] <= k
  int lo = 0, hi = nrows - 1;
  while (lo < hi) {
    int mid = (lo + hi + 1) >> 1;
    if (rowstart[mid] <= k) lo = mid; else hi = mid - 1;
  }
  c.i = lo;
  c.nt = (rowstart[lo + 1] - rowstart[lo]) / hkv;
  const int rel = k - rowstart[lo];
  c.g = rel / c.nt;
  c.s1 = rowstart[lo] + (c.g + 1) * c.nt;
}

// Move c to the first tile >= c.k that belongs to this warp (offset `w`
// from its segment's start within [lo, hi), stride W), crossing segments.
__device__ __forceinline__ void normalize(const int* rowstart, int hkv, int hi, int w, Cursor& c) {
  while (c.k >= min(c.s1, hi)) {
    if (c.s1 >= hi) { c.k = hi; return; }
    int s0 = c.s1;
    if (++c.g == hkv) {
      c.g = 0;
      ++c.i;
      c.nt = (rowstart[c.i + 1] - rowstart[c.i]) / hkv;
    }
    c.s1 = s0 + c.nt;
    c.k = s0 + w;
  }
}

}  // namespace oda
