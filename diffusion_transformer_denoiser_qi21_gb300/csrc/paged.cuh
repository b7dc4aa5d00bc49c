// Device side of a batch over a paged K/V cache (qi21_paged), shared by the
// append and the attention kernels.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace qi21 {

constexpr unsigned int kStatusPage = 2u;  // a page or row outside the cache

// The sequence of row t: the b in [0, nseq) with cu[b] <= t < cu[b + 1], or
// nseq if there is none. By one whole warp: 32 probes per round narrow the
// count of ends cu[1 ..] that are <= t, one round per factor of 32 of nseq
// (a binary search by one thread would wait for a load per factor of 2).
// Ends after a few rounds whatever cu holds.
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ cu, int nseq, int t, int lane) {
  int lo = 0, hi = nseq;  // the count is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step;
    const bool le = i <= hi && __ldg(cu + i) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    const int64_t end = lo + static_cast<int64_t>(n + 1) * step - 1;
    lo += n * step;
    hi = end < hi ? static_cast<int>(end) : hi;
  }
  if (lo < nseq && !(__ldg(cu + lo) <= t && t < __ldg(cu + lo + 1))) lo = nseq;
  return lo;
}

// Row (of the flattened pool) of own row `own` of sequence b; -1, with the
// status raised, if the row or its page is outside the cache.
__device__ __forceinline__ int64_t paged_row(const PagedArgs& p, int b, int own, unsigned int* status) {
  if (own >= 0 && own < p.table_rows) {
    const int pg = own / p.page_rows;
    const int id = __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + pg);
    if (id >= 0 && id < p.npages) return static_cast<int64_t>(id) * p.page_rows + (own - pg * p.page_rows);
  }
  atomicOr(status, kStatusPage);
  return -1;
}

}  // namespace qi21
