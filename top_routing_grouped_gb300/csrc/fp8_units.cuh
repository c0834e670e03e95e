// fp8_units.cuh -- where each segment's rows and units of work begin, found by every CTA of an 8-bit
// product from the segment counts themselves (at most 256 numbers, two barriers), so that a call
// needs no kernel for tables.
#pragma once
#include "device_common.cuh"

namespace moe {
namespace fp8 {

struct Segments {
  int row0[kMaxExperts + 1];   // first row of each segment
  int unit0[kMaxExperts + 1];  // first unit of each segment
  int64_t row_tot[8];          // the scans' warp totals
  uint32_t unit_tot[8];
};

// Inclusive scans over the first 256 threads (all threads call it): counts (null: one segment of
// `capacity` rows) -> sg; returns the units' number, or -1 when a count is negative or their sum is
// above the capacity.
template <typename UnitsOf>
__device__ __forceinline__ int scan_segments(Segments* sg, const int32_t* counts, int n_seg, int64_t capacity,
                                             UnitsOf units_of) {
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int cnt = i < n_seg ? (counts ? counts[i] : (int)capacity) : 0;
  int64_t rows = cnt < 0 ? (int64_t)1 << 40 : cnt;  // 64 bits: bad counts may sum to anything
  uint32_t units = cnt > 0 ? (uint32_t)units_of(cnt) : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, rows, o);
    const uint32_t y = __shfl_up_sync(0xffffffffu, units, o);
    if (lane >= o) {
      rows += x;
      units += y;
    }
  }
  if (warp < 8 && lane == 31) {
    sg->row_tot[warp] = rows;
    sg->unit_tot[warp] = units;
  }
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) {
      rows += sg->row_tot[w];
      units += sg->unit_tot[w];
    }
    all += sg->row_tot[w];
  }
  if (i < kMaxExperts) {
    sg->row0[i + 1] = (int)rows;
    sg->unit0[i + 1] = (int)units;
  }
  if (i == 0) sg->row0[0] = sg->unit0[0] = 0;
  __syncthreads();
  return all > capacity ? -1 : sg->unit0[n_seg];
}

// The segment of unit u: the last one whose first unit is at or below it.
__device__ __forceinline__ int segment_of(const Segments* sg, int n_seg, int u) {
  int lo = 0, hi = n_seg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sg->unit0[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The call's status word, set by its first launch (thread 0 of CTA 0).  Other CTAs record errors of
// their own only kMinTimeoutNs or more after they have started, that is, after this.
__device__ __forceinline__ void begin_status(const Ws& ws, bool bad, uint32_t site) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    ws.hdr[kHdrWhere] = bad ? site : 0u;
    ws.hdr[kHdrStatus] = bad ? (uint32_t)MOE_ERR_INTERNAL : 0u;
  }
}

}  // namespace fp8
}  // namespace moe
