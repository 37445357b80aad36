// Prefix sums over a CTA of 1024 threads, and the search in them.
#pragma once

#include <cstdint>

namespace mla {

constexpr int kScanWarps = 32;  // of the CTA: the second level of the scan is one warp

// Exclusive prefix of v over the CTA's threads, and the total. part: [kScanWarps] of shared memory.
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  long long w = part[lane];  // (one of each warp)
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();  // `part` may be written again
  return x - v + (warp > 0 ? before : 0);
}
// The last b of [lo, hi] with at[b] <= i (at non-decreasing, at[lo] <= i).
__device__ __forceinline__ int find_last(const int32_t* at, int lo, int hi, int32_t i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace mla
