// How the tiles of a batch are shared out by the block-scaled 8-bit decode and
// found again by its merge.
//
// The batch's visible runs, cut into tiles of 128 tokens request after request,
// are one line of T tiles. Gang j of J takes tiles [jT/J, (j+1)T/J) of it (one
// CTA of a gang per row group), so every gang works on the same number of tiles
// whatever the lengths, and lengths are read where they lie: no host plan, and
// a captured call follows contexts as they grow. A request that lies within
// one gang is finished there; one cut by gang borders has a part per gang: its
// first gang keeps it in entry 1 (that gang's open end), the others in entry
// 0, and the merge finds the gangs from the request's place on the line.
#pragma once

#include "device_common.cuh"

namespace mla {

constexpr int kQ8Tile = 128;

__device__ __forceinline__ int64_t q8_tiles(const DecodeQ8Params& p, int b) {
  const WindowView v = window_view(__ldcg(p.context_lens + b), p.q_len, p.bs, p.causal, p.window, p.sinks);
  return (static_cast<int64_t>(v.n) + kQ8Tile - 1) / kQ8Tile;
}

// Gangs that get tiles (all of them unless there are fewer tiles), gang j's first tile, and the gang of tile x.
__device__ __forceinline__ int64_t q8_live_gangs(int64_t T, int gangs) { return T < gangs ? T : gangs; }
__device__ __forceinline__ int64_t q8_gang_begin(int64_t j, int64_t T, int64_t J) { return j * T / J; }
__device__ __forceinline__ int q8_gang_of(int64_t x, int64_t T, int64_t J) {
  return static_cast<int>(((x + 1) * J - 1) / T);
}

// Exclusive prefix over the block's threads of each thread's `mine`, and the total. `scratch`: 33 values.
template <int kThreads>
__device__ __forceinline__ int64_t block_prefix(int64_t mine, int64_t* scratch, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    all += scratch[w];
  }
  __syncthreads();
  *total = all;
  return before + x - mine;
}

}  // namespace mla
