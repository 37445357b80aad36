// How the tiles of a batch are shared out by the block-scaled 8-bit decode and
// found again by its merge.
//
// The batch's visible runs, cut into tiles of p.tile tokens request after request,
// are one line of T tiles. Gang j of J takes T / J of it, the first T % J gangs
// one more (one CTA of a gang per row group), so every gang works on the same number of tiles
// whatever the lengths, and lengths are read where they lie: no host plan, and
// a captured call follows contexts as they grow. A request that lies within
// one gang is finished there; one cut by gang borders has a part per gang: its
// first gang keeps it in entry 1 (that gang's open end), the others in entry
// 0, and says in its first gang's entry of ws_cut how many there are.
#pragma once

#include "device_common.cuh"

namespace mla {

__device__ __forceinline__ WindowView q8_view(const DecodeQ8Params& p, int L) {
  return window_view(L, p.q_len, p.bs, p.causal, p.window, p.sinks);
}
__device__ __forceinline__ int q8_tiles(const WindowView& v, int tile) {
  return v.n / tile + (v.n % tile != 0 ? 1 : 0);
}
// Context lengths, the first of them kept in shared memory: the walks below read them one after the other.
constexpr int kQ8Lens = 640;
struct Q8Lens {
  const int32_t* global;
  const int32_t* cached;  // shared memory, kQ8Lens
  __device__ __forceinline__ int operator()(int b) const { return b < kQ8Lens ? cached[b] : __ldcg(global + b); }
};

// The line of T tiles among the gangs that get any (all of them unless there are fewer tiles).
struct Q8Line {
  int64_t base;      // tiles of a gang
  int32_t gangs, more;  // the first `more` gangs have one more
  __device__ __forceinline__ int64_t begin(int j) const { return base * j + min(j, more); }
  // the gang of tile x
  __device__ __forceinline__ int gang_of(int64_t x) const {
    const int64_t head = (base + 1) * more;
    return x < head ? static_cast<int>(div(x, base + 1)) : more + static_cast<int>(div(x - head, base));
  }
  // (32-bit division where it does)
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
  }
};
__device__ __forceinline__ Q8Line q8_line(int64_t T, int gangs) {
  Q8Line l;
  l.gangs = T < gangs ? static_cast<int32_t>(T) : gangs;
  l.base = l.gangs > 0 ? Q8Line::div(T, l.gangs) : 0;
  l.more = static_cast<int32_t>(T - l.base * l.gangs);
  return l;
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

// A gang's tiles, request after request.
struct Q8Walk {
  int b;            // request of the current segment
  int ta, tb;       // its tiles [ta, tb) are this gang's ...
  int n_tiles;      // ... of so many
  int64_t left;     // tiles behind the segment
  WindowView v;
};
__device__ __forceinline__ Q8Walk q8_walk(int b0, int64_t off0, int64_t tiles) {
  Q8Walk w;
  w.b = b0 - 1;
  w.ta = 0;
  w.tb = static_cast<int>(off0);  // (where the first segment starts)
  w.n_tiles = 0;
  w.left = tiles;
  return w;
}
// The next segment; false at the end. (Its search is one function for all roles: code that is met once costs what
// it takes to fetch, some ten cycles an instruction, and so it has been fetched after the first role's call.)
template <int kT>
__device__ __noinline__ Q8Walk q8_search(const int32_t* lens_global, const int32_t* lens_cached, int q_len, int bs,
                                         int causal, int window, int sinks, int b, int start, int64_t left) {
  const Q8Lens lens{lens_global, lens_cached};
  Q8Walk w;
  do {
    ++b;
    w.v = window_view(lens(b), q_len, bs, causal, window, sinks);
    w.n_tiles = q8_tiles(w.v, kT);
  } while (w.n_tiles == 0);
  w.b = b;
  w.ta = start;
  w.tb = static_cast<int>(w.n_tiles < start + left ? w.n_tiles : start + left);
  w.left = left - (w.tb - start);
  return w;
}
template <int kT>
__device__ __forceinline__ bool q8_next(const DecodeQ8Params& p, const Q8Lens& lens, Q8Walk& w, bool first) {
  if (w.left <= 0) return false;
  w = q8_search<kT>(lens.global, lens.cached, p.q_len, p.bs, p.causal, p.window, p.sinks, w.b, first ? w.tb : 0, w.left);
  return true;
}

}  // namespace mla
