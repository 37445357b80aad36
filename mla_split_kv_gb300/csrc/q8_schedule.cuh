// How the tiles of a batch are shared out by the block-scaled 8-bit decode and
// found again by its merge.
//
// The batch's visible runs, cut into tiles request after request,
// are one line, with a gap of a few cells between requests: what a gang spends on
// going from one request to the next (its output, the next one's queries, the
// first tiles' rescales: 8 us at 32 rows a CTA, 5 at 16, of tiles of 2600 cycles:
// six, and four) counts as tiles. Gang j of J takes L / J cells of the line's L, the first L % J gangs one
// more (one CTA of a gang per row group), so every gang works as long as the
// others whatever the lengths (without the gaps, gangs with one request ended
// after 55 us, those with two after 65 to 76; calls 4 to 7% slower). Lengths are
// read where they lie: no host plan, and a captured call follows contexts as they
// grow. A request that lies within one gang is finished there; one cut by gang
// borders has a part per gang: its first gang keeps it in entry 1 (that gang's
// open end), the others in entry 0, and ws_cut says how many there are.
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
template <int kCached>
struct Q8Lens {
  const int32_t* global;
  const int32_t* cached;  // shared memory, kCached
  __device__ __forceinline__ int operator()(int b) const { return b < kCached ? cached[b] : __ldcg(global + b); }
};

// A pair of counts in one sum: tiles (at most 65535 * 2^25 < 2^44) and the requests that have any.
constexpr int kQ8CountShift = 44;
constexpr int64_t kQ8Tiles = (int64_t{1} << kQ8CountShift) - 1;
// The gap. Measured with 4 / 5 / 6 / 7 tiles: 32 rows, 8 requests to 64K of 128 heads 141.4 / 140.6 / 139.7 / 138.9 us,
// 48 windows of 4096 of 64 heads 67.0 / 65.6 / 65.7 / 65.6, 4 requests of 9 fp16 rows 141.9 / 140.9 / 140.3 / 140.3; 16
// rows, 300 requests of 500 to 3000 tokens 69.0 / 69.1 / 70.2 / 71.5, 150 of 2K to 9K 90.2 / 90.4 / 91.5 / 92.7, 32 to 16K
// 42.6 with each.
template <int NR>
constexpr int kQ8Gap = NR == 16 ? 4 : 6;

// The line among the gangs that get any of it (all of them unless there are fewer tiles).
struct Q8Line {
  int64_t length, base;      // cells, and those of a gang
  int32_t gangs, more, gap;  // the first `more` gangs have one more
  __device__ __forceinline__ int64_t begin(int j) const { return base * j + min(j, more); }
  // the gang of cell x
  __device__ __forceinline__ int gang_of(int64_t x) const {
    const int64_t head = (base + 1) * more;
    return x < head ? static_cast<int>(div(x, base + 1)) : more + static_cast<int>(div(x - head, base));
  }
  // (32-bit division where it does)
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
  }
};
template <int kGap>
__device__ __forceinline__ Q8Line q8_line(int64_t tiles, int32_t requests, int gangs) {
  Q8Line l;
  // a gap is at most a fifth of a gang's tiles, so every gang has some
  const int64_t share = Q8Line::div(tiles, gangs);
  l.gap = share >= 5 * kGap ? kGap : static_cast<int32_t>(share) / 5;
  l.length = tiles + (requests > 1 ? static_cast<int64_t>(l.gap) * (requests - 1) : 0);
  l.gangs = l.length < gangs ? static_cast<int32_t>(l.length) : gangs;
  l.base = l.gangs > 0 ? Q8Line::div(l.length, l.gangs) : 0;
  l.more = static_cast<int32_t>(l.length - l.base * l.gangs);
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
template <int kT, int kCached>
__device__ __noinline__ Q8Walk q8_search(const int32_t* lens_global, const int32_t* lens_cached, int q_len, int bs,
                                         int causal, int window, int sinks, int B, int b, int start, int64_t left) {
  const Q8Lens<kCached> lens{lens_global, lens_cached};
  Q8Walk w;
  do {
    ++b;
    w.v = window_view(b < B ? lens(b) : 0, q_len, bs, causal, window, sinks);
    w.n_tiles = q8_tiles(w.v, kT);
  } while (w.n_tiles == 0 && b < B);
  if (b >= B) left = 0;  // (only when the lengths changed under the call: the walk ends, the waits run out)
  w.b = b;
  w.ta = start;
  w.tb = static_cast<int>(w.n_tiles < start + left ? w.n_tiles : start + left);
  w.left = left - (w.tb - start);
  return w;
}
template <int kT, int kCached>
__device__ __forceinline__ bool q8_next(const DecodeQ8Params& p, const Q8Lens<kCached>& lens, Q8Walk& w, bool first) {
  if (w.left <= 0) return false;
  w = q8_search<kT, kCached>(lens.global, lens.cached, p.q_len, p.bs, p.causal, p.window, p.sinks, p.B, w.b, first ? w.tb : 0, w.left);
  return true;
}

}  // namespace mla
