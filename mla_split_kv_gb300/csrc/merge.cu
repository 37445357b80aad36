// LSE-weighted merge of request-major partials (base-2 LSE).
//
// "feat(core): matrix-absorbed MLA decode over a compressed-latent KV cache",
// *How #898's merge kernel is reused*: partials of request b are rows
// o_indptr[b] .. o_indptr[b+1]-1, their LSE is base 2. "[kernel] Wire MLA
// split-KV decode", *What changed*: the reduce combines slices by their LSE so
// the result equals ordinary attention. MTPLX PR #639 commit log: a partial with
// LSE = -inf has weight 0, an all -inf row merges to zeros, and the fp32
// result is rounded once to the output dtype.
//
// One warp per (request, row, 128-column quarter); each lane owns 4 columns.
// The kernel is a programmatic dependent launch: it may be scheduled while the
// partial kernel that precedes it still runs, and waits for that grid before
// its first read, so its launch latency hides behind the partial kernel's end.
// The weights are computed lane-parallel (lane s holds partial s), the sum over
// partials runs in fixed order, so the result is bitwise reproducible.
#include <algorithm>

#include "device_common.cuh"

namespace mla {

namespace {

constexpr int kWarps = 2;

__global__ void __launch_bounds__(kWarps * 32) mla_merge_kernel(const MergeParams p) {
  // Launched as a programmatic dependent of the partial kernel: everything this
  // kernel reads may still be in flight until the wait returns. The next kernel
  // (the next layer's partial kernel) is released after the wait and may start
  // its set-up while this one works.
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long total = static_cast<long long>(p.B) * p.rows * 4;
  if (gw >= total) return;
  const int quarter = static_cast<int>(gw & 3);
  const long long br = gw >> 2;  // b * rows + row
  const int b = static_cast<int>(br / p.rows);
  const int row = static_cast<int>(br % p.rows);
  const int lo = p.o_indptr[b], hi = p.o_indptr[b + 1];
  const int n = hi - lo;

  const float* col = p.partials + static_cast<long long>(row) * kRank + quarter * 128 + lane * 4;
  const long long stride = static_cast<long long>(p.rows) * kRank;  // one partial slot
  // the first 8 partials' values do not depend on the weights: their loads go out with the LSE loads
  float4 v0[8];
#pragma unroll
  for (int jj = 0; jj < 8; ++jj)
    v0[jj] = (jj < n) ? *reinterpret_cast<const float4*>(col + (lo + jj) * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
  // maximum LSE over this row's partials; lane s keeps the LSE of partial s (s < 32)
  const float l0 = (lane < n) ? p.lse[static_cast<long long>(lo + lane) * p.rows + row] : -INFINITY;
  float M = l0;
  for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, p.lse[static_cast<long long>(lo + s) * p.rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));

  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int cnt = min(32, n - s0);
      float wl = 0.f;
      if (lane < cnt) {
        const float l = (s0 == 0) ? l0 : p.lse[static_cast<long long>(lo + s0 + lane) * p.rows + row];
        wl = (l == -INFINITY) ? 0.f : exp2f(l - M);
      }
      // batches of 8 partials: all loads of a batch in flight at once, then the
      // weighted sum in partial order
      for (int j0 = 0; j0 < cnt; j0 += 8) {
        float4 v[8];
#pragma unroll
        for (int jj = 0; jj < 8; ++jj)
          v[jj] = (s0 + j0 == 0) ? v0[jj]
                  : (j0 + jj < cnt) ? *reinterpret_cast<const float4*>(col + (lo + s0 + j0 + jj) * stride)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
          const float wj = __shfl_sync(0xffffffffu, wl, (j0 + jj) & 31);
          if (j0 + jj < cnt) {
            den += wj;
            acc.x = fmaf(wj, v[jj].x, acc.x);
            acc.y = fmaf(wj, v[jj].y, acc.y);
            acc.z = fmaf(wj, v[jj].z, acc.z);
            acc.w = fmaf(wj, v[jj].w, acc.w);
          }
        }
      }
    }
    acc = make_float4(acc.x / den, acc.y / den, acc.z / den, acc.w / den);
  }
  const long long o_off = br * kRank + quarter * 128 + lane * 4;
  if (p.out_dtype == 2) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o_off) = acc;
  } else {
    uint16_t h[4];
    const bool bf = (p.out_dtype == 1);
    const float f[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = bf ? f2h<true>(f[j]) : f2h<false>(f[j]);
    uint2 packed;
    packed.x = static_cast<uint32_t>(h[0]) | (static_cast<uint32_t>(h[1]) << 16);
    packed.y = static_cast<uint32_t>(h[2]) | (static_cast<uint32_t>(h[3]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o_off) = packed;
  }
  if (p.out_lse != nullptr && quarter == 0 && lane == 0)
    p.out_lse[br] = (M == -INFINITY) ? -INFINITY : M + log2f(den);
}

// The same merge, the same operations in the same order, for batches with rows to fill the device with fewer warps a
// (request, row): one, or two, a lane owning 4 columns of each of its warp's quarters, so the weights' code runs once
// (twice) a row instead of four times. A request of many partials goes through rounds of loads one behind the other
// whatever its batch, so from 2048 rows on, where one such request sets the time, two warps with eight partials in
// flight take a row, from 4096 on, or where no request can have many, one warp with two. Measured, one warp / two /
// four: 2048 rows with 2 partials a row 3.6 / 4.1 / 6.3 us, with 9 6.1 / 5.7 / 8.3, with 40 29 / 27.5 / 31, with 20 (60,
// 76) in one request of 16 and 1 (1, 2) in the others 5.6 (11.3, 14.1) / 4.2 (6.8, 8.2) / 6.5 (7.4, 8.3); 4096 rows with
// 60 in one request of 32 11.4 / 7.8 / 12.0, with 16 a row 25.8 / 21.9 / 24.8; behind a partial kernel two warps take
// longer than one, 2560 rows with 1 partial a row, whole calls 41.7 against 42.9 us, 3840 rows 25.3 against 26.8, 4096
// rows with 2 108.0 against 109.1. Below 2048 rows four warps are four chains of loads side by side: 1024 rows with 2 /
// 9 partials 2.6 / 4.0 us with one against 3.9 / 5.3, but 1 us more behind a partial kernel (fewer of its larger blocks
// are resident early); 512 rows 2.4 / 3.6 against 2.4 / 3.2.
constexpr long long kMinRows = 2048, kMinRowsOneWarp = 4096, kFewParts = 24;
template <int kRowWarps>  // warps a row
struct RowMerge {
  static constexpr int kQuarters = 4 / kRowWarps, kAhead = kRowWarps == 1 ? 2 : 8;
  static constexpr int kBlockRows = kRowWarps == 1 ? 4 : 1, kThreads = kBlockRows * kRowWarps * 32;
  static constexpr int kMinBlocks = kRowWarps == 1 ? 6 : 10;  // registers for six blocks of 128 threads, ten of 64: no spills
};

template <int kRowWarps>
__global__ void __launch_bounds__((RowMerge<kRowWarps>::kThreads), (RowMerge<kRowWarps>::kMinBlocks))
    mla_merge_rows_kernel(const MergeParams p) {
  using C = RowMerge<kRowWarps>;
  constexpr int kQuarters = C::kQuarters, kAhead = C::kAhead;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long br = static_cast<long long>(blockIdx.x) * C::kBlockRows + warp / kRowWarps;  // b * rows + row
  if (br >= static_cast<long long>(p.B) * p.rows) return;
  const int b = static_cast<int>(br / p.rows), row = static_cast<int>(br % p.rows);
  const int lo = p.o_indptr[b], n = p.o_indptr[b + 1] - lo;
  const int first_col = warp % kRowWarps * (kQuarters * 128) + lane * 4;
  const float* const col = p.partials + static_cast<long long>(row) * kRank + first_col;
  const long long stride = static_cast<long long>(p.rows) * kRank;  // one partial slot
  auto load = [&](float4 (&v)[kAhead][kQuarters], int j0, int cnt) {
#pragma unroll
    for (int jj = 0; jj < kAhead; ++jj)
#pragma unroll
      for (int q = 0; q < kQuarters; ++q)
        v[jj][q] = (j0 + jj < cnt) ? *reinterpret_cast<const float4*>(col + (lo + j0 + jj) * stride + q * 128)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 v[kAhead][kQuarters];
  load(v, 0, n);  // (they do not depend on the weights)
  const float l0 = (lane < n) ? p.lse[static_cast<long long>(lo + lane) * p.rows + row] : -INFINITY;
  float M = l0;
  for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, p.lse[static_cast<long long>(lo + s) * p.rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 acc[kQuarters];
#pragma unroll
  for (int q = 0; q < kQuarters; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  if (M != -INFINITY) {
    float wl = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += kAhead) {
      if (j0 % 32 == 0) {  // lane s holds the weight of partial j0 + s
        wl = 0.f;
        if (j0 + lane < n) {
          const float l = (j0 == 0) ? l0 : p.lse[static_cast<long long>(lo + j0 + lane) * p.rows + row];
          wl = (l == -INFINITY) ? 0.f : exp2f(l - M);
        }
      }
#pragma unroll
      for (int jj = 0; jj < kAhead; ++jj) {
        if (jj > 0 && jj % 2 == 0 && j0 + jj >= n) break;
        const float wj = __shfl_sync(0xffffffffu, wl, (j0 + jj) & 31);
        if (j0 + jj < n) {
          den += wj;
#pragma unroll
          for (int q = 0; q < kQuarters; ++q) {
            acc[q].x = fmaf(wj, v[jj][q].x, acc[q].x);
            acc[q].y = fmaf(wj, v[jj][q].y, acc[q].y);
            acc[q].z = fmaf(wj, v[jj][q].z, acc[q].z);
            acc[q].w = fmaf(wj, v[jj][q].w, acc[q].w);
          }
        }
      }
      if (j0 + kAhead < n) load(v, j0 + kAhead, n);
    }
#pragma unroll
    for (int q = 0; q < kQuarters; ++q) acc[q] = make_float4(acc[q].x / den, acc[q].y / den, acc[q].z / den, acc[q].w / den);
  }
#pragma unroll
  for (int q = 0; q < kQuarters; ++q) store_out4(p.out, p.out_dtype, br * kRank + first_col + q * 128, acc[q]);
  if (p.out_lse != nullptr && lane == 0 && warp % kRowWarps == 0) p.out_lse[br] = (M == -INFINITY) ? -INFINITY : M + log2f(den);
}

// sum_e w_e l_e of a row from its entries' second copies, over the warp
__device__ __forceinline__ float second_sum(const float* ml1, long long mlstride, int e0, int e1, float M, int lane) {
  float s = 0.f;
  for (int e = e0 + lane; e < e1; e += 32) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(ml1 + e * mlstride));
    s = fmaf((ml.x == -INFINITY) ? 0.f : exp2f(ml.x - M), ml.y, s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The merge of the paired kernel's pair entries into the output (mla_decode's default on that
// kernel). Entry e holds one CTA pair's unnormalized O (its tokens, all 512 columns: each CTA of
// the pair wrote its 256), its row maximum m_e and its row sum l_e relative to m_e. Per (request,
// row): M = max_e m_e, w_e = 2^(m_e - M) (0 for m_e = -inf), out = sum_e w_e O_e / sum_e w_e l_e,
// out_lse = M + log2 sum_e w_e l_e -- the merge of the pages' contract, applied to unnormalized
// parts. One warp per (request, row, 16 columns): lane = 4 g + q takes column quad q of the entries
// g, g + 8, g + 16, ... (up to 12 per lane, 96 entries, in one round of loads), sums them in entry
// order, and the warp adds the eight entry groups with a fixed shuffle tree, so the result is the
// same bits on every call.
//
// Residency: a CTA is 128 threads of at most 128 registers and no shared memory, so one fits on an
// SM beside a CTA of the paired kernel (384 threads x 128 registers, 226 KB). The merge of call n
// is therefore resident while its partial kernel runs, and it releases its own dependent (the next
// call's partial kernel) at once: that kernel waits for this one to complete before it reads
// anything, and its CTAs take each SM as the partial CTA there leaves, beside this merge's CTA.
constexpr int kEntryWarps = 4;
constexpr int kEntryGroups = 8;                  // entry groups per warp
constexpr int kEntriesPerLane = 12;              // per round of loads
constexpr int kEntryRound = kEntryGroups * kEntriesPerLane;

// One warp's 16 columns of a (request, row): the request's entries [e0, e1).
__device__ __forceinline__ void merge_entry_columns(const EntryMergeParams& p, long long br, int row, int cb, int e0, int e1,
                                                    int lane) {
  const int g = lane >> 2, q = lane & 3;
  const int col = 16 * cb + 4 * q;
  const long long ostride = static_cast<long long>(p.rows) * kRank;  // one entry's O
  const float* const obase = p.ws_partials + static_cast<long long>(row) * kRank + col;
  const float* const mlbase = p.ws_lse + static_cast<long long>(row) * 2;  // copy 0 of the entry's m, l
  const long long mlstride = 4LL * p.rows;                                  // one entry's two copies
  // round 0: the first 96 entries' m, l and values (the values do not depend on the weights)
  float2 ml0[kEntriesPerLane];
  float4 v0[kEntriesPerLane];
#pragma unroll
  for (int j = 0; j < kEntriesPerLane; ++j) {
    const int e = e0 + g + kEntryGroups * j;
    const bool in = e < e1;
    ml0[j] = in ? __ldcg(reinterpret_cast<const float2*>(mlbase + e * mlstride)) : make_float2(-INFINITY, 0.f);
    v0[j] = in ? __ldcg(reinterpret_cast<const float4*>(obase + e * ostride)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
#pragma unroll
  for (int j = 0; j < kEntriesPerLane; ++j) M = fmaxf(M, ml0[j].x);
  for (int base = e0 + kEntryRound; base < e1; base += kEntryRound)
#pragma unroll
    for (int j = 0; j < kEntriesPerLane; ++j) {
      const int e = base + g + kEntryGroups * j;
      if (e < e1) M = fmaxf(M, __ldcg(mlbase + e * mlstride));
    }
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 4));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY) {
    for (int base = e0; base < e1; base += kEntryRound) {
#pragma unroll
      for (int j = 0; j < kEntriesPerLane; ++j) {
        const int e = base + g + kEntryGroups * j;
        float2 ml;
        float4 v;
        if (base == e0) {
          ml = ml0[j];
          v = v0[j];
        } else {
          const bool in = e < e1;
          ml = in ? __ldcg(reinterpret_cast<const float2*>(mlbase + e * mlstride)) : make_float2(-INFINITY, 0.f);
          v = in ? __ldcg(reinterpret_cast<const float4*>(obase + e * ostride)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float w = (ml.x == -INFINITY) ? 0.f : exp2f(ml.x - M);
        den = fmaf(w, ml.y, den);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    den += __shfl_xor_sync(0xffffffffu, den, o);
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  float den_lse = den;
  if (p.exact_lse && cb == 0 && M != -INFINITY) den_lse = second_sum(mlbase + 2 * p.rows, mlstride, e0, e1, M, lane);
  if (g != 0) return;
  float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY) out = make_float4(acc.x / den, acc.y / den, acc.z / den, acc.w / den);
  store_out4(p.out, p.out_dtype, br * kRank + col, out);
  if (p.out_lse != nullptr && cb == 0 && q == 0) p.out_lse[br] = merged_lse(M, den_lse);
}

__global__ void __launch_bounds__(kEntryWarps * 32, 4) mla_merge_entries_kernel(const EntryMergeParams p) {
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = static_cast<long long>(blockIdx.x) * kEntryWarps + warp;
  const bool active = gw < static_cast<long long>(p.B) * p.rows * 32;
  const int cb = static_cast<int>(gw & 31);  // columns [16 cb, 16 cb + 16)
  const long long br = gw >> 5;              // b * rows + row
  const int b = static_cast<int>(br / p.rows), row = static_cast<int>(br % p.rows);
  // the offsets are an input of the call, not data of the partial kernel: with tables_ready (complete
  // before that kernel started) they are read before the wait, so the entries' loads follow it at once
  int e0 = 0, e1 = 0;
  if (active && p.tables_ready) {
    e0 = __ldg(p.o_indptr + b) * p.epc;
    e1 = __ldg(p.o_indptr + b + 1) * p.epc;
  }
  pdl_wait();  // the entries are complete once the partial kernel has
  if (!active) return;
  if (!p.tables_ready) {
    e0 = p.o_indptr[b] * p.epc;
    e1 = p.o_indptr[b + 1] * p.epc;
  }
  merge_entry_columns(p, br, row, cb, e0, e1, lane);
}

// The same for batches, whose requests have few entries each: two warps a (request, row), 8 columns a lane, the same
// operations in the same order (entry groups g, g + 8 summed in entry order, then added in the shuffles' order).
// A warp of the kernel above looks after 12 entries a lane whether they are there or not; 32 of them a row, a thousand
// rows are 13 waves of blocks.
constexpr int kEntryRowWarps = 2, kEntryRowLoads = 4 / kEntryRowWarps;
// Measured as whole calls of 16 rows, against the kernel above: 4 requests with 8 / 18 entries each 11.5 / 17.3 us
// against 12.0 / 14.5, 8 with 4 / 9 entries 11.8 / 16.2 against 14.2 / 17.1, 32 with 2 entries 12.9 against 26.0,
// 64 with one 13.2 against 41.5. So a request of more than 12 entries is merged as above, request by request (the host
// knows no request's count, only their sum): the grid's last blocks look such requests up in the offsets and share
// their (row, 16 columns) out. One of 131,072 tokens, 40 entries, beside seven of 2000: 62.8 us, 67.1 by rows; 16
// requests of 4096 tokens, where the last blocks find nothing, 25.2 (26.7 with a list of 528 bytes of shared memory,
// for which an SM has no room beside the paired kernel).
constexpr long long kMinEntryRows = 128;
constexpr int kMaxRowEntries = 12, kLongBlocks = 256;

__global__ void __launch_bounds__(kEntryWarps * 32, 4)
    mla_merge_entries_rows_kernel(const EntryMergeParams p, uint32_t row_blocks) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= row_blocks) {
    // long requests: of 32 in a row, one a lane, shared with the warps that look at the same ones (no shared memory,
    // see above)
    const int warps = (gridDim.x - row_blocks) * kEntryWarps, me = (blockIdx.x - row_blocks) * kEntryWarps + warp;
    const int portions = (p.B + 31) / 32, portion = me % portions, b = portion * 32 + lane;
    pdl_wait();
    const uint32_t found = __ballot_sync(
        0xffffffffu, b < p.B && (__ldcg(p.o_indptr + b + 1) - __ldcg(p.o_indptr + b)) * p.epc > kMaxRowEntries);
    const int per_request = p.rows * 32, units = __popc(found) * per_request;
    const int step = (warps - portion + portions - 1) / portions;
    for (int u = me / portions; u < units; u += step) {
      const int which = portion * 32 + static_cast<int>(__fns(found, 0, u / per_request + 1)), row = u % per_request / 32;
      merge_entry_columns(p, static_cast<long long>(which) * p.rows + row, row, u % 32, __ldcg(p.o_indptr + which) * p.epc,
                          __ldcg(p.o_indptr + which + 1) * p.epc, lane);
    }
    return;
  }
  const long long gw = static_cast<long long>(blockIdx.x) * kEntryWarps + warp;
  const long long br = gw / kEntryRowWarps;  // b * rows + row
  const bool active = br < static_cast<long long>(p.B) * p.rows;
  const int b = static_cast<int>(br / p.rows), row = static_cast<int>(br % p.rows);
  int e0 = 0, e1 = 0;
  if (active && p.tables_ready) {
    e0 = __ldg(p.o_indptr + b) * p.epc;
    e1 = __ldg(p.o_indptr + b + 1) * p.epc;
  }
  pdl_wait();  // the entries are complete once the partial kernel has
  if (!active) return;
  if (!p.tables_ready) {
    e0 = p.o_indptr[b] * p.epc;
    e1 = p.o_indptr[b + 1] * p.epc;
  }
  if (e1 - e0 > kMaxRowEntries) return;  // a long request
  const int col = static_cast<int>(gw % kEntryRowWarps) * (kRank / kEntryRowWarps) + 4 * lane;
  const long long ostride = static_cast<long long>(p.rows) * kRank;  // one entry's O
  const float* const obase = p.ws_partials + static_cast<long long>(row) * kRank + col;
  const float* const mlbase = p.ws_lse + static_cast<long long>(row) * 2;  // copy 0 of the entry's m, l
  const long long mlstride = 4LL * p.rows;                                  // one entry's two copies
  // the first entries' values (they do not depend on the weights)
  float4 v[kEntryGroups];
  auto load = [&](int base, int k) {
#pragma unroll
    for (int g = 0; g < kEntryGroups; ++g)
      v[g] = base + g < e1 ? __ldcg(reinterpret_cast<const float4*>(obase + (base + g) * ostride + 128 * k))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(e0, 0);
  // lane x weighs entry e0 + x
  const float2 ml = e0 + lane < e1 ? __ldcg(reinterpret_cast<const float2*>(mlbase + (e0 + lane) * mlstride)) : make_float2(-INFINITY, 0.f);
  float M = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float w = (ml.x == -INFINITY) ? 0.f : exp2f(ml.x - M);
  auto tree = [](const float* a) -> float { return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7])); };
  float den = 0.f;
#pragma unroll 1
  for (int k = 0; k < kEntryRowLoads; ++k) {
    float d[kEntryGroups], ax[kEntryGroups], ay[kEntryGroups], az[kEntryGroups], aw[kEntryGroups];
#pragma unroll
    for (int g = 0; g < kEntryGroups; ++g) d[g] = ax[g] = ay[g] = az[g] = aw[g] = 0.f;
    if (M != -INFINITY) {
#pragma unroll 1
      for (int base = e0; base < e1; base += kEntryGroups) {
        if (base != e0 || k != 0) load(base, k);
#pragma unroll
        for (int g = 0; g < kEntryGroups; ++g) {
          const float we = __shfl_sync(0xffffffffu, w, base - e0 + g), le = __shfl_sync(0xffffffffu, ml.y, base - e0 + g);
          d[g] = fmaf(we, le, d[g]);
          ax[g] = fmaf(we, v[g].x, ax[g]);
          ay[g] = fmaf(we, v[g].y, ay[g]);
          az[g] = fmaf(we, v[g].z, az[g]);
          aw[g] = fmaf(we, v[g].w, aw[g]);
        }
      }
    }
    den = tree(d);
    float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) out = make_float4(tree(ax) / den, tree(ay) / den, tree(az) / den, tree(aw) / den);
    store_out4(p.out, p.out_dtype, br * kRank + col + 128 * k, out);
  }
  if (p.out_lse != nullptr && gw % kEntryRowWarps == 0) {
    if (p.exact_lse && M != -INFINITY) den = second_sum(mlbase + 2 * p.rows, mlstride, e0, e1, M, lane);
    if (lane == 0) p.out_lse[br] = merged_lse(M, den);
  }
}

}  // namespace

cudaError_t launch_merge_entries(const EntryMergeParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.rows;
  // by rows where most requests are short (all of them, or all but a few: the sum of the counts is at most 12 a request)
  const bool by_row = rows >= kMinEntryRows && p.entries <= static_cast<long long>(kMaxRowEntries) * p.B;
  const long long warps = rows * (by_row ? kEntryRowWarps : 32);
  long long blocks = (warps + kEntryWarps - 1) / kEntryWarps;
  if (blocks <= 0) return cudaSuccess;
  const uint32_t row_blocks = static_cast<uint32_t>(blocks);
  if (by_row && !p.uniform) {  // as many blocks as the long requests that there may be can use
    const long long most = p.entries / (kMaxRowEntries + 1) * p.rows * (32 / kEntryWarps);
    const long long portions = (p.B + 31) / 32, least = most > 0 ? (portions + kEntryWarps - 1) / kEntryWarps : 0;
    blocks += std::max(least, std::min<long long>(most, kLongBlocks));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kEntryWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return by_row ? cudaLaunchKernelEx(&cfg, mla_merge_entries_rows_kernel, p, row_blocks)
                : cudaLaunchKernelEx(&cfg, mla_merge_entries_kernel, p);
}

cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.rows;
  const bool few = p.most_parts > 0 && p.most_parts <= kFewParts;
  const int row_warps = rows < kMinRows ? 4 : rows >= kMinRowsOneWarp || few ? 1 : 2;
  const int per_block = row_warps == 1 ? RowMerge<1>::kThreads / 32 : row_warps == 2 ? RowMerge<2>::kThreads / 32 : kWarps;
  const long long blocks = (rows * row_warps + per_block - 1) / per_block;
  if (blocks <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(per_block) * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, row_warps == 1   ? mla_merge_rows_kernel<1>
                                  : row_warps == 2 ? mla_merge_rows_kernel<2> : mla_merge_kernel, p);
}

}  // namespace mla
