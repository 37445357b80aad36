// A step's block tables and slot map from the requests' lengths, and the cache write through the slot map, sm_103a.
//
// Request b has L_b tokens and gets (or, negative, gives back) n_b. With P(x) = ceil(x / bs) pages for x tokens:
//  - back_b = P(L_b) - P(L_b + n_b) pages of each shrinking request go onto the stack of free pages, in the
//    requests' order; top = count + sum back_b;
//  - take_b = P(L_b + n_b) - P(L_b) pages of each growing request come from the stack's top, in the requests'
//    order: with T_b = sum over growing requests before b of take, the j-th new page is stack[top - 1 - T_b - j];
//  - new token i of request b is token t = L_b + i, slot page * bs + t % bs, at place Q_b + i, Q_b the new
//    tokens of the requests before b.
// Three exclusive prefix sums over the requests, then independent work per page given back and per new token (a new
// page's first token is a new token, which writes the page's table entry). A page that another request has just
// given back is looked up where that request's row still has it (the place on the stack tells which), so no thread
// waits for another's write. What bounds it is latency: launch, one round of loads, the scans (two barriers each),
// one search in shared memory, one or two dependent loads. A step of 256 single tokens takes 5.5 us a call in a
// replayed graph.
//
// One CTA does all of a small step. Where there are more than 4096 places in `slots`, it leaves them to a second kernel
// over the whole device, which reads offsets, lengths and tables back (256 requests: 4096 places 7.8 us a call with one
// kernel, 8.6 with two; 8192: 11.6, 9.9; 16,384: 18.3, 10.2):
// 512 requests, 30% of which give pages back, and 100,147 new tokens in all: 13.7 us a call; 23.1 us with a cluster of
// eight CTAs that scanned the requests each and wrote the slots, too.
//
// mla_cache_append_slots: a copy of 1152 bytes a token, HBM-bound: a warp a token (four tokens a warp, all their loads in
// flight together, took as long from 16,384 tokens on and longer below). 65,536 tokens: 22.6 us, 6.7 TB/s, the rate of a
// plain copy; 24 tokens: 1 us in a replayed graph.
#include "block_scan.cuh"
#include "device_common.cuh"

namespace mla {

namespace {

constexpr int kFewSlots = 4096;  // up to so many places in `slots`: one CTA
constexpr int kThreads = 1024;
static_assert(kThreads == 32 * kScanWarps, "block_scan's");
constexpr int kEach = 4;  // pages that a thread looks up before it stores any

struct Request {
  long long len;   // tokens before the step
  long long base;  // tokens that stay: before the new ones, or after those given back
  long long next;  // tokens that are asked for
  long long held, want;  // pages before and after
  long long back, take, grow;
};

__device__ __forceinline__ Request request_of(const TablesParams& p, int b) {
  Request r;
  const long long len = max(p.lens[b], 0), d = max(static_cast<long long>(p.changes[b]), -len);
  r.len = len;
  r.next = len + d;
  r.base = min(len, r.next);
  r.held = (len + p.bs - 1) >> p.bs_shift;
  r.want = (r.next + p.bs - 1) >> p.bs_shift;
  const long long width = p.max_blocks;
  r.back = d < 0 ? max(min(r.held, width) - r.want, 0ll) : 0;  // (a row holds no more than its width)
  r.take = d > 0 ? r.want - r.held : 0;
  r.grow = d > 0 ? d : 0;
  return r;
}

// The cache row of token t in its page; -1 for a page outside the pool.
__device__ __forceinline__ long long slot_of(const TablesParams& p, int32_t page, int t, bool* bad) {
  const bool ok = page >= 0 && page < p.num_blocks;
  *bad |= !ok;
  return ok ? (static_cast<long long>(page) << p.bs_shift) + (t & (p.bs - 1)) : -1ll;
}

// kSlots: the slots, too; else the next kernel writes them.
template <bool kSlots>
__global__ void __launch_bounds__(kThreads, 1) mla_update_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t sh[];
  __shared__ long long part[kScanWarps];
  __shared__ int first_misfit;
  __shared__ long long misfit_q, misfit_take;
  const int B = p.B, tid = threadIdx.x;
  int32_t* const q_at = sh;                // [B + 1] new tokens of the requests before
  int32_t* const take_at = q_at + B + 1;   // [B] pages taken by them
  int32_t* const back_at = take_at + B;    // [B + 1] pages given back by them
  int32_t* const base_of = back_at + B + 1;  // [B]
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) first_misfit = B;

  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long back = 0, take = 0, grow = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    back += r.back;
    take += r.take;
    grow += r.grow;
  }
  const long long count = min(max(*p.free_count, 0), p.num_blocks);
  long long all_back, all_take, all_grow;
  back = block_scan(back, part, &all_back);
  take = block_scan(take, part, &all_take);
  grow = block_scan(grow, part, &all_grow);
  // (more than the pool has: a page given back twice)
  if (tid == 0 && count + all_back > p.num_blocks) flag_error(MLA_DEVERR_BAD_PAGE);
  const long long top = min(count + all_back, static_cast<long long>(p.num_blocks));

  // the first growing request that does not fit; those from it on do not grow
  {
    long long t = take, q = grow;
    for (int b = b0; b < b1; ++b) {
      const Request r = request_of(p, b);
      if (r.grow > 0 && (t + r.take > top || r.want > p.max_blocks || q + r.grow > p.capacity || r.next > 0x7fffffffll)) {
        atomicMin(&first_misfit, b);
        break;
      }
      t += r.take;
      q += r.grow;
    }
  }
  __syncthreads();
  const int served = first_misfit;
  long long lens = 0;
  {
    long long t = take, q = grow, k = back;
    for (int b = b0; b < b1; ++b) {
      const Request r = request_of(p, b);
      if (b == served) {
        misfit_q = q;
        misfit_take = t;
      }
      if (b <= served) {  // (bounded by the capacity and the pool there)
        q_at[b] = static_cast<int32_t>(q);
        take_at[b] = static_cast<int32_t>(t);
      }
      back_at[b] = static_cast<int32_t>(min(k, 0x7fffffffll));
      base_of[b] = static_cast<int32_t>(r.base);
      lens += r.grow > 0 && b >= served ? r.len : r.next;
      t += r.take;
      q += r.grow;
      k += r.back;
    }
  }
  __syncthreads();
  const int32_t tokens = static_cast<int32_t>(served < B ? misfit_q : all_grow);
  const long long taken = served < B ? misfit_take : all_take;
  for (int b = tid; b < B; b += kThreads)
    if (b > served) q_at[b] = tokens;
  if (tid == 0) {
    q_at[B] = tokens;
    back_at[B] = static_cast<int32_t>(min(all_back, 0x7fffffffll));
  }
  long long all_lens;
  lens = block_scan(lens, part, &all_lens);  // (its barriers also publish what was written above)

  // the inputs are read before outputs that may be the same memory are written
  int32_t keep_len[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (b0 + j < b1) {
      const Request r = request_of(p, b0 + j);
      keep_len[j] = static_cast<int32_t>(r.grow > 0 && b0 + j >= served ? r.len : r.next);
    }
  }
  __syncthreads();
  long long s = lens;
  bool over = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (b0 + j < b1) {
      const int b = b0 + j;
      over |= s > 0x7fffffffll;
      p.lens_out[b] = keep_len[j];
      p.q_indptr[b] = q_at[b];
      p.kv_indptr[b] = static_cast<int32_t>(min(s, 0x7fffffffll));
      s += keep_len[j];
    }
  }
  if (tid == 0) {
    over |= all_lens > 0x7fffffffll;
    p.q_indptr[B] = tokens;
    p.kv_indptr[B] = static_cast<int32_t>(min(all_lens, 0x7fffffffll));
    *p.free_count_out = static_cast<int32_t>(top - taken);
    *p.served = served;
  }
  if (over) flag_error(MLA_DEVERR_BAD_PAGE);
  const int shift = p.bs_shift;
  // pages given back: the k-th of the step goes to stack[count + k]
  auto given_back = [&](int k) {
    const int b = find_last(back_at, 0, B - 1, k);
    const int col = ((base_of[b] + p.bs - 1) >> shift) + (k - back_at[b]);
    return p.block_table[static_cast<long long>(b) * p.max_blocks + col];
  };
  for (int k0 = tid; count + k0 < top; k0 += kEach * kThreads) {
    int32_t page[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (count + k0 + j * kThreads < top) page[j] = given_back(k0 + j * kThreads);
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (count + k0 + j * kThreads < top) p.pages[count + k0 + j * kThreads] = page[j];
  }
  // the j-th page that request b takes
  auto page_taken = [&](int b, int j) {
    const int at = static_cast<int>(top) - 1 - take_at[b] - j;
    return at < count ? p.pages[at] : given_back(at - static_cast<int>(count));
  };
  if constexpr (!kSlots) {
    for (int i0 = tid; i0 < taken; i0 += kEach * kThreads) {
      int32_t page[kEach];
      int32_t* entry[kEach];
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int i = i0 + k * kThreads;
        if (i >= taken) continue;
        // (as many requests as were served: those behind have no places in take_at)
        const int b = find_last(take_at, 0, min(served, B - 1), i), j = i - take_at[b];
        entry[k] = p.block_table + static_cast<long long>(b) * p.max_blocks + ((base_of[b] + p.bs - 1) >> shift) + j;
        page[k] = page_taken(b, j);
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (i0 + k * kThreads < taken) *entry[k] = page[k];
    }
  } else {
    bool bad = false;
    for (int i = tid; i < tokens; i += kThreads) {
      const int b = find_last(q_at, 0, B - 1, i);
      const int t = base_of[b] + (i - q_at[b]);
      const int col = t >> shift, held = static_cast<int>((static_cast<long long>(base_of[b]) + p.bs - 1) >> shift);
      int32_t* const entry = p.block_table + static_cast<long long>(b) * p.max_blocks + col;
      int32_t page;
      if (col < held) {
        page = *entry;
      } else {
        page = page_taken(b, col - held);
        if ((t & (p.bs - 1)) == 0) *entry = page;
      }
      p.slots[i] = slot_of(p, page, t, &bad);
    }
    for (long long i = static_cast<long long>(tokens) + tid; i < p.capacity; i += kThreads) p.slots[i] = -1;
    if (bad) flag_error(MLA_DEVERR_BAD_PAGE);
  }
}

// The slots of a step with many places, from the tables that the kernel above has written.
constexpr int kSlotThreads = 256, kSlotsEach = 4;

__global__ void __launch_bounds__(kSlotThreads) mla_step_slots_kernel(const TablesParams p) {
  extern __shared__ int32_t q_at[];  // [B + 1]
  pdl_wait();
  pdl_launch_dependents();
  for (int b = threadIdx.x; b <= p.B; b += kSlotThreads) q_at[b] = p.q_indptr[b];
  __syncthreads();
  const int tokens = q_at[p.B];
  bool bad = false;
  const long long step = static_cast<long long>(gridDim.x) * kSlotThreads * kSlotsEach;
  for (long long i0 = static_cast<long long>(blockIdx.x) * kSlotThreads * kSlotsEach + threadIdx.x; i0 < p.capacity; i0 += step) {
    long long slot[kSlotsEach];
#pragma unroll
    for (int k = 0; k < kSlotsEach; ++k) {
      const long long i = i0 + k * kSlotThreads;
      slot[k] = -1;
      if (i >= tokens) continue;
      const int b = find_last(q_at, 0, p.B - 1, static_cast<int32_t>(i));
      const int t = p.lens_out[b] - (q_at[b + 1] - static_cast<int>(i));  // (its new tokens are its last)
      slot[k] = slot_of(p, p.block_table[static_cast<long long>(b) * p.max_blocks + (t >> p.bs_shift)], t, &bad);
    }
#pragma unroll
    for (int k = 0; k < kSlotsEach; ++k)
      if (i0 + k * kSlotThreads < p.capacity) p.slots[i0 + k * kSlotThreads] = slot[k];
  }
  if (bad) flag_error(MLA_DEVERR_BAD_PAGE);
}

constexpr int kCopyWarps = 8;

// A warp a token. Lane l holds its columns 8 l.. and 256 + 8 l.., and of the rope columns 8 l.. (l < 8).
__global__ void __launch_bounds__(kCopyWarps * 32) mla_cache_append_slots_kernel(const AppendSlotsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long tok = static_cast<long long>(blockIdx.x) * kCopyWarps + warp;
  if (tok >= p.tokens) return;
  const long long slot = p.slots[tok];
  if (slot < 0) return;
  if (slot >= p.rows) {
    if (lane == 0) flag_error(MLA_DEVERR_BAD_PAGE);
    return;
  }
  const uint4* const from = reinterpret_cast<const uint4*>(p.ckv_new + tok * p.ckv_stride);
  const uint4 c0 = from[lane], c1 = from[lane + 32];
  uint4 r;
  if (lane < 8) r = reinterpret_cast<const uint4*>(p.kpe_new + tok * p.kpe_stride)[lane];
  uint4* const to = reinterpret_cast<uint4*>(p.ckv + slot * kRank);
  to[lane] = c0;
  to[lane + 32] = c1;
  if (lane < 8) reinterpret_cast<uint4*>(p.kpe + slot * kRope)[lane] = r;
}

template <class Params>
cudaError_t launch_dependent(void (*kernel)(const Params), unsigned grid, unsigned block, size_t smem, const Params& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_update_tables(const TablesParams& p, cudaStream_t stream) {
  static DeviceOnce once, once_slots;
  const bool few = p.capacity <= kFewSlots;
  const auto kernel = few ? &mla_update_tables_kernel<true> : &mla_update_tables_kernel<false>;
  const size_t smem = (static_cast<size_t>(p.B) * 4 + 2) * sizeof(int32_t);
  cudaError_t e = set_attribute_once(few ? once_slots : once, reinterpret_cast<const void*>(kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (kMaxStepRequests * 4 + 2) * static_cast<int>(sizeof(int32_t)));
  if (e != cudaSuccess) return e;
  e = launch_dependent(kernel, 1, kThreads, smem, p, stream);
  if (e != cudaSuccess || few) return e;
  constexpr int kMostCtas = 1024;
  const long long ctas = (static_cast<long long>(p.capacity) + kSlotThreads * kSlotsEach - 1) / (kSlotThreads * kSlotsEach);
  return launch_dependent(mla_step_slots_kernel, static_cast<unsigned>(ctas < kMostCtas ? ctas : kMostCtas), kSlotThreads,
                          (static_cast<size_t>(p.B) + 1) * sizeof(int32_t), p, stream);
}

cudaError_t launch_append_slots(const AppendSlotsParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.tokens + kCopyWarps - 1) / kCopyWarps);
  return launch_dependent(mla_cache_append_slots_kernel, grid, kCopyWarps * 32, 0, p, stream);
}

cudaError_t step_tables_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
