// Attention over a block-scaled 8-bit cache, sm_103a.
//
// For each row of a request, over the tokens t that it sees,
//   s_t = scale * z_t * (q_abs . c_t + q_pe . k_t)
//   out = sum_t softmax(s)_t * z_t * c_t,   lse = log2 sum_t exp(s_t)
// with c_t, k_t the E4M3 values of the token's bytes and z_t its block's scale.
//
// The tensor core takes the bytes as they are (kind::f8f6f4, E4M3 x E4M3 with
// fp32 sums): nothing is widened, and a 96-token tile of the whole latent is
// 54 KB, so one CTA holds it for both products and no CTA waits on another.
// What is not 8-bit is split into E4M3 terms, each the rounding of what the
// terms before it leave: x = t1 + 2^-5 t2 + 2^-10 t3 + ... A term keeps 4
// significant bits and leaves at most 2^-4 of its value, so three terms hold
// an fp16 query exactly (11 bits) and two a bf16 one (8 bits), as long as its
// magnitude is above 2^-14 of the row's largest (the row is first scaled by a
// power of two to [128, 256)), and below that to 2^-23 of the largest; the
// weights of the value product, three terms (four for 16 rows), to 2^-14 + 2^-16
// (2^-16) of themselves or 2^-26 of the largest. The terms are further columns
// of the MMA's N side:
//   S^T[tok, (term, row)]  = [c | k][tok, :] . Qterms^T    M=128 tokens, K=576
//   O^T[d, (term, row)]   += c^T[d, tok] . Wterms^T        M=128 columns x 4, K=tokens
// An MMA's time is that of reading its operands from shared memory, 4 KB of A
// (47 cycles up to N = 48, 57 at 96), which the terms share.
//
// A token's scale goes with its weight: with y_t = s_t log2 e + log2 z_t the
// weights are w_t = 2^(y_t - m), m a running maximum of y, so they stay in
// range whatever the scales; out = sum w_t c_t / sum (w_t / z_t), and the LSE
// is m + log2 of that same sum.
//
// NR rows a CTA: 16, or 32 for calls with more (a group of CTAs, a gang, then
// shares each tile through L2). O^T is 4 x kTerms NR columns of tensor memory,
// 384 of the 512 at 32 rows. The tiles of the batch are one line, shared out
// evenly over the gangs (q8_schedule.cuh), and a second kernel merges the
// requests that gang borders cut.
//
// The pipeline. Three tile slots of 54 to 57 KB. A tile's weights take the place of its rope columns, which the scores
// have read by then. One thread issues the score products, another the value
// products (one for both spent the MMAs' time on asking whose inputs were
// there). The softmax warps write weights as 8-byte words of their token's row
// (the value product reads them N-major); byte stores of the K-major layout
// took longer than the MMAs. Four warps share 8 rows and meet once a tile; only
// when a score passes its row's reference by 2^kTau do they take maxima and
// rescale O. After a request's last tile they split the next one's queries
// first, while its last value product runs, then write its output.
//
// What bounds it, in cycles of an SM (2070 MHz) for a 96-token tile: HBM's share
// 2570; the MMAs 1550 with nothing else on shared memory, 2300 as they run. At
// 16 rows a tile takes 2600: HBM. At 32 rows it takes 2600, with the references
// that move early in a request (1700 more each time) 2900 on average: a slot's
// round of load, scores, weights and value product, three at a time. A call has
// some 10 us around that: the lengths and the schedule 1.5 to 2 us, the first
// tiles from HBM 3 us, the last output and the merge 5 us; a good part of it
// is the fetch of code that is met once (ten cycles an instruction), so what
// runs once per call or request is kept short.
//
// Measured (us a call, captured back to back; scaling by HBM alone in brackets):
// 131,072 tokens, 16 fp16 heads 25.5 (11.1); 32 requests up to 16K, 16 bf16 heads
// 42.7 (25.8); 8 requests up to 64K, 128 bf16 heads 139.7 (26.2; the formula's
// products at the card's 16-bit matrix rate 44); 9 causal fp16 rows over 16 heads,
// 4 requests up to 82K, 140.5 (19.9 and 38); 48 requests through a window of 4096,
// 64 bf16 heads, 66.4 (17.3); 37 tokens 10.1.
//
// Warp roles: softmax, rescale and output (thread = token; 8 rows a thread: 8
// warps for 16 rows, 16 for 32), one warp each that issues the score and the
// value products, one that loads pages.
#include "q8_schedule.cuh"

namespace mla {

namespace {

constexpr int kGroupBytes = 8 * kRank;            // 4 KB: 8 tokens, four swizzled [8 x 128] atoms
constexpr int kT = 96;                            // tokens per tile
constexpr int kStep = 32;                         // tokens of an MMA step of the value product
constexpr int kSlots = 3;
constexpr int RH = 8;                             // rows per softmax thread
constexpr float kTermStep = 32.0f, kTermInv = 1.0f / 32.0f;

template <int kLens>
struct Small {
  uint64_t full[kSlots], empty[kSlots];  // tile slots
  uint64_t sfull[2], sfree[2];           // score buffers
  uint64_t pfull[kSlots];                // weights per slot
  uint64_t qfull, ofree, drain[2];
  int64_t scratch[33];
  int64_t off0, first_tile, last_tile;
  int b0;
  uint32_t tmem_base;
  int32_t abort_flag;
  alignas(16) float factor[2][32];       // per row: score scale over the query's power of two, log2 units
  alignas(16) float red[2][4][32];       // per tile parity and token quadrant, rows' maxima (then their sums)
  int32_t lens[kLens];
};

template <int NR, bool BF16>
struct Cfg {
  // terms of a query, of a weight. Four for the weights of 16 rows: 64 columns take the MMA no longer than 48.
  static constexpr int kQTerms = BF16 ? 2 : 3, kTerms = NR == 16 ? 4 : 3;
  // A row's reference lies 2^kWeightExp below the maximum it was taken from and moves when a score passes that by
  // more than kTau, so weights are at most 2^(kTau + kWeightExp), within E4M3's 448, and its subnormals reach down to
  // 2^-25 of the maximum in the last term.
  static constexpr float kTau = NR == 16 ? 7.0f : 2.0f, kWeightExp = NR == 16 ? 1.0f : 6.0f;
  static constexpr int kNS = NR * kQTerms, kNP = NR * kTerms;      // N of the two products
  static constexpr int kSBufs = (4 * kNP + 2 * kNS <= 512) ? 2 : 1;  // score buffers in tensor memory
  // Weights: [kT tokens x kNP] bytes, N-major, a thread storing its token's row as words, in the place of the tile's
  // rope columns, which only the scores read: for 16 rows in rows of 64 bytes with the swizzle of that width, for 32
  // a run of 32-byte rows per term, 3 KB of a slot more than its rope columns.
  static constexpr uint32_t kPRow = NR == 16 ? 64 : 32, kPBytes = kT * kNP;
  static constexpr uint32_t kCkvBytes = kT * kRank;
  static constexpr uint32_t kTileSlot = kCkvBytes + (kPBytes > kT * kRope ? kPBytes : kT * kRope);
  static constexpr uint32_t kQChunk = kNS * 128;                   // [kNS x 128 columns], swizzled
  static constexpr uint32_t kQBytes = kNS * kQkDim;                // four chunks, then [kNS x 64] (64-byte swizzle)
  static constexpr int kLens = NR == 32 && !BF16 ? 64 : 640;       // context lengths kept in shared memory
  static constexpr uint32_t kOffQ = kSlots * kTileSlot;
  static constexpr uint32_t kOffSmall = kOffQ + kQBytes;
  static constexpr uint32_t kSmem = kOffSmall + sizeof(Small<kLens>);
  static constexpr uint32_t kTmemO = 0, kTmemS = 4 * kNP;
  // warps
  static constexpr int kSoftmaxWarps = NR / RH * 4, kScoreWarp = kSoftmaxWarps, kValueWarp = kScoreWarp + 1;
  static constexpr int kLoadWarp = kValueWarp + 1, kThreads = (kLoadWarp + 1) * 32;
  static_assert(kQBytes % 1024 == 0 && kQChunk % 1024 == 0 && kOffSmall % 16 == 0, "swizzle atoms stay aligned");
  static_assert(kTileSlot % 1024 == 0 && kCkvBytes % 1024 == 0, "tile slots");
  static_assert(kPRow == 32 ? NR == 32 : kNP == static_cast<int>(kPRow), "layouts");
  static_assert(kTmemS + kSBufs * kNS <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// (x - v) * 32 for the two fp16 values of a pair
__device__ __forceinline__ uint32_t next_term(uint32_t x, uint32_t v) {
  const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&v)),
                            __float2half2_rn(kTermStep));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// x = t1 + t2 / 32 + ... for a pair of fp16 values of at most 256, each term two E4M3 bytes: x has 11 bits, so
// what a term leaves, and that times 32, are fp16 values themselves, and the third term leaves nothing
template <int N>
__device__ __forceinline__ void split_f16(uint32_t x, uint16_t* t) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = f16x2_to_e4m3x2(x);
    if (i + 1 < N) x = next_term(x, e4m3x2_to_f16x2(t[i]));
  }
}
// The same for two weights of at most 256. The first term and what it leaves (at most 2^-4 of the weight, times 32 at
// most 256) are taken in fp32, the rest of it in fp16 (off by 2^-16 of the weight): three terms are off by at most
// 2^-14 + 2^-16 of the weight, four by 2^-16. (A weight rounded to fp16 before its three terms was
// off by up to 2^-11; many heads 139.0 us with that, 139.6 with this.)
template <int N>
__device__ __forceinline__ void split_weights(float a, float b, uint16_t* t) {
  t[0] = e4m3x2(a, b);
  const float2 v = e4m3x2_values(t[0]);
  const __half2 rest = __hmul2(__floats2half2_rn(a - v.x, b - v.y), __float2half2_rn(kTermStep));
  split_f16<N - 1>(*reinterpret_cast<const uint32_t*>(&rest), t + 1);
}

// NaN bytes of tokens [t0, t1) of a tile to zero: tokens that some row does not see. Its weight for them is 0,
// and every other byte is finite; for a row that does see one, the score has already made the weight NaN.
__device__ __forceinline__ void clear_nan_bytes(uint8_t* ckv, int t0, int t1, int tid, int nthreads) {
  for (int x = tid; x < (t1 - t0) * 32; x += nthreads) {
    const int t = t0 + (x >> 5);
    uint4* const at = reinterpret_cast<uint4*>(ckv + (t >> 3) * kGroupBytes + ((x >> 3) & 3) * 1024 + (t & 7) * 128 + (x & 7) * 16);
    uint4 v = *at;
    uint32_t* const w = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t nan = (((w[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in each NaN byte
      w[j] &= ~(nan * 255u);
    }
    *at = v;
  }
}

template <int NR, bool BF16>
__global__ void __launch_bounds__((Cfg<NR, BF16>::kThreads), 1)
    mla_decode_q8_kernel(const __grid_constant__ CUtensorMap tm_ckv, const __grid_constant__ CUtensorMap tm_kpe,
                         const DecodeQ8Params p) {
  using C = Cfg<NR, BF16>;
  constexpr int kTerms = C::kTerms, kThreads = C::kThreads, kSoftmaxWarps = C::kSoftmaxWarps;
  constexpr uint32_t kCkvBytes = C::kCkvBytes, kTileSlot = C::kTileSlot;
  extern __shared__ uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need it; the size leaves no slack to align it
    if (threadIdx.x == 0) flag_error(MLA_DEVERR_CONFIG);
    return;
  }
  auto* const sm = reinterpret_cast<Small<C::kLens>*>(smem + C::kOffSmall);
  volatile int32_t* abort_flag = &sm->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gang = blockIdx.y;
  const int rows_total = p.q_len * p.H;
  const int row0 = blockIdx.x * NR, nrows = min(NR, rows_total - row0);

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
      mbar_init(&sm->pfull[s], kSoftmaxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm->sfull[s], 1);
      mbar_init(&sm->sfree[s], kSoftmaxWarps);
    }
    mbar_init(&sm->qfull, kSoftmaxWarps);
    mbar_init(&sm->ofree, kSoftmaxWarps);
    mbar_init(&sm->drain[0], 1);
    mbar_init(&sm->drain[1], 1);
    sm->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kScoreWarp) {
    tmem_alloc(&sm->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tm_ckv);
    tma_prefetch_desc(&tm_kpe);
  }
  pdl_wait();
  pdl_launch_dependents();

  // Data of the call: what the kernel before may have written until the wait above returned (scales by the cache's
  // write, tables and lengths on the device) is read past L1, whose lines may be older than that.
  // This gang's place on the line of tiles
  const Q8Lens<C::kLens> lens{p.context_lens, sm->lens};
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0, T = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int L = __ldcg(p.context_lens + b);
    if (b < C::kLens) sm->lens[b] = L;
    const int n = q8_tiles(q8_view(p, L), kT);
    mine += n + (n > 0 ? int64_t{1} << kQ8CountShift : 0);
  }
  const int64_t prefix = block_prefix<kThreads>(mine, sm->scratch, &T);
  const Q8Line line = q8_line<kQ8Gap<NR>>(T & kQ8Tiles, static_cast<int32_t>(T >> kQ8CountShift), p.gangs);
  const bool work = gang < line.gangs;
  const int64_t lo = work ? line.begin(gang) : 0, hi = work ? line.begin(gang + 1) : 0;
  {  // the thread whose requests the gang starts (ends) in finds the place: its request and tile, tiles before it
    int64_t tiles = prefix & kQ8Tiles, at = tiles + line.gap * (prefix >> kQ8CountShift);
    const int64_t end = at + (mine & kQ8Tiles) + line.gap * (mine >> kQ8CountShift);
    if (work && ((lo >= at && lo < end) || (hi >= at && hi < end))) {
      for (int b = b_lo; b < b_hi; ++b) {
        const int n = q8_tiles(q8_view(p, lens(b)), kT);
        const int64_t next = at + n + (n > 0 ? line.gap : 0);
        if (lo >= at && lo < next) {
          const bool in_gap = lo - at >= n;
          sm->b0 = in_gap ? b + 1 : b;
          sm->off0 = in_gap ? 0 : lo - at;
          sm->first_tile = tiles + min(lo - at, static_cast<int64_t>(n));
        }
        if (hi >= at && hi < next) sm->last_tile = tiles + min(hi - at, static_cast<int64_t>(n));
        at = next;
        tiles += n;
      }
    }
    if (tid == 0 && hi == line.length) sm->last_tile = T & kQ8Tiles;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  const int N = work ? static_cast<int>(sm->last_tile - sm->first_tile) : 0;  // this gang's tiles
  Q8Walk w = q8_walk(work ? sm->b0 : 0, work ? sm->off0 : 0, N);
  uint64_t tmo = p.timeout_ns;
  asm volatile("" : "+l"(tmo));

  // One row of request b's queries to its terms, by one warp: a lane takes latent columns 8 lane .. and 256 + 8
  // lane .., and in lanes 0-7 8 rope columns. In two steps, so that rows' loads overlap.
  struct QueryRow {
    uint4 v[3];
  };
  auto load_query = [&](int b, int r) -> QueryRow {
    QueryRow q;
#pragma unroll
    for (int x = 0; x < 3; ++x) q.v[x] = make_uint4(0u, 0u, 0u, 0u);
    if (r < nrows) {
      const long long at = static_cast<long long>(b) * rows_total + row0 + r;
      q.v[0] = __ldcg(reinterpret_cast<const uint4*>(p.q_abs + at * kRank) + lane);
      q.v[1] = __ldcg(reinterpret_cast<const uint4*>(p.q_abs + at * kRank) + 32 + lane);
      if (lane < kRope / 8) q.v[2] = __ldcg(reinterpret_cast<const uint4*>(p.q_pe + at * kRope) + lane);
    }
    return q;
  };
  auto split_query = [&](const QueryRow& qr, int seg, int r) {
    uint8_t* const q = smem + C::kOffQ;
    const uint32_t* const u = reinterpret_cast<const uint32_t*>(qr.v);
    // the row's largest magnitude (its bits: 15 of them order both types, NaN and infinity on top)
    uint32_t top = 0;
#pragma unroll
    for (int x = 0; x < 12; ++x) top = __vmaxu2(top, u[x] & 0x7fff7fffu);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    const float amax = h2f<BF16>(static_cast<uint16_t>(top));
    // 2^e takes it to [128, 256); a row below 2^-119 stays under it
    const int e = min(126, 134 - static_cast<int>(__float_as_uint(amax) >> 23));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if (lane == 0)
      sm->factor[seg & 1][r] = (amax < INFINITY) ? p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23)
                                                     : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      if (x == 2 && lane >= kRope / 8) break;
      uint16_t t[4][C::kQTerms];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t w = u[4 * x + y];
        const __half2 f = __floats2half2_rn(h2f<BF16>(static_cast<uint16_t>(w & 0xffffu)) * up,
                                            h2f<BF16>(static_cast<uint16_t>(w >> 16)) * up);
        split_f16<C::kQTerms>(*reinterpret_cast<const uint32_t*>(&f), t[y]);
      }
      // columns 8 lane .. + 7 of latent half x (or of the rope part)
      uint8_t* at = x < 2 ? q + (2 * x + (lane >> 4)) * C::kQChunk + r * 128 + (((lane >> 1) ^ r) & 7) * 16 + (lane & 1) * 8
                          : q + 4 * C::kQChunk + r * 64 + (((lane >> 1) ^ (r >> 1)) & 3) * 16 + (lane & 1) * 8;
#pragma unroll
      for (int n = 0; n < C::kQTerms; ++n)  // (NR rows on: the same swizzle)
        *reinterpret_cast<uint2*>(at + n * NR * (x < 2 ? 128 : 64)) = make_uint2(pack16(t[0][n], t[1][n]), pack16(t[2][n], t[3][n]));
    }
  };
  if (warp == C::kLoadWarp) {
    // ------------------------------------------------------------------ page loads
    const uint64_t pol = l2_policy_evict_first();
    // One lane a unit of a tile: a page, or half of one of 64 tokens, so that units fill a tile.
    const int unit_shift = min(p.bs_shift, 5), unit = 1 << unit_shift;
    const int tok = lane << unit_shift;            // its first token in the tile
    // the table's entry for this lane's unit (looked at when it is used: its load has a tile's time)
    auto entry_of = [&](const Q8Walk& w, int tile) -> int {
      const uint32_t at = run_position(tile, kT, tok);
      if (tok >= kT || at >= static_cast<uint32_t>(w.v.n)) return -1;
      const int u = static_cast<int>(at);
      const int pg = (u >> p.bs_shift) + (u >= w.v.sa ? w.v.skip >> p.bs_shift : 0);
      return pg < p.max_blocks ? __ldcg(p.block_table + static_cast<long long>(w.b) * p.max_blocks + pg) : -1;
    };
    struct Unit {
      int entry, sub, count;  // this lane's entry and first row in its page; units of the tile
    };
    // the walk's tiles, one after the other
    bool live = q8_next<kT>(p, lens, w, true);
    int tile = w.ta;
    auto next_unit = [&]() -> Unit {
      if (!live) return Unit{-1, 0, 0};
      const Unit r{entry_of(w, tile), static_cast<int>(run_position(tile, kT, tok)) & (p.bs - 1), (min(kT, w.v.n - tile * kT) + unit - 1) >> unit_shift};
      if (++tile == w.tb) {
        live = q8_next<kT>(p, lens, w, false);
        tile = w.ta;
      }
      return r;
    };
    // (an entry ahead of the loads; asking L2 for pages further on made calls 1 to 5% slower)
    Unit cur = next_unit();
    int issued = -1;
    bool stop = false;
    for (int i = 0; i < N && !stop; ++i) {
      const int s = i % kSlots;
      // an entry outside the pool or the table row reads zeros
      const Unit nxt = next_unit();
      int pid = cur.entry;
      if (lane < cur.count && (pid < 0 || pid >= p.num_blocks)) {
        flag_error(MLA_DEVERR_BAD_PAGE);
        pid = -1;
      }
      uint8_t* const slot = smem + s * kTileSlot;
      const int row = (pid << p.bs_shift) + (pid < 0 ? 0 : cur.sub);
      const bool mine = lane < cur.count;
      // Once the value product of tile i - kSlots has left the slot. (Given up, the loads are issued all the same, so
      // that the barrier completes.)
      if (i >= kSlots && !__all_sync(0xffffffffu, mbar_wait(&sm->empty[s], (i / kSlots - 1) & 1, tmo) && !*abort_flag)) {
        stop = true;
        *abort_flag = 1;
      }
      if (lane == 0) mbar_arrive_expect_tx(&sm->full[s], static_cast<uint32_t>((cur.count << unit_shift) * kQkDim));
      __syncwarp();
      if (mine) {
        tma_load_4d(slot + tok * kRank, &tm_ckv, 0, 0, 0, row >> 3, &sm->full[s], pol);
        tma_load_2d(slot + kCkvBytes + tok * kRope, &tm_kpe, 0, row, &sm->full[s], pol);
      }
      issued = i;
      cur = nxt;
    }
    // after an abort, loads in flight land before shared memory is released
    if (lane == 0 && *abort_flag)
      for (int t = max(0, issued - (kSlots - 1)); t <= issued; ++t) mbar_wait(&sm->full[t % kSlots], (t / kSlots) & 1, kDrainTimeoutNs);
  } else if (warp == C::kScoreWarp) {
    // ------------------------------------------------------------------ score products
    // One thread issues them in tile order as tiles land, another one the value products: each waits for its
    // own inputs only, and its issue (some 60 cycles an MMA) overlaps the other's waits.
    constexpr uint32_t idesc = idesc_e4m3_f32(128, C::kNS, false, false);
    const uint32_t base = smem_u32(smem);
    if (lane == 0) {
      int i = 0;
      bool first = true, ok = true;
      // gangs that a request which starts in this one is cut into
      auto parts_of = [&](const Q8Walk& w) -> int {
        return w.tb < w.n_tiles ? line.gang_of(hi + (w.n_tiles - w.tb) - 1) - gang + 1 : 1;
      };
      for (int seg = 0; ok && q8_next<kT>(p, lens, w, first); ++seg, first = false) {
        const uint32_t q = base + C::kOffQ;
        const Desc2 bd = desc2(smem_desc_sw128(q, 16, 1024)), bk = desc2(smem_desc_sw64(q + 4 * C::kQChunk, 512));
        if (p.cuts_by_request && w.ta == 0 && blockIdx.x == 0)  // a request that starts here: its gangs, for the merge
          p.ws_cut[w.b] = make_int2(gang, parts_of(w));
        ok = mbar_wait(&sm->qfull, seg & 1, tmo);
        for (int tile = w.ta; ok && tile < w.tb; ++tile, ++i) {
          ok = mbar_wait(&sm->full[i % kSlots], (i / kSlots) & 1, tmo) &&
               (i < C::kSBufs || mbar_wait(&sm->sfree[i % C::kSBufs], (i / C::kSBufs - 1) & 1, tmo)) && !*abort_flag;
          if (!ok) break;
          tc_fence_after();
          const uint32_t slot = base + (i % kSlots) * kTileSlot;
          const Desc2 ad = desc2(smem_desc_sw128(slot, 16, kGroupBytes)), ak = desc2(smem_desc_sw64(slot + kCkvBytes, 512));
          const uint32_t d = tmem + C::kTmemS + (i % C::kSBufs) * C::kNS;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma8_ss(d, ad, (c * 1024 + kk * 32) >> 4, bd, (c * C::kQChunk + kk * 32) >> 4, idesc, (c | kk) != 0 ? 1u : 0u);
          umma8_ss(d, ak, 0, bk, 0, idesc, 1u);
          umma8_ss(d, ak, 32 >> 4, bk, 32 >> 4, idesc, 1u);
          umma_commit(&sm->sfull[i % C::kSBufs]);
        }
      }
      if (!ok) *abort_flag = 1;
      // ... and (after the last segment) the request at this gang's open end
      if (!p.cuts_by_request && blockIdx.x == 0) p.ws_cut[gang] = make_int2(w.b, N > 0 && w.ta == 0 ? parts_of(w) : 0);
      umma_commit(&sm->drain[0]);  // every MMA issued has completed before TMEM is freed
      mbar_wait(&sm->drain[0], 0, kDrainTimeoutNs);
    }
    __syncwarp();
  } else if (warp == C::kValueWarp) {
    // ------------------------------------------------------------------ value products
    constexpr uint32_t idesc = idesc_e4m3_f32(128, C::kNP, true, true);
    const uint32_t base = smem_u32(smem);
    if (lane == 0) {
      int i = 0;
      bool first = true, ok = true;
      for (int seg = 0; ok && q8_next<kT>(p, lens, w, first); ++seg, first = false) {
        if (seg > 0) ok = mbar_wait(&sm->ofree, (seg - 1) & 1, tmo);  // the last segment's O has been read
        for (int tile = w.ta; ok && tile < w.tb; ++tile, ++i) {
          ok = mbar_wait(&sm->pfull[i % kSlots], (i / kSlots) & 1, tmo) && !*abort_flag;
          if (!ok) break;
          tc_fence_after();
          const uint32_t slot = base + (i % kSlots) * kTileSlot;
          const uint32_t wts = slot + kCkvBytes;
          const Desc2 pb = desc2(C::kPRow == 32 ? smem_desc_sw32(wts, kT * 32, 256) : smem_desc_sw64(wts, 512));
          const Desc2 a0 = desc2(smem_desc_sw128(slot, 1024, kGroupBytes));
          const int ksteps = (min(kT, w.v.n - tile * kT) + kStep - 1) / kStep;
#pragma unroll 1
          for (int ks = 0; ks < ksteps; ++ks) {
#pragma unroll
            for (int blk = 0; blk < 4; ++blk)
              umma8_ss(tmem + C::kTmemO + blk * C::kNP, a0, (blk * 1024 + ks * 4 * kGroupBytes) >> 4, pb, (ks * kStep * C::kPRow) >> 4, idesc,
                       (tile == w.ta && ks == 0) ? 0u : 1u);
          }
          umma_commit(&sm->empty[i % kSlots]);
        }
      }
      if (!ok) *abort_flag = 1;
      umma_commit(&sm->drain[1]);
      mbar_wait(&sm->drain[1], 0, kDrainTimeoutNs);
    }
    __syncwarp();
  } else if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------------ softmax
    const int q4 = warp & 3, h = warp >> 2;
    const int tl = 32 * q4 + lane;  // this thread's token of each tile, and latent column of each block of O
    const uint32_t lane_base = static_cast<uint32_t>(32 * q4) << 16;
    const bool has_tokens = 32 * q4 < kT;  // (a 96-token tile leaves the last quadrant's warps without)
    const uint32_t bar = 1 + h;  // the four warps of a run of rows meet by themselves
    constexpr uint32_t kMeet = 128;
    constexpr float kNone = -3.402823466e38f;  // the reference of a row that has seen no token: finite, below any score
    // this thread's page of a tile, and its token's scale there: loads a tile ahead of their use each, so
    // neither looks at what it loaded
    auto page_at = [&](const Q8Walk& w, int tile) -> int {
      const uint32_t at = run_position(tile, kT, tl);
      if (!has_tokens || at >= static_cast<uint32_t>(w.v.n)) return -1;
      const int u = static_cast<int>(at);
      const int pg = (u >> p.bs_shift) + (u >= w.v.sa ? w.v.skip >> p.bs_shift : 0);
      return pg < p.max_blocks ? __ldcg(p.block_table + (static_cast<long long>(w.b) * p.max_blocks + pg)) : -1;
    };
    auto scale_at = [&](int pid, int tile) -> float {  // 1 where there is no page
      if (pid < 0 || pid >= p.num_blocks) return 1.f;
      const int row = (pid << p.bs_shift) + (static_cast<int>(run_position(tile, kT, tl)) & (p.bs - 1));  // (a pool has fewer than 2^31 tokens)
      return __ldcg(p.scales + (row >> p.g_shift));
    };
    // The value product of tile t: it has left the slot. (The phase before on that barrier, tile t - kSlots,
    // was complete before tile t was loaded, so its parity cannot be taken for this one's.)
    auto product_done = [&](int t) -> bool { return mbar_wait(&sm->empty[t % kSlots], (t / kSlots) & 1, tmo); };
    int i = 0;  // tile count
    // Each round: a request's tiles, the split of the next one's queries (while the last value product runs), then
    // the request's output. The first round only splits.
    Q8Walk next = w;
    bool more = q8_next<kT>(p, lens, next, true);
    float z_raw = 1.f;  // the scale of this thread's token in the next tile, and its page in the one after that
    int pid = -1;
    for (int seg = -1;; ++seg) {
     bool stop = false;
     float lsum[RH], mr[RH];
     if (seg >= 0) {
#pragma unroll
      for (int k = 0; k < RH; ++k) {
        lsum[k] = 0.f;
        mr[k] = kNone;
      }
      // rows' positions: the first and last row of this CTA, and what their windows leave out
      const int pos_first = p.causal ? w.v.n - p.q_len + (row0 >> p.h_shift) : w.v.n - 1;
      const int pos_last = p.causal ? w.v.n - p.q_len + ((row0 + nrows - 1) >> p.h_shift) : w.v.n - 1;
      const int low_last = p.window > 0 ? window_floor(pos_last, p.window) : -1;
      // tiles of which every row sees every token (rows past the last, zeros, may see what they like: nothing of
      // theirs is written)
      const int plain_lo = low_last < 0 ? 0 : low_last / kT + 1, plain_hi = max(0, pos_first + 1) / kT;
      for (int tile = w.ta; tile < w.tb; ++tile, ++i) {
        // NaN for a scale that is neither NaN nor in range
        const float z = (z_raw >= 0x1p-60f && z_raw <= 0x1p60f) ? z_raw : __uint_as_float(0x7fc00000u);
        // (approximate: their errors, 2^-22, make a token's weight and its share of the sum wrong alike)
        const float lz = __log2f(z), iz = z == z ? fast_rcp(z) : 0.f;  // (NaN: who sees the token has a NaN weight)
        z_raw = tile + 1 < w.tb ? scale_at(pid, tile + 1) : 1.f;
        pid = tile + 2 < w.tb ? page_at(w, tile + 2) : -1;
        const int sb = i % C::kSBufs;
        bool ok = mbar_wait(&sm->sfull[sb], (i / C::kSBufs) & 1, tmo);
        float x[RH];
        ok = __all_sync(0xffffffffu, ok);
        if (ok && has_tokens) {
          tc_fence_after();
          float t2[RH], t3[RH];
          const uint32_t sa = tmem + lane_base + C::kTmemS + sb * C::kNS + RH * h;
          tmem_ld8(sa, x);
          tmem_ld8(sa + NR, t2);
          if constexpr (C::kQTerms == 3) tmem_ld8(sa + 2 * NR, t3);
          float factor[RH];
#pragma unroll
          for (int k = 0; k < RH; k += 4)
            *reinterpret_cast<float4*>(factor + k) = *reinterpret_cast<const float4*>(&sm->factor[seg & 1][RH * h + k]);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->sfree[sb]);
#pragma unroll
          for (int k = 0; k < RH; k += 2) {
            const float2 inv = make_float2(kTermInv, kTermInv);
            float2 t = make_float2(t2[k], t2[k + 1]);
            if constexpr (C::kQTerms == 3) t = fma2(make_float2(t3[k], t3[k + 1]), inv, t);
            t = mul2(fma2(t, inv, make_float2(x[k], x[k + 1])), make_float2(factor[k], factor[k + 1]));
            t = fma2(t, make_float2(z, z), make_float2(lz, lz));
            x[k] = t.x;
            x[k + 1] = t.y;
          }
          if (__builtin_expect(tile < plain_lo || tile >= plain_hi, 0)) {
            const int u0 = tile * kT, nvalid = min(kT, w.v.n - u0);
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              const int r = row0 + RH * h + k;
              const uint32_t u = run_position(tile, kT, tl);
              const int pos = p.causal ? w.v.n - p.q_len + (r >> p.h_shift) : w.v.n - 1;
              bool vis = tl < nvalid && static_cast<int>(u) <= pos;
              if (p.window > 0) vis = vis && (static_cast<int>(u) > window_floor(pos, p.window) || static_cast<int>(u) < p.sinks);
              if (!vis) x[k] = -INFINITY;
            }
            // tokens that some row does not see: below the last row's window, behind the first row, and the
            // rest of the tail's last step
            uint8_t* const slot = smem + (i % kSlots) * kTileSlot;
            const int a0 = min(kT, max(0, p.sinks - u0)), a1 = min(kT, low_last + 1 - u0);
            const int b0 = max(0, min(kT, min(w.v.n, pos_first + 1) - u0)), b1 = (nvalid + 31) & ~31;
            if (a0 < a1) clear_nan_bytes(slot, a0, a1, h * kT + tl, NR / RH * kT);
            if (b0 < b1) clear_nan_bytes(slot, b0, b1, h * kT + tl, NR / RH * kT);
          }
        } else {
          if (!ok) *abort_flag = 1;
          if (lane == 0) mbar_arrive(&sm->sfree[sb]);
#pragma unroll
          for (int k = 0; k < RH; ++k) x[k] = -INFINITY;
        }
        // Does a score pass its row's reference by more than kTau? One barrier of the four warps that share the rows;
        // only then are the rows' maxima taken, and the references move to them, with the sums and O.
        bool need = false;
#pragma unroll
        for (int k = 0; k < RH; k += 2) {
          const float2 d = fma2(make_float2(mr[k], mr[k + 1]), make_float2(-1.f, -1.f), make_float2(x[k], x[k + 1]));
          need |= d.x > C::kTau + C::kWeightExp || d.y > C::kTau + C::kWeightExp;
        }
        need = named_bar_sync_or(bar, kMeet, need || !ok || *abort_flag != 0);
        float al[RH];
        if (need) {
          float v[RH];
#pragma unroll
          for (int k = 0; k < RH; ++k) v[k] = warp_max(x[k]);
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < RH; k += 4)
              *reinterpret_cast<float4*>(&sm->red[i & 1][q4][RH * h + k]) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
          if (named_bar_sync_or(bar, kMeet, !ok || *abort_flag != 0)) {
            stop = true;
            break;
          }
#pragma unroll
          for (int k = 0; k < RH; k += 4) {
            float4 m4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) m4[q] = *reinterpret_cast<const float4*>(&sm->red[i & 1][q][RH * h + k]);
            v[k] = fmaxf(fmaxf(m4[0].x, m4[1].x), fmaxf(m4[2].x, m4[3].x));
            v[k + 1] = fmaxf(fmaxf(m4[0].y, m4[1].y), fmaxf(m4[2].y, m4[3].y));
            v[k + 2] = fmaxf(fmaxf(m4[0].z, m4[1].z), fmaxf(m4[2].z, m4[3].z));
            v[k + 3] = fmaxf(fmaxf(m4[0].w, m4[1].w), fmaxf(m4[2].w, m4[3].w));
          }
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            const float m = fmaxf(mr[k], v[k] - C::kWeightExp);
            al[k] = fast_exp2(mr[k] - m);
            mr[k] = m;
            lsum[k] *= al[k];
          }
        }
        if (has_tokens) {
          uint16_t term[RH / 2][kTerms];
#pragma unroll
          for (int k = 0; k < RH; k += 2) {
            const float2 d = fma2(make_float2(mr[k], mr[k + 1]), make_float2(-1.f, -1.f), make_float2(x[k], x[k + 1]));
            const float2 wt = make_float2(fast_exp2(d.x), fast_exp2(d.y));  // hidden tokens (-inf) give 0
            const float2 l = fma2(wt, make_float2(iz, iz), make_float2(lsum[k], lsum[k + 1]));
            lsum[k] = l.x;
            lsum[k + 1] = l.y;
            split_weights<kTerms>(wt.x, wt.y, term[k / 2]);
          }
          uint8_t* const pb = smem + (i % kSlots) * kTileSlot + kCkvBytes;  // (the scores are done with what lay there)
          // columns n * NR + 8 h .. + 7 of this token's row: half of one 16-byte piece
#pragma unroll
          for (int n = 0; n < kTerms; ++n) {
            const int piece = (n * NR + RH * h) >> 4;
            const int at = C::kPRow == 32 ? (piece >> 1) * kT * 32 + tl * 32 + ((piece ^ (tl >> 2)) & 1) * 16
                                          : tl * 64 + ((piece ^ (tl >> 1)) & 3) * 16;
            *reinterpret_cast<uint2*>(pb + at + (h & 1) * 8) = make_uint2(pack16(term[0][n], term[1][n]), pack16(term[2][n], term[3][n]));
          }
          fence_proxy_async_smem();
        }
        if (need && tile > w.ta) {  // O: the value product of the tile before must be complete
          if (__all_sync(0xffffffffu, product_done(i - 1))) {
            tc_fence_after();
#pragma unroll 1
            for (int blk = 0; blk < 4; ++blk) {
              float v[kTerms][RH];
              const uint32_t a = tmem + lane_base + C::kTmemO + blk * C::kNP + RH * h;
#pragma unroll
              for (int n = 0; n < kTerms; ++n) tmem_ld8(a + n * NR, v[n]);
              tmem_wait_ld();
#pragma unroll
              for (int n = 0; n < kTerms; ++n) {
#pragma unroll
                for (int k = 0; k < RH; k += 2) {
                  const float2 y = mul2(make_float2(v[n][k], v[n][k + 1]), make_float2(al[k], al[k + 1]));
                  v[n][k] = y.x;
                  v[n][k + 1] = y.y;
                }
                tmem_st8(a + n * NR, v[n]);
              }
            }
            tmem_wait_st();
          } else {
            *abort_flag = 1;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->pfull[i % kSlots]);
      }
     }
     if (stop) break;
     if (more) {
      // (their scores done, nothing reads the last request's queries any more)
      pid = page_at(next, next.ta);
      QueryRow row = load_query(next.b, warp);
#pragma unroll 1
      for (int r = warp; r < NR; r += kSoftmaxWarps) {
        const QueryRow ahead = load_query(next.b, r + kSoftmaxWarps);  // (past the last: zeros)
        split_query(row, seg + 1, r);
        row = ahead;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->qfull);
      z_raw = scale_at(pid, next.ta);
      pid = next.ta + 1 < next.tb ? page_at(next, next.ta + 1) : -1;
     }
     if (seg >= 0) {
      // the segment's end: its sums, and O once its last value product is complete
      const bool ended = product_done(i - 1);
      if (!ended) *abort_flag = 1;
      // rows' sums over the warp's tokens: at each of three steps a lane hands half of its rows to its partner
#pragma unroll
      for (int o = 16, n = RH / 2; n > 0; o >>= 1, n >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const float mine = up ? lsum[k + n] : lsum[k], his = up ? lsum[k] : lsum[k + n];
          lsum[k] = mine + __shfl_xor_sync(0xffffffffu, his, o);
        }
      }
      lsum[0] += __shfl_xor_sync(0xffffffffu, lsum[0], 2);
      lsum[0] += __shfl_xor_sync(0xffffffffu, lsum[0], 1);
      if ((lane & 3) == 0) sm->red[(i - 1) & 1][q4][RH * h + (lane >> 2)] = lsum[0];
      if (named_bar_sync_or(bar, kMeet, !ended || *abort_flag != 0)) break;
      const bool whole = w.ta == 0 && w.tb == w.n_tiles;
      const long long orow = whole ? static_cast<long long>(w.b) * rows_total + row0 + RH * h
                                   : (static_cast<long long>(gang) * 2 + (w.ta == 0 ? 1 : 0)) * p.row_pad + row0 + RH * h;
      const int my_rows = nrows - RH * h;
      const bool f32 = !whole || p.out_dtype == 2;
      void* const dst = whole ? p.out : p.ws_o;
      const long long first_off = orow * kRank + tl;
      // lane k (mod 8) works out row k's factor
      float m = mr[0];
#pragma unroll
      for (int k = 1; k < RH; ++k)
        if ((lane & (RH - 1)) == k) m = mr[k];
      const int r = RH * h + (lane & (RH - 1));
      const auto& sum = sm->red[(i - 1) & 1];
      const float l = (sum[0][r] + sum[1][r]) + (sum[2][r] + sum[3][r]);
      const float my_inv = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);  // (no visible token: every weight was 0)
      if (q4 == 0 && lane < my_rows && lane < RH) {
        if (!whole) {
          *reinterpret_cast<float2*>(p.ws_ml + (orow + lane) * 2) = make_float2(m == kNone ? -INFINITY : m, l);
        } else if (p.out_lse != nullptr) {
          p.out_lse[orow + lane] = l == 0.f ? -INFINITY : (m == kNone ? 0.f : m) + log2f(l);
        }
      }
      float inv[RH];
#pragma unroll
      for (int k = 0; k < RH; ++k) inv[k] = __shfl_sync(0xffffffffu, my_inv, k);
      tc_fence_after();
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk) {
        float o[kTerms][RH];
        const uint32_t a = tmem + lane_base + C::kTmemO + blk * C::kNP + RH * h;
#pragma unroll
        for (int n = 0; n < kTerms; ++n) tmem_ld8(a + n * NR, o[n]);
        tmem_wait_ld();
        if (blk == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->ofree);
        }
#pragma unroll
        for (int k = 0; k < RH; k += 2) {
          float2 v = make_float2(o[kTerms - 1][k], o[kTerms - 1][k + 1]);
#pragma unroll
          for (int n = kTerms - 2; n >= 0; --n) v = fma2(v, make_float2(kTermInv, kTermInv), make_float2(o[n][k], o[n][k + 1]));
          v = mul2(v, make_float2(inv[k], inv[k + 1]));
          o[0][k] = v.x;
          o[0][k + 1] = v.y;
        }
        // (rows and blocks of columns at fixed distances: one address a thread)
        if (f32) {
          float* const at = static_cast<float*>(dst) + first_off + blk * 128;
#pragma unroll
          for (int k = 0; k < RH; ++k)
            if (k < my_rows) at[k * kRank] = o[0][k];
        } else {
          uint16_t* const at = static_cast<uint16_t*>(dst) + first_off + blk * 128;
#pragma unroll
          for (int k = 0; k < RH; ++k)
            if (k < my_rows) at[k * kRank] = p.out_dtype == 1 ? f2h<true>(o[0][k]) : f2h<false>(o[0][k]);
        }
      }
     }
     if (!more) break;
     w = next;
     more = q8_next<kT>(p, lens, next, false);
    }
  }
  // requests with nothing to see
  for (int b = gang; b < p.B; b += p.gangs) {
    if (q8_view(p, lens(b)).n != 0) continue;
    if (p.cuts_by_request && blockIdx.x == 0 && tid == 0) p.ws_cut[b] = make_int2(gang, 0);
    for (int x = tid; x < nrows * (kRank / 4); x += kThreads) {
      const long long at = static_cast<long long>(b) * rows_total + row0 + x / (kRank / 4);
      store_out4(p.out, p.out_dtype, at * kRank + 4 * (x % (kRank / 4)), make_float4(0.f, 0.f, 0.f, 0.f));
      if (x % (kRank / 4) == 0 && p.out_lse != nullptr) p.out_lse[at] = -INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The requests cut by gang borders: per (request, row) the parts of its gangs,
//   M = max m_j, w_j = 2^(m_j - M), out = sum w_j O_j / sum w_j l_j, lse = M + log2 sum w_j l_j.
// Two kernels, by what there is to share out; in both, sums are added in a fixed order: the same bits on every call.
// Their time is one chain of loads (an entry of ws_cut, then a row's parts) and the fetch and issue of their code, so
// both keep it short, and a warp asks for its own entry of ws_cut only (a list of all entries made by every block:
// the same lines asked for by a thousand blocks, 1 to 3 us).
constexpr int kMergeThreads = 128, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBlocks = 8;  // per SM: one wave

// a part's weight: one without a visible token has l = 0; one whose every score is NaN has no maximum, and l NaN
__device__ __forceinline__ float part_weight(float m, float l, float ref) {
  return l == 0.f ? 0.f : (m == -INFINITY ? 1.f : exp2f(m - ref));
}
__device__ __forceinline__ void fma4(float4& acc, float w, const float4 v) {
  acc.x = fmaf(w, v.x, acc.x);
  acc.y = fmaf(w, v.y, acc.y);
  acc.z = fmaf(w, v.z, acc.z);
  acc.w = fmaf(w, v.w, acc.w);
}

// the parts of row `row` of a request whose first gang is j0: gang j0's in entry 1, the others' in entry 0
struct MergeParts {
  const float2* ml;
  const float* o;
  long long slot0, pitch;
  __device__ __forceinline__ MergeParts(const DecodeQ8Params& p, int j0, int row)
      : ml(reinterpret_cast<const float2*>(p.ws_ml)), o(p.ws_o),
        slot0(static_cast<long long>(j0) * 2 * p.row_pad + row), pitch(p.row_pad) {}
  __device__ __forceinline__ long long slot(int x) const { return slot0 + (x == 0 ? 1 : 2 * x) * pitch; }
  __device__ __forceinline__ float2 max_sum(int x) const { return __ldcg(ml + slot(x)); }
  __device__ __forceinline__ float4 values(int x, int col) const {
    return __ldcg(reinterpret_cast<const float4*>(o + slot(x) * kRank + col));
  }
};
// (a call that gave up has left entries as they were: they lead nowhere outside the buffers)
__device__ __forceinline__ bool merge_entry_ok(const DecodeQ8Params& p, int b, int j0, int n) {
  return n > 1 && n <= p.gangs && j0 >= 0 && j0 <= p.gangs - n && b >= 0 && b < p.B;
}
__device__ __forceinline__ void merge_out(const DecodeQ8Params& p, long long br, int col, float4 acc, float inv) {
  store_out4(p.out, p.out_dtype, br * kRank + col, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

// Batches whose rows fill the device: kRowWarps warps a (gang, row), which end at once where no request with that
// gang as its first is cut. Lane x weighs part x, then the parts' columns go by, 8 float4 a lane in flight.
constexpr int kRowWarps = 2, kRowLoads = 4 / kRowWarps, kRowParts = 8 / kRowLoads;
__global__ void __launch_bounds__(kMergeThreads, kMergeBlocks) mla_merge_q8_rows_kernel(const DecodeQ8Params p) {
  const int lane = threadIdx.x & 31;
  const uint32_t rows_total = p.q_len * p.H, per_gang = rows_total * kRowWarps, units = p.gangs * per_gang;
  pdl_wait();
  pdl_launch_dependents();
  for (uint32_t unit = blockIdx.x * kMergeWarps + (threadIdx.x >> 5); unit < units; unit += gridDim.x * kMergeWarps) {
    const int j0 = unit / per_gang, row = unit % per_gang / kRowWarps, col = unit % kRowWarps * (kRank / kRowWarps) + 4 * lane;
    const int2 cut = __ldcg(p.ws_cut + j0);
    const int n = cut.y;
    if (!merge_entry_ok(p, cut.x, j0, n)) continue;
    const MergeParts parts(p, j0, row);
    float4 v[kRowParts][kRowLoads];
    auto load = [&](int x0) {
#pragma unroll
      for (int y = 0; y < kRowParts; ++y)
#pragma unroll
        for (int k = 0; k < kRowLoads; ++k)
          v[y][k] = x0 + y < n ? parts.values(x0 + y, col + 128 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);  // (they do not depend on the weights)
    float M = -INFINITY, den = 0.f, w = 0.f;
    float4 acc[kRowLoads];
#pragma unroll
    for (int k = 0; k < kRowLoads; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += kRowParts) {
      if (x0 % 32 == 0) {  // lane x weighs part x0 + x
        const float2 ml = x0 + lane < n ? parts.max_sum(x0 + lane) : make_float2(-INFINITY, 0.f);
        const float m = fmaxf(M, warp_max(ml.x)), ref = m == -INFINITY ? 0.f : m;
        const float al = M == -INFINITY ? 1.f : exp2f(M - ref);  // (nothing summed before the first, or only NaN)
        w = part_weight(ml.x, ml.y, ref);
        float sum = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        den = fmaf(den, al, sum);
        M = m;
#pragma unroll
        for (int k = 0; k < kRowLoads; ++k) acc[k] = make_float4(acc[k].x * al, acc[k].y * al, acc[k].z * al, acc[k].w * al);
      }
#pragma unroll
      for (int y = 0; y < kRowParts; ++y) {
        const float wx = __shfl_sync(0xffffffffu, w, (x0 + y) & 31);  // (0 past the last part)
#pragma unroll
        for (int k = 0; k < kRowLoads; ++k) fma4(acc[k], wx, v[y][k]);
      }
      if (x0 + kRowParts < n) load(x0 + kRowParts);
    }
    const long long br = static_cast<long long>(cut.x) * rows_total + row;
    const bool none = den == 0.f;
    const float inv = none ? 0.f : 1.f / den;
#pragma unroll
    for (int k = 0; k < kRowLoads; ++k) merge_out(p, br, col + 128 * k, acc[k], inv);
    if (p.out_lse != nullptr && col == 0) p.out_lse[br] = none ? -INFINITY : (M == -INFINITY ? 0.f : M) + log2f(den);
  }
}

// Few rows (one long request: each in as many parts as there are gangs): a block 16 columns of a row, the parts
// shared by 32 lanes, a lane's loads of a round in flight at once.
constexpr int kPartLanes = 32, kColLanes = kMergeThreads / kPartLanes, kColUnits = kRank / (4 * kColLanes);
constexpr int kMergeLoads = 5;   // 160 gangs in a round
__global__ void __launch_bounds__(kMergeThreads, kMergeBlocks) mla_merge_q8_parts_kernel(const DecodeQ8Params p) {
  __shared__ float4 sm_acc[kMergeWarps][kColLanes];
  __shared__ float sm_m[kMergeWarps], sm_den[kMergeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e = tid / kColLanes, rows_total = p.q_len * p.H;
  const uint32_t per_request = rows_total * kColUnits, units = per_request * p.B;
  pdl_wait();
  pdl_launch_dependents();
  for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int b = unit / per_request, rest = unit % per_request, row = rest / kColUnits;
    const int2 cut = __ldcg(p.ws_cut + b);
    const int n = cut.y, col = rest % kColUnits * 4 * kColLanes + 4 * (tid % kColLanes);
    if (!merge_entry_ok(p, b, cut.x, n)) continue;
    const MergeParts parts(p, cut.x, row);
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int x0 = e; x0 < n; x0 += kPartLanes * kMergeLoads) {
      float2 ml[kMergeLoads];
      float4 v[kMergeLoads];
      float m = M;
#pragma unroll
      for (int y = 0; y < kMergeLoads; ++y) {
        const int x = x0 + kPartLanes * y;
        ml[y] = x < n ? parts.max_sum(x) : make_float2(-INFINITY, 0.f);
        v[y] = x < n ? parts.values(x, col) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int y = 0; y < kMergeLoads; ++y) m = fmaxf(m, ml[y].x);
      const float ref = m == -INFINITY ? 0.f : m;
      const float al = M == -INFINITY ? 1.f : exp2f(M - ref);  // (nothing summed before the first, or only NaN)
      den *= al;
      acc = make_float4(acc.x * al, acc.y * al, acc.z * al, acc.w * al);
      M = m;
#pragma unroll
      for (int y = 0; y < kMergeLoads; ++y) {
        const float w = part_weight(ml[y].x, ml[y].y, ref);
        den = fmaf(w, ml[y].y, den);
        fma4(acc, w, v[y]);
      }
    }
    // lanes' sums, each a part of its own: over the warp's 8 part lanes, then over the warps
    float m = M;
#pragma unroll
    for (int o = kColLanes; o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sm_m[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    const float w = part_weight(M, den, m == -INFINITY ? 0.f : m);
    float s[5] = {den * w, acc.x * w, acc.y * w, acc.z * w, acc.w * w};
#pragma unroll
    for (int o = kColLanes; o < 32; o *= 2)
#pragma unroll
      for (int k = 0; k < 5; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if (lane < kColLanes) sm_acc[warp][lane] = make_float4(s[1], s[2], s[3], s[4]);
    if (lane == 0) sm_den[warp] = s[0];
    __syncthreads();
    if (e == 0) {
      den = (sm_den[0] + sm_den[1]) + (sm_den[2] + sm_den[3]);
      acc = sm_acc[0][lane];
#pragma unroll
      for (int k = 1; k < kMergeWarps; ++k) fma4(acc, 1.f, sm_acc[k][lane]);
      const long long br = static_cast<long long>(b) * rows_total + row;
      const bool none = den == 0.f;
      merge_out(p, br, col, acc, none ? 0.f : 1.f / den);
      if (p.out_lse != nullptr && col == 0) p.out_lse[br] = none ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(den);
    }
    __syncthreads();
  }
}

template <int NR, bool BF16>
cudaError_t launch(cudaLaunchConfig_t cfg, const CUtensorMap& tm_ckv, const CUtensorMap& tm_kpe, const DecodeQ8Params& p) {
  static DeviceOnce once;
  const cudaError_t e = set_attribute_once(once, reinterpret_cast<const void*>(&mla_decode_q8_kernel<NR, BF16>),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NR, BF16>::kSmem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(p.groups), static_cast<unsigned>(p.gangs), 1);
  cfg.blockDim = dim3(Cfg<NR, BF16>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<NR, BF16>::kSmem;
  return cudaLaunchKernelEx(&cfg, mla_decode_q8_kernel<NR, BF16>, tm_ckv, tm_kpe, p);
}

}  // namespace

int q8_rows_per_cta(int total_rows) { return total_rows <= 16 ? 16 : 32; }
int q8_gangs(int total_rows, int sms) {
  const int nr = q8_rows_per_cta(total_rows), groups = (total_rows + nr - 1) / nr;
  const int gangs = sms > groups ? sms / groups : 1;
  return gangs;
}

cudaError_t launch_decode_q8(const CUtensorMap& tm_ckv, const CUtensorMap& tm_kpe, const DecodeQ8Params& p, bool bf16,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (q8_rows_per_cta(p.q_len * p.H) == 16)
    e = bf16 ? launch<16, true>(cfg, tm_ckv, tm_kpe, p) : launch<16, false>(cfg, tm_ckv, tm_kpe, p);
  else
    e = bf16 ? launch<32, true>(cfg, tm_ckv, tm_kpe, p) : launch<32, false>(cfg, tm_ckv, tm_kpe, p);
  if (e != cudaSuccess) return e;
  if (p.gangs == 1) return cudaSuccess;  // nothing is cut
  const int64_t rows = static_cast<int64_t>(p.q_len) * p.H;
  const int64_t blocks = p.cuts_by_request ? rows * p.B * kColUnits : (rows * p.gangs * kRowWarps + kMergeWarps - 1) / kMergeWarps;
  const int64_t wave = static_cast<int64_t>(kMergeBlocks) * p.gangs * p.groups;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < wave ? blocks : wave), 1, 1);
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, p.cuts_by_request ? mla_merge_q8_parts_kernel : mla_merge_q8_rows_kernel, p);
}

cudaError_t decode_q8_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
