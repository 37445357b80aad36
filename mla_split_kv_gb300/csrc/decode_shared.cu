// Decode attention of a batch whose contexts start with the same tokens, sm_103a.
//
// Absorbed latent attention (keys [ckv | kpe], values ckv) of B requests of q_len rows and H heads each, of whose tokens
// the first P are common: those are read and multiplied once, for all rows of the batch in groups of 128, and each
// request's own tokens once for its own rows:
//   s_t = scale (q_abs . ckv_t + q_pe . kpe_t),  out = sum_t softmax(s)_t ckv_t,  lse = log2 sum_t exp(s_t)
// over pieces of either, merged by their LSE. 2176 operations a (row, token): with the 1152 bytes of a token shared by
// 128 rows or more, the common part is tensor-core bound, each CTA's own shared memory right behind.
//
// An item is a group of up to 128 rows and a run of tokens, as two units: one CTA computes the scores of the group and
// one half of the value columns (O for all 512 would fill tensor memory), so that CTAs share nothing and wait for
// none. Tiles of 64 tokens; a unit's tensor memory: O [128 x 256] fp32, S [128 x 64] fp32, the weights [128 x 64] in 16
// bits as the value product's A operand, and 320 of the 576 query columns as the score product's (the other 256 are in
// shared memory, 64 KB; with two terms 256 and 320: a product that reads A there takes 49 cycles in place of 33). The products go
//   S(i+1) PV(i) S(i+2) PV(i+1) ...
// each issued by a warp of its own, PV(i) only behind S(i+1): S(i+1) is read out of its one buffer beside PV(i), and
// S(i)'s softmax runs beside PV(i-1) and S(i+1). (With PV(i) as soon as its weights are there it ran in the middle of
// S(i+1), and the tensor cores idled behind that: 2340 cycles a tile, 2100 in turns, of which the products take 1960.)
// A tile is 72 KB: the half of its latents that only the score product reads, with the rotary keys (two slots of 40 KB,
// free after S), and the half that is the values too (a ring of five pieces of 128 columns, 16 KB, free after PV): what
// the next score product needs last has been on its way longest.
//
// Four warps of their own read the next unit's queries while the last tiles of a unit are in the works, write them as
// soon as its last score product is done, and take its output out of tensor memory beside the next unit's first scores.
// 65,536 common tokens, 2432 rows: 296 us, 1.79 PFLOP/s of products as they run (the scores once in each of two CTAs).
//
// The running maximum moves only when a tile's passes it by more than 2^15 (fp16, the room its weights have above 1) or
// 2^30 (bf16), since with it all of O moves, for some row of a warp every few tiles. 64 requests, 32,768 common tokens,
// bf16, random latents: 116 us with 2^15, 109 with 2^20, 98 with 2^30 and with 2^60, which would leave values less room
// below fp32's end. Sums are of the unrounded weights, in fp32; the weights are rounded once to the cache's type (by half a
// step: 2^-11 of themselves in fp16, 2^-8 in bf16), as an output of that type is. Beside fp32 and fp16 outputs a bf16 weight is
// two terms, 2^-16 of itself (kTwo): rounded once, it leaves 0.7e-3 to 1.5e-3 of an output, where fp32 results are to keep
// 1e-3. The second term is a second value product over the same tile (captured: 64 requests as above 130 us, 98 with bf16
// outputs; 24 requests of 2 x 128 rows, 8192 common tokens 179 and 132), with 16 KB less of the ring and 64 fewer query columns
// in tensor memory.
// Tokens that some row of a group does not see (behind a shorter context or, in a window, behind the row) have weight 0
// there, and values that are not finite are taken out of such tiles. For a row that does see one of them its score is not
// finite either: a weight that is NaN, which makes all of the row so, or, with a score of -inf, one of 0, which times the
// value is NaN in that column: there the CTA writes NaN at its end (Small::dirty), as the product does in other tiles.
//
// Units are shared out by the host plan (plan_shared.cpp). The merge is a kernel of its own.
//
// Warps: 0-3 softmax (thread = row), 4 score products, 6 value products, 5 and 7 loads (of the two parts of a tile, each as
// soon as there is room), 8-11 queries and partial output (thread = row).
#include <type_traits>

#include "device_common.cuh"
#include "umma_issue.cuh"

namespace mla {

namespace {

constexpr int kT = 64;                    // tokens a tile
constexpr int kRows = 128;
constexpr int kHalf = kRank / 2;          // value columns of a unit
constexpr int kOther = kT * kHalf * 2;    // 32 KB: the other half of a tile's latents
constexpr int kPe = kT * kRope * 2;       // 8 KB
constexpr int kSlotA = kOther + kPe;
constexpr int kPiece = kT * 128 * 2;      // 16 KB: 128 of the unit's own columns
constexpr int kQChunk = kRows * 128;      // 16 KB: [128 rows x 64 columns]
constexpr int kScoreWarp = 4, kLoadWarpA = 5, kValueWarp = 6, kLoadWarpB = 7;
constexpr int kThreads = 384;
// Registers: launched with 120 a thread.
constexpr int kSoftmaxRegs = 168, kIssueRegs = 64, kAuxRegs = 128;
static_assert(kSoftmaxRegs + kIssueRegs + kAuxRegs <= 3 * 120, "what the block was launched with");
constexpr uint32_t kSmallBytes = 2048;
// Where things lie. With the weights as two terms (kTwo) their second 32 columns of tensor memory come from the queries', whose
// place in shared memory comes from the ring.
template <bool kTwo>
struct Shape {
  static constexpr int kRingB = kTwo ? 4 : 5;
  static constexpr int kQTmemBlocks = kTwo ? 4 : 5;  // blocks of 64 query columns in tensor memory; the others and the rotary one are not
  static constexpr int kQSmemChunks = kRank / kBoxCols - kQTmemBlocks + 1;
  static constexpr uint32_t kOffA = kQSmemChunks * kQChunk;
  static constexpr uint32_t kOffB = kOffA + 2 * kSlotA;
  static constexpr uint32_t kOffSmall = kOffB + kRingB * kPiece;
  static constexpr uint32_t kSmem = kOffSmall + kSmallBytes + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  static constexpr uint32_t kTmemQ = kTwo ? 384 : 352;
  static_assert(kTmemQ + 32 * kQTmemBlocks == 512, "tensor memory's columns");
};
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemP = 320, kTmemLow = 352;

constexpr float kLowest = -3.402823466e38f;  // LSE of a part that has no score above -inf

struct Small {
  uint64_t a_full[2], a_empty[2], b_full[4], b_empty[5], q_full, q_empty, s_full, s_empty, s_issued[2], p_full, pv_done, stat_full[2], o_empty, drain[2];
  float inv[2][kRows];  // 1 / sum, of the units in turn
  int32_t dirty;        // a value that some row sees was taken out of a tile
  uint32_t tmem_base;
  int32_t abort_flag;
};
static_assert(sizeof(Small) <= kSmallBytes, "small smem region");

__device__ __forceinline__ void tma_load_pages(void* dst, const CUtensorMap* map, int32_t block, int32_t group, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(0), "r"(0), "r"(block), "r"(group), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int32_t y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(0), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void store32(float* dst, const float* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void issue_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
}

struct Unit {
  int row0, rows, request, t0, t1, slot, half, tiles, least;  // least: tokens that every row of the group sees
};

// Tokens that flat row `row` ([B, q_len, H]) sees.
__device__ __forceinline__ int visible(const SharedParams& p, int row) {
  const int per = p.q_len * p.H, b = row / per;
  const int L = max(p.context_lens[b], 0);
  return p.causal ? max(0, L - p.q_len + (row % per) / p.H + 1) : L;
}

// The k-th unit of this CTA, by a whole warp. False behind the last one.
__device__ __forceinline__ bool unit_of(const SharedParams& p, int k, int lane, Unit& w) {
  const int at = __ldg(p.cta_indptr + blockIdx.x) + k;
  if (at >= __ldg(p.cta_indptr + blockIdx.x + 1)) return false;
  const int4* const unit = reinterpret_cast<const int4*>(p.units) + 2 * at;
  const int4 x = __ldg(unit), y = __ldg(unit + 1);
  w.row0 = x.x;
  w.rows = max(0, min(min(x.y, kRows), p.rows - x.x));
  w.request = x.z;
  w.t0 = x.w;
  w.slot = y.y;
  w.half = y.z & 1;
  int most = 0, least = 0x7fffffff;
  for (int r = lane; r < w.rows; r += 32) {
    const int v = visible(p, w.row0 + r);
    most = max(most, v);
    least = min(least, v);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  w.least = __reduce_min_sync(0xffffffffu, least);
  w.t1 = max(w.t0, min(min(y.x, most), w.request < 0 ? p.shared_tokens : 0x7fffffff));
  w.tiles = (w.t1 - w.t0 + kT - 1) / kT;
  return true;
}

// Values that are not finite in the unit's pieces of a tile (two of [64 tokens x 128 columns], eight tokens' rows of 64
// columns beside the same tokens' next 64) become 0; *dirty is set where one of them belongs to a token before `seen`.
template <bool BF16>
__device__ __forceinline__ void clean_values(uint8_t* p0, uint8_t* p1, int r, int tok0, int seen, volatile int32_t* dirty) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll 4
  for (int it = 0; it < 16; ++it) {
    const int idx = it * kRows + r;  // 16-byte pieces, 1024 a piece
    const uint32_t at = smem_u32((idx >= 1024 ? p1 : p0) + (idx & 1023) * 16);
    const uint4 v = lds128(at);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & (kExp * 0x10001u));
    if (__builtin_expect((m & 0xffffu) == kExp || (m >> 16) == kExp, 0)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((w[j] & kExp) == kExp) w[j] &= 0xffff0000u;
        if ((w[j] & (kExp << 16)) == (kExp << 16)) w[j] &= 0xffffu;
      }
      if (tok0 + ((idx & 1023) >> 7) * 8 + ((idx & 63) >> 3) < seen) *dirty = 1;
      sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

// Of a unit whose partial output this warp has written (rows from row0 on), the columns in which a row sees a value that was
// taken out of a masked tile become NaN: a token a round, eight columns a lane.
template <bool BF16>
__device__ __forceinline__ void spoil_output(const SharedParams& p, const Unit& w, int lane, int row0) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  const int32_t* const table = w.request < 0 ? p.shared_table : p.block_table + static_cast<long long>(w.request) * p.max_blocks;
  const int columns = w.request < 0 ? p.shared_tokens / p.bs : p.max_blocks;
  const int sees = row0 + lane < w.rows ? min(visible(p, w.row0 + row0 + lane), w.t1) : 0;
  const int most = __reduce_max_sync(0xffffffffu, sees);
  float* const out = p.part_o + (static_cast<long long>(w.slot) * kRows + row0) * kRank + kHalf * w.half + 8 * lane;
  __syncwarp();  // behind the rows' stores by other lanes
  for (int t = w.t0 + max(0, min(w.least, w.t1) - w.t0) / kT * kT; t < most; ++t) {
    const int col = t / p.bs, pid = col < columns ? table[col] : -1;
    if (pid < 0 || pid >= p.num_blocks) continue;  // (zeros)
    const uint16_t* const from = p.ckv + (static_cast<long long>(pid) * p.bs + t % p.bs) * kRank + kHalf * w.half + 8 * lane;
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= ((word[j / 2] >> (16 * (j & 1)) & kExp) == kExp ? 1u : 0u) << j;
    if (!__any_sync(0xffffffffu, bad != 0)) continue;
    for (int r = 0; r < 32; ++r) {
      if (__shfl_sync(0xffffffffu, sees, r) <= t) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (bad >> j & 1) out[static_cast<long long>(r) * kRank + j] = __int_as_float(0x7fffffff);
    }
  }
}

// 120 registers a thread at launch: a CTA of the merge then fits on an SM beside this kernel's one and waits there.
// kTwo (bf16): the weights as two terms.
template <bool BF16, bool kTwo>
__global__ void __maxnreg__(120)
    mla_decode_shared_kernel(const __grid_constant__ CUtensorMap tm_half, const __grid_constant__ CUtensorMap tm_piece,
                             const __grid_constant__ CUtensorMap tm_kpe, const __grid_constant__ SharedParams p) {
  using Place = Shape<kTwo>;
  constexpr int kRingB = Place::kRingB, kQTmemBlocks = Place::kQTmemBlocks, kQSmemChunks = Place::kQSmemChunks;
  constexpr uint32_t kOffA = Place::kOffA, kOffB = Place::kOffB, kTmemQ = Place::kTmemQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = align1024(smem_raw);
  Small* const sm = reinterpret_cast<Small*>(smem + Place::kOffSmall);
  volatile int32_t* const abort_flag = &sm->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm->a_full[s], 1);
      mbar_init(&sm->a_empty[s], 1);
    }
    // one arrival a piece; of four tiles, since pieces of the tile after next may be on their way while the score product
    // still waits for the second one of this
    for (int s = 0; s < 4; ++s) mbar_init(&sm->b_full[s], 2);
    for (int s = 0; s < kRingB; ++s) mbar_init(&sm->b_empty[s], 1);
    mbar_init(&sm->q_full, 4);
    mbar_init(&sm->q_empty, 1);
    mbar_init(&sm->stat_full[0], 4);
    mbar_init(&sm->stat_full[1], 4);
    mbar_init(&sm->o_empty, 4);
    mbar_init(&sm->s_full, 1);
    mbar_init(&sm->s_issued[0], 1);
    mbar_init(&sm->s_issued[1], 1);
    mbar_init(&sm->s_empty, 4);
    mbar_init(&sm->p_full, 4);
    mbar_init(&sm->pv_done, 1);
    mbar_init(&sm->drain[0], 1);
    mbar_init(&sm->drain[1], 1);
    sm->abort_flag = 0;
    sm->dirty = 0;
    fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    tmem_alloc(&sm->tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  const uint64_t tmo = p.timeout_ns;
  Unit w;

  if (warp == kLoadWarpA || warp == kLoadWarpB) {
    // ---------------------------------------------------------------- loads
    issue_registers();
    const bool first = warp == kLoadWarpA;  // the half that is only keys, and the rotary keys; else the values' half
    uint32_t tile = 0;
    bool ok = true;
    for (int k = 0; ok && unit_of(p, k, lane, w); ++k) {
      const int32_t* const table = w.request < 0 ? p.shared_table : p.block_table + static_cast<long long>(w.request) * p.max_blocks;
      const int columns = w.request < 0 ? p.shared_tokens / p.bs : p.max_blocks;
      for (int i = 0; i < w.tiles && ok; ++i, ++tile) {
        const int tok = w.t0 + i * kT;
        const int pages = (min(kT, w.t1 - tok) + p.bs - 1) / p.bs;  // (tok starts a page)
        int pid = -1;
        if (lane < pages) {
          const int col = tok / p.bs + lane;
          pid = col < columns ? table[col] : -1;  // (no __ldg: the kernel before this one may write tables while this one waits)
          if (pid < 0 || pid >= p.num_blocks) {
            flag_error(MLA_DEVERR_BAD_PAGE);
            pid = -1;  // (lies before the cache: zeros)
          }
        }
        const int group = pid * (p.bs / 8);
        if (first) {
          const uint32_t s = tile & 1;
          if (tile >= 2) ok = mbar_wait_warp(&sm->a_empty[s], ((tile >> 1) - 1) & 1, tmo);
          if (!ok) break;
          uint8_t* const a = smem + kOffA + s * kSlotA;
          if (lane == 0) mbar_arrive_expect_tx(&sm->a_full[s], pages * p.bs * (kHalf + kRope) * 2);
          __syncwarp();
          if (lane < pages) {
            tma_load_rows(a + kOther + lane * p.bs * 128, &tm_kpe, pid * p.bs, &sm->a_full[s]);
            tma_load_pages(a + lane * p.bs * (kHalf * 2), &tm_half, 4 * (w.half ^ 1), group, &sm->a_full[s]);
          }
          continue;
        }
#pragma unroll
        for (uint32_t x = 0; x < 2; ++x) {
          const uint32_t piece = 2 * tile + x, b = piece % kRingB;
          if (piece >= kRingB) ok = ok && mbar_wait_warp(&sm->b_empty[b], (piece / kRingB - 1) & 1, tmo);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm->b_full[tile & 3], pages * p.bs * 256);
          __syncwarp();
          if (lane < pages)
            tma_load_pages(smem + kOffB + b * kPiece + lane * p.bs * 256, &tm_piece, 4 * w.half + 2 * x, group, &sm->b_full[tile & 3]);
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == kScoreWarp) {
    // ---------------------------------------------------------------- score products: the warp in step (umma_issue.cuh)
    issue_registers();
    const uint32_t leader = elect_one();
    const uint32_t idesc = idesc_f16_f32(kRows, kT, BF16, false, false);
    const uint64_t q0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t a0 = smem_desc_sw128(smem_u32(smem + kOffA), 16, 4096);  // the other half, rows of tokens
    const uint64_t pe0 = smem_desc_sw128(smem_u32(smem + kOffA + kOther), 16, 1024);
    const uint64_t k0 = smem_desc_sw128(smem_u32(smem + kOffB), 16, 2048);  // a piece as keys
    uint32_t tile0 = 0, unit = 0;
    bool ok = true;
    auto block = [&](int cb, uint64_t keys) {  // a block of 64 latent columns
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (cb < kQTmemBlocks)
          issue_ts(leader, tmem + kTmemS, tmem + kTmemQ + 32 * cb + 8 * kk, keys + 2 * kk, idesc, 1);
        else
          issue_ss(leader, tmem + kTmemS, q0 + (cb - kQTmemBlocks) * (kQChunk / 16) + 2 * kk, keys + 2 * kk, idesc, 1);
      }
    };
    auto scores = [&](int i, auto half_of) {
      constexpr int half = decltype(half_of)::value;
      const uint32_t t = tile0 + i, s = t & 1;
      ok = ok && mbar_wait_warp(&sm->a_full[s], (t >> 1) & 1, tmo);
      if (t > 0) ok = ok && mbar_wait_warp(&sm->s_empty, (t - 1) & 1, tmo);
      if (!ok) return;
      tc_fence_after();
      const uint64_t pe = pe0 + s * (kSlotA / 16), a = a0 + s * (kSlotA / 16);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) issue_ss(leader, tmem + kTmemS, q0 + (kQSmemChunks - 1) * (kQChunk / 16) + 2 * kk, pe + 2 * kk, idesc, kk > 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) block(4 * (half ^ 1) + j, a + j * 64);
      issue_commit(leader, &sm->a_empty[s]);
      ok = ok && mbar_wait_warp(&sm->b_full[t & 3], (t >> 2) & 1, tmo);
      if (!ok) return;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t b = (2 * t + x) % kRingB;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (x == 1 && j == 1 && lane == 0) mbar_arrive(&sm->s_issued[t & 1]);
          __syncwarp();
          block(4 * half + 2 * x + j, k0 + b * (kPiece / 16) + j * 64);
        }
      }
      issue_commit(leader, &sm->s_full);
      if (i + 1 == w.tiles) issue_commit(leader, &sm->q_empty);
    };
    for (int k = 0; ok && unit_of(p, k, lane, w); ++k) {
      if (w.tiles == 0) continue;
      ok = mbar_wait_warp(&sm->q_full, unit & 1, tmo);
      ++unit;
      if (w.half == 0) {
        for (int i = 0; i < w.tiles && ok; ++i) scores(i, std::integral_constant<int, 0>{});
      } else {
        for (int i = 0; i < w.tiles && ok; ++i) scores(i, std::integral_constant<int, 1>{});
      }
      tile0 += w.tiles;
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
    issue_commit(leader, &sm->drain[0]);  // every product is done before tensor memory is freed
    mbar_wait(&sm->drain[0], 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp == kValueWarp) {
    // ---------------------------------------------------------------- value products: a warp of their own, so that what one
    // of the two waits for is hidden behind the other's products
    issue_registers();
    const uint32_t leader = elect_one();
    const uint32_t idesc = idesc_f16_f32(kRows, 128, BF16, false, true);
    const uint64_t v0 = smem_desc_sw128(smem_u32(smem + kOffB), 1024, 2048);  // a piece as values
    uint32_t t = 0, unit = 0;
    bool ok = true;
    for (int k = 0; ok && unit_of(p, k, lane, w); ++k) {
      if (w.tiles == 0) continue;
      if (unit > 0) ok = mbar_wait_warp(&sm->o_empty, (unit - 1) & 1, tmo);
      ++unit;
      for (int i = 0; i < w.tiles && ok; ++i, ++t) {
        ok = mbar_wait_warp(&sm->p_full, t & 1, tmo);  // (its scores are done: the tile is there)
        // behind the next tile's scores, whose softmax then runs beside this product
        if (i + 1 < w.tiles) ok = ok && mbar_wait_warp(&sm->s_issued[(t + 1) & 1], ((t + 1) >> 1) & 1, tmo);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t b = (2 * t + x) % kRingB;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            issue_ts(leader, tmem + kTmemO + 128 * x, tmem + kTmemP + 8 * kk, v0 + b * (kPiece / 16) + kk * 256, idesc, i > 0 || kk > 0);
          if constexpr (kTwo) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              issue_ts(leader, tmem + kTmemO + 128 * x, tmem + kTmemLow + 8 * kk, v0 + b * (kPiece / 16) + kk * 256, idesc, 1);
          }
          if (x == 0) issue_commit(leader, &sm->b_empty[b]);
        }
        issue_commit(leader, &sm->pv_done);
        issue_commit(leader, &sm->b_empty[(2 * t + 1) % kRingB]);
      }
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
    issue_commit(leader, &sm->drain[1]);
    mbar_wait(&sm->drain[1], 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp < kScoreWarp) {
    // ---------------------------------------------------------------- softmax: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int r = tid;
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const float scale = p.scale_log2;
    constexpr float kSlack = BF16 ? 30.f : 15.f;
    uint32_t tile0 = 0, unit = 0;
    bool ok = true;
    for (int k = 0; ok && unit_of(p, k, lane, w); ++k) {
      const bool real = r < w.rows;
      const long long row = w.row0 + (real ? r : 0);
      const long long slot_row = static_cast<long long>(w.slot) * kRows + r;
      if (w.tiles == 0) {
        if (real && w.half == 0) p.part_lse[slot_row] = -INFINITY;  // (the merge does not read the values)
        continue;
      }
      const int seen = real ? visible(p, static_cast<int>(row)) : 0x7fffffff;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < w.tiles; ++i) {
        const uint32_t t = tile0 + i;
        const int tok = w.t0 + i * kT;
        ok = mbar_wait_warp(&sm->s_full, t & 1, tmo);
        if (!ok) break;
        tc_fence_after();
        float x[kT];
        ld32(tmem + lanes + kTmemS, x);
        ld32(tmem + lanes + kTmemS + 32, x + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->s_empty);
        const int limit = min(w.t1, w.least);  // tokens that every row sees
        const bool masked = tok + kT > limit;
        float f = scale;
        if (masked) {
          const int nvis = min(seen, w.t1) - tok;
#pragma unroll
          for (int j = 0; j < kT; ++j) x[j] = j < nvis ? x[j] * scale : -INFINITY;
          f = 1.f;
        }
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int j = 4; j < kT; j += 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = fmaxf(m4[q], x[j + q]);
        }
        // (a negative scale: the largest score is the smallest product's)
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f;
        if (!masked && scale < 0.f) {
          float lo = x[0];
#pragma unroll
          for (int j = 1; j < kT; ++j) lo = fminf(lo, x[j]);
          mx = lo * f;
        }
        const bool need = mx > m + kSlack;
        const float m_new = need ? mx : m;
        const float mm = m_new == -INFINITY ? 0.f : -m_new;
        const float2 f2 = make_float2(f, f), m2 = make_float2(mm, mm);
        float2 sum = make_float2(0.f, 0.f), sum_b = sum;
        uint32_t h[kT / 2], low[kTwo ? kT / 2 : 1];
#pragma unroll
        for (int j = 0; j < kT / 2; ++j) {
          float2 e = fma2(make_float2(x[2 * j], x[2 * j + 1]), f2, m2);
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          if (j & 1) sum_b = add2(sum_b, e);
          else sum = add2(sum, e);
          h[j] = pack2<BF16>(e.x, e.y);
          if constexpr (kTwo) low[j] = pack2<BF16>(e.x - __uint_as_float(h[j] << 16), e.y - __uint_as_float(h[j] & 0xffff0000u));
        }
        sum = add2(sum, sum_b);
        if (t > 0) {  // the weights' buffer, and (but for a unit's first tile) O, are free
          ok = mbar_wait_warp(&sm->pv_done, (t - 1) & 1, tmo);
          if (!ok) break;
          tc_fence_after();
        }
        if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
          const float alpha = need ? (m == -INFINITY ? 0.f : exp2f(m - m_new)) : 1.f;
          if (i > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < kHalf / 16; ++q) {
              float o[16];
              tmem_ld16(tmem + lanes + kTmemO + 16 * q, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= alpha;
              tmem_st16(tmem + lanes + kTmemO + 16 * q, o);
            }
            tmem_wait_st();
          }
          l *= alpha;
          m = m_new;
        }
        l += sum.x + sum.y;
        if (masked) {  // (b_full is complete: so are the scores)
          const uint32_t b = 2 * t, c = b + 1;
          ok = mbar_wait_warp(&sm->b_full[t & 3], (t >> 2) & 1, tmo);
          if (!ok) break;
          clean_values<BF16>(smem + kOffB + (b % kRingB) * kPiece, smem + kOffB + (c % kRingB) * kPiece, r, tok, w.t1, &sm->dirty);
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(h[16 * j + c]);
          tmem_st16(tmem + lanes + kTmemP + 16 * j, v);
          if constexpr (kTwo) {
#pragma unroll
            for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(low[16 * j + c]);
            tmem_st16(tmem + lanes + kTmemLow + 16 * j, v);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full);
      }
      if (!ok) break;
      const bool any = m != -INFINITY;
      sm->inv[unit & 1][r] = any ? 1.f / l : 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->stat_full[unit & 1]);
      // (-inf is for what was not written: a part whose scores are all -inf counts with weight 0, its NaN among its values)
      if (real && w.half == 0) p.part_lse[slot_row] = any ? m + log2f(l) : (l != l ? l : kLowest);
      ++unit;
      tile0 += w.tiles;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ---------------------------------------------------------------- queries and partial output: thread = row
    // While a unit's last tiles are still in the works, the next one's queries are read, and written as soon as its last
    // score product is done; its first scores and their softmax run beside the output of the unit before.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
    const int r = tid & (kRows - 1);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    uint32_t unit = 0, tile0 = 0;
    int slot = 0, rows = 0, half = 0;  // of the unit before
    bool ok = true;
    auto output = [&](auto last_of) {  // of unit - 1, whose last tile is tile0 - 1
      constexpr bool last = decltype(last_of)::value;
      // (a barrier a unit in turns: the unit after may be through its softmax, the one behind that waits for this output)
      ok = mbar_wait_warp(&sm->stat_full[(unit - 1) & 1], ((unit - 1) >> 1) & 1, tmo);
      ok = ok && mbar_wait_warp(&sm->pv_done, (tile0 - 1) & 1, tmo);
      if (!ok) return;
      tc_fence_after();
      const float inv = sm->inv[(unit - 1) & 1][r];
      float* const out = p.part_o + (static_cast<long long>(slot) * kRows + r) * kRank + kHalf * half;
      const uint32_t stage = smem_u32(smem + kOffA) + 4096 * (warp & 3);
#pragma unroll 1
      for (int q = 0; q < kHalf / 32; ++q) {
        float o[32];
        ld32(tmem + lanes + kTmemO + 32 * q, o);
        tmem_wait_ld();
        if constexpr (last) {
          // nothing else runs any more: through 4 KB a warp of the tiles' place, rows of 128 bytes out, four to an
          // instruction (a thread a row, 32 bytes each, takes the memory pipeline longer)
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sts128(stage + lane * 128 + ((j ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(o[4 * j] * inv), __float_as_uint(o[4 * j + 1] * inv), __float_as_uint(o[4 * j + 2] * inv), __float_as_uint(o[4 * j + 3] * inv)));
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = 4 * j + (lane >> 3), c = lane & 7;  // row, 16-byte piece
            const uint4 v = lds128(stage + at * 128 + ((c ^ (at & 7)) << 4));
            if (32 * (warp & 3) + at < rows) *reinterpret_cast<uint4*>(out + static_cast<long long>(at - lane) * kRank + 32 * q + 4 * c) = v;
          }
          continue;
        }
        if (q == kHalf / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->o_empty);
        }
        if (r < rows) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = o[8 * j + i] * inv;
            store32(out + 32 * q + 8 * j, v);
          }
        }
      }
    };
    for (int k = 0; ok && unit_of(p, k, lane, w); ++k) {
      const bool real = r < w.rows;
      const long long row = w.row0 + (real ? r : 0);
      if (w.tiles == 0) continue;
      const uint4* const src = reinterpret_cast<const uint4*>(p.q_abs + row * kRank);
      const uint4 none = make_uint4(0, 0, 0, 0);
      constexpr int kPieces = 4 * kQTmemBlocks;
      static_assert(kQTmemBlocks * 8 == 2 * kPieces, "two rounds of loads");
      uint4 x[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) x[j] = real ? src[j] : none;
      if (unit > 0) ok = mbar_wait_warp(&sm->q_empty, (unit - 1) & 1, tmo);
      if (!ok) break;
      tc_fence_after();
      // the blocks of shared memory, eight lanes a row's 128 bytes, all in flight; those of tensor memory beside them, a
      // thread a row, in two rounds of 16-byte pieces
      for (int at = r; at < kQSmemChunks * kRows * 8; at += kRows) {
        const int c = at / (kRows * 8), rr = at / 8 % kRows, j = at % 8;
        const bool in = rr < w.rows;
        const long long from = w.row0 + (in ? rr : 0);
        const uint16_t* const piece = c < kQSmemChunks - 1 ? p.q_abs + from * kRank + (kQTmemBlocks + c) * kBoxCols + 8 * j : p.q_pe + from * kRope + 8 * j;
        cp_async16(smem + c * kQChunk + rr * 128 + ((j ^ (rr & 7)) << 4), piece, in ? 16u : 0u);
      }
#pragma unroll
      for (int round = 0; round < 2; ++round) {
#pragma unroll
        for (int g = 0; g < kPieces / 4; ++g) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[4 * j] = __uint_as_float(x[4 * g + j].x);
            v[4 * j + 1] = __uint_as_float(x[4 * g + j].y);
            v[4 * j + 2] = __uint_as_float(x[4 * g + j].z);
            v[4 * j + 3] = __uint_as_float(x[4 * g + j].w);
          }
          tmem_st16(tmem + lanes + kTmemQ + 16 * (round * (kPieces / 4) + g), v);
        }
        if (round == 0) {
#pragma unroll
          for (int j = 0; j < kPieces; ++j) x[j] = real ? src[kPieces + j] : none;
        }
      }
      cp_async_wait_all();
      tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_full);
      if (unit > 0) output(std::false_type{});
      slot = w.slot;
      rows = w.rows;
      half = w.half;
      tile0 += w.tiles;
      ++unit;
    }
    if (ok && unit > 0) output(std::true_type{});
    if (__builtin_expect(ok && *const_cast<volatile int32_t*>(&sm->dirty) != 0, 0)) {
      for (int k = 0; unit_of(p, k, lane, w); ++k)
        if (w.tiles > 0) spoil_output<BF16>(p, w, lane, 32 * (warp & 3));
    }
    tc_fence_before();
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) settle_in_flight(3000000ull);  // copies in flight land before shared memory goes
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, 512);
}

// kSplit warps a row, each a share of its columns: the parts in order (the common tokens' pieces, then its own tokens'),
// M = max lse, weights 2^(lse - M). Latency: the offsets (the plan's) are read before the decode kernel ends, the first
// parts' values beside their LSE, and 4 KB a warp are in flight. Four warps a row up to 2048 rows, one with more (64 rows
// of 17 parts: 13.9 us a call with four, 16.5 with one; 1024 rows: 105.9, 109.2; 6144: 148.5, 145.2).
constexpr int kMergeThreads = 128;
constexpr int kMergeFewRows = 2048;
template <int kSplit>
__global__ void __launch_bounds__(kMergeThreads, 6) mla_decode_shared_merge_kernel(const SharedParams p) {
  constexpr int kCols = 4 / kSplit;       // times 4 columns a lane
  constexpr int kMergeDepth = 2 * kSplit;  // parts in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * (4 / kSplit) + warp / kSplit, col = kRank / kSplit * (warp % kSplit) + 4 * lane;
  const int per = p.q_len * p.H, b = row / per, r = row % per;
  const int own = b * ((per + kRows - 1) / kRows) + r / kRows;
  const bool in = row < p.rows;
  const int s0 = in ? p.own_indptr[own] : 0, n = in ? p.shared_parts + p.own_indptr[own + 1] - s0 : 0;
  pdl_wait();
  pdl_launch_dependents();
  if (!in) return;
  // the row of part j in the slots
  auto at = [&](int j) -> long long {
    return j < p.shared_parts ? (static_cast<long long>(row / kRows) * p.shared_parts + j) * kRows + row % kRows
                              : static_cast<long long>(s0 + j - p.shared_parts) * kRows + r % kRows;
  };
  // a group of parts' values and, in as many lanes, their LSE
  float lse;
  float4 v[kMergeDepth][kCols];
  auto load = [&](int j0) {
    lse = lane < kMergeDepth && j0 + lane < n ? p.part_lse[at(j0 + lane)] : -INFINITY;
#pragma unroll
    for (int j = 0; j < kMergeDepth; ++j) {
      const float* const from = p.part_o + at(min(j0 + j, n - 1)) * kRank + col;
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[j][c] = *reinterpret_cast<const float4*>(from + 128 * c);
    }
  };
  load(0);
  float M = lse;
  for (int j = kMergeDepth + lane; j < n; j += 32) M = max_nan(M, p.part_lse[at(j)]);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, d));
  float4 acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  const bool none = M <= kLowest;  // no score above -inf
  if (!none) {
    for (int j0 = 0; j0 < n; j0 += kMergeDepth) {
      if (j0 > 0) load(j0);
      const float w = lse == -INFINITY ? -1.f : exp2f(lse - M);
#pragma unroll
      for (int j = 0; j < kMergeDepth; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        if (wj == -1.f) continue;  // (nothing was written there)
        den += wj;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          acc[c].x = fmaf(wj, v[j][c].x, acc[c].x);
          acc[c].y = fmaf(wj, v[j][c].y, acc[c].y);
          acc[c].z = fmaf(wj, v[j][c].z, acc[c].z);
          acc[c].w = fmaf(wj, v[j][c].w, acc[c].w);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = make_float4(acc[c].x / den, acc[c].y / den, acc[c].z / den, acc[c].w / den);
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) store_out4(p.out, p.out_dtype, static_cast<long long>(row) * kRank + col + 128 * c, acc[c]);
  if (lane == 0 && warp % kSplit == 0 && p.out_lse != nullptr) p.out_lse[row] = none ? -INFINITY : merged_lse(M, den);
}

cudaError_t launch_dependent(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaSuccess;
}

template <bool BF16, bool kTwo>
cudaError_t launch_units(const CUtensorMap& tm_half, const CUtensorMap& tm_piece, const CUtensorMap& tm_kpe, const SharedParams& p,
                         cudaStream_t stream) {
  static DeviceOnce once;
  constexpr uint32_t kSmem = Shape<kTwo>::kSmem;
  const cudaError_t e = set_attribute_once(once, reinterpret_cast<const void*>(&mla_decode_shared_kernel<BF16, kTwo>),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  launch_dependent(cfg, attr, p.num_ctas, kThreads, kSmem, stream);
  return cudaLaunchKernelEx(&cfg, mla_decode_shared_kernel<BF16, kTwo>, tm_half, tm_piece, tm_kpe, p);
}

}  // namespace

cudaError_t launch_decode_shared(const CUtensorMap& tm_half, const CUtensorMap& tm_piece, const CUtensorMap& tm_kpe,
                                 const SharedParams& p, bool bf16, cudaStream_t stream) {
  // (bf16 caches, and outputs that hold more than bf16 does: the weights as two terms)
  const cudaError_t e = !bf16              ? launch_units<false, false>(tm_half, tm_piece, tm_kpe, p, stream)
                        : p.out_dtype != 1 ? launch_units<true, true>(tm_half, tm_piece, tm_kpe, p, stream)
                                           : launch_units<true, false>(tm_half, tm_piece, tm_kpe, p, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  if (p.rows <= kMergeFewRows) {
    launch_dependent(cfg, attr, p.rows, kMergeThreads, 0, stream);
    return cudaLaunchKernelEx(&cfg, mla_decode_shared_merge_kernel<4>, p);
  }
  launch_dependent(cfg, attr, (p.rows + 3) / 4, kMergeThreads, 0, stream);
  return cudaLaunchKernelEx(&cfg, mla_decode_shared_merge_kernel<1>, p);
}

cudaError_t decode_shared_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
