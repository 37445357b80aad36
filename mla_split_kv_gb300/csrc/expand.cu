// Keys and values of every head from cached latents (the expanded form of latent attention), sm_103a.
//
// For token t of a request, head h, with c_t its latent [512]:
//   k_nope[t, h, :] = W_UK[h] c_t      ([128, 512])
//   v[t, h, :]      = W_UV^T[h]^T c_t  ([512, 128] transposed)
// accumulated in fp32 and rounded once to the cache's type; the rotary key, shared by the heads, is copied.
//
// One product [tokens x 512] . [512 x 256 H]: 262,144 H operations a token against 512 H bytes written, so
// tensor-core bound for many heads, with writes at about half the memory's rate beside it. K is only 512: a tile's
// outputs have to be drained as fast as four thousand cycles of products make them.
//
// A pair of CTAs (cta_group::2, M = 256) takes blocks of 256 tokens of one request, 128 rows a CTA, and walks over
// the heads two at a time, their keys, then their values (N = 256): the latents of a block stay in shared memory (128
// KB a CTA, loaded page by page through the block table, 128-byte swizzle) while the heads' weights stream through a
// ring of four 16 KB stages, each 64 latent columns of one head a CTA (the pair shares B): W_UK as it lies, W_UV^T
// with the operand's other dimension contiguous. Shared memory sets the tile: at 128 bytes a cycle, products of N =
// 256 read 64 (N = 128, a head's keys beside its values: 96), the refills write 32 and the way out takes 32.
// Accumulators of two tiles alternate in tensor memory (2 x 256 columns): eight warps drain one through 4 KB each of
// shared memory and TMA stores of [32 tokens x 64 columns], while the next is computed. (32 bytes a thread, every
// thread another token, straight to memory: 527 us against 352 without any stores, of 16,384 tokens and 128 heads.)
// Every pair takes an equal run of the (block, two heads, keys or values) tiles (Walk). A block's tile costs the same 2.3 us
// however few of its 256 rows are tokens: 32 requests of 18 tokens under 128 heads take 132 us, as one request 25.
//
// Warps: 0-7 epilogue (0-3 the first head, 4-7 the second), 8 loads, 9 products (of the pair's first CTA).
#include "device_common.cuh"
#include "umma_issue.cuh"

namespace mla {

namespace {

constexpr int kBlock = 256;               // tokens a pair takes at a time
constexpr int kRows = 128;                // of them a CTA
constexpr int kHeadCols = 128;            // key (without rotation) and value columns of a head
constexpr int kChunks = kRank / kBoxCols; // 8 column blocks of 64
constexpr int kAChunk = kRows * 128;      // 16 KB: [128 tokens x 64 columns]
constexpr int kStage = kHeadCols * 128;   // 16 KB: [128 x 64] of W_UK, or two [64 x 64] of W_UV^T
constexpr int kStages = 4;
static_assert(kChunks % kStages == 0, "the products' addresses are known when they are compiled");
constexpr int kEpiWarps = 8;
constexpr int kOutBox = 32 * 128;         // 4 KB: [32 tokens x 64 columns] on the way out
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr uint32_t kOffRing = kChunks * kAChunk;
constexpr uint32_t kOffOut = kOffRing + kStages * kStage;
constexpr uint32_t kOffSmall = kOffOut + kEpiWarps * kOutBox;
constexpr uint32_t kSmem = kOffSmall + 1024 + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");

struct Small {
  uint64_t full[kStages], empty[kStages], a_full, a_empty, t_full[2], t_empty[2];
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t first_b, first_blk, last_b, last_blk;
  int32_t part[kThreads / 32];
};
static_assert(sizeof(Small) <= 1024, "small smem region");

// A tile into this CTA's shared memory that completes on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma2_load_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
// A box from shared memory out; the thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z, const void* src,
                                             uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(
                   map),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src)), "l"(policy)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_last() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
  const float x = __uint_as_float(a), y = __uint_as_float(b);
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// First packed row and number of tokens of request b, within the outputs.
__device__ __forceinline__ int2 request_rows(const ExpandParams& p, int b) {
  const int k0 = p.kv_indptr[b], k1 = min(p.kv_indptr[b + 1], p.max_tokens);
  return k0 < 0 || k1 <= k0 ? make_int2(0, 0) : make_int2(k0, k1 - k0);
}
__host__ __device__ constexpr int tiles_per_block(int H) { return 2 * ((H + 1) / 2); }
__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }

// The tiles of a pair: of a block, two heads' keys (h even), then their values (h odd). The run's last block comes
// first, if the run ends inside it, then the others in order: all runs are equally long, so all pairs then go through
// the heads at the same time, and the weights that one has brought into L2 serve the others before the outputs that
// stream through it have pushed them out.
struct Walk {
  int b, blk, h, per_block, left, jump;
  int2 rows;
  bool fresh;  // the first tile of a block
  __device__ __forceinline__ void at(const ExpandParams& p, int b0, int blk0, int h0) {
    b = b0;
    blk = blk0;
    h = h0;
    rows = request_rows(p, b);
    fresh = true;
  }
  __device__ __forceinline__ void start(const ExpandParams& p, const Small* sm, int n, int h0) {
    per_block = tiles_per_block(p.H);
    left = n;
    const int tail = (h0 + n) % per_block;  // tiles of the last block, if the run ends inside it
    jump = h0 + n > per_block && tail > 0 ? n - tail : 0;  // that many are left behind them
    if (jump > 0) at(p, sm->last_b, sm->last_blk, 0);
    else at(p, sm->first_b, sm->first_blk, h0);
  }
  __device__ __forceinline__ void next(const ExpandParams& p, const Small* sm, int h0) {
    fresh = false;
    if (--left == jump && jump > 0) {
      at(p, sm->first_b, sm->first_blk, h0);
      return;
    }
    if (++h < per_block) return;
    h = 0;
    fresh = true;
    if (++blk < blocks_of(rows.y)) return;
    blk = 0;
    do {
      ++b;
      rows = b < p.B ? request_rows(p, b) : make_int2(0, 0);
    } while (b < p.B && rows.y == 0);
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_expand_kv_kernel(const __grid_constant__ CUtensorMap tm_ckv, const __grid_constant__ CUtensorMap tm_uk,
                         const __grid_constant__ CUtensorMap tm_uv, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = align1024(smem_raw);
  Small* const sm = reinterpret_cast<Small*>(smem + kOffSmall);
  volatile int32_t* const abort_flag = &sm->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
    }
    mbar_init(&sm->a_full, 1);
    mbar_init(&sm->a_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm->t_full[s], 1);
      mbar_init(&sm->t_empty[s], 2 * kEpiWarps);
    }
    sm->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm->tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == kLoadWarp) {
    // all weights into L2, a share of them by each CTA: pairs in step would wait for memory together at every tile
    // (16,384 tokens, 128 heads: 421 us without)
    constexpr uint32_t kPiece = 4096;
    const long long pieces = static_cast<long long>(p.H) * kHeadCols * kRank * 2 / kPiece;  // of either
    for (long long i = static_cast<long long>(blockIdx.x) * 32 + lane; i < 2 * pieces; i += static_cast<long long>(gridDim.x) * 32)
      bulk_prefetch_l2((i < pieces ? p.w_uk + i * kPiece : p.w_uv_t + (i - pieces) * kPiece), kPiece);
  }
  pdl_wait();
  pdl_launch_dependents();

  // how many blocks there are, and where this pair's run of tiles starts
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    mine += blocks_of(request_rows(p, b).y);
    bad |= p.kv_indptr[b] < 0 || p.kv_indptr[b + 1] < p.kv_indptr[b] || p.kv_indptr[b + 1] > p.max_tokens;
  }
  if (bad && blockIdx.x == 0) flag_error(MLA_DEVERR_BAD_PAGE);
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += y;
  }
  if (lane == 31) sm->part[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int blocks = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm->part[w];
    blocks += sm->part[w];
  }
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const int per_block = tiles_per_block(p.H);
  const long long tiles = static_cast<long long>(blocks) * per_block;
  const long long g0 = tiles * pair / pairs, g1 = tiles * (pair + 1) / pairs;
  const int n = static_cast<int>(g1 - g0);
  const int first = static_cast<int>(g0 / per_block), h0 = static_cast<int>(g0 % per_block);
  const int last = static_cast<int>((g1 - 1) / per_block);
  if (n > 0 && last >= before && first < before + mine) {  // this thread's requests have one of the two blocks
    int at = before;
    for (int b = b0; b < b1; ++b) {
      const int nb = blocks_of(request_rows(p, b).y);
      if (first >= at && first < at + nb) {
        sm->first_b = b;
        sm->first_blk = first - at;
      }
      if (last >= at && last < at + nb) {
        sm->last_b = b;
        sm->last_blk = last - at;
      }
      at += nb;
    }
  }
  cluster_sync();  // the barriers of both CTAs are set up
  const uint32_t tmem = sm->tmem_base;
  const uint64_t tmo = p.timeout_ns;
  Walk w;
  if (n > 0) w.start(p, sm, n, h0);

  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loads
    uint32_t use = 0, block = 0;
    bool ok = true;
    const uint64_t once = l2_policy_evict_first(), often = l2_policy_evict_last();  // latents; weights
    for (int i = 0; i < n && ok; ++i, w.next(p, sm, h0)) {
      if (w.fresh) {
        if (block > 0) {
          if (lane == 0) ok = mbar_wait(&sm->a_empty, (block - 1) & 1, tmo) && !*abort_flag;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
        }
        ++block;
        const int t0 = w.blk * kBlock;
        const int pages0 = (min(w.rows.y - t0, kRows) + p.bs - 1) / p.bs;                    // of the first CTA's rows
        const int pages1 = (min(max(w.rows.y - t0 - kRows, 0), kRows) + p.bs - 1) / p.bs;   // of the second's
        const int own = rank == 0 ? pages0 : pages1;
        if (rank == 0 && lane == 0)
          mbar_arrive_expect_tx(&sm->a_full, static_cast<uint32_t>((pages0 + pages1) * p.bs * kRank * 2));
        __syncwarp();
        const uint32_t bar = dsmem_addr(&sm->a_full, 0);
        if (lane < own) {
          const int col = (t0 + rank * kRows) / p.bs + lane;
          int pid = col < p.max_blocks ? p.block_table[static_cast<long long>(w.b) * p.max_blocks + col] : -1;
          if (pid < 0 || pid >= p.num_blocks) {
            flag_error(MLA_DEVERR_BAD_PAGE);
            pid = -1;  // (lies before the cache: zeros)
          }
          for (int c = 0; c < kChunks; ++c)
            tma2_load_2d(smem + c * kAChunk + lane * p.bs * 128, &tm_ckv, c * kBoxCols, pid * p.bs, bar, once);
        }
        __syncwarp();
      }
      if (lane == 0) {
        for (int c = 0; c < kChunks; ++c, ++use) {
          const int s = use % kStages;
          if (use >= kStages && !(mbar_wait(&sm->empty[s], (use / kStages - 1) & 1, tmo) && !*abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* const at = smem + kOffRing + s * kStage;
          const uint32_t bar = dsmem_addr(&sm->full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&sm->full[s], 2 * kStage);
          const int head = (w.h & ~1) + rank;  // (past the last one: zeros)
          if ((w.h & 1) == 0) {
            tma2_load_2d(at, &tm_uk, c * kBoxCols, head * kHeadCols, bar, often);
          } else {
            tma2_load_2d(at, &tm_uv, 0, head * kRank + c * kBoxCols, bar, often);
            tma2_load_2d(at + kStage / 2, &tm_uv, kBoxCols, head * kRank + c * kBoxCols, bar, often);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (!ok && lane == 0) *abort_flag = 1;
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    if (rank == 0) {  // the whole warp in step; one lane's instructions count
      const uint32_t leader = elect_one();
      const uint32_t idesc_k = idesc_f16_f32(kBlock, 2 * kHeadCols, BF16, false, false);
      const uint32_t idesc_v = idesc_f16_f32(kBlock, 2 * kHeadCols, BF16, false, true);
      const uint64_t a0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k0 = smem_desc_sw128(smem_u32(smem + kOffRing), 16, 1024);
      const uint64_t v0 = smem_desc_sw128(smem_u32(smem + kOffRing), kStage / 2, 1024);
      uint32_t use = 0, block = 0;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        if (w.fresh) {
          ok = mbar_wait_warp(&sm->a_full, block & 1, tmo);
          ++block;
        }
        const int buf = i & 1;
        if (i >= 2) ok = ok && __all_sync(0xffffffffu, mbar_wait_cluster(&sm->t_empty[buf], ((i >> 1) - 1) & 1, tmo));
        if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * 2 * kHeadCols;
        const bool keys = (w.h & 1) == 0;
        w.next(p, sm, h0);
        const bool block_done = w.fresh;
        auto stages = [&](const uint64_t b0, const uint32_t step, const uint32_t idesc) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c, ++use) {
            const int s = c % kStages;  // (a tile's chunks go round the ring a whole number of times)
            ok = ok && mbar_wait_warp(&sm->full[s], (use / kStages) & 1, tmo);
            const uint64_t a = a0 + c * (kAChunk / 16), b = b0 + s * (kStage / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) issue2_ss(leader, d, a + 2 * kk, b + step * kk, idesc, c > 0 || kk > 0);
            issue2_commit(leader, &sm->empty[s]);
          }
        };
        if (keys) stages(k0, 2, idesc_k);
        else stages(v0, 128, idesc_v);
        if (block_done) issue2_commit(leader, &sm->a_empty);
        issue2_commit(leader, &sm->t_full[buf]);
      }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int part = warp >> 2;  // head of the two
    const int row = rank * kRows + 32 * (warp & 3);  // the warp's first token of the block
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint64_t once = l2_policy_evict_first();  // the outputs pass through L2 and leave the weights there
    uint8_t* const stage = smem + kOffOut + warp * kOutBox;
    const uint32_t mine_at = smem_u32(stage) + lane * 128;
    for (int i = 0; i < n; ++i, w.next(p, sm, h0)) {
      const int buf = i & 1;
      if (w.h == 0) {  // the block's rotary keys: eight lanes a token
        for (int r = tid >> 3; r < kRows; r += kEpiWarps * 4) {
          const int t = w.blk * kBlock + rank * kRows + r;
          if (t >= w.rows.y) break;
          const int col = t / p.bs;
          const int pid = col < p.max_blocks ? p.block_table[static_cast<long long>(w.b) * p.max_blocks + col] : -1;
          uint4 x = make_uint4(0, 0, 0, 0);  // (a page outside the pool: flagged by the loads)
          if (pid >= 0 && pid < p.num_blocks)
            x = reinterpret_cast<const uint4*>(p.kpe + (static_cast<long long>(pid) * p.bs + t % p.bs) * kRope)[tid & 7];
          reinterpret_cast<uint4*>(p.k_pe + static_cast<long long>(w.rows.x + t) * kRope)[tid & 7] = x;
        }
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&sm->t_full[buf], (i >> 1) & 1, tmo) && !*abort_flag;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const int t = w.blk * kBlock + row, head = (w.h & ~1) + part;
      const bool whole = t + 32 <= w.rows.y;  // else the rows behind the last token are someone else's
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t x[kBoxCols / 2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t r[32];
          tmem_ld32(tmem + lanes + (2 * buf + part) * kHeadCols + kBoxCols * half + 32 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) x[16 * q + j] = pack2<BF16>(r[2 * j], r[2 * j + 1]);
        }
        if (half == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(dsmem_addr(&sm->t_empty[buf], 0));
        }
        if (head >= p.H || t >= w.rows.y) continue;
        if (whole) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the box before is read
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sts128(mine_at + ((j ^ (lane & 7)) << 4), make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_3d((w.h & 1) == 0 ? &tm_k : &tm_v, kBoxCols * half, head, w.rows.x + t, stage, once);
        } else if (t + lane < w.rows.y) {
          uint16_t* const at = ((w.h & 1) == 0 ? p.k_nope : p.v) + (static_cast<long long>(w.rows.x + t + lane) * p.H + head) * kHeadCols + kBoxCols * half;
#pragma unroll
          for (int q = 0; q < 4; ++q) store32(at + 16 * q, x + 8 * q);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) settle_in_flight(3000000ull);  // copies and products in flight land before shared memory goes
  tc_fence_before();
  cluster_sync();  // the peer's arrivals here, and the pair's products on its tensor memory, are over
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <bool BF16>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const CUtensorMap& tm_ckv, const CUtensorMap& tm_uk,
                   const CUtensorMap& tm_uv, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const ExpandParams& p) {
  static DeviceOnce once;
  const cudaError_t e = set_attribute_once(once, reinterpret_cast<const void*>(&mla_expand_kv_kernel<BF16>),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, mla_expand_kv_kernel<BF16>, tm_ckv, tm_uk, tm_uv, tm_k, tm_v, p);
}

}  // namespace

cudaError_t launch_expand_kv(const CUtensorMap& tm_ckv, const CUtensorMap& tm_uk, const CUtensorMap& tm_uv,
                             const CUtensorMap& tm_k, const CUtensorMap& tm_v, const ExpandParams& p, bool bf16,
                             int sms, cudaStream_t stream) {
  // no more pairs than there can be tiles: every request may add a block that is not full
  const int64_t tiles = (static_cast<int64_t>(p.max_tokens) / kBlock + p.B) * tiles_per_block(p.H);
  const int64_t pairs = sms / 2 < tiles ? sms / 2 : tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (pairs > 0 ? pairs : 1)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return bf16 ? launch<true>(cfg, tm_ckv, tm_uk, tm_uv, tm_k, tm_v, p) : launch<false>(cfg, tm_ckv, tm_uk, tm_uv, tm_k, tm_v, p);
}

cudaError_t expand_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
