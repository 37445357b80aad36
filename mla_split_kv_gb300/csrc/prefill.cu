// Attention of prompts over expanded keys and values (128 + 64 key columns, 128 value columns a head), sm_103a.
//
// For row i of request b's n newest tokens (position L - n + i of its L tokens) and head h:
//   s_t = scale (q_nope . k_nope[t, h] + q_pe . k_pe[t]),   t <= L - n + i when causal
//   out = sum_t softmax(s)_t v[t, h],   lse = log2 sum_t exp(s_t)
// 640 operations per (row, token, head) against a few bytes: tensor-core bound but for the shortest calls.
//
// A CTA takes 256 rows of a request and a head as two subtiles of 128 (the MMA's M) and walks over the tokens in tiles
// of 128, reading each tile once for both. Tensor memory (512 columns) holds per subtile the scores S [128 x 128] fp32,
// which the probabilities P overwrite in 16 bits as the A operand of the value product, and O [128 x 128]. The
// subtiles alternate: while one's scores are exponentiated, the other's products run,
//   PV0(i) S0(i+1) PV1(i) S1(i+1) ...,
// so a subtile's softmax has the other's 1280 cycles of products to hide behind. The products of one thread execute in
// the order of issue, so S(i+1) may follow PV(i) over the same columns without a wait. P is handed over in halves of 64
// tokens: the value product starts on the first while the second is exponentiated.
//
// Two subtiles' tile is 2600 cycles of products and 2690 of shared memory (operands 2050, refills 640), and takes 3200 to
// 3500: 8192 causal rows, 64 heads, bf16, 912 to 980 us, 1400 to 1500 TFLOP/s at the GPU's power limit (1.65 GHz).
// Slower: score and value products from a warp each (925 to 1130 us), two threads a row (1165), the first half of a
// tile weighed beside the search for its maximum (1014), keys and values asked into L2 ahead (1000).
//
// Shared memory: both subtiles' queries (96 KB) and a ring of eight 16 KB chunks [128 x 64 columns] (keys: two of 64
// columns without rotation, one of rotary columns) or [64 tokens x 128 columns] (values: two a tile), five a tile,
// each with barriers of its own, so that a chunk is refilled as soon as its last product is done. A tile's keys and
// values together are 80 KB: two whole ones would not fit beside the queries, eight chunks are 1.6.
//
// The running maximum is moved only when a tile's maximum passes it by more than 2^15, the room that fp16 has for weights
// above 1 (more, in bf16, is no faster), so O is hardly ever rescaled; the sums are those of the unrounded weights in fp32.
// P is rounded once to 16 bits (by half a step, 2^-8 of itself in bf16, 2^-11 in fp16, as the output is).
//
// What lies in a tile behind a row's last visible token counts for nothing, infinities and NaN included: its weight is
// an exact 0, and where a tile has tokens that some row of the subtile does not see, its values are searched for
// numbers that are not finite, which are set to 0 in shared memory; if one of them belongs to a token that other rows
// do see, those rows take it from the values themselves at the end.
//
// Units (256 rows, head, run of tiles) go to the CTAs longest first, in turns. Where there are too few of them for the
// GPU, long runs are cut into pieces whose normalized outputs and LSE are merged by a kernel of their own
// (mla_prefill_merge_kernel). The list comes from a kernel before this one (mla_prefill_plan_kernel), or, in small
// calls, from this one's start.
//
// A unit of up to 128 rows uses the first subtile alone, and its queries are loaded once the unit before is through its last
// score product, so that short units follow each other at a load's latency and a softmax each: 16 prompts of 30 rows, 128
// heads, 14 units a CTA, 74 us for 10 us of bytes.
//
// Warps: 0-3 and 4-7 softmax and output of the two subtiles (thread = row), 8 products, 9 loads.
#include "block_scan.cuh"
#include "device_common.cuh"
#include "umma_issue.cuh"

namespace mla {

namespace {

constexpr int kTile = 128;                 // tokens a tile
constexpr int kSub = 128;                  // rows a subtile
constexpr int kUnitRows = 2 * kSub;
constexpr int kDim = 128;                  // key columns without rotation, and value columns
constexpr int kChunk = 16384;
constexpr int kRing = 8;
constexpr int kTileChunks = 5;             // keys 0, 1, rotary, values 0, 1
constexpr int kQBytes = 3 * kChunk;        // of a subtile
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 12 * 32;          // (the last two warps only make the third warpgroup whole)
// Registers: launched with 168 a thread (64,512 in all); the softmax warps take 224, the third warpgroup keeps 56.
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= 168 * kThreads, "what the block was launched with");
constexpr int kDirect = 64;                // items of a call that plans for itself
constexpr int kDirectCost = 36;            // half tiles of its longest
constexpr uint32_t kOffRing = 2 * kQBytes;
constexpr uint32_t kOffSmall = kOffRing + kRing * kChunk;
constexpr uint32_t kSmem = kOffSmall + 2048 + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // + 128 * subtile

struct Small {
  uint64_t k_full[2], v_full[2], empty[kRing], q_full[2], q_empty[2], s_full[2], p_full[2][2], pv_done[2], drain;
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t items;
  int32_t dirty[8];  // by unit of this CTA: 1 + the unit in which a value that is not finite was taken out
  int4 list[kDirect];
};
static_assert(sizeof(Small) <= 2048, "small smem region");

// A run of tiles [j0, j1) of the 256 rows from q0 on of request b; slot >= 0: a piece, whose result goes there.
struct Item {
  int32_t b, q0, j0, j1, slot, pad[3];
};

struct Unit {
  int h, q0, j0, slot;
  int n, L;              // the request's rows and tokens
  int qrow, kvrow;       // its first row and token in the packed tensors
  int tiles[2], rows[2]; // of the subtiles
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// the largest of three (NaN passed over)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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
__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

// A request's rows and tokens in the packed tensors, within them.
struct Request {
  int qrow, n, kvrow, L;
};
__device__ __forceinline__ Request request_of(const PrefillParams& p, int b) {
  const int q0 = p.q_indptr[b], q1 = min(p.q_indptr[b + 1], p.T), k0 = p.kv_indptr[b], k1 = min(p.kv_indptr[b + 1], p.S);
  Request r;
  r.qrow = q0;
  r.n = q0 < 0 || q1 <= q0 ? 0 : q1 - q0;
  r.kvrow = k0;
  r.L = k0 < 0 || k1 <= k0 ? 0 : k1 - k0;
  return r;
}
__device__ __forceinline__ bool request_bad(const PrefillParams& p, int b) {
  return p.q_indptr[b] < 0 || p.q_indptr[b + 1] < p.q_indptr[b] || p.q_indptr[b + 1] > p.T || p.kv_indptr[b] < 0 ||
         p.kv_indptr[b + 1] < p.kv_indptr[b] || p.kv_indptr[b + 1] > p.S;
}
// Tokens that row i of a request sees.
__device__ __forceinline__ int visible(const PrefillParams& p, int n, int L, int i) {
  return p.causal ? max(0, min(L, L - n + i + 1)) : L;
}
// Tiles that the rows [q0, q0 + rows) see.
__device__ __forceinline__ int tiles_of(const PrefillParams& p, int n, int L, int q0, int rows) {
  return rows > 0 ? (visible(p, n, L, q0 + rows - 1) + kTile - 1) / kTile : 0;
}
__device__ __forceinline__ int item_tiles(const PrefillParams& p, const Request& r, int q0) {
  return tiles_of(p, r.n, r.L, q0, min(r.n - q0, kUnitRows));
}

// (A Unit stays in registers: nothing takes its address or indexes it by a variable. Local memory is behind L2 here.)
__device__ __forceinline__ Unit unit_of(const PrefillParams& p, const Small* sm, int u) {
  Unit w;
  Item it;
  const int at = u / p.H;
  if (p.items != nullptr) {
    const int4 x = reinterpret_cast<const int4*>(p.items)[2 * at];  // (no __ldg: the list may be written while this kernel waits)
    it.b = x.x;
    it.q0 = x.y;
    it.j0 = x.z;
    it.j1 = x.w;
    it.slot = p.items[8 * at + 4];
  } else {
    const int4 x = sm->list[at];
    it.b = x.x;
    it.q0 = x.y;
    it.j0 = 0;
    it.j1 = x.z;
    it.slot = -1;
  }
  w.h = u % p.H;
  w.rows[0] = w.rows[1] = w.tiles[0] = w.tiles[1] = 0;
  w.q0 = w.j0 = w.n = w.L = w.qrow = w.kvrow = 0;
  w.slot = -1;
  if (it.b < 0) return w;
  const Request r = request_of(p, it.b);
  w.q0 = it.q0;
  w.j0 = it.j0;
  w.slot = it.slot;
  w.n = r.n;
  w.L = r.L;
  w.qrow = r.qrow;
  w.kvrow = r.kvrow;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    w.rows[s] = max(0, min(kSub, r.n - it.q0 - s * kSub));
    w.tiles[s] = max(0, min(it.j1, tiles_of(p, r.n, r.L, it.q0 + s * kSub, w.rows[s])) - it.j0);
  }
  return w;
}
// The k-th unit of this CTA: in turns, every second one backwards, so that what is left over evens out.
__device__ __forceinline__ int unit_index(int k) {
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  return k * g + ((k & 1) ? g - 1 - c : c);
}

// Values that are not finite in the tile at chunks c0, c1 (two of 64 tokens x 128 columns, each as two swizzled
// [64 x 64] boxes) become 0; *dirty = mark first, where one of them belongs to a token before `seen`.
template <bool BF16>
__device__ __forceinline__ void clean_values(uint8_t* c0, uint8_t* c1, int tok0, int seen, int r, volatile int32_t* dirty, int mark) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll 4
  for (int it = 0; it < 16; ++it) {
    const int idx = it * kSub + r;  // 16-byte pieces, 1024 a chunk
    uint8_t* const at = (idx >= 1024 ? c1 : c0) + (idx & 1023) * 16;
    const uint4 v = lds128(smem_u32(at));
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
      const int tok = tok0 + ((idx >= 1024) ? 64 : 0) + ((idx & 511) >> 3);
      if (tok < seen) {
        *dirty = mark;
        __threadfence_block();
      }
      sts128(smem_u32(at), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qpe,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kpe,
                       const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = align1024(smem_raw);
  Small* const sm = reinterpret_cast<Small*>(smem + kOffSmall);
  volatile int32_t* const abort_flag = &sm->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&sm->empty[s], 1);
      sm->dirty[s] = 0;
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm->k_full[s], 3);  // one arrival a chunk
      mbar_init(&sm->v_full[s], 2);
      mbar_init(&sm->q_full[s], 1);
      mbar_init(&sm->q_empty[s], 1);
      mbar_init(&sm->s_full[s], 1);
      mbar_init(&sm->p_full[s][0], 4);
      mbar_init(&sm->p_full[s][1], 4);
      mbar_init(&sm->pv_done[s], 1);
    }
    mbar_init(&sm->drain, 1);
    sm->abort_flag = 0;
    sm->items = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sm->tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.items == nullptr) {
    // at most kDirect items: laid out in the requests' order, then ranked by length
    if (warp == 0) {
      int at = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        Request r{0, 0, 0, 0};
        if (b < p.B) {
          r = request_of(p, b);
          if (blockIdx.x == 0 && request_bad(p, b)) flag_error(MLA_DEVERR_BAD_PAGE);
        }
        const int mine = (r.n + kUnitRows - 1) / kUnitRows;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += y;
        }
        for (int j = 0; j < mine; ++j) {
          const int i = at + upto - mine + j;
          if (i < kDirect) sm->list[i] = make_int4(b, j * kUnitRows, item_tiles(p, r, j * kUnitRows), 0);
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
      }
      __syncwarp();
      const int n = min(at, kDirect);
      int4 own[2];
      int rank[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        rank[k] = -1;
        if (i < n) {
          own[k] = sm->list[i];
          rank[k] = 0;
          for (int j = 0; j < n; ++j) {
            const int c = sm->list[j].z;
            rank[k] += c > own[k].z || (c == own[k].z && j < i);
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (rank[k] >= 0) sm->list[rank[k]] = own[k];
      if (lane == 0) sm->items = n;
    }
    __syncthreads();
  }
  const uint32_t tmem = sm->tmem_base;
  const uint64_t tmo = p.timeout_ns;
  const int units = (p.items != nullptr ? *p.num_items : sm->items) * p.H;

  if (warp == kLoadWarp) {
    // ---------------------------------------------------------------- loads
    fewer_registers();
    if (lane == 0) {
      uint32_t c = 0, tile = 0, used[2] = {0, 0};
      bool ok = true;
      auto chunk = [&](uint64_t* bar) -> uint8_t* {  // the next chunk of the ring, free and armed
        const int s = c % kRing;
        if (c >= kRing && !mbar_wait(&sm->empty[s], (c / kRing - 1) & 1, tmo)) ok = false;
        if (!ok) return nullptr;
        mbar_arrive_expect_tx(bar, kChunk);
        return smem + kOffRing + s * kChunk;
      };
      for (int k = 0; ok; ++k) {
        const int u = unit_index(k);
        if (u >= units) {
          if (k * static_cast<int>(gridDim.x) >= units) break;
          continue;
        }
        const Unit w = unit_of(p, sm, u);
        const int nt = max(w.tiles[0], w.tiles[1]);
        auto queries = [&](int s) {
          if (w.tiles[s] == 0 || !ok) return;
          if (used[s] > 0 && !mbar_wait(&sm->q_empty[s], (used[s] - 1) & 1, tmo)) {
            ok = false;
            return;
          }
          ++used[s];
          uint8_t* const at = smem + s * kQBytes;
          const int row = w.qrow + w.q0 + s * kSub;
          mbar_arrive_expect_tx(&sm->q_full[s], kQBytes);
          tma_load_3d(at, &tm_q, 0, w.h, row, &sm->q_full[s]);
          tma_load_3d(at + kChunk, &tm_q, 64, w.h, row, &sm->q_full[s]);
          tma_load_3d(at + 2 * kChunk, &tm_qpe, 0, w.h, row, &sm->q_full[s]);
        };
        for (int i = 0; i < nt && ok; ++i, ++tile) {
          const int tok = w.kvrow + (w.j0 + i) * kTile;
          if (i == 0) queries(0);
          for (int x = 0; x < kTileChunks && ok; ++x, ++c) {
            uint64_t* const bar = x < 3 ? &sm->k_full[tile & 1] : &sm->v_full[tile & 1];
            uint8_t* const at = chunk(bar);
            if (at == nullptr) break;
            if (x < 2) {
              tma_load_3d(at, &tm_k, 64 * x, w.h, tok, bar);
            } else if (x == 2) {
              tma_load_rows(at, &tm_kpe, 0, tok, bar);
              if (i == 0) queries(1);
            } else {
              tma_load_3d(at, &tm_v, 0, w.h, tok + 64 * (x - 3), bar);
              tma_load_3d(at + kChunk / 2, &tm_v, 64, w.h, tok + 64 * (x - 3), bar);
            }
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    // The whole warp runs this; one lane's instructions count (umma_issue.cuh).
    fewer_registers();
    const uint32_t leader = elect_one();
    const uint32_t idesc_s = idesc_f16_f32(kSub, kTile, BF16, false, false) | (p.negate ? 1u << 13 : 0u);
    const uint32_t idesc_o = idesc_f16_f32(kSub, kDim, BF16, false, true);
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + kOffRing), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + kOffRing), kChunk / 2, 1024);
    uint32_t tile0 = 0;                       // tiles before this unit
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};  // units and tiles of each subtile so far
    bool ok = true;
    int tiles0 = 0, tiles1 = 0;  // of the unit
    auto scores = [&](int s, int i) {  // S of tile i; the first of the subtiles waits for the keys
      const uint32_t x = kTileChunks * (tile0 + i), t = tile0 + i;
      const bool last = s == 1 || i >= tiles1, first = s == 0 || i >= tiles0;
      if (first) ok = ok && mbar_wait_warp(&sm->k_full[t & 1], (t >> 1) & 1, tmo);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int y = 0; y < 3; ++y) {
        const uint32_t slot = (x + y) % kRing;
        const uint64_t a = q_desc + ((s * kQBytes + y * kChunk) >> 4), b = k_desc + ((slot * kChunk) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          issue_ss(leader, tmem + kTmemS + s * kTile, a + 2 * kk, b + 2 * kk, idesc_s, y > 0 || kk > 0);
        if (last && y < 2) issue_commit(leader, &sm->empty[slot]);
      }
      issue_commit(leader, &sm->s_full[s]);
      if (last) issue_commit(leader, &sm->empty[(x + 2) % kRing]);
      if (i + 1 == (s == 0 ? tiles0 : tiles1)) issue_commit(leader, &sm->q_empty[s]);
    };
    auto values = [&](int s, int i) {
      const uint32_t x = kTileChunks * (tile0 + i) + 3, t = tile0 + i;
      const bool last = s == 1 || i >= tiles1, first = s == 0 || i >= tiles0;
      if (first) ok = ok && mbar_wait_warp(&sm->v_full[t & 1], (t >> 1) & 1, tmo);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        ok = ok && mbar_wait_warp(&sm->p_full[s][y], pn[s] & 1, tmo);
        if (!ok) return;
        tc_fence_after();
        const uint32_t slot = (x + y) % kRing;
        const uint64_t b = v_desc + ((slot * kChunk) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          issue_ts(leader, tmem + kTmemO + s * kDim, tmem + kTmemS + s * kTile + 32 * y + 8 * kk, b + 128 * kk, idesc_o,
                   i > 0 || y > 0 || kk > 0);
        if (last && y == 0) issue_commit(leader, &sm->empty[slot]);
      }
      issue_commit(leader, &sm->pv_done[s]);
      if (last) issue_commit(leader, &sm->empty[(x + 1) % kRing]);
      ++pn[s];
    };
    for (int k = 0; ok; ++k) {
      const int u = unit_index(k);
      if (u >= units) {
        if (k * static_cast<int>(gridDim.x) >= units) break;
        continue;
      }
      const Unit w = unit_of(p, sm, u);
      tiles0 = w.tiles[0];
      tiles1 = w.tiles[1];
      const int nt = max(tiles0, tiles1);
      if (nt == 0) continue;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if ((s == 0 ? tiles0 : tiles1) == 0 || !ok) continue;
        ok = mbar_wait_warp(&sm->q_full[s], qn[s] & 1, tmo);
        ++qn[s];
        if (ok) scores(s, 0);
      }
      for (int i = 0; i < nt && ok; ++i) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (i >= (s == 0 ? tiles0 : tiles1) || !ok) continue;
          values(s, i);
          if (ok && i + 1 < (s == 0 ? tiles0 : tiles1)) scores(s, i + 1);
        }
      }
      tile0 += nt;
    }
    if (!ok) *abort_flag = 1;
    // every product issued so far is done before tensor memory is freed
    __syncwarp();
    issue_commit(leader, &sm->drain);
    mbar_wait(&sm->drain, 0, kDrainTimeoutNs);
    __syncwarp();
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- softmax, output: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2, r = tid & (kSub - 1);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + kTmemS + s * kTile, to = tmem + lanes + kTmemO + s * kDim;
    const float scale = p.scale_log2;
    constexpr float kSlack = 15.f;
    uint32_t done = 0;   // tiles of this subtile so far
    uint32_t tile0 = 0;  // tiles of all units before this one
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int u = unit_index(k);
      if (u >= units) {
        if (k * static_cast<int>(gridDim.x) >= units) break;
        continue;
      }
      const Unit w = unit_of(p, sm, u);
      const int nt = s == 0 ? w.tiles[0] : w.tiles[1], rows = s == 0 ? w.rows[0] : w.rows[1], q0 = w.q0 + s * kSub;
      if (rows > 0) {
        const int seen = visible(p, w.n, w.L, q0 + min(r, rows - 1));  // tokens that this row sees
        const int all = visible(p, w.n, w.L, q0);                      // that every row of the subtile sees
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < nt; ++i, ++done) {
          const int tok0 = (w.j0 + i) * kTile;
          ok = mbar_wait_warp(&sm->s_full[s], done & 1, tmo);
          if (!ok) break;
          tc_fence_after();
          float x[kTile];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, x + 32 * q);
          tmem_wait_ld();
          float f = scale;
          const bool masked = tok0 + kTile > all;
          if (masked) {
            const int nvis = seen - tok0;
#pragma unroll
            for (int t = 0; t < kTile; ++t) x[t] = t < nvis ? x[t] * scale : -INFINITY;
            f = 1.f;
          }
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int t = 4; t < kTile - 4; t += 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m4[j] = max3(m4[j], x[t + j], x[t + 4 + j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], x[kTile - 4 + j]);
          const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * f;
          const bool need = mx > m + kSlack;
          if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
            const float m_new = need ? mx : m;
            const float alpha = need ? (m == -INFINITY ? 0.f : exp2f(m - m_new)) : 1.f;
            if (i > 0) {
              ok = mbar_wait_warp(&sm->pv_done[s], (done - 1) & 1, tmo);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                float o[32];
                tmem_ld32(to + 32 * q, o);
                tmem_wait_ld();
                uint32_t b[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) b[j] = __float_as_uint(o[j] * alpha);
                tmem_st32(to + 32 * q, b);
              }
              tmem_wait_st();
            }
            l *= alpha;
            m = m_new;
          }
          if (masked) {
            const uint32_t t = tile0 + i, c = kTileChunks * t + 3;
            ok = mbar_wait_warp(&sm->v_full[t & 1], (t >> 1) & 1, tmo);
            if (!ok) break;
            clean_values<BF16>(smem + kOffRing + (c % kRing) * kChunk, smem + kOffRing + ((c + 1) % kRing) * kChunk, tok0, w.L, r,
                               &sm->dirty[k & 7], k + 1);
            fence_proxy_async_smem();  // (the product waits for all four warps' weights, so for all of the search)
          }
          const float mm = m == -INFINITY ? 0.f : -m;
          const float2 f2 = make_float2(f, f), m2 = make_float2(mm, mm);
          float2 sum = make_float2(0.f, 0.f), sum_b = sum;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t b[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int t = 64 * half + 2 * j;
              float2 e = fma2(make_float2(x[t], x[t + 1]), f2, m2);
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              if (j & 1) sum_b = add2(sum_b, e);
              else sum = add2(sum, e);
              b[j] = pack2<BF16>(e.x, e.y);
            }
            tmem_st32(ts + 32 * half, b);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->p_full[s][half]);
          }
          sum = add2(sum, sum_b);
          l += sum.x + sum.y;
        }
        if (!ok) break;
        if (nt > 0) {
          ok = mbar_wait_warp(&sm->pv_done[s], (done - 1) & 1, tmo);
          if (!ok) break;
          tc_fence_after();
        }
        const bool any = nt > 0 && m != -INFINITY;
        const float inv = any ? 1.f / l : 0.f;
        const float lse = any ? m + log2f(l) : (l != l ? l : -INFINITY);  // (every score NaN: no maximum)
        // (a piece without a score above -inf counts with weight 0 in the merge, and its infinite values are NaN there)
        const bool counts = any || (nt > 0 && w.slot >= 0);
        // (a later unit's mark, from a subtile that is eight units ahead, may lie over this one's: looked for in vain at worst)
        const bool dirty = counts && *const_cast<volatile int32_t*>(&sm->dirty[k & 7]) > k;
        // the tiles that were searched, of either subtile, as far as this row sees
        const int first = max(w.j0 * kTile, visible(p, w.n, w.L, w.q0) / kTile * kTile);
        const int last = min(seen, (w.j0 + nt) * kTile);
        const long long row = static_cast<long long>(w.qrow) + q0 + r;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float o[32];
          if (nt > 0) {
            tmem_ld32(to + 32 * q, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = counts ? o[j] * inv : (l != l ? l : 0.f);
          if (__builtin_expect(dirty, 0)) {
            // values that are not finite were taken out of the searched tiles: those that this row sees belong to its sum
            // (weights are positive; infinities of both signs, or a NaN, give NaN)
            constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll 1
            for (int t = first; t < last; ++t) {
              const uint16_t* const v = p.v + (static_cast<long long>(w.kvrow + t) * p.H + w.h) * kDim + 32 * q;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if ((v[j] & kExp) == kExp) o[j] += h2f<BF16>(v[j]);
            }
          }
          if (r < rows) {
            if (w.slot < 0) {
              uint32_t b[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) b[j] = pack2<BF16>(o[2 * j], o[2 * j + 1]);
              uint16_t* const at = static_cast<uint16_t*>(p.out) + (row * p.H + w.h) * kDim + 32 * q;
              store32(at, b);
              store32(at + 16, b + 8);
            } else {
              uint32_t b[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) b[j] = __float_as_uint(o[j]);
              float* const at = p.part_o + ((static_cast<long long>(w.slot) * kUnitRows + s * kSub + r) * p.H + w.h) * kDim + 32 * q;
#pragma unroll
              for (int j = 0; j < 4; ++j) store32(at + 8 * j, b + 8 * j);
            }
          }
        }
        tc_fence_before();
        if (r < rows) {
          if (w.slot >= 0) p.part_lse[(static_cast<long long>(w.slot) * kUnitRows + s * kSub + r) * p.H + w.h] = lse;
          else if (p.out_lse != nullptr) p.out_lse[row * p.H + w.h] = lse;
        }
      }
      tile0 += max(w.tiles[0], w.tiles[1]);
    }
    if (!ok) *abort_flag = 1;
  } else {
    fewer_registers();
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) settle_in_flight(3000000ull);  // copies in flight land before shared memory goes
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The list of units' runs of tiles, longest first (by counting, 256 steps of length): one CTA.
constexpr int kPlanThreads = 1024;
constexpr int kSteps = 256;
constexpr int kLeastPiece = 12;  // half tiles (of 128 rows): a piece's start and its share of the merge cost about two
constexpr int kFewRuns = 2048;

// Tiles a piece of a run of so many tiles: even ones, of no more than the target's cost as far as tiles are whole.
__device__ __forceinline__ int piece_length(int cost, int tiles, int target) {
  const int pieces = (cost + target - 1) / target;
  return max(1, (tiles + pieces - 1) / pieces);
}

__global__ void __launch_bounds__(kPlanThreads, 1) mla_prefill_plan_kernel(const PrefillParams p, const PrefillPlanParams pl) {
  extern __shared__ int32_t tile_at[];  // [B + 1]
  __shared__ long long part[32];
  __shared__ unsigned long long sum_cost;
  __shared__ int longest, slots, merges, hist[kSteps], cursor[kSteps], aims[32];
  __shared__ int2 runs[kFewRuns];  // cost, tiles
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) {
    sum_cost = 0;
    longest = 1;
    slots = merges = 0;
  }
  if (tid < kSteps) hist[tid] = 0;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0, all;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    mine += (request_of(p, b).n + kUnitRows - 1) / kUnitRows;
    bad |= request_bad(p, b);
  }
  if (bad) flag_error(MLA_DEVERR_BAD_PAGE);
  long long at = block_scan(mine, part, &all);
  for (int b = b0; b < b1; ++b) {
    tile_at[b] = static_cast<int>(min(at, 0x7fffffffll));
    at += (request_of(p, b).n + kUnitRows - 1) / kUnitRows;
  }
  __syncthreads();
  const int n = static_cast<int>(min(all, static_cast<long long>(pl.max_tiles)));  // (more: offsets that overlap)
  // a run's cost in half tiles
  auto cost_of = [&](int i, int* b, int* q0, int* tiles) {
    *b = find_last(tile_at, 0, p.B - 1, i);
    const Request r = request_of(p, *b);
    *q0 = (i - tile_at[*b]) * kUnitRows;
    *tiles = item_tiles(p, r, *q0);
    return *tiles * (r.n - *q0 > kSub ? 2 : 1) + 2;
  };
  int b, q0, tiles;
  unsigned long long cost = 0;
  int most = 0;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int c = cost_of(i, &b, &q0, &tiles);
    if (n <= kFewRuns) runs[i] = make_int2(c, tiles);
    cost += c;
    most = max(most, c);
  }
  atomicAdd(&sum_cost, cost);
  atomicMax(&longest, most);
  __syncthreads();
  // How runs are cut: each into as many pieces as its cost holds targets. With few enough runs a warp a candidate: the
  // longest into 1 to 16 pieces, or all into as many as fill 1 to 16 rounds of the GPU's CTAs. A CTA's time is the average,
  // or more where the units at least as long as x take whole rounds of x; merging a piece costs about a twelfth of a half
  // tile, and the first one six. (With the average and the longest unit for the time, 4000 causal rows of 16 heads were cut
  // in two and took 116 us; whole, 77.)
  // (1000 and 670 rows behind 29,192 and 31,316 tokens, 16 heads: 112 units as long as 492 half tiles into 448, three rounds
  // of 152, 396 us; into pieces of a quarter of a CTA's share, 672 of them, 442 us.)
  if (n <= kFewRuns) {
    const int k = tid >> 5, lane = tid & 31;
    const long long r = static_cast<long long>(k - 15) * pl.sms / max(1ll, static_cast<long long>(n) * p.H);
    const int wanted = static_cast<int>(k < 16 ? k + 1 : max(1ll, min(r, 1ll << 20)));
    const int aim = max(1, (longest + wanted - 1) / wanted);
    int parts = 0, most_of = 0;
    long long sum = 0;
    for (int i = lane; i < n; i += 32) {
      const int2 run = runs[i];
      const int len = piece_length(run.x, run.y, aim), count = max(1, (run.y + len - 1) / len);
      parts += count > 1 ? count : 0;
      sum += run.x + 2 * (count - 1);
      most_of = max(most_of, (run.x - 2) / max(1, run.y) * min(len, run.y) + 2);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    parts = __reduce_add_sync(0xffffffffu, parts);
    most_of = __reduce_max_sync(0xffffffffu, most_of);
    int at_least[8] = {};  // units of no less than an eighth, two, ... of the longest
    for (int i = lane; i < n; i += 32) {
      const int2 run = runs[i];
      const int len = piece_length(run.x, run.y, aim), count = max(1, (run.y + len - 1) / len), each = (run.x - 2) / max(1, run.y);
      const int full = each * len + 2, rest = each * (run.y - (count - 1) * len) + 2;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        at_least[j] += (8 * full >= (j + 1) * most_of ? count - 1 : 0) + (8 * rest >= (j + 1) * most_of ? 1 : 0);
    }
    int units = 0;  // lane j: of the j-th kind
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int all = __reduce_add_sync(0xffffffffu, at_least[j]);
      if (lane == j) units = all;
    }
    // (a way that is weighed has at most 16 pieces a run, or 16 rounds of them: 31 bits hold units times heads)
    const unsigned rounds = (static_cast<unsigned>(units) * p.H + pl.sms - 1) / static_cast<unsigned>(pl.sms);
    const long long whole = static_cast<long long>(rounds) * (static_cast<long long>(lane + 1) * most_of / 8);
    long long time = max(sum * p.H / pl.sms, static_cast<long long>(__reduce_max_sync(0xffffffffu, static_cast<int>(min(whole, 0x7fffffffll)))));
    if (parts > 0) time += static_cast<long long>(parts) * p.H / 12 + 6;
    const bool fits = k == 0 || (aim >= kLeastPiece && parts <= pl.max_slots);
    if (lane == 0) {
      part[k] = fits ? time : 0x7fffffffffffffffll;
      aims[k] = aim;
    }
    __syncthreads();
  }
  int target;
  bool slack = false;
  if (n <= kFewRuns) {
    long long time = part[tid & 31];
    int best = tid & 31;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      const long long time_of = __shfl_xor_sync(0xffffffffu, time, d);
      const int other = __shfl_xor_sync(0xffffffffu, best, d);
      if (time_of < time || (time_of == time && other < best)) {
        time = time_of;
        best = other;
      }
    }
    target = aims[best];
  } else {  // four units a CTA, if that takes cutting
    const long long fair = static_cast<long long>((sum_cost * p.H + 4 * pl.sms - 1) / (4 * pl.sms));
    target = static_cast<int>(max(static_cast<long long>(kLeastPiece), min(fair, 0x3fffffffll)));
    slack = true;
  }
  auto pieces_of = [&](int c, int tiles) {  // tiles a piece
    return slack && 2ll * c <= 3ll * target ? max(1, tiles) : piece_length(c, tiles, target);
  };
  const int top = longest;
  auto step_of = [&](int c, int tiles, int len) {
    const long long each = static_cast<long long>(c) * len / max(1, tiles);
    return static_cast<int>(kSteps - 1 - min(static_cast<long long>(kSteps - 1), each * (kSteps - 1) / top));
  };
  for (int i = tid; i < n; i += kPlanThreads) {
    const int c = cost_of(i, &b, &q0, &tiles);
    const int len = pieces_of(c, tiles);
    atomicAdd(&hist[step_of(c, tiles, len)], max(1, (tiles + len - 1) / len));
  }
  __syncthreads();
  if (tid < 32) {
    int before = 0;
    for (int k = tid; k < kSteps; k += 32) {
      const int v = hist[k];
      int x = v;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (tid >= d) x += y;
      }
      cursor[k] = before + x - v;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (tid == 0) *pl.num_items = min(before, pl.max_items);
  }
  __syncthreads();
  int4* const items = reinterpret_cast<int4*>(pl.items);
  for (int i = tid; i < n; i += kPlanThreads) {
    const int c = cost_of(i, &b, &q0, &tiles);
    int len = pieces_of(c, tiles);
    const int count = max(1, (tiles + len - 1) / len);
    const int to = atomicAdd(&cursor[step_of(c, tiles, len)], count);
    int slot = -1;
    if (count > 1) {
      slot = atomicAdd(&slots, count);
      if (slot + count > pl.max_slots) {  // (does not happen: max_slots is what the rule above can give)
        slot = -1;
        len = tiles;
      } else {
        const Request r = request_of(p, b);
        pl.merge[atomicAdd(&merges, 1)] = make_int4(r.qrow + q0, min(kUnitRows, r.n - q0), slot, count);
      }
    }
    for (int j = 0; j < count; ++j) {
      if (to + j >= pl.max_items) break;
      const bool real = slot >= 0 || j == 0;
      items[2 * (to + j)] = make_int4(real ? b : -1, q0, j * len, min(tiles, (j + 1) * len));
      items[2 * (to + j) + 1] = make_int4(slot >= 0 ? slot + j : -1, 0, 0, 0);
    }
  }
  __syncthreads();
  if (tid == 0) *pl.num_merges = merges;
}

// Cut runs: a warp a (row, head), the pieces in order, M = max lse, weights 2^(lse - M).
constexpr int kMergeThreads = 256;
constexpr int kMergeDepth = 8;  // pieces in flight
__global__ void __launch_bounds__(kMergeThreads, 3) mla_prefill_merge_kernel(const PrefillParams p, const PrefillPlanParams pl, int bf16) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long total = static_cast<long long>(*pl.num_merges) * kUnitRows * p.H;
  const long long warps = static_cast<long long>(gridDim.x) * (kMergeThreads / 32);
  for (long long i = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5); i < total; i += warps) {
    const int h = static_cast<int>(i % p.H), r = static_cast<int>(i / p.H % kUnitRows);
    const int4 e = pl.merge[i / p.H / kUnitRows];
    if (r >= e.y) continue;
    const long long first = (static_cast<long long>(e.z) * kUnitRows + r) * p.H + h, stride = static_cast<long long>(kUnitRows) * p.H;
    // a group of pieces' values and, in as many lanes, their LSE; the first on its way while the maximum is found
    float lse;
    float4 v[kMergeDepth];
    auto load = [&](int j0) {
      lse = lane < kMergeDepth && j0 + lane < e.w ? p.part_lse[first + (j0 + lane) * stride] : -INFINITY;
#pragma unroll
      for (int j = 0; j < kMergeDepth; ++j)
        v[j] = j0 + j < e.w ? reinterpret_cast<const float4*>(p.part_o + (first + (j0 + j) * stride) * kDim)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float M = lse;
    for (int j = kMergeDepth + lane; j < e.w; j += 32) M = max_nan(M, p.part_lse[first + j * stride]);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, d));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    if (M != -INFINITY) {
      for (int j0 = 0; j0 < e.w; j0 += kMergeDepth) {
        if (j0 > 0) load(j0);
        const float w = lse == -INFINITY ? 0.f : exp2f(lse - M);
#pragma unroll
        for (int j = 0; j < kMergeDepth; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, j);
          den += wj;
          acc.x = fmaf(wj, v[j].x, acc.x);
          acc.y = fmaf(wj, v[j].y, acc.y);
          acc.z = fmaf(wj, v[j].z, acc.z);
          acc.w = fmaf(wj, v[j].w, acc.w);
        }
      }
      acc = make_float4(acc.x / den, acc.y / den, acc.z / den, acc.w / den);
    }
    const long long row = static_cast<long long>(e.x) + r;
    store_out4(p.out, bf16, (row * p.H + h) * kDim + 4 * lane, acc);
    if (lane == 0 && p.out_lse != nullptr) p.out_lse[row * p.H + h] = merged_lse(M, den);
  }
}

template <class... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                             const Args&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// The pieces of all cut runs together, at most. With many runs: a run is cut where it costs more than 3/2 of the target,
// into no more than cost / target + 1 <= 5/3 cost / target pieces, and the costs of all runs, H times, are at most 4 sms
// targets. With few, ways of cutting that would take more are not taken.
int prefill_max_slots(int H, int sms) { return (4 * sms * 5 / 3) / H + 2; }
int prefill_max_tiles(int B, int T) { return T / kUnitRows + B; }
bool prefill_direct(int B, int T, int S) {
  // planned in the kernel itself: few runs, and none so long that cutting it would save the ten microseconds of the planning
  // kernel and the merge (16 heads, planned here and there: 300 rows 13.0 and 23.8 us, 2000 rows 37.1 and 47.6, 16 rows
  // behind 2100 tokens 31.8 and 41.4, 512 rows 40.5 and 37.6; behind 4000 tokens 53 to 66 and 34 to 43)
  return prefill_max_tiles(B, T) <= kDirect && 2 * ((S + kTile - 1) / kTile) + 2 <= kDirectCost;
}

cudaError_t launch_prefill(const PrefillMaps& maps, const PrefillParams& p, const PrefillPlanParams& pl, bool bf16,
                           int sms, cudaStream_t stream) {
  static DeviceOnce once_plan, once_f16, once_bf16;
  const void* const fn = bf16 ? reinterpret_cast<const void*>(&mla_prefill_kernel<true>)
                              : reinterpret_cast<const void*>(&mla_prefill_kernel<false>);
  cudaError_t e = set_attribute_once(bf16 ? once_bf16 : once_f16, fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  if (p.items != nullptr) {
    e = set_attribute_once(once_plan, reinterpret_cast<const void*>(&mla_prefill_plan_kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (kMaxStepRequests + 1) * 4);
    if (e != cudaSuccess) return e;
    e = launch_dependent(mla_prefill_plan_kernel, 1, kPlanThreads, (p.B + 1) * 4, stream, p, pl);
    if (e != cudaSuccess) return e;
  }
  const int64_t units = (p.items != nullptr ? static_cast<int64_t>(pl.max_items) : prefill_max_tiles(p.B, p.T)) * p.H;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  e = bf16 ? launch_dependent(mla_prefill_kernel<true>, grid, kThreads, kSmem, stream, maps.q, maps.qpe, maps.k, maps.kpe, maps.v, p)
           : launch_dependent(mla_prefill_kernel<false>, grid, kThreads, kSmem, stream, maps.q, maps.qpe, maps.k, maps.kpe, maps.v, p);
  if (e != cudaSuccess || p.items == nullptr) return e;
  return launch_dependent(mla_prefill_merge_kernel, static_cast<unsigned>(4 * sms), kMergeThreads, 0, stream, p, pl, bf16 ? 1 : 0);
}

cudaError_t prefill_read_clear_error(uint32_t* out) { return read_clear_device_error(out); }

}  // namespace mla
