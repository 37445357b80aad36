// Internal interface between the C-ABI layer and the kernels (not installed).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mla {

constexpr int kRank = 512;        // kv_lora_rank: width of ckv
constexpr int kRope = 64;         // rope dim: width of kpe
constexpr int kQkDim = kRank + kRope;
constexpr int kTileTokens = 64;   // tokens per pipeline tile
constexpr int kBoxCols = 64;      // 16-bit columns per TMA box (128 bytes)
constexpr int kBoxesPerTile = kQkDim / kBoxCols;  // 8 ckv boxes + 1 kpe box
constexpr int kBoxBytes = kTileTokens * kBoxCols * 2;  // 8 KB
constexpr int kTileBytes = kBoxesPerTile * kBoxBytes;  // 72 KB

// Device error bits (the per-file g_device_error words).
constexpr uint32_t MLA_DEVERR_TIMEOUT = 1u;
constexpr uint32_t MLA_DEVERR_BAD_PAGE = 2u;
constexpr uint32_t MLA_DEVERR_CONFIG = 4u;  // a kernel found its launch unusable (shared memory alignment)

struct PartialParams {
  const uint16_t* q_abs;       // [B, q_len, H, 512]
  const uint16_t* q_pe;        // [B, q_len, H, 64]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* context_lens; // [B]
  const uint8_t* ckv;          // ckv cache base: page g at g * bs * 1024 bytes
  const uint8_t* kpe;          // kpe cache base: page g at g * bs * 128 bytes
  const void* chunks;          // device int4 {b, t0, t1, slot} per chunk, or null
  float* partials;             // [slots, q_len, H, 512]
  float* lse;                  // [slots, q_len, H]
  float scale_log2;            // softmax scale * log2(e)
  int32_t B, H, q_len, bs, max_blocks, num_blocks;
  int32_t num_parts;           // uniform split when chunks == null
  int32_t causal;
  int32_t tables_ready;        // chunks / context_lens / block_table may be read before the dependency wait
  int32_t fp8;                 // E4M3 caches (the paired kernel): loaded as bytes, converted to fp16 in the slot
  float cache_scale;           // E4M3: the value of byte x is e4m3(x) * cache_scale (folded into scale_log2 and O)
  int32_t prefix_ready;        // cache rows before each request's window may be read before the dependency wait
  int32_t xchg16;              // the 128-row kernel: 1 partial scores cross the pair as fp16, 2 none cross
  uint64_t timeout_ns;
  // a chunk spread over `subs` clusters (the paired 16-row kernel): grid.y = chunks * subs.
  // One entry per CTA pair of a chunk (subs * cluster / 2 of them): its unnormalized O^T in
  // ws_partials and its row maxima / sums in ws_lse; two tickets per chunk (one per column
  // half). Tickets are zero between calls.
  int32_t subs;
  float* ws_partials;          // [entries, q_len, H, 512]
  float* ws_lse;               // [entries, 2, q_len, H, 2]
  uint32_t* ws_tickets;        // [chunks, 2]
  // Single-launch decode (out != null): once a request's chunk partials are written, the CTA
  // that finishes last for a column slice of the request merges that slice of all of them into
  // `out`, with the merge kernel's arithmetic. Tickets: [B][kSliceTickets], zero between calls.
  // lse_copy: [slots, q_len, H], the second column half's copy of each chunk's LSE (spread plans).
  const int32_t* o_indptr;     // [B+1] request-major chunk offsets (device)
  void* out;                   // [B, q_len, H, 512] of out_dtype, or null
  float* out_lse;              // [B, q_len, H], or null
  int32_t out_dtype;           // MLA_F16 / MLA_BF16 / MLA_F32
  uint32_t* req_tickets;
  float* lse_copy;
  // the paired kernel writes every CTA pair's part (unnormalized O^T, row maxima and sums) as an
  // entry of ws_partials / ws_lse and nothing else; the entries merge kernel combines them
  int32_t entries_only;
  // a sliding window beside the first `sinks` tokens (0: none); chunks, lengths and positions are then those
  // of the requests' visible runs (WindowView)
  int32_t window, sinks;
};
constexpr int kSliceTickets = 16;  // per request: one per column slice (cluster rank) or column half

// The merge of the paired kernel's pair entries (entries_only): request b's entries are
// [o_indptr[b] * epc, o_indptr[b+1] * epc), epc = entries per chunk.
struct EntryMergeParams {
  const float* ws_partials;    // [entries, rows, 512] unnormalized O
  const float* ws_lse;         // [entries, 2, rows, 2] row maximum and sum (two equal copies)
  const int32_t* o_indptr;     // [B+1]
  void* out;                   // [B, rows, 512] of out_dtype
  float* out_lse;              // [B, rows] or null
  int32_t B, rows, epc, out_dtype;
  int32_t tables_ready;        // o_indptr complete before the partial kernel started: read before the wait
  int64_t entries;             // of all requests
  int32_t uniform;             // as many in each
  int32_t exact_lse;           // the entries' second copies hold sums of their own, for the LSE
};
cudaError_t launch_merge_entries(const EntryMergeParams& p, cudaStream_t stream);

struct MergeParams {
  const float* partials;
  const float* lse;
  const int32_t* o_indptr;
  void* out;
  float* out_lse;
  int32_t B, rows;  // rows = q_len * H
  int32_t out_dtype;
  int64_t most_parts;  // the most partials that a request can have (0: not known)
};

// The cache write of a layer call: token i of request b's q_len new tokens goes to logical
// position context_lens[b] - q_len + i.
struct AppendParams {
  const uint16_t* ckv_new;     // [B, q_len, 512]
  const uint16_t* kpe_new;     // [B, q_len, 64]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* context_lens; // [B]
  uint16_t* ckv;               // [num_blocks, bs, 512]
  uint16_t* kpe;               // [num_blocks, bs, 64]
  int32_t B, q_len, bs, max_blocks, num_blocks;
};

// Merge of each request's partials, then the unembed W_UV^T of each head.
struct UnembedParams {
  const float* partials;       // [N, q_len, H, 512] normalized O, or [E, q_len, H, 512] pair entries' O
  const float* lse;            // [N, q_len, H] log2 LSE, or [E, 2, q_len, H, 2] entries' (m, l)
  const int32_t* o_indptr;     // [B+1]
  const uint16_t* w_uv_t;      // [H, 512, v_head]
  void* out;                   // [B, q_len, H, v_head] of out_dtype
  float* out_lse;              // [B, q_len, H] or null
  int32_t B, q_len, H, v_head, out_dtype;
  int32_t entries;             // 1: pair entries (epc per chunk), 0: chunk partials (epc 1)
  int32_t epc;
  int32_t tables_ready;        // o_indptr complete before the preceding kernel started: read before the wait
};

// What the rows of a request see of its L tokens through a sliding window beside its first `sinks`
// tokens: the pages of the sinks, then, `skip` tokens further on, the pages from the first token that
// the earliest row's window reaches. The n tokens of both, one after the other, are the request's
// visible run; position u of the run is token u below `sa` and token u + skip from there on, both
// page-aligned. window = 0: the whole request. Whether row i sees position u is, in the run's own
// positions, the rule on tokens: with n for L, u <= n - q_len + i (causal) and (u > pos - window or
// u < sinks), pos the row's own position: `skip` shifts a token and its row alike, and where skip > 0
// every position below sa is below every row's window.
struct WindowView {
  int32_t n, sa, skip;
};
#ifdef __CUDACC__
#define MLA_HOST_DEVICE __host__ __device__
#else
#define MLA_HOST_DEVICE
#endif
MLA_HOST_DEVICE inline WindowView window_view(int32_t L, int32_t q_len, int32_t bs, int32_t causal, int32_t window,
                                              int32_t sinks) {
  WindowView v{L > 0 ? L : 0, 0, 0};
  if (window <= 0 || L <= 0) return v;
  const int64_t first = static_cast<int64_t>(L) - (causal ? q_len : 1);  // the earliest row's position
  const int64_t low = first - window + 1;                                // the first token its window reaches
  if (low <= 0) return v;
  const int64_t page = ~static_cast<int64_t>(bs - 1);  // (bs is a power of two)
  const int64_t low_page = low & page, sink_end = (static_cast<int64_t>(sinks) + bs - 1) & page;
  v.sa = static_cast<int32_t>(sink_end < low_page ? sink_end : low_page);
  v.skip = static_cast<int32_t>(low_page - v.sa);
  v.n = L - v.skip;
  return v;
}

// The last position that the window of the row at position `pos` leaves out (-1: none). A row before the request's
// first token (pos < 0) sees nothing whatever this says.
MLA_HOST_DEVICE inline int32_t window_floor(int32_t pos, int32_t window) {
  const int32_t low = (pos > -1 ? pos : -1) - window;  // (no less than -2^31)
  return low > -1 ? low : -1;
}
// Position of token t of a tile of a run, without a sign: a tile at the end of the longest run passes 2^31.
MLA_HOST_DEVICE inline uint32_t run_position(int32_t tile, int32_t tile_tokens, int32_t t) {
  return static_cast<uint32_t>(tile) * static_cast<uint32_t>(tile_tokens) + static_cast<uint32_t>(t);
}

// Block-scaled 8-bit caches: the value of a cached byte x of token row r is e4m3(x) * scales[r >> g_shift].
struct AppendQ8Params {
  const uint16_t* ckv_new;     // [B, q_len, 512]
  const uint16_t* kpe_new;     // [B, q_len, 64]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* context_lens; // [B]
  uint8_t* ckv;                // [num_blocks, bs, 512]
  uint8_t* kpe;                // [num_blocks, bs, 64]
  float* scales;               // [num_blocks, bs / g]
  int32_t B, q_len, bs, max_blocks, num_blocks, g;
};
cudaError_t launch_append_q8(const AppendQ8Params& p, bool bf16, cudaStream_t stream);
cudaError_t append_q8_read_clear_error(uint32_t* out);

struct DecodeQ8Params {
  const uint16_t* q_abs;       // [B, q_len, H, 512]
  const uint16_t* q_pe;        // [B, q_len, H, 64]
  const uint8_t* ckv;          // [num_blocks, bs, 512]
  const uint8_t* kpe;          // [num_blocks, bs, 64]
  const float* scales;         // [num_blocks, bs >> g_shift]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* context_lens; // [B]
  void* out;                   // [B, q_len, H, 512] of out_dtype
  float* out_lse;              // [B, q_len, H] or null
  float* ws_o;                 // [gangs, 2, row_pad, 512] unnormalized O of a gang's two open ends
  float* ws_ml;                // [gangs, 2, row_pad, 2] their row maxima and sums
  int2* ws_cut;                // by gang, the request that starts there and goes on in others, and its parts (0: none); with
                               // cuts_by_request by request, its first gang and its parts
  float scale_log2;            // softmax scale * log2(e)
  int32_t B, H, h_shift, q_len, bs, bs_shift, max_blocks, num_blocks, g_shift, causal, window, sinks, out_dtype;
  int32_t gangs;               // CTAs that share the tiles of the batch, one per row group each
  int32_t groups, row_pad;     // row groups; rows padded to whole groups
  int32_t cuts_by_request;     // the batch has fewer rows than the grid has CTAs
  uint64_t timeout_ns;
};
// Rows per CTA and gangs of the launch for q_len * H rows on a device of `sms` SMs.
int q8_rows_per_cta(int total_rows);
int q8_gangs(int total_rows, int sms);
// tm_ckv: boxes of one page of the byte cache, [8 rows x 128 columns] swizzled atoms, four column blocks to a
// row group; tm_kpe: boxes of one page's 64 rope columns with the 64-byte swizzle.
cudaError_t launch_decode_q8(const CUtensorMap& tm_ckv, const CUtensorMap& tm_kpe, const DecodeQ8Params& p, bool bf16,
                             cudaStream_t stream);
cudaError_t decode_q8_read_clear_error(uint32_t* out);

// A step's tables from the requests' lengths (mla_update_tables).
constexpr int kMaxStepRequests = 8192;  // MLA_MAX_STEP_REQUESTS
struct TablesParams {
  const int32_t* changes;      // [B]
  const int32_t* lens;         // [B]
  int32_t* lens_out;           // [B], may be lens
  int32_t* block_table;        // [B, max_blocks]
  int32_t* pages;              // [num_blocks], the stack of free ones
  const int32_t* free_count;   // [1]
  int32_t* free_count_out;     // [1], may be free_count
  int32_t* q_indptr;           // [B+1]
  int32_t* kv_indptr;          // [B+1]
  int64_t* slots;              // [capacity]
  int32_t* served;             // [1]
  int32_t B, bs, bs_shift, num_blocks, max_blocks, capacity;
};
cudaError_t launch_update_tables(const TablesParams& p, cudaStream_t stream);
struct AppendSlotsParams {
  const uint16_t* ckv_new;
  const uint16_t* kpe_new;
  const int64_t* slots;        // [tokens]
  uint16_t* ckv;               // [rows, 512]
  uint16_t* kpe;               // [rows, 64]
  int64_t ckv_stride, kpe_stride, tokens, rows;
};
cudaError_t launch_append_slots(const AppendSlotsParams& p, cudaStream_t stream);
cudaError_t step_tables_read_clear_error(uint32_t* out);

// Keys and values of every head from cached latents (mla_expand_kv): maps of boxes of 64 columns, a page high over the
// [rows, 512] cache, 128 rows high over w_uk as [H * 128, 512], 64 over w_uv_t as [H * 512, 128], 32 rows of one head
// high over the outputs, 128-byte swizzle.
struct ExpandParams {
  const uint16_t* kpe;         // [num_blocks, bs, 64]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* kv_indptr;    // [B+1]
  const uint8_t* w_uk;         // [H, 128, 512] 16-bit
  const uint8_t* w_uv_t;       // [H, 512, 128] 16-bit
  uint16_t* k_nope;            // [max_tokens, H, 128]
  uint16_t* v;                 // [max_tokens, H, 128]
  uint16_t* k_pe;              // [max_tokens, 64]
  int32_t B, H, bs, max_blocks, num_blocks, max_tokens;
  uint64_t timeout_ns;
};
cudaError_t launch_expand_kv(const CUtensorMap& tm_ckv, const CUtensorMap& tm_uk, const CUtensorMap& tm_uv,
                             const CUtensorMap& tm_k, const CUtensorMap& tm_v, const ExpandParams& p, bool bf16,
                             int sms, cudaStream_t stream);
cudaError_t expand_read_clear_error(uint32_t* out);

// Attention of prompts (mla_prefill). The maps, 128-byte swizzle, 64 columns a box: q and qpe [T, H, 128 / 64] and k [S,
// H, 128] with boxes of 128 rows of one head, kpe [S, 64] of 128 rows, v [S, H, 128] of 64 rows of one head.
struct PrefillMaps {
  CUtensorMap q, qpe, k, kpe, v;
};
struct PrefillParams {
  const int32_t* q_indptr;     // [B+1]
  const int32_t* kv_indptr;    // [B+1]
  const uint16_t* v;           // [S, H, 128]
  void* out;                   // [T, H, 128]
  float* out_lse;              // [T, H] or null
  const int32_t* items;        // the plan's list, eight words an item, or null: planned in the kernel
  const int32_t* num_items;
  float* part_o;               // [slots, 256, H, 128]
  float* part_lse;             // [slots, 256, H]
  float scale_log2;            // |softmax scale| * log2(e)
  int32_t negate;              // the scale is negative
  int32_t B, H, T, S, causal;
  uint64_t timeout_ns;
};
struct PrefillPlanParams {
  int32_t* items;
  int32_t* num_items;
  int32_t* num_merges;
  int4* merge;                 // {first row of out, rows, first slot, pieces}
  int32_t max_items, max_slots, max_tiles, sms;
};
int prefill_max_slots(int H, int sms);
int prefill_max_tiles(int B, int T);
bool prefill_direct(int B, int T, int S);
cudaError_t launch_prefill(const PrefillMaps& maps, const PrefillParams& p, const PrefillPlanParams& pl, bool bf16,
                           int sms, cudaStream_t stream);
cudaError_t prefill_read_clear_error(uint32_t* out);

// A batch whose contexts start with the same tokens (mla_decode_shared). Maps over the [rows, 512] cache as (64 columns,
// 8 rows, 8 column blocks, row groups), a page high, four (tm_half) and two (tm_piece) column blocks a box, and over
// the [rows, 64] one, 128-byte swizzle.
struct SharedParams {
  const uint16_t* q_abs;       // [rows, 512]
  const uint16_t* q_pe;        // [rows, 64]
  const uint16_t* ckv;         // [num_blocks, bs, 512]
  const int32_t* shared_table; // [shared_tokens / bs]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* context_lens; // [B]
  const int32_t* units;        // eight words a unit (mla_shared_unit_t)
  const int32_t* own_indptr;   // [B * groups of a request + 1]
  const int32_t* cta_indptr;   // [num_ctas + 1]
  void* out;                   // [rows, 512] of out_dtype
  float* out_lse;              // [rows] or null
  float* part_o;               // [slots, 128, 512]
  float* part_lse;             // [slots, 128]
  float scale_log2;
  int32_t B, H, q_len, rows, bs, max_blocks, num_blocks, causal, shared_tokens, shared_parts, num_ctas, out_dtype;
  uint64_t timeout_ns;
};
cudaError_t launch_decode_shared(const CUtensorMap& tm_half, const CUtensorMap& tm_piece, const CUtensorMap& tm_kpe,
                                 const SharedParams& p, bool bf16, cudaStream_t stream);
cudaError_t decode_shared_read_clear_error(uint32_t* out);

// What the files of entry points share (api.cu).
void count_launch(int counter, uint64_t n = 1);
int32_t rejected(int32_t status);  // counts it and gives it back
uint64_t wait_timeout_ns();
bool is_aligned(const void* p, uintptr_t a);
// A map over 16-bit elements: `rank` dimensions innermost first, strides in bytes of all but the innermost, 128-byte
// swizzle, zeros outside. False where the driver refuses it.
bool encode_map16(CUtensorMap* out, const void* base, bool bf16, int rank, const uint64_t* dims,
                  const uint64_t* strides, const uint32_t* box);

// Launchers return cudaSuccess or the launch error. grid.x = cluster of
// `cluster` CTAs, grid.y = chunks, grid.z = row groups.
cudaError_t launch_partial_simt(const CUtensorMap& tm_ckv, const CUtensorMap& tm_kpe, const PartialParams& p,
                                int num_chunks, int cluster, bool bf16, cudaStream_t stream);
// tm_pages: 4D map of the ckv cache whose box is one half (256 columns) of a page;
// tm_kpe_half: kpe boxes of 32 columns with the 64-byte swizzle.
cudaError_t launch_partial_tc(const CUtensorMap& tm_ckv, const CUtensorMap& tm_kpe, const CUtensorMap& tm_pages,
                              const CUtensorMap& tm_kpe_half, const PartialParams& p, int num_chunks, int cluster,
                              bool bf16, cudaStream_t stream);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);
// 128-token-tile tensor-core kernel for CTAs of at most 16 rows (fp16, bf16, or E4M3 caches),
// CTAs in pairs that split the latent columns (cluster of 2..16 CTAs).
// tm_kpe_half: kpe boxes of 32 columns with the 64-byte swizzle.
bool tc128_supports(int total_rows, bool bf16, int cluster);
cudaError_t launch_partial_tc128(const CUtensorMap& tm_pages, const CUtensorMap& tm_kpe_half, const PartialParams& p,
                                 int num_chunks, int cluster, bool bf16, cudaStream_t stream);
int tc128_max_active_clusters(int cluster);
// 64-token-tile tensor-core kernel for groups of 128 rows (q_len * H > 16, the last group
// padded), fp16 or bf16, each group on a cluster of one CTA pair that split the latent columns.
bool mh_supports(int total_rows, int cluster);
// The 128-row groups without a score exchange (xchg16 == 2): every CTA of a pair computes the full scores.
cudaError_t launch_partial_mh_nx(const CUtensorMap& tm_pages, const CUtensorMap& tm_kpe_half, const PartialParams& p,
                                 int num_chunks, bool bf16, cudaStream_t stream);
cudaError_t mh_nx_read_clear_error(uint32_t* out);
cudaError_t launch_partial_mh(const CUtensorMap& tm_pages, const CUtensorMap& tm_kpe_half, const PartialParams& p,
                              int num_chunks, bool bf16, cudaStream_t stream);

// Query rows per CTA for q_len x H rows (SIMT: always 16).
int simt_rows_per_cta();
int tc_rows_per_cta(int total_rows, bool bf16);
// Occupancy: co-resident clusters of `cluster` CTAs of the tensor-core kernel.
int tc_max_active_clusters(int cluster, int rows_per_cta, bool bf16);

cudaError_t simt_read_clear_error(uint32_t* out);
cudaError_t tc_read_clear_error(uint32_t* out);
cudaError_t tc128_read_clear_error(uint32_t* out);
cudaError_t mh_read_clear_error(uint32_t* out);
cudaError_t wrap_read_clear_error(uint32_t* out);

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_merge_unembed(const UnembedParams& p, bool w_bf16, cudaStream_t stream);

}  // namespace mla
