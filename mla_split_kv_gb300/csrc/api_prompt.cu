// C ABI entry points of a serving step and its prompts: argument checks (before any launch) and dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "kernels.h"
#include "mla_split_kv.h"

namespace {

mla_status_t reject(mla_status_t s) { return static_cast<mla_status_t>(mla::rejected(s)); }

bool valid_page(int32_t bs) { return bs == 16 || bs == 32 || bs == 64; }

mla_status_t launched(cudaError_t e, int counter) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  mla::count_launch(counter);
  return MLA_OK;
}

// A dense [rows, cols] matrix of 16-bit elements in boxes of 64 columns.
bool rows_map(CUtensorMap* out, const void* base, bool bf16, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const uint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
  const uint32_t box[2] = {mla::kBoxCols, box_rows};
  return mla::encode_map16(out, base, bf16, 2, dims, strides, box);
}

// Boxes of 64 columns of one head, `box_rows` rows high, of a [rows, H, cols] tensor.
bool heads_map(CUtensorMap* out, const void* base, bool bf16, uint64_t rows, uint64_t H, uint64_t cols,
               int64_t row_stride, int64_t head_stride, uint32_t box_rows) {
  const uint64_t dims[3] = {cols, H, rows};
  const uint64_t strides[2] = {static_cast<uint64_t>(head_stride) * 2, static_cast<uint64_t>(row_stride) * 2};
  const uint32_t box[3] = {mla::kBoxCols, 1, box_rows};
  return mla::encode_map16(out, base, bf16, 3, dims, strides, box);
}

// mla_prefill's workspace: the plan's counts and lists, then the cut runs' pieces.
struct PrefillSpace {
  uint64_t items, merge, part_o, part_lse, bytes;
  int max_items, max_slots, max_tiles;
};
PrefillSpace prefill_space(int32_t B, int32_t H, int32_t T, int sms) {
  auto round256 = [](uint64_t x) { return (x + 255) / 256 * 256; };
  PrefillSpace w;
  w.max_slots = mla::prefill_max_slots(H, sms);
  w.max_tiles = mla::prefill_max_tiles(B, T);
  w.max_items = w.max_tiles + w.max_slots;
  const uint64_t rows = static_cast<uint64_t>(w.max_slots) * 256 * H;
  w.items = 256;
  w.merge = w.items + round256(static_cast<uint64_t>(w.max_items) * 32);
  w.part_o = w.merge + round256(static_cast<uint64_t>(w.max_slots) * 16);
  w.part_lse = w.part_o + rows * MLA_V_HEAD_DIM * 4;
  w.bytes = w.part_lse + rows * 4;
  return w;
}

int current_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sms;
}

}  // namespace

extern "C" {

mla_status_t mla_update_tables(const int32_t* changes, const int32_t* context_lens, int32_t* context_lens_out,
                               int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                               int32_t* free_count_out, int32_t* q_indptr, int32_t* kv_indptr, int64_t* slots,
                               int32_t* served, const mla_step_desc_t* d) {
  if (d == nullptr || changes == nullptr || context_lens == nullptr || context_lens_out == nullptr ||
      block_table == nullptr || free_pages == nullptr || free_count == nullptr || free_count_out == nullptr ||
      q_indptr == nullptr || kv_indptr == nullptr || slots == nullptr || served == nullptr)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests < 1 || d->num_blocks < 1 || d->max_blocks_per_req < 1 || d->capacity < 1)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests > MLA_MAX_STEP_REQUESTS || !valid_page(d->block_size)) return reject(MLA_ERR_UNSUPPORTED);
  const int32_t* const words[] = {changes, context_lens, context_lens_out, block_table, free_pages, free_count,
                                  free_count_out, q_indptr, kv_indptr, served};
  for (const int32_t* w : words)
    if (!mla::is_aligned(w, 4)) return reject(MLA_ERR_INVALID_ARG);
  if (!mla::is_aligned(slots, 8)) return reject(MLA_ERR_INVALID_ARG);
  mla::TablesParams p;
  p.changes = changes;
  p.lens = context_lens;
  p.lens_out = context_lens_out;
  p.block_table = block_table;
  p.pages = free_pages;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.q_indptr = q_indptr;
  p.kv_indptr = kv_indptr;
  p.slots = slots;
  p.served = served;
  p.B = d->num_requests;
  p.bs = d->block_size;
  p.bs_shift = d->block_size == 16 ? 4 : d->block_size == 32 ? 5 : 6;
  p.num_blocks = d->num_blocks;
  p.max_blocks = d->max_blocks_per_req;
  p.capacity = d->capacity;
  return launched(mla::launch_update_tables(p, static_cast<cudaStream_t>(d->stream)), MLA_CTR_STEP);
}

mla_status_t mla_cache_append_slots(const void* ckv_new, int64_t ckv_stride, const void* kpe_new, int64_t kpe_stride,
                                    const int64_t* slots, int64_t num_tokens, int32_t block_size, int32_t num_blocks,
                                    void* ckv_cache, void* kpe_cache, void* stream) {
  if (ckv_new == nullptr || kpe_new == nullptr || slots == nullptr || ckv_cache == nullptr || kpe_cache == nullptr)
    return reject(MLA_ERR_INVALID_ARG);
  if (num_tokens < 1 || num_tokens > 0x7fffffffll || num_blocks < 1) return reject(MLA_ERR_INVALID_ARG);
  if (!valid_page(block_size)) return reject(MLA_ERR_UNSUPPORTED);
  if (ckv_stride < mla::kRank || kpe_stride < mla::kRope || ckv_stride % 8 != 0 || kpe_stride % 8 != 0)
    return reject(MLA_ERR_INVALID_ARG);
  if (!mla::is_aligned(ckv_new, 16) || !mla::is_aligned(kpe_new, 16) || !mla::is_aligned(ckv_cache, 16) ||
      !mla::is_aligned(kpe_cache, 16) || !mla::is_aligned(slots, 8))
    return reject(MLA_ERR_INVALID_ARG);
  mla::AppendSlotsParams p;
  p.ckv_new = static_cast<const uint16_t*>(ckv_new);
  p.kpe_new = static_cast<const uint16_t*>(kpe_new);
  p.slots = slots;
  p.ckv = static_cast<uint16_t*>(ckv_cache);
  p.kpe = static_cast<uint16_t*>(kpe_cache);
  p.ckv_stride = ckv_stride;
  p.kpe_stride = kpe_stride;
  p.tokens = num_tokens;
  p.rows = static_cast<int64_t>(num_blocks) * block_size;
  return launched(mla::launch_append_slots(p, static_cast<cudaStream_t>(stream)), MLA_CTR_STEP);
}

mla_status_t mla_expand_kv(const void* ckv_cache, const void* kpe_cache, const int32_t* block_table,
                           const int32_t* kv_indptr, const void* w_uk, const void* w_uv_t, void* k_nope, void* v,
                           void* k_pe, const mla_expand_desc_t* d) {
  if (d == nullptr || ckv_cache == nullptr || kpe_cache == nullptr || block_table == nullptr || kv_indptr == nullptr ||
      w_uk == nullptr || w_uv_t == nullptr || k_nope == nullptr || v == nullptr || k_pe == nullptr)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests < 1 || d->num_blocks < 1 || d->max_blocks_per_req < 1 || d->max_tokens < 1)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_heads < 1 || d->num_heads > 256 || !valid_page(d->block_size)) return reject(MLA_ERR_UNSUPPORTED);
  if (d->dtype != MLA_F16 && d->dtype != MLA_BF16) return reject(MLA_ERR_UNSUPPORTED);
  if (!mla::is_aligned(ckv_cache, 16) || !mla::is_aligned(kpe_cache, 16) || !mla::is_aligned(w_uk, 16) ||
      !mla::is_aligned(w_uv_t, 16) || !mla::is_aligned(k_nope, 32) || !mla::is_aligned(v, 32) ||
      !mla::is_aligned(k_pe, 16) || !mla::is_aligned(block_table, 4) || !mla::is_aligned(kv_indptr, 4))
    return reject(MLA_ERR_INVALID_ARG);
  const uint64_t rows = static_cast<uint64_t>(d->num_blocks) * static_cast<uint64_t>(d->block_size);
  if (rows > 0x7fffffffull) return reject(MLA_ERR_UNSUPPORTED);
  const bool bf16 = d->dtype == MLA_BF16;
  const int sms = current_sms();
  CUtensorMap tm_ckv, tm_uk, tm_uv, tm_k, tm_v;
  const int64_t dense = static_cast<int64_t>(d->num_heads) * MLA_V_HEAD_DIM;
  if (sms < 2 || !rows_map(&tm_ckv, ckv_cache, bf16, rows, mla::kRank, d->block_size) ||
      !rows_map(&tm_uk, w_uk, bf16, static_cast<uint64_t>(d->num_heads) * MLA_NOPE_DIM, mla::kRank, 128) ||
      !heads_map(&tm_k, k_nope, bf16, d->max_tokens, d->num_heads, MLA_NOPE_DIM, dense, MLA_NOPE_DIM, 32) ||
      !heads_map(&tm_v, v, bf16, d->max_tokens, d->num_heads, MLA_V_HEAD_DIM, dense, MLA_V_HEAD_DIM, 32) ||
      !rows_map(&tm_uv, w_uv_t, bf16, static_cast<uint64_t>(d->num_heads) * mla::kRank, MLA_V_HEAD_DIM, mla::kBoxCols))
    return reject(MLA_ERR_CUDA);
  mla::ExpandParams p;
  p.kpe = static_cast<const uint16_t*>(kpe_cache);
  p.block_table = block_table;
  p.kv_indptr = kv_indptr;
  p.w_uk = static_cast<const uint8_t*>(w_uk);
  p.w_uv_t = static_cast<const uint8_t*>(w_uv_t);
  p.k_nope = static_cast<uint16_t*>(k_nope);
  p.v = static_cast<uint16_t*>(v);
  p.k_pe = static_cast<uint16_t*>(k_pe);
  p.B = d->num_requests;
  p.H = d->num_heads;
  p.bs = d->block_size;
  p.max_blocks = d->max_blocks_per_req;
  p.num_blocks = d->num_blocks;
  p.max_tokens = d->max_tokens;
  p.timeout_ns = mla::wait_timeout_ns();
  return launched(mla::launch_expand_kv(tm_ckv, tm_uk, tm_uv, tm_k, tm_v, p, bf16, sms, static_cast<cudaStream_t>(d->stream)),
                  MLA_CTR_PREFILL);
}

uint64_t mla_prefill_workspace_bytes(const mla_device_info_t* dev, int32_t num_requests, int32_t num_heads,
                                     int32_t max_q_tokens) {
  if (dev == nullptr || dev->num_sms < 1 || num_requests < 1 || num_requests > MLA_MAX_STEP_REQUESTS || num_heads < 1 ||
      num_heads > 256 || max_q_tokens < 1)
    return 0;
  return prefill_space(num_requests, num_heads, max_q_tokens, dev->num_sms).bytes;
}

mla_status_t mla_prefill(const void* q_nope, const void* q_pe, const void* k_nope, const void* k_pe, const void* v,
                         const int32_t* q_indptr, const int32_t* kv_indptr, float scale, void* out, float* out_lse,
                         const mla_prefill_desc_t* d) {
  if (d == nullptr || q_nope == nullptr || q_pe == nullptr || k_nope == nullptr || k_pe == nullptr || v == nullptr ||
      q_indptr == nullptr || kv_indptr == nullptr || out == nullptr)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests < 1 || d->max_q_tokens < 1 || d->max_kv_tokens < 1 || (d->causal != 0 && d->causal != 1) ||
      !std::isfinite(scale))
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests > MLA_MAX_STEP_REQUESTS || d->num_heads < 1 || d->num_heads > 256)
    return reject(MLA_ERR_UNSUPPORTED);
  if (d->dtype != MLA_F16 && d->dtype != MLA_BF16) return reject(MLA_ERR_UNSUPPORTED);
  // work items are counted, and positions held, in 31 bits
  if (d->max_kv_tokens > 0x7fffffff - 256 ||
      (static_cast<int64_t>(mla::prefill_max_tiles(d->num_requests, d->max_q_tokens)) + 1024) * d->num_heads > 0x3fffffff)
    return reject(MLA_ERR_UNSUPPORTED);
  const int64_t* const strides[2] = {d->q_nope_stride, d->q_pe_stride};
  const int64_t least[2] = {MLA_NOPE_DIM, mla::kRope};
  for (int k = 0; k < 2; ++k)
    for (int j = 0; j < 2; ++j)
      if (strides[k][j] < least[k] || strides[k][j] % 8 != 0 || strides[k][j] >= (1ll << 38))
        return reject(MLA_ERR_INVALID_ARG);
  if (!mla::is_aligned(q_nope, 16) || !mla::is_aligned(q_pe, 16) || !mla::is_aligned(k_nope, 16) ||
      !mla::is_aligned(k_pe, 16) || !mla::is_aligned(v, 16) || !mla::is_aligned(q_indptr, 4) ||
      !mla::is_aligned(kv_indptr, 4) || !mla::is_aligned(out, 32) || (out_lse != nullptr && !mla::is_aligned(out_lse, 4)))
    return reject(MLA_ERR_INVALID_ARG);
  const int sms = current_sms();
  if (sms < 1) return reject(MLA_ERR_CUDA);
  const int B = d->num_requests, H = d->num_heads, T = d->max_q_tokens, S = d->max_kv_tokens;
  const PrefillSpace space = prefill_space(B, H, T, sms);
  if (d->workspace == nullptr || !mla::is_aligned(d->workspace, 256) || d->workspace_bytes < space.bytes)
    return reject(MLA_ERR_INVALID_ARG);
  const bool bf16 = d->dtype == MLA_BF16;
  mla::PrefillMaps maps;
  const uint64_t dims[2] = {static_cast<uint64_t>(mla::kRope), static_cast<uint64_t>(S)}, pitch[1] = {mla::kRope * 2};
  const uint32_t box[2] = {mla::kBoxCols, 128};
  const int64_t dense = static_cast<int64_t>(H) * MLA_V_HEAD_DIM;
  if (!heads_map(&maps.q, q_nope, bf16, T, H, MLA_NOPE_DIM, d->q_nope_stride[0], d->q_nope_stride[1], 128) ||
      !heads_map(&maps.qpe, q_pe, bf16, T, H, mla::kRope, d->q_pe_stride[0], d->q_pe_stride[1], 128) ||
      !heads_map(&maps.k, k_nope, bf16, S, H, MLA_NOPE_DIM, dense, MLA_NOPE_DIM, 128) ||
      !heads_map(&maps.v, v, bf16, S, H, MLA_V_HEAD_DIM, dense, MLA_V_HEAD_DIM, 64) ||
      !mla::encode_map16(&maps.kpe, k_pe, bf16, 2, dims, pitch, box))
    return reject(MLA_ERR_CUDA);
  uint8_t* const ws = static_cast<uint8_t*>(d->workspace);
  mla::PrefillPlanParams pl;
  pl.num_items = reinterpret_cast<int32_t*>(ws);
  pl.num_merges = pl.num_items + 1;
  pl.items = reinterpret_cast<int32_t*>(ws + space.items);
  pl.merge = reinterpret_cast<int4*>(ws + space.merge);
  pl.max_items = space.max_items;
  pl.max_slots = space.max_slots;
  pl.max_tiles = space.max_tiles;
  pl.sms = sms;
  mla::PrefillParams p;
  p.q_indptr = q_indptr;
  p.kv_indptr = kv_indptr;
  p.v = static_cast<const uint16_t*>(v);
  p.out = out;
  p.out_lse = out_lse;
  p.items = mla::prefill_direct(B, T, S) ? nullptr : pl.items;
  p.num_items = pl.num_items;
  p.part_o = reinterpret_cast<float*>(ws + space.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + space.part_lse);
  p.scale_log2 = std::fabs(scale) * 1.4426950408889634f;
  p.negate = scale < 0 ? 1 : 0;
  p.B = B;
  p.H = H;
  p.T = T;
  p.S = S;
  p.causal = d->causal;
  p.timeout_ns = mla::wait_timeout_ns();
  return launched(mla::launch_prefill(maps, p, pl, bf16, sms, static_cast<cudaStream_t>(d->stream)), MLA_CTR_PREFILL);
}

uint64_t mla_decode_shared_workspace_bytes(int32_t num_slots) {
  if (num_slots < 1) return 0;
  return static_cast<uint64_t>(num_slots) * 128 * (mla::kRank + 1) * 4;
}

mla_status_t mla_decode_shared(const void* q_absorbed, const void* q_pe, const void* ckv_cache, const void* kpe_cache,
                               const int32_t* shared_table, const int32_t* block_table, const int32_t* context_lens,
                               float scale, void* out, float* out_lse, const mla_shared_desc_t* d) {
  if (d == nullptr || q_absorbed == nullptr || q_pe == nullptr || ckv_cache == nullptr || kpe_cache == nullptr ||
      shared_table == nullptr || block_table == nullptr || context_lens == nullptr || out == nullptr ||
      d->units == nullptr || d->own_indptr == nullptr || d->cta_indptr == nullptr)
    return reject(MLA_ERR_INVALID_ARG);
  if (d->num_requests < 1 || d->num_blocks < 1 || d->max_blocks_per_req < 1 || (d->causal != 0 && d->causal != 1) ||
      !std::isfinite(scale) || d->num_units < 1 || d->num_slots < 1 || d->shared_parts < 1 || d->num_ctas < 1)
    return reject(MLA_ERR_INVALID_ARG);
  if ((d->num_heads != 16 && d->num_heads != 64 && d->num_heads != 128) || d->q_len < 1 || d->q_len > MLA_MAX_Q_LEN ||
      !valid_page(d->block_size))
    return reject(MLA_ERR_UNSUPPORTED);
  if (d->dtype != MLA_F16 && d->dtype != MLA_BF16) return reject(MLA_ERR_UNSUPPORTED);
  if (d->out_dtype != MLA_F16 && d->out_dtype != MLA_BF16 && d->out_dtype != MLA_F32) return reject(MLA_ERR_UNSUPPORTED);
  if (d->shared_tokens < d->block_size || d->shared_tokens % d->block_size != 0) return reject(MLA_ERR_INVALID_ARG);
  const int64_t rows = static_cast<int64_t>(d->num_requests) * d->q_len * d->num_heads;
  const uint64_t cached = static_cast<uint64_t>(d->num_blocks) * static_cast<uint64_t>(d->block_size);
  if (rows > (1ll << 28) || cached > 0x7fffffffull || d->num_units > (1 << 28) || d->num_ctas > 65535) return reject(MLA_ERR_UNSUPPORTED);
  if (!mla::is_aligned(q_absorbed, 16) || !mla::is_aligned(q_pe, 16) || !mla::is_aligned(ckv_cache, 16) ||
      !mla::is_aligned(kpe_cache, 16) || !mla::is_aligned(out, 16) || !mla::is_aligned(shared_table, 4) ||
      !mla::is_aligned(block_table, 4) || !mla::is_aligned(context_lens, 4) || !mla::is_aligned(d->units, 16) ||
      !mla::is_aligned(d->own_indptr, 4) || !mla::is_aligned(d->cta_indptr, 4) || (out_lse != nullptr && !mla::is_aligned(out_lse, 4)))
    return reject(MLA_ERR_INVALID_ARG);
  // (partial outputs are stored 32 bytes at a time, at multiples of 32 from its start)
  if (d->workspace == nullptr || !mla::is_aligned(d->workspace, 32) ||
      d->workspace_bytes < mla_decode_shared_workspace_bytes(d->num_slots))
    return reject(MLA_ERR_INVALID_ARG);
  const bool bf16 = d->dtype == MLA_BF16;
  // the latent cache as (64 columns, 8 rows, 8 column blocks, row groups)
  const uint64_t dims[4] = {mla::kBoxCols, 8, mla::kRank / mla::kBoxCols, cached / 8};
  const uint64_t strides[3] = {mla::kRank * 2, mla::kBoxCols * 2, mla::kRank * 2 * 8};
  const uint32_t height = static_cast<uint32_t>(d->block_size / 8);
  const uint32_t half[4] = {mla::kBoxCols, 8, 4, height}, piece[4] = {mla::kBoxCols, 8, 2, height};
  CUtensorMap tm_half, tm_piece, tm_kpe;
  if (!mla::encode_map16(&tm_half, ckv_cache, bf16, 4, dims, strides, half) ||
      !mla::encode_map16(&tm_piece, ckv_cache, bf16, 4, dims, strides, piece) ||
      !rows_map(&tm_kpe, kpe_cache, bf16, cached, mla::kRope, d->block_size))
    return reject(MLA_ERR_CUDA);
  mla::SharedParams p;
  p.q_abs = static_cast<const uint16_t*>(q_absorbed);
  p.q_pe = static_cast<const uint16_t*>(q_pe);
  p.ckv = static_cast<const uint16_t*>(ckv_cache);
  p.shared_table = shared_table;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.units = reinterpret_cast<const int32_t*>(d->units);
  p.own_indptr = d->own_indptr;
  p.cta_indptr = d->cta_indptr;
  p.out = out;
  p.out_lse = out_lse;
  p.part_o = static_cast<float*>(d->workspace);
  p.part_lse = p.part_o + static_cast<uint64_t>(d->num_slots) * 128 * mla::kRank;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.B = d->num_requests;
  p.H = d->num_heads;
  p.q_len = d->q_len;
  p.rows = static_cast<int32_t>(rows);
  p.bs = d->block_size;
  p.max_blocks = d->max_blocks_per_req;
  p.num_blocks = d->num_blocks;
  p.causal = d->causal;
  p.shared_tokens = d->shared_tokens;
  p.shared_parts = d->shared_parts;
  p.num_ctas = d->num_ctas;
  p.out_dtype = d->out_dtype == MLA_F32 ? 2 : d->out_dtype == MLA_BF16 ? 1 : 0;
  p.timeout_ns = mla::wait_timeout_ns();
  return launched(mla::launch_decode_shared(tm_half, tm_piece, tm_kpe, p, bf16, static_cast<cudaStream_t>(d->stream)),
                  MLA_CTR_DECODE_SHARED);
}

}  // extern "C"
