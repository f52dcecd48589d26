// extern "C" entry points of the paged KV cache, of attention over its pages and
// of attention over packed prompts: planning, argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "abi_util.h"
#include "kernels.h"
#include "mla_split.h"

namespace {

using skv::ptr_aligned;

constexpr int kDim = 128;
constexpr int kMaxHeads = 1 << 24;   // of the append that rotates, the read-back and 4-bit pages: heads are counted in int32

uint64_t round_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

// Bytes of an element of Q, and of a stride's unit of K and V.
int q_size(int dtype) { return dtype == SDPA_E4M3 ? 1 : 2; }
int elem_size(int dtype) { return dtype == SDPA_BF16 ? 2 : 1; }

// An element stride that TMA and 16-byte loads can take.
bool stride_ok(int64_t s, int esz) { return s > 0 && (s * esz) % 16 == 0 && s < (int64_t{1} << 40) / esz; }

bool out_ok(const void* out, int out_dtype, float inv_scale) {
  if (out == nullptr || !ptr_aligned(out, 16)) return false;
  if (out_dtype != MLA_OUT_F32 && out_dtype != MLA_OUT_BF16 && out_dtype != MLA_OUT_E4M3) return false;
  return out_dtype != MLA_OUT_E4M3 || std::isfinite(inv_scale);
}

// Pointers of fp32 and int32 data that may be null.
bool words_ok(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!ptr_aligned(p, 4)) return false;
  return true;
}

int check_heads(int batch, int h_q, int h_kv, int d, int dtype) {
  if (d != kDim) return MLA_ERR_UNSUPPORTED;
  if (dtype != SDPA_BF16 && dtype != SDPA_E4M3 && dtype != SDPA_E2M1) return MLA_ERR_UNSUPPORTED;
  if (batch < 1 || h_kv < 1 || h_q < 1 || h_q % h_kv != 0) return MLA_ERR_INVALID_ARG;
  if (h_q / h_kv > 128) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

int check_pages(const kv_pages_t* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->dtype != SDPA_BF16 && p->dtype != SDPA_E4M3 && p->dtype != SDPA_E2M1) return MLA_ERR_UNSUPPORTED;
  if (p->d != kDim) return MLA_ERR_UNSUPPORTED;
  if (p->k == nullptr || p->v == nullptr || !ptr_aligned(p->k, 16) || !ptr_aligned(p->v, 16)) return MLA_ERR_INVALID_ARG;
  if (p->num_pages < 1 || p->h_kv < 1) return MLA_ERR_INVALID_ARG;
  if (p->page_size < 16 || p->page_size > 65536 || (p->page_size & (p->page_size - 1)) != 0) return MLA_ERR_UNSUPPORTED;
  const int e = elem_size(p->dtype);
  if (!stride_ok(p->page_stride, e) || !stride_ok(p->row_stride, e) || !stride_ok(p->head_stride, e))
    return MLA_ERR_INVALID_ARG;
  if (p->dtype == SDPA_E2M1) {
    if (p->k_scales == nullptr || p->v_scales == nullptr || !ptr_aligned(p->k_scales, 16) || !ptr_aligned(p->v_scales, 16))
      return MLA_ERR_INVALID_ARG;
    if (!stride_ok(p->scale_page_stride, 1) || !stride_ok(p->scale_head_stride, 1)) return MLA_ERR_INVALID_ARG;
    if (p->h_kv > kMaxHeads) return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  cudaGetLastError();
  return MLA_ERR_CUDA;
}

// Q as [total_q][h_q][128] in boxes of one row block: group heads of 128 / group tokens.
int encode_q(CUtensorMap* m, int dtype, const void* q, int64_t ts, int64_t hs, int h_q, int group, int total_q) {
  auto enc = skv::tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t e = q_size(dtype);
  const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(h_q), static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[2] = {hs * e, ts * e};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / e), static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(128 / group)};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, e == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
             const_cast<void*>(q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK
             : MLA_ERR_CUDA;
}

// K or V as [heads][pages][rows][128] in boxes of `box_rows` rows of one page and head.
int encode_kv(CUtensorMap* m, int dtype, const void* base, int64_t rows, int64_t row_stride, int64_t pages,
              int64_t page_stride, int heads, int64_t head_stride, int box_rows) {
  auto enc = skv::tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t e = elem_size(dtype);
  const cuuint64_t dims[4] = {kDim, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(pages),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {row_stride * e, page_stride * e, head_stride * e};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / e), static_cast<cuuint32_t>(box_rows), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, dtype == SDPA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK
             : MLA_ERR_CUDA;
}

// bf16 K or V pages as {64 dims, 8 rows, column blocks, row groups, pages}: a box takes both 64-dim column blocks of
// its rows, so a page of 16 rows is one copy of 4 KB. `wide` as in AttnArgs.
int encode_kv_wide(CUtensorMap* m, const kv_pages_t* p, const void* base, int wide, int box_rows) {
  auto enc = skv::tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t heads = static_cast<cuuint64_t>(p->h_kv), groups = static_cast<cuuint64_t>(p->page_size / 8);
  const cuuint64_t dims[5] = {64, 8, wide == 1 ? 2 * heads : 2, wide == 1 ? groups : groups * heads,
                              static_cast<cuuint64_t>(p->num_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(p->row_stride) * 2;
  const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(p->page_stride) * 2};
  const cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>(box_rows / 8), 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK
             : MLA_ERR_CUDA;
}

// K or V codes of 4-bit pages in boxes of `box_rows` rows of one page and head, and their scales, two words a row.
int encode_kv4(CUtensorMap* m, const kv_pages_t* p, const void* base, int box_rows) {
  auto enc = skv::tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t dims[4] = {kDim / 2, static_cast<cuuint64_t>(p->page_size), static_cast<cuuint64_t>(p->num_pages),
                              static_cast<cuuint64_t>(p->h_kv)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p->row_stride), static_cast<cuuint64_t>(p->page_stride),
                                 static_cast<cuuint64_t>(p->head_stride)};
  const cuuint32_t box[4] = {kDim / 2, static_cast<cuuint32_t>(box_rows), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK
             : MLA_ERR_CUDA;
}
int encode_scales(CUtensorMap* m, const kv_pages_t* p, const void* base, int box_rows) {
  auto enc = skv::tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t page = static_cast<cuuint64_t>(p->scale_page_stride);
  const cuuint64_t dims[4] = {2 * static_cast<cuuint64_t>(p->page_size), 1, static_cast<cuuint64_t>(p->num_pages),
                              static_cast<cuuint64_t>(p->h_kv)};
  const cuuint64_t strides[3] = {page, page, static_cast<cuuint64_t>(p->scale_head_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(2 * box_rows), 1, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK
             : MLA_ERR_CUDA;
}

// The most (sequence, query tile) pairs of `tokens` tokens that total_q rows of `batch` sequences can make.
int64_t tiles_bound(int total_q, int batch, int tokens) { return total_q / tokens + std::min(total_q, batch); }

// Query rows of a job, and the tokens in them (row_kernel: as in the plan).
int job_rows(int row_kernel) { return row_kernel == 2 ? 8 : row_kernel == 1 ? skv::kRowRows : skv::kTileRows; }
int job_tokens(int row_kernel, int group) { return row_kernel ? job_rows(row_kernel) / group : 2 * (128 / group); }

// Equal shares: of a wave's CTAs as many for each of `side` KV heads, the largest divisor of h_kv that leaves at most
// one in sixteen without work.
int heads_side(int wave, int h_kv) {
  for (int side = std::min(wave, h_kv); side > 1; --side)
    if (h_kv % side == 0 && wave % side <= wave / 16) return side;
  return 1;
}
int64_t share_ctas(int wave, int h_kv) {
  const int side = heads_side(wave, h_kv);
  return static_cast<int64_t>(wave / side) * side;
}

// The workspace of a plan with more than one split, from its other fields; false where its partial rows pass an int32.
bool plan_layout(sdpa_paged_plan_t* p) {
  if (p->num_sms > (1 << 24)) return false;   // (three waves' rows pass it, and twice the count would not be an int)
  const int group = p->h_q / p->h_kv;
  const bool rows16 = p->row_kernel != 0;
  const int wave = rows16 ? p->num_sms * skv::kRowCtasPerSm : p->num_sms;
  const int slot_rows = rows16 ? skv::kRowRows : skv::kTileRows;
  const int64_t unsplit = tiles_bound(p->total_q_max, p->batch, job_tokens(p->row_kernel, group)) * p->h_kv;
  // split jobs: as many as forced; two pieces of cut jobs a CTA; at most so many waves (the rule keeps to that)
  const int64_t slots = !p->adaptive_splits ? unsplit * p->num_splits
                        : rows16            ? 2 * share_ctas(wave, p->h_kv)
                                            : static_cast<int64_t>(wave) * skv::kTileSplitWaves;
  if (slots * slot_rows > 0x7FFFFFFFll) return false;
  const uint64_t rows = static_cast<uint64_t>(slots) * slot_rows;
  p->o_acc_bytes = rows * kDim * 4;
  p->lse_acc_offset = round_up(p->o_acc_bytes, 256);
  p->lse_acc_bytes = rows * 4;
  p->map_offset = round_up(p->lse_acc_offset + p->lse_acc_bytes, 256);
  p->workspace_bytes = round_up(p->map_offset + static_cast<uint64_t>(p->total_q_max) * p->h_kv * 8, 256);
  return true;
}

int shift_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

// What the append and the read-back take of a cache.
void set_pages(skv::PagesAppendArgs* a, const kv_pages_t* p) {
  a->k = p->k;
  a->v = p->v;
  a->page_stride = p->page_stride;
  a->row_stride = p->row_stride;
  a->cache_head_stride = p->head_stride;
  if (p->dtype == SDPA_E2M1) {   // (other types: the descriptor may end before these)
    a->k_scales = static_cast<uint8_t*>(p->k_scales);
    a->v_scales = static_cast<uint8_t*>(p->v_scales);
    a->scale_page_stride = p->scale_page_stride;
    a->scale_head_stride = p->scale_head_stride;
  }
  a->num_slots = static_cast<int64_t>(p->num_pages) * p->page_size;
  a->page_shift = shift_of(p->page_size);
  a->h_kv = p->h_kv;
}

}  // namespace

extern "C" {

int kv_pages_map(int batch, int page_size, const int32_t* held_lens, const int32_t* new_lens,
                 const int32_t* cu_seqlens_q, int total_q, int32_t* block_table, int table_width, int32_t* free_pages,
                 int free_capacity, const int32_t* free_in, int32_t* free_out, int64_t* slot_map, int32_t* positions,
                 void* stream) {
  if (batch < 1 || page_size < 1 || table_width < 1 || free_capacity < 1 || total_q < 0) return MLA_ERR_INVALID_ARG;
  if (held_lens == nullptr || new_lens == nullptr || cu_seqlens_q == nullptr || block_table == nullptr ||
      free_pages == nullptr || free_in == nullptr || free_out == nullptr || (slot_map == nullptr && total_q > 0))
    return MLA_ERR_INVALID_ARG;
  if (!words_ok({held_lens, new_lens, cu_seqlens_q, block_table, free_pages, free_in, free_out, positions}) ||
      !ptr_aligned(slot_map, 8))
    return MLA_ERR_INVALID_ARG;
  if (batch > KV_PAGES_MAX_BATCH) return MLA_ERR_UNSUPPORTED;
  // (the kernel's page ordinals, and their sum with the list's count, are int32)
  if (static_cast<int64_t>(batch) * table_width > KV_PAGES_MAX_ENTRIES || free_capacity > KV_PAGES_MAX_ENTRIES)
    return MLA_ERR_UNSUPPORTED;
  skv::DeviceInfo dev;
  const int st = skv::current_device(&dev);
  if (st != MLA_OK) return st;
  skv::PagesMapArgs a{};
  a.batch = batch;
  a.page_size = page_size;
  a.held = held_lens;
  a.lens = new_lens;
  a.cu_q = cu_seqlens_q;
  a.total_q = total_q;
  a.table = block_table;
  a.width = table_width;
  a.free_pages = free_pages;
  a.capacity = free_capacity;
  a.free_in = free_in;
  a.free_out = free_out;
  a.slots = slot_map;
  a.positions = positions;
  return cuda_status(skv::launch_pages_map(a, static_cast<cudaStream_t>(stream)));
}

int kv_pages_write(const kv_pages_t* pages, int64_t rows, const void* k_new, const void* v_new, int64_t token_stride,
                   int64_t head_stride, const int64_t* slot_map, const float* descale_k, const float* descale_v,
                   void* stream) {
  int st = check_pages(pages);
  if (st != MLA_OK) return st;
  if (rows < 0 || rows > 0x7FFFFFFFll) return MLA_ERR_INVALID_ARG;
  if (rows == 0) return MLA_OK;
  if (k_new == nullptr || v_new == nullptr || slot_map == nullptr) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(k_new, 16) || !ptr_aligned(v_new, 16) || !ptr_aligned(slot_map, 8)) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(token_stride, 2) || !stride_ok(head_stride, 2)) return MLA_ERR_INVALID_ARG;
  if (!words_ok({descale_k, descale_v})) return MLA_ERR_INVALID_ARG;
  if (rows * pages->h_kv > (int64_t{1} << 35)) return MLA_ERR_INVALID_ARG;
  skv::DeviceInfo dev;
  st = skv::current_device(&dev);
  if (st != MLA_OK) return st;
  if (pages->dtype == SDPA_E2M1) {
    skv::PagesAppendArgs a{};
    set_pages(&a, pages);
  a.num_sms = dev.num_sms;
    a.k_new = static_cast<const uint16_t*>(k_new);
    a.v_new = static_cast<const uint16_t*>(v_new);
    a.token_stride = token_stride;
    a.head_stride = head_stride;
    a.slots = slot_map;
    a.rows = rows;
    a.descale_k = descale_k;
    a.descale_v = descale_v;
    return cuda_status(skv::launch_pages_append(a, pages->dtype, static_cast<cudaStream_t>(stream)));
  }
  skv::PagesWriteArgs a{};
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.slots = slot_map;
  a.rows = rows;
  a.k = pages->k;
  a.v = pages->v;
  a.page_stride = pages->page_stride;
  a.row_stride = pages->row_stride;
  a.cache_head_stride = pages->head_stride;
  a.num_slots = static_cast<int64_t>(pages->num_pages) * pages->page_size;
  a.page_shift = shift_of(pages->page_size);
  a.h_kv = pages->h_kv;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  return cuda_status(skv::launch_pages_write(a, pages->dtype, static_cast<cudaStream_t>(stream)));
}

int kv_pages_write_rotary(const kv_pages_t* pages, int64_t rows, int h_q, const void* q, int64_t q_token_stride,
                          int64_t q_head_stride, const void* k_new, const void* v_new, int64_t token_stride, int64_t head_stride,
                          const int32_t* positions, const float* cos_sin, int64_t num_positions, int rotary_dim, int interleaved,
                          const int64_t* slot_map, const float* descale_q, const float* descale_k, const float* descale_v,
                          int q_out_dtype, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                          int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
  int st = check_pages(pages);
  if (st != MLA_OK) return st;
  if (rows < 0 || rows > 0x7FFFFFFFll || h_q < 0 || h_q > kMaxHeads || pages->h_kv > kMaxHeads) return MLA_ERR_INVALID_ARG;
  if (rotary_dim < 32 || rotary_dim > kDim || rotary_dim % 32 != 0) return MLA_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return MLA_ERR_INVALID_ARG;
  if (num_positions < 1 || num_positions > (int64_t{1} << 31)) return MLA_ERR_INVALID_ARG;
  if (rows == 0) return MLA_OK;
  if (k_new == nullptr || v_new == nullptr || slot_map == nullptr || positions == nullptr || cos_sin == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(k_new, 16) || !ptr_aligned(v_new, 16) || !ptr_aligned(slot_map, 8) || !ptr_aligned(cos_sin, 16))
    return MLA_ERR_INVALID_ARG;
  if (!stride_ok(token_stride, 2) || !stride_ok(head_stride, 2)) return MLA_ERR_INVALID_ARG;
  if (!words_ok({positions, descale_q, descale_k, descale_v})) return MLA_ERR_INVALID_ARG;
  if (h_q > 0) {
    if (q == nullptr || q_out == nullptr || !ptr_aligned(q, 16) || !ptr_aligned(q_out, 16)) return MLA_ERR_INVALID_ARG;
    if (q_out_dtype != SDPA_BF16 && q_out_dtype != SDPA_E4M3) return MLA_ERR_INVALID_ARG;
    const int e = q_size(q_out_dtype);
    if (!stride_ok(q_token_stride, 2) || !stride_ok(q_head_stride, 2) || !stride_ok(q_out_token_stride, e) ||
        !stride_ok(q_out_head_stride, e))
      return MLA_ERR_INVALID_ARG;
  }
  if (k_out != nullptr && (!ptr_aligned(k_out, 16) || !stride_ok(k_out_token_stride, 2) || !stride_ok(k_out_head_stride, 2)))
    return MLA_ERR_INVALID_ARG;
  if (rows * (h_q + 2ll * pages->h_kv) > (int64_t{1} << 35)) return MLA_ERR_INVALID_ARG;
  skv::DeviceInfo dev;
  if ((st = skv::current_device(&dev)) != MLA_OK) return st;
  skv::PagesAppendArgs a{};
  set_pages(&a, pages);
  a.num_sms = dev.num_sms;
  a.q = static_cast<const uint16_t*>(q);
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.slots = slot_map;
  a.rows = rows;
  a.h_q = h_q;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.num_positions = num_positions;
  a.rot = rotary_dim;
  a.interleaved = interleaved;
  a.q_out = q_out;
  a.q_out_e4m3 = q_out_dtype == SDPA_E4M3;
  a.qo_ts = q_out_token_stride;
  a.qo_hs = q_out_head_stride;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.ko_ts = k_out_token_stride;
  a.ko_hs = k_out_head_stride;
  a.descale_q = descale_q;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  return cuda_status(skv::launch_pages_append(a, pages->dtype, static_cast<cudaStream_t>(stream)));
}

int kv_pages_read(const kv_pages_t* pages, int64_t rows, const int64_t* slot_map, const float* descale_k, const float* descale_v,
                  void* k_out, void* v_out, int64_t token_stride, int64_t head_stride, void* stream) {
  int st = check_pages(pages);
  if (st != MLA_OK) return st;
  if (rows < 0 || rows > 0x7FFFFFFFll || pages->h_kv > kMaxHeads) return MLA_ERR_INVALID_ARG;
  if (rows == 0) return MLA_OK;
  if (k_out == nullptr || v_out == nullptr || slot_map == nullptr) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(k_out, 16) || !ptr_aligned(v_out, 16) || !ptr_aligned(slot_map, 8)) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(token_stride, 2) || !stride_ok(head_stride, 2)) return MLA_ERR_INVALID_ARG;
  if (!words_ok({descale_k, descale_v})) return MLA_ERR_INVALID_ARG;
  if (rows * pages->h_kv > (int64_t{1} << 35)) return MLA_ERR_INVALID_ARG;
  skv::DeviceInfo dev;
  if ((st = skv::current_device(&dev)) != MLA_OK) return st;
  skv::PagesAppendArgs a{};
  set_pages(&a, pages);
  a.num_sms = dev.num_sms;
  a.slots = slot_map;
  a.rows = rows;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.ko_ts = token_stride;
  a.ko_hs = head_stride;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  return cuda_status(skv::launch_pages_read(a, pages->dtype, static_cast<cudaStream_t>(stream)));
}

int sdpa_paged_plan(int batch, int h_q, int h_kv, int d, int dtype, int max_q_per_seq, int total_q_max, int max_kv,
                    int num_sms, int max_splits, int force_splits, sdpa_paged_plan_t* out) {
  if (out == nullptr) return MLA_ERR_INVALID_ARG;
  std::memset(out, 0, sizeof(*out));
  int st = check_heads(batch, h_q, h_kv, d, dtype);
  if (st != MLA_OK) return st;
  if (max_q_per_seq < 1 || total_q_max < 1 || max_kv < 1 || num_sms < 0) return MLA_ERR_INVALID_ARG;
  if (max_splits < 0 || max_splits > MLA_MAX_SPLITS || force_splits < 0 || force_splits > MLA_MAX_SPLITS)
    return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(total_q_max) * h_q > 0x7FFFFFFFll) return MLA_ERR_INVALID_ARG;
  if (num_sms == 0) {
    skv::DeviceInfo dev;
    if ((st = skv::current_device(&dev)) != MLA_OK) return st;
    num_sms = dev.num_sms;
  }
  const int group = h_q / h_kv;
  int S = force_splits;
  int adaptive = 0;
  if (S == 0) {
    const int cap = max_splits > 0 ? max_splits : MLA_MAX_SPLITS;
    S = std::min(cap, (max_kv + 127) / 128);
    adaptive = S > 1 ? 1 : 0;
  }
  // few rows a sequence: the kernel of 16-row jobs, of which an SM holds two
  const bool rows16 = static_cast<int64_t>(max_q_per_seq) * group <= skv::kRowRows;
  out->batch = batch;
  out->h_q = h_q;
  out->h_kv = h_kv;
  out->d = d;
  out->dtype = dtype;
  out->max_q_per_seq = max_q_per_seq;
  out->total_q_max = total_q_max;
  out->max_kv = max_kv;
  out->num_splits = S;
  out->num_sms = num_sms;
  out->adaptive_splits = adaptive;
  out->row_kernel = !rows16 ? 0 : dtype == SDPA_E2M1 && static_cast<int64_t>(max_q_per_seq) * group <= 8 ? 2 : 1;
  if (S > 1 && !plan_layout(out)) {
    std::memset(out, 0, sizeof(*out));
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

int sdpa_paged(const sdpa_paged_plan_t* plan, int total_q, const void* q, int64_t q_token_stride,
               int64_t q_head_stride, const kv_pages_t* pages, const int32_t* block_table, int table_width,
               const int32_t* kv_lens, const int32_t* cu_seqlens_q, const float* descale_q, const float* descale_k,
               const float* descale_v, float sm_scale, int out_dtype, float out_inv_scale, void* out, float* lse_out,
               float* amax_out, void* workspace, void* stream) {
  if (plan == nullptr) return MLA_ERR_INVALID_ARG;
  int st = check_heads(plan->batch, plan->h_q, plan->h_kv, plan->d, plan->dtype);
  if (st != MLA_OK) return st;
  if ((st = check_pages(pages)) != MLA_OK) return st;
  if (pages->dtype != plan->dtype || pages->h_kv != plan->h_kv || pages->d != plan->d) return MLA_ERR_INVALID_ARG;
  if (plan->num_splits < 1 || plan->num_splits > MLA_MAX_SPLITS || plan->num_sms < 1) return MLA_ERR_INVALID_ARG;
  if (plan->adaptive_splits != 0 && plan->num_splits < 2) return MLA_ERR_INVALID_ARG;
  if (plan->row_kernel < 0 || plan->row_kernel > (plan->dtype == SDPA_E2M1 ? 2 : 1)) return MLA_ERR_INVALID_ARG;
  if (plan->row_kernel != 0 && plan->h_q / plan->h_kv > job_rows(plan->row_kernel)) return MLA_ERR_INVALID_ARG;
  if (total_q < 1 || total_q > plan->total_q_max || table_width < 1) return MLA_ERR_INVALID_ARG;
  if (q == nullptr || block_table == nullptr || kv_lens == nullptr || cu_seqlens_q == nullptr) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !words_ok({block_table, kv_lens, cu_seqlens_q, descale_q, descale_k, descale_v, lse_out, amax_out}))
    return MLA_ERR_INVALID_ARG;
  const int e = q_size(plan->dtype);
  if (!stride_ok(q_token_stride, e) || !stride_ok(q_head_stride, e)) return MLA_ERR_INVALID_ARG;
  if (!out_ok(out, out_dtype, out_inv_scale) || !std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  if (plan->num_splits > 1) {
    // the kernels write where the plan says, so it has to be what the planner makes of its other fields
    sdpa_paged_plan_t same = *plan;
    if (!plan_layout(&same) || same.o_acc_bytes != plan->o_acc_bytes || same.lse_acc_offset != plan->lse_acc_offset ||
        same.lse_acc_bytes != plan->lse_acc_bytes || same.map_offset != plan->map_offset ||
        same.workspace_bytes != plan->workspace_bytes)
      return MLA_ERR_WORKSPACE;
    if (workspace == nullptr || !ptr_aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  }
  skv::DeviceInfo dev;
  if ((st = skv::current_device(&dev)) != MLA_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (amax_out != nullptr && (st = cuda_status(cudaMemsetAsync(amax_out, 0, sizeof(float), cs))) != MLA_OK) return st;
  skv::AttnArgs a{};
  a.q = q;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.table = block_table;
  a.table_width = table_width;
  a.page_shift = shift_of(pages->page_size);
  a.num_pages = pages->num_pages;
  a.cu_q = cu_seqlens_q;
  a.kv_lens = kv_lens;
  a.descale_q = descale_q;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  a.batch = plan->batch;
  a.h_q = plan->h_q;
  a.h_kv = plan->h_kv;
  a.group = plan->h_q / plan->h_kv;
  a.total_q = total_q;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_dtype = out_dtype;
  a.inv_scale = out_inv_scale;
  a.lse_out = lse_out;
  a.amax = amax_out;
  a.num_splits = plan->num_splits;
  const bool rows16 = plan->row_kernel != 0;
  a.num_sms = rows16 ? plan->num_sms * skv::kRowCtasPerSm : plan->num_sms;
  a.max_slots = static_cast<int>(plan->o_acc_bytes / ((rows16 ? skv::kRowRows : skv::kTileRows) * kDim * 4ull));
  if (plan->num_splits > 1) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.o_part = reinterpret_cast<float*>(ws);
    a.lse_part = reinterpret_cast<float*>(ws + plan->lse_acc_offset);
    a.row_map = reinterpret_cast<int2*>(ws + plan->map_offset);
  }
  a.status = dev.status;
  a.wait_limit_ns = skv::wait_limit_ns();
  a.drain_limit_ns = skv::drain_limit_ns();
  CUtensorMap tq, tk, tv, tks, tvs;
  const bool four = plan->dtype == SDPA_E2M1;
  const int box = rows16 && !four ? skv::attn_row_box(plan->dtype, pages->page_size)
                                  : std::min(pages->page_size, rows16 ? skv::kRow4Box : 128);
  if (!rows16 && plan->dtype == SDPA_BF16) {
    // (with one head its stride says nothing)
    if (pages->h_kv == 1 || pages->head_stride == kDim) a.kv_wide = 1;
    else if (pages->head_stride == pages->page_size * pages->row_stride) a.kv_wide = 2;
  }
  auto encode = [&](CUtensorMap* m, const void* base) {
    if (four) return encode_kv4(m, pages, base, box);
    if (a.kv_wide) return encode_kv_wide(m, pages, base, a.kv_wide, box);
    return encode_kv(m, plan->dtype, base, pages->page_size, pages->row_stride, pages->num_pages, pages->page_stride,
                     pages->h_kv, pages->head_stride, box);
  };
  if (!rows16 && (st = encode_q(&tq, plan->dtype, q, q_token_stride, q_head_stride, a.h_q, a.group, total_q)) != MLA_OK)
    return st;
  if ((st = encode(&tk, pages->k)) != MLA_OK || (st = encode(&tv, pages->v)) != MLA_OK) return st;
  if (four && rows16 && ((st = encode_scales(&tks, pages, pages->k_scales, box)) != MLA_OK ||
                         (st = encode_scales(&tvs, pages, pages->v_scales, box)) != MLA_OK))
    return st;
  const int64_t unsplit = tiles_bound(total_q, a.batch, job_tokens(plan->row_kernel, a.group)) * a.h_kv;
  int64_t grid = unsplit * a.num_splits;
  // Equal shares balance best, but let query tiles of one sequence read the same keys at different times. Decode has one
  // query tile a sequence. With more rows, the keys of e4m3 still come from DRAM fast enough (32 KB a tile and SM in
  // 1.4 us: 3.5 TB/s), those of bf16 do not (1,024 tokens over 65,536 keys: 641 -> 729 us); unsplit jobs that fit one
  // wave have no second one to even out (8 x 16 over 8,192 e4m3 keys: 40.5 -> 44.6 us); and the two cut jobs of
  // every CTA (256 rows each, and their combine) have to be small beside a sequence (e4m3, 2 x 2,048 tokens over 4,096 keys 145 ->
  // 157 us, 8,192 308 -> 296, 16,384 638 -> 579; 4 x 300 over 9,000 169 -> 129; 40 x 16 over 9,000 185 -> 144).
  // The length is the plan's bound: 2 x 2,048 over 4,096 under a plan for 131,072 keys take 150 us instead of 139.
  constexpr int kLongKeys = 6144;
  // 4 bits, sequences of one query tile each, as decode: whole jobs leave too few pieces to even out (16 x 1 to 16 tokens over 1,024 to
  // 16,384 keys by length 133 us, in shares 98; 8 x 8 over 8,192 55 and 52; 40 x 1 to 16 over 1,000 to 5,500 126 and 111; 8 of 256 to
  // 1,024 23.9 and 24.1, 8 of 128 to 300 20.6 and 26.6). Chunks gain or lose with the keys an SM has (1 x 512 over 32,768 202 and 180,
  // 2 x 300 over 16,384 72 and 88), which the host does not know, and keep to the rule of e4m3.
  constexpr int kFewKeys = 1024;
  if (plan->adaptive_splits) {
    const bool one_tile = four && plan->max_q_per_seq <= job_tokens(0, a.group) && plan->max_kv >= kFewKeys;
    const bool shares = rows16 || one_tile || (plan->dtype != SDPA_BF16 && unsplit > a.num_sms && plan->max_kv >= kLongKeys);
    a.adaptive = shares ? skv::kShares : skv::kByLength;
  }
  if (a.adaptive == skv::kByLength) {
    grid = unsplit <= a.num_sms ? a.num_sms : unsplit + static_cast<int64_t>(skv::kTileSplitWaves) * a.num_sms;
  } else if (a.adaptive == skv::kShares) {
    // the units of all jobs have to add up to an int32
    const int64_t tiles = std::min<int64_t>((static_cast<int64_t>(table_width) << a.page_shift) / 128, 1 << 24);
    a.side = heads_side(a.num_sms, a.h_kv);
    // (4 bits: 256 keys are a block for each of a CTA's four warps; cut at 128, two of them idle at a piece's end: 8 ragged
    // sequences 28.4 us, 26.8 so, 96 149 and 145)
    if (four && rows16) a.share_shift = 1;
    while (unsplit / a.side * (2 * (tiles >> a.share_shift) + 32) > 0x7FFFFFFFll)
      if (++a.share_shift > 16) return MLA_ERR_UNSUPPORTED;   // (four million jobs)
    grid = share_ctas(a.num_sms, a.h_kv);
    a.part_gap = static_cast<int>(grid) * (rows16 ? skv::kRowRows : skv::kTileRows);
  }
  skv::KvScales scales = {};
  if (four)
    scales = {static_cast<const uint8_t*>(pages->k_scales), static_cast<const uint8_t*>(pages->v_scales), pages->scale_page_stride,
              pages->scale_head_stride};
  st = cuda_status(rows16 && four ? skv::launch_attn_row4(tk, tv, tks, tvs, a, job_rows(plan->row_kernel), grid, cs)
                   : rows16       ? skv::launch_attn_row(tk, tv, a, plan->dtype, grid, cs)
                   : four         ? skv::launch_attn_tile4(tq, tk, tv, a, scales, grid, cs)
                                  : skv::launch_attn_tile(tq, tk, tv, a, plan->dtype, grid, cs));
  if (st != MLA_OK || a.num_splits == 1) return st;
  return cuda_status(skv::launch_attn_combine(a, rows16 ? skv::kRowRows : skv::kTileRows, cs));
}

int sdpa_prompt(int batch, int h_q, int h_kv, int d, int dtype, int total_q, int64_t total_kv, const void* q,
                int64_t q_token_stride, int64_t q_head_stride, const void* k, const void* v, int64_t kv_token_stride,
                int64_t kv_head_stride, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                const float* descale_q, const float* descale_k, const float* descale_v, float sm_scale, int out_dtype,
                float out_inv_scale, void* out, float* lse_out, float* amax_out, void* stream) {
  int st = check_heads(batch, h_q, h_kv, d, dtype);
  if (st == MLA_OK && dtype == SDPA_E2M1) st = MLA_ERR_UNSUPPORTED;   // (a form of caches; kv_pages_read gives bf16 rows)
  if (st != MLA_OK) return st;
  if (total_q < 1 || total_kv < 1 || total_kv > 0x7FFFFFFFll) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(total_q) * h_q > 0x7FFFFFFFll) return MLA_ERR_INVALID_ARG;
  if (q == nullptr || k == nullptr || v == nullptr || cu_seqlens_q == nullptr || cu_seqlens_kv == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(k, 16) || !ptr_aligned(v, 16) ||
      !words_ok({cu_seqlens_q, cu_seqlens_kv, descale_q, descale_k, descale_v, lse_out, amax_out}))
    return MLA_ERR_INVALID_ARG;
  const int e = elem_size(dtype);
  if (!stride_ok(q_token_stride, e) || !stride_ok(q_head_stride, e) || !stride_ok(kv_token_stride, e) ||
      !stride_ok(kv_head_stride, e))
    return MLA_ERR_INVALID_ARG;
  if (!out_ok(out, out_dtype, out_inv_scale) || !std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  skv::DeviceInfo dev;
  if ((st = skv::current_device(&dev)) != MLA_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (amax_out != nullptr && (st = cuda_status(cudaMemsetAsync(amax_out, 0, sizeof(float), cs))) != MLA_OK) return st;
  skv::AttnArgs a{};
  a.q = q;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.cu_q = cu_seqlens_q;
  a.cu_kv = cu_seqlens_kv;
  a.descale_q = descale_q;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  a.batch = batch;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.group = h_q / h_kv;
  a.total_q = total_q;
  a.total_kv = static_cast<int>(total_kv);
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_dtype = out_dtype;
  a.inv_scale = out_inv_scale;
  a.lse_out = lse_out;
  a.amax = amax_out;
  a.num_splits = 1;
  a.num_sms = dev.num_sms;
  a.status = dev.status;
  a.wait_limit_ns = skv::wait_limit_ns();
  a.drain_limit_ns = skv::drain_limit_ns();
  CUtensorMap tq, tk, tv;
  if ((st = encode_q(&tq, dtype, q, q_token_stride, q_head_stride, h_q, a.group, total_q)) != MLA_OK ||
      (st = encode_kv(&tk, dtype, k, total_kv, kv_token_stride, 1, kv_token_stride, h_kv, kv_head_stride, 128)) != MLA_OK ||
      (st = encode_kv(&tv, dtype, v, total_kv, kv_token_stride, 1, kv_token_stride, h_kv, kv_head_stride, 128)) != MLA_OK)
    return st;
  const int64_t grid = tiles_bound(total_q, batch, 2 * (128 / a.group)) * h_kv;
  return cuda_status(skv::launch_attn_tile(tq, tk, tv, a, dtype, grid, cs));
}

}  // extern "C"
