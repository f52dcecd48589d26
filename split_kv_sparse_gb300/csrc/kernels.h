// Host-side launch interface between the C ABI (abi.cu) and the kernel
// translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace skv {

constexpr int kMlaHeads = 64;
constexpr int kMlaDqk = 576;
constexpr int kMlaDv = 512;
constexpr int kMlaBlockRows = 64;   // top-k entries per block (split unit and pipeline step)

// Per-launch arguments of the sparse-MLA decode kernel (split or direct epilogue).
struct MlaArgs {
  const uint8_t* kv;    // [n_kv][576] bf16 rows of 1152 B
  const int32_t* idx;   // [s_q][topk]
  int s_q;
  int topk;
  int n_kv;
  int num_splits;       // uniform schedule: splits per token (1 for the direct path)
  int num_blocks;       // ceil(topk / 64): 64-row blocks per token
  int dim_groups;       // uniform schedule: CTAs per (token, split) job (1, 2 or 4); CTA
                        // g of a job computes the same scores and softmax and the
                        // output dims [512 g / dim_groups, 512 (g + 1) / dim_groups)
  int sched;            // 0: (token, split) jobs, grid s_q * num_splits * dim_groups;
                        // 1: balanced, the s_q * num_blocks blocks cut into num_ctas
                        //    near-equal contiguous ranges, one per CTA (grid num_ctas)
  int num_ctas;         // balanced schedule: CTAs (<= s_q * num_blocks)
  int direct_whole;     // a job that covers a whole token writes the final output
                        // (sink, cast, LSE, amax) instead of a partial
  int tail_first;       // uniform schedule with tail_splits > 0: tokens 0 .. tail_first - 1
  int tail_splits;      // run whole on CTAs 0 .. tail_first - 1; tokens tail_first .. s_q - 1
                        // are cut into tail_splits splits, CTA tail_first + k running split
                        // k % tail_splits of tail token k / tail_splits, whose partial goes to
                        // slot (split, tail token) of the workspace (needs num_splits ==
                        // dim_groups == 1); 0: no tail
  int check_idx;        // 1: a loader that meets an index outside {-1} and [0, n_kv) sets
                        // status bit 0x10 (the row stays masked either way)
  int tail_dgroups;     // uniform schedule, tail_splits == 0: tokens tail_first .. s_q - 1 run
                        // whole on tail_dgroups (2 or 4) CTAs each, CTA tail_first + k taking
                        // dim group k % tail_dgroups of tail token k / tail_dgroups and
                        // writing its final rows (needs num_splits == dim_groups == 1); 0: no
  float scale_log2;     // sm_scale * log2(e)
  // Partial workspace: [slot][s_q][64][512] and [slot][s_q][64]. Uniform: slot =
  // the split. Balanced: slot = a piece's place among the pieces of its token
  // (a token cut by range boundaries); whole tokens write their final rows.
  float* o_acc;         // fp32, or bf16 values when partial_bf16
  float* lse_acc;
  int partial_bf16;     // O partials stored as bf16 (LSE partials stay fp32)
  // direct path: final output
  void* out;            // [s_q][64][512] of out_dtype
  int out_dtype;
  float inv_scale;
  float* lse_out;       // [s_q][64] or null
  const float* sink;    // [64] or null
  float* amax;          // scalar or null (zeroed by the launcher)
  uint32_t* status;     // device status words [2]
  uint64_t wait_limit_ns;   // a pipeline wait that runs longer records a timeout and aborts the CTA
  uint64_t drain_limit_ns;  // how long an aborting CTA waits for its own copies and MMAs in flight
};

// Balanced schedule arithmetic, shared by the host and the decode kernel: U
// units (64-row blocks, token-major) cut into P contiguous ranges, the first
// U % P of them one unit longer. Requires 1 <= P <= U.
__host__ __device__ inline int bal_begin(int p, int U, int P) {
  const int base = U / P, rem = U % P;
  return p * base + (p < rem ? p : rem);
}
// The range (CTA) that holds unit u.
__host__ __device__ inline int bal_cta_of(int u, int U, int P) {
  const int base = U / P, rem = U % P;
  const int big = rem * (base + 1);
  return u < big ? u / (base + 1) : rem + (u - big) / base;
}

// Dynamic shared memory the MLA decode kernel needs.
int mla_decode_smem_bytes();
// One-time per-device set-up (shared-memory opt-in of the kernels); called by the
// ABI the first time it sees a device, outside any stream capture.
cudaError_t prepare_mla_kernels();
cudaError_t prepare_sdpa_kernels();

// tm_q: Q viewed as 2-D [s_q*64 rows][576] bf16, box 64x64, 128B swizzle.
cudaError_t launch_mla_decode(const CUtensorMap& tm_q, const MlaArgs& a, cudaStream_t stream);

// Log-sum-exp combine over `rows` output rows of width d (512 or 128).
struct CombineArgs {
  const float* o_acc;   // [S][rows][d], fp32 or (partial_bf16) bf16 values
  const float* lse_acc; // [S][rows]
  int partial_bf16;
  int num_splits;
  int rows;             // tokens * heads
  int heads;            // head index = row % heads (for the sink)
  int d;
  const float* sink;    // [heads] or null
  void* out;
  int out_dtype;
  float inv_scale;
  float* lse_out;       // [rows] or null
  float* amax;          // scalar or null
  // Balanced sparse-MLA schedule (bal_ctas > 0): row r belongs to token r / heads,
  // whose split count is the number of CTA ranges its bal_nb blocks fall in (the
  // blocks of all tokens, bal_units of them, cut into bal_ctas ranges); a token in
  // one range was finished by the decode kernel and is left alone.
  int bal_nb, bal_units, bal_ctas;
  int num_sms;          // SMs of the device (caps the grid; 0: one CTA per 8 items)
  int sparse_splits;    // most split slots of most rows are empty (LSE -inf): load a
                        // slice only once its weight is known to be non-zero
};
// zero_amax: clear *amax first (a memset on the stream); pdl: launch as a
// programmatic dependent of the preceding kernel on the stream.
cudaError_t launch_combine(const CombineArgs& a, bool zero_amax, bool pdl, cudaStream_t stream);

// Bounded-wait self test: one CTA waits on a barrier nobody arrives on.
cudaError_t launch_wait_selftest(uint32_t* status, uint64_t limit_ns, cudaStream_t stream);

// Dense FP8 split-KV SDPA decode.
struct SdpaArgs {
  const uint8_t* q;             // [total_q][h_q][128] e4m3
  const int32_t* cu_q;          // [batch+1]
  const int32_t* cu_kv;         // [batch+1]
  const float* descale_q;       // device scalars or null
  const float* descale_k;
  const float* descale_v;
  int batch, h_q, h_kv, total_q, num_splits;
  int adaptive;                 // per-sequence split counts (<= num_splits) from the KV lengths
  int num_sms;                  // SM count the adaptive rule spreads the work over
  float scale_log2;
  float* o_acc;                 // split path [S][total_q][h_q][128]
  float* lse_acc;               // [S][total_q][h_q]
  void* out;                    // direct path [total_q][h_q][128]
  int out_dtype;
  float inv_scale;
  float* lse_out;
  float* amax;
  uint32_t* status;
  uint64_t wait_limit_ns;   // as in MlaArgs
  uint64_t drain_limit_ns;
};
int sdpa_decode_smem_bytes();
// tm_q: Q viewed as 3-D [total_q][h_q][128] e4m3, box {128 d, group heads, 64/group tokens}.
// tm_k / tm_v: K and V viewed as 3-D [total_kv][h_kv][128] e4m3, box {128 d, 1 head, 128 keys}.
cudaError_t launch_sdpa_decode(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const SdpaArgs& a, bool direct, cudaStream_t stream);

// Attention of packed queries over a paged cache or over packed K and V.
constexpr int kByLength = 1, kShares = 2;   // rules of AttnArgs::adaptive
struct AttnArgs {
  const void* q;                // element (token, head, x) at token * q_ts + head * q_hs + x
  int64_t q_ts, q_hs;           // (K and V are read through tensor maps)
  const int32_t* table;         // paged: [batch][table_width]; null: packed
  int table_width, page_shift, num_pages;
  const int32_t* cu_q;          // [batch + 1]
  const int32_t* kv_lens;       // paged: [batch]
  const int32_t* cu_kv;         // packed: [batch + 1]
  const float* descale_q;       // device scalars or null
  const float* descale_k;
  const float* descale_v;
  int kv_wide;                  // tile kernel, bf16 pages: tm_k / tm_v take both 64-dim column blocks of a row in one box
                                // (1: heads beside one another in a row, 2: pages of one head after the other)
  int batch, h_q, h_kv, group, total_q;
  int total_kv;                 // packed
  float scale_log2;
  void* out;                    // [total_q][h_q][128]
  int out_dtype;
  float inv_scale;
  float* lse_out;
  float* amax;
  int num_splits;               // the most splits a sequence gets
  int adaptive;                 // its count follows from the lengths: kByLength or kShares (0: exactly num_splits)
  int num_sms;                  // jobs of one wave, over which the adaptive rules spread the work
  int max_slots;                // split jobs that the workspace holds
  int side;                     // kShares: KV heads whose CTAs walk the same keys side by side
  int share_shift;              // kShares: log2 of the key tiles of a unit of work
  int part_gap;                 // kShares: rows that a sequence's splits after its first lie nearer to the front
  float* o_part;                // num_splits > 1: partial rows [slot][rows of a job][128], normalised
  float* lse_part;              // their log2 LSE
  int2* row_map;                // [total_q][h_kv]: first partial row of the token's group, and its split
                                // count (0: the final rows were written)
  uint32_t* status;
  uint64_t wait_limit_ns, drain_limit_ns;   // as in MlaArgs
};
// Query rows (tokens x group) and partial rows per job of each kernel.
constexpr int kTileRows = 256;
constexpr int kRowRows = 16;
// Split jobs of the tile kernel that an automatic plan's workspace holds, in waves.
constexpr int kTileSplitWaves = 3;
// tm_q: Q as 3-D [total_q][h_q][128], box {128 bytes, group heads, 128 / group tokens}; tm_k / tm_v: K and V as 4-D
// {128, rows, pages, heads} (packed: one page of total_kv rows), box {128 bytes, min(page, 128) rows, 1, 1}; with
// kv_wide as 5-D {64, 8 rows, column blocks, row groups, pages}, box {64, 8, 2, min(page, 128) / 8, 1}.
cudaError_t launch_attn_tile(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const AttnArgs& a, int dtype, int64_t grid, cudaStream_t stream);
// 4-bit pages. tm_k / tm_v: codes, box {64 bytes, min(page, 128) rows, 1, 1}, 64-byte swizzle.
struct KvScales {
  const uint8_t *k, *v;
  int64_t page_stride, head_stride;   // bytes; a row is 8
};
cudaError_t launch_attn_tile4(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a,
                              const KvScales& scales, int64_t grid, cudaStream_t stream);
// Box of tm_k / tm_v: {128 bytes, attn_row_box(dtype, page size) rows, 1, 1}.
cudaError_t launch_attn_row(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a, int dtype,
                            int64_t grid, cudaStream_t stream);
int attn_row_box(int dtype, int page_size);
// 4-bit pages; rows: of a job, 8 or 16. tm_k / tm_v as in launch_attn_tile4, boxes of min(page, kRow4Box) rows; tm_ks / tm_vs: scales
// as 4-D {rows * 2 words, 1, pages, heads}, boxes of as many rows.
cudaError_t launch_attn_row4(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_ks, const CUtensorMap& tm_vs,
                             const AttnArgs& a, int rows, int64_t grid, cudaStream_t stream);
constexpr int kRow4Box = 64;
// CTAs of the row kernel that an SM holds.
constexpr int kRowCtasPerSm = 2;
// Folds the partial rows of every split token; a.num_splits > 1. rows_per_slot: kTileRows or kRowRows.
cudaError_t launch_attn_combine(const AttnArgs& a, int rows_per_slot, cudaStream_t stream);

struct PagesMapArgs {
  int batch, page_size;
  const int32_t* held;
  const int32_t* lens;
  const int32_t* cu_q;
  int total_q;
  int32_t* table;
  int width;
  int32_t* free_pages;
  int capacity;
  const int32_t* free_in;
  int32_t* free_out;
  int64_t* slots;
  int32_t* positions;           // or null
};
cudaError_t launch_pages_map(const PagesMapArgs& a, cudaStream_t stream);

struct PagesWriteArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t token_stride, head_stride;
  const int64_t* slots;
  int64_t rows;
  void* k;
  void* v;
  int64_t page_stride, row_stride, cache_head_stride;
  int64_t num_slots;
  int page_shift, h_kv;
  const float* descale_k;
  const float* descale_v;
};
cudaError_t launch_pages_write(const PagesWriteArgs& a, int dtype, cudaStream_t stream);

// Rows with arithmetic on the way: the append that rotates, the append into 4-bit pages, the read-back.
struct PagesAppendArgs {
  const uint16_t* q;            // [rows][h_q][128] (h_q may be 0)
  int64_t q_ts, q_hs;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t token_stride, head_stride;
  const int64_t* slots;
  int64_t rows;
  int h_q, h_kv;
  const int32_t* positions;     // null: no rotation
  const float* cos_sin;         // [num_positions][rot]: rot / 2 cosines, then the sines
  int64_t num_positions;
  int rot, interleaved;
  void* q_out;                  // bf16, or e4m3 codes
  int q_out_e4m3;
  int64_t qo_ts, qo_hs;
  uint16_t* k_out;              // append: rotated rows of k, or null; read: rows of k
  uint16_t* v_out;              // read: rows of v, of k_out's strides
  int64_t ko_ts, ko_hs;
  void* k;
  void* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int64_t page_stride, row_stride, cache_head_stride;   // (4-bit pages: in bytes)
  int64_t scale_page_stride, scale_head_stride;
  int64_t num_slots;
  int page_shift;
  int num_sms;
  const float* descale_q;
  const float* descale_k;
  const float* descale_v;
};
// dtype: of the cache.
cudaError_t launch_pages_append(const PagesAppendArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_pages_read(const PagesAppendArgs& a, int dtype, cudaStream_t stream);

cudaError_t prepare_paged_kernels();
cudaError_t prepare_attn_tile();
cudaError_t prepare_attn_row();
cudaError_t prepare_attn_row4();

}  // namespace skv
