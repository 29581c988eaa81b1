// params.cuh -- parameter blocks passed from the host ABI to the kernels,
// and the launch functions of each kernel file.
#pragma once

#include <utility>

#include "mla_device.cuh"

namespace mla {

// Element type of the cached rows (mla_cache_dtype): bf16 values, INT8 codes
// with a per-token (scale, zero point), FP8 E4M3 codes with a per-token
// scale, or FP4 E2M1 codes with a power-of-two scale per 32 values in the row.
enum CacheCode : int { kCodeBf16 = 0, kCodeInt8 = 1, kCodeE4m3 = 2, kCodeE2m1 = 3 };

// FP4 rows (MLA_CACHE_FP4): 18 blocks of 32 codes, 16 bytes each, then their
// scale bytes (2^(byte - 127); 255: NaN), then zeros up to whole sectors.
constexpr int kFp4Blocks = kRow / 32;        // 18
constexpr int kFp4Scales = kFp4Blocks * 16;  // offset of the scale bytes: 288
constexpr int kFp4RowBytes = 320;

// Bytes of one cached row without per-token parameters kept elsewhere.
constexpr int cache_row_bytes(int code) {
  return code == kCodeBf16 ? 2 * kRow : code == kCodeE2m1 ? kFp4RowBytes : kRow;
}

// Multi-token decode (q_len query tokens per sequence) runs the same kernels
// over "rows": row v = t * heads_w + h of a sequence is query token t, head
// h.  `heads` below counts rows (q_len * heads_w); the weights have heads_w
// heads and row v uses head v % heads_w.
struct AbsorbParams {
  const __nv_bfloat16* q_nope;  // [B, heads, 128]
  const __nv_bfloat16* q_pe;    // [B, heads, 64]
  const __nv_bfloat16* W_UK;    // [heads_w, 128, 512]
  __nv_bfloat16* q_full;        // [B, H, 576] (fp16 bit patterns for 1-byte caches)
  float* q_sum;                 // [B, H, kQSumParts]
  // plan
  const int* seq_lens;
  int* tile_start;
  int* seg_base;
  int* len_checked;
  int* status;
  int batch, heads, heads_w, max_len, num_splits;
  int reset_status;  // 1: the plan starts the call's status word at MLA_OK (0: a kernel before it did)
  // The absorption GEMM's view of the rows: row v = t * heads_w + h of
  // sequence b is column b * q_len + t of weight head h, so each head's
  // product covers every (sequence, token) column at once; cols = batch *
  // q_len, q_nope / q_full / q_sum rows are at (column * heads_w + h).
  int cols;
};

// Sparse (top-k) decode: the listed rows of each sequence, compacted in list
// order into pages_per_seq pages of the gathered cache (sequence b owns pages
// [b pages_per_seq, (b + 1) pages_per_seq)), its length and page-table row.
struct GatherParams {
  const void* cache;         // bf16, int8 or e4m3 [num_pages, P, 576], or FP4 rows [num_pages, P, 320 bytes]
  const float* scale_zero;   // [num_pages, P, 2] (INT8) or [num_pages, P] (FP8)
  const int* block_table;    // [B, max_pages]
  const int* seq_lens;       // [B]
  const int* indices;        // [B, top_k], -1 = padding
  void* out_cache;           // [B * pages_per_seq, P, 576]
  float* out_scale_zero;     // [B * pages_per_seq, P, 2] (INT8) or [.., P] (FP8)
  int* out_table;            // [B, pages_per_seq]
  int* out_lens;             // [B]
  int* status;               // MLA_ERR_DEVICE_BOUNDS for bad entries (zeroed on the stream before the launch)
  int batch, top_k, max_pages, num_pages, page_size, pages_per_seq;
};

struct AppendParams {
  void* cache;                   // bf16, int8 or e4m3 [num_pages, P, 576], or FP4 rows [num_pages, P, 320 bytes]
  float* scale_zero;             // [num_pages, P, 2] (INT8) or [num_pages, P] (FP8)
  const int* block_table;        // [num_seqs, max_pages]
  const int* seq_ids;            // [N]   (chunk == 0)
  const int* positions;          // [N]   (chunk == 0)
  const int* seq_lens;           // [num_seqs] (chunk > 0: token i is token i % chunk of sequence
                                 // i / chunk, at position seq_lens[b] - chunk + i % chunk)
  int chunk;                     // 0: explicit seq_ids / positions; > 0: prefill chunk per sequence
  const __nv_bfloat16* c_kv;     // [N, 512]
  const __nv_bfloat16* k_pe;     // [N, 64]
  int* status;                   // optional
  double rope_theta;
  double inv_freq[kRope / 2];    // theta^(-2i/64), evaluated on the host in fp64
  uint64_t turn[kRope / 2];      // FP4: the fraction of inv_freq / (2 pi) in units of 2^-64
  int rotate;                    // FP4: rope_theta > 0
  int n_tokens, num_seqs, max_pages, num_pages, page_size;
  int run;                       // FP4: tokens of a warp (1 .. 32)
};

// Packed rows read back out of the cache (mla_cache_read).
struct CacheReadParams {
  const void* cache;         // bf16, int8 or e4m3 [num_pages, P, 576], or FP4 rows [num_pages, P, 320 bytes]
  const float* scale_zero;   // [num_pages, P, 2] (INT8) or [num_pages, P] (FP8)
  const int* block_table;    // [num_seqs, max_pages]
  const int* starts;         // [num_seqs] first position, or null: 0
  const int* cu_rows;        // [num_seqs + 1]
  __nv_bfloat16* c_kv;       // [n_rows, 512]
  __nv_bfloat16* k_pe;       // [n_rows, 64]
  int* status;               // optional
  int num_seqs, max_pages, num_pages, page_size, n_rows;
};

// Latents expanded to per-head keys and values (mla_expand_kv).
struct ExpandParams {
  const __nv_bfloat16* c_kv;  // [n_rows, 512]
  const __nv_bfloat16* W_UK;  // [heads, 128, 512]
  const __nv_bfloat16* W_UV;  // [heads, 128, 512]
  __nv_bfloat16* k_nope;      // [n_rows, heads, 128]
  __nv_bfloat16* v;           // [n_rows, heads, 128]
  int* status;                // optional
  int n_rows, heads;
  int sm_count;               // sizes the grid
  int inject_wait_timeout;    // test hook: 16 bytes of the first streamed box never delivered
};

// Causal attention over packed prompts (mla_prompt_attention).  The plan
// kernel lists the work, longest first: one item per block of up to 256 query
// rows of a sequence, or several over parts of its keys where there are few
// blocks; the attention kernel runs every item for every head.
struct alignas(16) PromptItem {
  int q_row0, rows;      // first packed token and number of rows (1..256): row i is token i >> pack, head i mod 2^pack
  int k_row0;            // first packed key row of the sequence
  int vis0;              // keys that row 0 sees (row i sees vis0 + (i >> pack); none if that is <= 0)
  int kv_begin, kv_end;  // key range of this item, relative to k_row0
  int pieces, piece;     // items that share the block's keys, and which one this is
  int partial;           // pieces > 1: first partial row of the block
  int head;              // the unit's head (in the attention kernel's copy)
  int pad[2];
};
struct PromptSplit {     // a block whose keys are split, for the merge
  int q_row0, rows, pieces, partial;
  int row_start;         // rows of the split blocks before
};
constexpr int kPromptRows = 256;         // query rows of a block
constexpr int kPromptMaxPieces = 32;     // pieces of one block
constexpr int kPromptMaxSplit = 512;     // blocks of a call that may be split
constexpr int kPromptExtraItems = 512;   // items beyond one per block
// partial rows of one call: two rounds of blocks on 152 SMs
constexpr int kPromptPartialRows = 2 * 152 * kPromptRows;
struct PromptParams {
  const int* cu_q;           // [num_seqs + 1]
  const int* cu_k;           // [num_seqs + 1]
  const __nv_bfloat16 *q_nope, *q_pe, *k_nope, *k_pe, *v;
  __nv_bfloat16* out;        // [n_q, heads, 128]
  float* lse_out;            // [n_q, heads] or null
  int* status;               // workspace: status word, items, units taken, split blocks and their rows
  int* seq_first;            // workspace: [num_seqs] first item of each sequence
  int* block_start;          // workspace: [num_seqs + 1] first block of each sequence
  PromptItem* items;         // workspace: [(n_q << pack) / 256 + num_seqs + kPromptExtraItems]
  PromptSplit* splits;       // workspace: [kPromptMaxSplit]
  float* partial_o;          // workspace: [partial_rows][128] unnormalised outputs
  float2* partial_ml;        // workspace: [partial_rows] reference maximum (unscaled) and sum
  int n_q, n_k, num_seqs, heads, kv_heads, sm_count, partial_rows;
  int may_split;             // keys may be split (set by the launch)
  int pack, heads_v;         // log2 of the heads packed into rows, and heads >> pack
  float scale_log2;          // softmax_scale * log2(e)
  float scale;
  int inject_wait_timeout;   // test hook: 16 bytes of the first key tile never delivered
};

struct CombineUVParams {
  const float* partial_o;     // [NSEG, H, 512]
  const float* partial_lse;   // [NSEG, H]
  const int* seg_base;        // [B + 1]
  const __nv_bfloat16* W_UV;  // [heads_w, 128, 512]
  __nv_bfloat16* out;         // [B, heads, 128]
  float* lse_out;             // [B, heads] or null
  int* status;
  int batch, heads, heads_w;
  int q_len;                  // rows per sequence = q_len * heads_w; column c = b * q_len + t
  int sm_count;               // sizes the grid
};

struct CombineParams {
  const float* partial_o;    // [B, S, H, D]
  const float* partial_lse;  // [B, S, H]
  float* o_lat;              // [B, H, D]
  float* lse_out;            // [B, H] or null
  int batch, splits, heads, dim;
};

cudaError_t launch_absorb(const AbsorbParams& p, bool fp16_out, cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, int code, cudaStream_t stream);
cudaError_t launch_combine_uv(const CombineUVParams& p, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheReadParams& p, int code, cudaStream_t stream);
cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream);
cudaError_t launch_prompt_attention(PromptParams p, cudaStream_t stream);
cudaError_t launch_gather(const GatherParams& p, int code, cudaStream_t stream);
cudaError_t launch_decode_tc(const DecodeParams& p, int hc, int code, int grid, cudaStream_t stream);
int decode_head_group(int heads, bool byte_cache);
// FP4 caches, groups of 16 or 32 query rows: one CTA per SM.
cudaError_t launch_decode_fp4(const DecodeParams& p, int hc, int grid, cudaStream_t stream);
// Launches `kernel` with programmatic dependent launch (and, if cluster_x > 1,
// thread-block clusters of cluster_x CTAs).  The kernels of the decode step
// (append, absorb, attention, merge + up-projection) set up their shared
// memory, barriers and tensor memory, then call griddep_wait() before their
// first global-memory access and griddep_launch_dependents() after it, so
// each launch and prologue overlaps the tail of the kernel before it.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              unsigned cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster_x;
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// bf16 caches: CTA-cluster kernel.  Capacity = clusters resident at once (0 if none).
int decode_pair_capacity(int hc);
cudaError_t launch_decode_pair(const DecodeParams& p, int hc, int clusters_per_group, cudaStream_t stream);
// Groups of 128 query rows, any cache format (CacheCode): CTA-pair kernel
// with the rows on the MMA's M extent.  Capacity = pairs resident at once (0 if none).
int decode_rows128_capacity(int code);
cudaError_t launch_decode_rows128(const DecodeParams& p, int code, int clusters_per_group, cudaStream_t stream);

}  // namespace mla
