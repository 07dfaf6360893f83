// Host-side launchers of the paged-attention kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"

namespace pa {

// Cache types, numbered as pa_kv_dtype.
constexpr int kKvBf16 = 0, kKvE4m3 = 1, kKvFp4 = 2;

// Split-KV launch geometry: grid = (max_partitions, num_kv_heads, num_seqs).
struct Launch {
  int head_dim;
  int group;  // num_q_heads / num_kv_heads
  bool fp8;
  cudaStream_t stream;
  int kv = kKvBf16;  // cache type (fp8: kv == kKvE4m3)
  int form = kFormAll;
  bool join = false;  // a row's partitions are one cluster, which joins them (no partials, no merge)
};
constexpr int kJoinCtas = kJoinMax;      // partitions of a cluster at most (the portable size)
// Bytes of kept scores of a CTA at most: they take room from the ring stages of other CTAs (64 contexts of up to 16384
// tokens, bf16, 32 KB of scores a CTA: 428 us where scores in scratch take 392).
constexpr int kJoinScores = 8 << 10;

// Each returns cudaSuccess or the launch error.  Unsupported combinations return
// cudaErrorInvalidConfiguration (the caller has already checked them).
cudaError_t launch_decode(const AttnParams& p, const Launch& l);
// Decode on mma.sync (same grid, partitions and partial layout as launch_decode): E4M3 caches for
// every group, bf16 caches for groups of 1, 2 and 4.  tk / tv: 2-D TMA maps of the K and V pools
// viewed as [num_blocks * Hkv * bs, d] with 16-row boxes of 128-byte rows and the 128-byte swizzle
// (bf16: 64-dim boxes, as for verify; E4M3 d = 128: one box per page), or for E4M3 d = 64 one box
// of 64-byte rows with the 64-byte swizzle.
cudaError_t launch_decode_mma(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
// Verify: planner + persistent tcgen05 kernel + segment merge, all on l.stream.  `scratch` holds
// verify_scratch_bytes(...) bytes; ncta = verify_resident_ctas(num_sms) persistent CTAs.
// tk / tv: 2-D TMA maps of the bf16 K and V pools viewed as [num_blocks * Hkv * bs, d] with
// 16 x 64 boxes and the 128-byte swizzle.
int verify_resident_ctas(int num_sms);
size_t verify_scratch_bytes(int num_seqs, int q_len, int num_q_heads, int num_kv_heads, int head_dim, int ncta);
cudaError_t launch_verify_tc(const AttnParams& p, const Launch& l, void* scratch, int ncta, const CUtensorMap& tk,
                             const CUtensorMap& tv);
cudaError_t launch_merge(const AttnParams& p, const Launch& l);
// Paged prefill (varlen queries, p.query_start_loc / p.total_q set; p.q_len = the host bound on
// any sequence's new rows): a planner orders the (sequence, 128-row tile) pairs by work, then one
// tcgen05 CTA per (kv head, pair).  scratch holds prefill_scratch_bytes(...) bytes.
size_t prefill_scratch_bytes(int num_seqs, int max_q_len, int group);
// Verify / tree verify (p.tree_mask) with bf16 caches and 65-128 rows per kv head on the prefill
// kernel split like decode: grid (partition, kv head, sequence) from p.pages_per_partition (a
// multiple of 4 pages) / p.max_partitions, partials in p.part_o / p.part_lse for launch_merge.
cudaError_t launch_verify_split(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t launch_prefill_tc(const AttnParams& p, const Launch& l, int max_q_len, void* scratch, const CUtensorMap& tk,
                              const CUtensorMap& tv);
// Its parts: the planner's work list, and the tile kernel's forms with a window and over 4-bit caches
// (tiles null: the split form).
cudaError_t launch_prefill_plan(const AttnParams& p, int tiles_per_row, int32_t* tiles, cudaStream_t st);
cudaError_t prefill_window_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles,
                                const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t prefill_fp4_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles);
// A few rows per kv head (group * q_len at most kRowsMax, bf16 kRowsMaxBf16) on mma.sync: 4-bit caches, and window forms of
// bf16 and E4M3 caches; same grid, partitions (any page count) and partials as launch_decode_mma.
constexpr int kRowsMax = 32, kRowsMaxBf16 = 16;
// CTAs of it that share an SM, by the rows per kv head (its accumulators' registers).
constexpr int rows_resident_ctas(int rows) { return rows <= 8 ? 4 : rows <= 16 ? 3 : 2; }
cudaError_t rows_fp4_form(const AttnParams& p, const Launch& l);
cudaError_t rows_window_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
// The forms over listed blocks, over what lies behind a shared prefix and with kept scores: of the decode kernel, the
// rows kernel (every cache type) and the tile kernel (more rows than that takes).
cudaError_t decode_blocks_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t decode_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t decode_scores_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t rows_blocks_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t rows_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t rows_scores_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
cudaError_t tiles_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
// The shared prefixes of p.num_groups groups, in at most prefix_tiles(...) tiles of 128 rows (prefix_tile_tokens new tokens) per
// kv head: a bound without the groups' sizes, as each but one may leave a tile part full.
int prefix_tile_tokens(int group);
int prefix_tiles(int num_seqs, int q_len, int group, int num_groups);
cudaError_t launch_prefix(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv);
// KV append (bf16 scatter, fp8 with per-(block, head) rescaling, or E2M1 codes with a scale for each
// 16 dims of a token); arguments already checked.
cudaError_t launch_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                          const int32_t* block_table, const int32_t* context_lens, int num_seqs, int n_new,
                          int max_blocks_per_seq, int num_blocks, int num_kv_heads, int head_dim, int kv_dtype,
                          float* k_scale, float* v_scale, unsigned* err, cudaStream_t stream);

// Read the last n tokens of every sequence back as bf16 rows; arguments already checked.
struct ReadParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_table;
  const int32_t* context_lens;
  const float* k_scale;   // as the cache type's (E2M1: [Hkv] or null)
  const float* v_scale;
  __nv_bfloat16* k_out;   // [B, n, Hkv, d]
  __nv_bfloat16* v_out;
  unsigned* err;
  int num_seqs, n, max_blocks_per_seq, num_blocks, num_kv_heads;
};
cudaError_t launch_read_kv(const ReadParams& p, int head_dim, int kv_dtype, cudaStream_t st);

// Bounds of the keys of each block that holds one of a sequence's last n tokens; arguments already checked.
struct BoundsParams {
  const uint8_t* k_cache;
  const int32_t* block_table;
  const int32_t* context_lens;
  const float* k_scale;   // as the cache type's (E2M1: [Hkv] or null)
  int8_t* bounds;         // [NB, Hkv, 2, d]: codes of the largest, then of the smallest
  float* bound_scale;     // [NB, Hkv]: a power of two
  unsigned* err;
  int num_seqs, n, max_blocks_per_seq, num_blocks, num_kv_heads;
};
cudaError_t launch_block_bounds(const BoundsParams& p, int head_dim, int kv_dtype, int num_sms, cudaStream_t st);

// The highest-scoring blocks of each (sequence, kv head).  scratch holds select_scratch_bytes(...) bytes.
struct SelectParams {
  const __nv_bfloat16* q;       // [B, q_len, Hq, d]
  const int8_t* bounds;
  const float* bound_scale;
  const int32_t* block_table;
  const int32_t* context_lens;
  int32_t* blocks;              // [B, Hkv, count]
  float* scores;                // [B, Hkv, max_cols]
  unsigned* err;
  int num_seqs, q_len, num_q_heads, num_kv_heads, max_blocks_per_seq, num_blocks, max_context_len, max_cols;
  int count, sinks, recent;     // in blocks
};
constexpr int kSelectMaxRows = 32;  // q_len * group
size_t select_scratch_bytes(int num_seqs, int num_kv_heads, int max_context_len, int num_sms);
cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, int num_sms, cudaStream_t st);

// The step's softmax weights from the kept scores and the rows' log2-sum-exps, folded into the tokens' sums.
struct WeightParams {
  const float* scores;          // [B, Hkv, max_context_len, G]
  const float* lse;             // [B, Hq]
  float* weights;               // [NB, Hkv, 16]
  const int32_t* block_table;
  const int32_t* context_lens;
  int num_seqs, num_kv_heads, group, max_blocks_per_seq, num_blocks, max_context_len;
  float decay;
};
cudaError_t launch_fold_weights(const WeightParams& p, cudaStream_t st);

// Eviction: the tokens of the largest sums move to the blocks of new_table.  scratch holds evict_scratch_bytes(...).
struct EvictParams {
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;               // E4M3: [NB, Hkv]
  float* v_scale;
  float* weights;               // [NB, Hkv, 16]
  const int32_t* block_table;
  const int32_t* context_lens;
  const int32_t* new_table;     // [B, new_blocks]
  int32_t* new_lens;            // [B]
  int32_t* kept;                // scratch: [B, Hkv, keep] positions, then the keys of long contexts
  unsigned* err;
  int num_seqs, max_blocks_per_seq, new_blocks, num_blocks, num_kv_heads, max_context_len, keep, sinks, recent;
};
size_t evict_scratch_bytes(int num_seqs, int num_kv_heads, int keep, int max_context_len);
cudaError_t launch_evict(const EvictParams& p, int head_dim, int kv_dtype, int num_sms, cudaStream_t st);

// RMS norm and rotation of the query and key head rows; strides in elements between tokens.
struct RopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* q_weight;  // [d]
  const __nv_bfloat16* k_weight;
  const float* cos_sin;           // [max_position, rotary]
  const int32_t* positions;       // [T]
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  unsigned* err;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int num_tokens, num_q_heads, num_kv_heads, rotary, max_position;
  float eps;
};
cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, bool interleaved, cudaStream_t st);

// Speculative acceptance: scan kernel over vocabulary chunks, then the pick kernel (programmatic
// dependent).  chunk_sums holds accept_scratch_bytes(num_seqs, vocab) bytes.
size_t accept_scratch_bytes(int num_seqs, int vocab);
cudaError_t launch_accept(const float* p, const float* q, const int32_t* draft, const float* u_accept,
                          const uint32_t* words, int num_seqs, int num_draft, int vocab, int32_t* out_tokens,
                          int32_t* num_accepted, void* scratch, unsigned* err, cudaStream_t stream);
// Programmatic dependent launch of `fn` on `st` (cudaLaunchKernelExC with the
// programmatic-stream-serialisation attribute).
cudaError_t launch_pdl(const void* fn, dim3 grid, dim3 block, int smem, cudaStream_t st, void** args);

// launch_pdl for kernels whose every CTA waits (griddepcontrol.wait) before its first read of what the kernel before
// it wrote, and before it returns; and for those over own tokens, which read nothing of it and whose first CTA waits.
cudaError_t launch_dependent(const void* fn, dim3 grid, dim3 block, int smem, cudaStream_t st, void** args);

// Launch in clusters of `ctas` along x (at most 8).
cudaError_t launch_clusters(const void* fn, dim3 grid, dim3 block, int smem, int ctas, cudaStream_t st, void** args);

// Raise a kernel's dynamic shared-memory limit on the current device (first call per device
// and kernel only; later calls are a table lookup).
cudaError_t set_smem_once(const void* kernel, int bytes);

// Host-side argument checks of paged_attn_decode (a pa_status), and the current device's
// error-word address; neither allocates.
int validate_decode_args(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                         const int32_t* context_lens, int num_seqs, int max_blocks_per_seq, int num_blocks,
                         int max_context_len, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                         int block_size, int kv_dtype, const float* k_scale, const float* v_scale,
                         const void* out);
cudaError_t error_word_address(unsigned** out);

}  // namespace pa
