/*
 * paged_attn.h -- C ABI of the GB300 (sm_103a) paged-KV GQA attention library.
 *
 * Operation.  For every sequence b, new-token row i in [0, q_len) and query head h:
 *   g   = h / (num_q_heads / num_kv_heads)            GQA: contiguous groups of query heads
 *                                                       share one K/V head (studybook
 *                                                       fde-roadmap ch.10 "production latency
 *                                                       and cost", section 10.1.2)
 *   L   = context_lens[b]                              tokens in the cache, new ones included
 *   n   = L - q_len + i + 1                            causal: row i sees itself and everything
 *                                                       before it (sirzzang "Speculative
 *                                                       Decoding", parallel verification and
 *                                                       its causal-mask figure)
 *   k_j = K[block_table[b][j / bs], g, j % bs, :]      paged gather through the block table
 *   v_j = V[block_table[b][j / bs], g, j % bs, :]      (section 10.4.2, figure 10.4.2; aegloslab
 *                                                       servingai 5.3.7)
 *   s_j = scale * <q[b, i, h, :], k_j>,  j < n
 *   out[b, i, h, :] = sum_j softmax(s)_j v_j           attention over the cached K/V
 *                                                       (section 10.3.1), computed tile by tile
 *                                                       with an online softmax (10.1.2)
 * fp8 caches hold OCP E4M3 bytes; the value of a byte is e4m3(byte) * k_scale[block, g] (or
 * v_scale) with one fp32 scale per (physical block, kv head) -- the symmetric scale
 * quantisation of section 10.8.2.
 *
 * Layouts (row-major, contiguous, element sizes in brackets):
 *   q            [num_seqs, q_len, num_q_heads, head_dim]        bf16 [2]
 *   k_cache,
 *   v_cache      [num_blocks, num_kv_heads, block_size, head_dim] bf16 [2] or E4M3 [1]
 *   k_scale,
 *   v_scale      [num_blocks, num_kv_heads]                      fp32 [4]; NULL for bf16
 *   block_table  [num_seqs, max_blocks_per_seq]                   int32; entries past
 *                                                                 ceil(L / block_size) are
 *                                                                 never read
 *   context_lens [num_seqs]                                       int32
 *   out          [num_seqs, q_len, num_q_heads, head_dim]        bf16 [2]
 *
 * Ownership.  Every pointer argument is a device pointer owned by the caller; the library
 * never frees or retains one after the call returns.  Calls are asynchronous on `stream`
 * (a cudaStream_t; NULL is the legacy default stream) and do not synchronise it.
 *
 * Scratch.  When a sequence's context is split into several partitions the library keeps
 * per-partition partial results in stream-ordered scratch memory that it allocates from a
 * memory pool of its own (one per device) on `stream` and frees on `stream` after the merge.
 *
 * Errors.  Every entry point returns a pa_status.  Argument checks run on the host before any
 * launch; a failed check launches nothing.  PA_OK from an attention call means the kernels were
 * launched.  Conditions only the device can see (a block id outside [0, num_blocks), a
 * sequence with fewer than q_len tokens, an asynchronous copy that did not complete within
 * its wait limit) never fault: the affected page is skipped or the affected rows are written
 * as zeros, and a per-device error word records it for paged_attn_check_device_errors.
 */
#ifndef PAGED_ATTN_H_
#define PAGED_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,   /* a null pointer, a negative size, Hq % Hkv != 0, ...            */
  PA_ERR_UNSUPPORTED = 2,   /* a valid shape the kernels are not built for                     */
  PA_ERR_CUDA = 3,          /* a CUDA runtime call or a launch failed                          */
  PA_ERR_NO_MEMORY = 4,     /* the split-KV scratch could not be allocated                     */
  PA_ERR_DEVICE_BOUNDS = 5, /* device-side: a block id was out of range or a context too short */
  PA_ERR_DEVICE_TIMEOUT = 6, /* device-side: an asynchronous copy wait hit its iteration limit */
  PA_ERR_SCRATCH_LIMIT = 7   /* the static-scratch decode needs more than its fixed array      */
} pa_status;

typedef enum { PA_KV_BF16 = 0, PA_KV_FP8_E4M3 = 1, PA_KV_FP4_E2M1 = 2 } pa_kv_dtype;

/*
 * 4-bit caches (PA_KV_FP4_E2M1).  Each 16 consecutive dims of one token's head row are stored as 16
 * OCP E2M1 codes (two a byte, the lower dim in the low nibble) and one OCP E4M3 scale; the value of a
 * code is e2m1(code) * e4m3(scale) * k_scale[g] (or v_scale[g]), with one fp32 scale per kv head:
 *   k_cache, v_cache  [num_blocks, num_kv_heads, 16, 9 * head_dim / 16] bytes, 16-byte aligned.  A
 *                     (block, head) page of 9 * head_dim bytes holds the codes of its 16 tokens
 *                     (head_dim / 2 bytes each), then their scales (head_dim / 16 bytes each).
 *   k_scale, v_scale  [num_kv_heads] fp32, device, positive and finite; NULL means 1.  Static: a
 *                     value near amax / (6 * 448) over the head's expected keys (values) centres the
 *                     E4M3 scales.
 * Accepted by paged_attn_append_kv, paged_attn_read_kv, paged_attn_decode, paged_attn_verify,
 * paged_attn_tree_verify, paged_attn_prefill and the window forms.  Attention turns a page into f16
 * operands exactly (code * scale has at most six significant bits); q is re-encoded as f16 as for E4M3
 * caches, weights are f16, sums and softmax statistics fp32.  Decode and verify of up to 32 rows per kv
 * head run the rows kernel (mma.sync), anything else the prefill kernel.
 */

/*
 * Single-token decode for a continuous batch with ragged context lengths (studybook section
 * 10.2.2: one new token per step reads the whole cache; aegloslab servingai 5.3.1).
 *   q_len must be 1.  head_dim in {64, 128}; block_size 16; num_q_heads / num_kv_heads at most
 *   64; kv_dtype a pa_kv_dtype (k_scale/v_scale required for fp8, ignored for bf16).  max_context_len is a host-known upper bound of context_lens (it sizes the grid
 *   without reading device memory); it must not exceed max_blocks_per_seq * block_size.
 *   `scale` multiplies q.k (1/sqrt(head_dim) for standard attention).
 * Kernel: split-KV partitions (paged_attn_plan) merged by log-sum-exp; within a partition both
 * products run on the warp-level tensor-core instruction (mma.sync m16n8k16, fp32 accumulation,
 * the G heads as the columns of an 8-wide tile): bf16 caches in bf16, with each softmax weight
 * carried as a bf16 high part plus its rounded remainder (~16 significant bits); E4M3 caches
 * converted exactly to f16 pairs in registers, weights in f16 with each page's V scale folded in,
 * and q re-encoded as f16 after a power of two per query head that brings its largest |q| just
 * below 2^15 (exact for every element within 2^28 of the largest; the scores are scaled back),
 * so any bf16 q is accepted.  That kernel serves groups of 1, 2, 4 and
 * 8 query heads; any other group (3, 5, 7, 16, ...) runs the tcgen05 kernel of paged_attn_verify
 * with q_len = 1 (its balanced persistent split).
 */
int paged_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                      int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                      float scale, int kv_dtype, const float* k_scale, const float* v_scale,
                      void* out, void* stream);

/*
 * (K+1)-query causal verify forward of speculative decoding: the target scores the q_len =
 * K+1 newest tokens (K drafts plus the bonus position) in one call, row i masked to the
 * tokens up to itself (sirzzang "Speculative Decoding", parallel verification; aegloslab
 * servingai 5.3.9).  The new tokens' K/V must already be in the cache and context_lens counts
 * them.  Same arguments and limits as paged_attn_decode, with 1 <= q_len <= 16 and
 * (num_q_heads / num_kv_heads) * q_len <= 128 (rows beyond 64 per kv head -- e.g. 8 drafts under
 * groups of 8 -- run the chunked-prefill kernel, split into partitions like decode and merged
 * the same way).  bf16 caches run the products in bf16; E4M3 caches are converted exactly to
 * f16 in shared memory and the products run in f16 (each Q row re-encoded as f16 after the power
 * of two that keeps it in range, as for decode; each page's scales are applied to its scores and
 * weights), fp32 accumulation in both.
 */
int paged_attn_verify(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                      int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                      float scale, int kv_dtype, const float* k_scale, const float* v_scale,
                      void* out, void* stream);

/*
 * Tree verification: paged_attn_verify with the causal mask over the q_len new tokens replaced
 * by an ancestor mask, so that one forward scores a tree of draft branches (tree attention,
 * aegloslab servingai 5.3.13; Medusa-style candidate trees, sirzzang "Speculative Decoding").
 *   tree_mask [num_seqs, q_len] uint32, device: bit t of tree_mask[b * q_len + i] set means new
 *   token i attends to new token t (normally t = i and i's ancestors); every context token
 *   before the q_len new ones is visible to every row.  The chain mask (bits 0..i) reproduces
 *   paged_attn_verify.  A row whose mask and prefix are both empty comes out as zeros.
 * Same arguments, limits and errors as paged_attn_verify; a NULL tree_mask is
 * PA_ERR_INVALID_ARG.
 */
int paged_attn_tree_verify(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_table, const int32_t* context_lens,
                           const uint32_t* tree_mask, int num_seqs, int max_blocks_per_seq,
                           int num_blocks, int max_context_len, int q_len, int num_q_heads,
                           int num_kv_heads, int head_dim, int block_size, float scale,
                           int kv_dtype, const float* k_scale, const float* v_scale, void* out,
                           void* stream);

/*
 * Paged attention over packed, variable-length query rows: chunked prefill (a prompt chunk
 * attends to everything cached before it and causally within itself; aegloslab servingai 5.3.15,
 * Sarathi-style chunking with piggybacked decode) and, in the same call, decode (1 row) or verify
 * (K + 1 rows) sequences.  FlashAttention tiling with an online softmax (studybook fde-roadmap
 * ch.10, section 10.1.2) on the tensor cores, 128-row tiles of (token, query head) per kv head.
 *   q                [total_q, num_q_heads, head_dim] bf16, device, 16-byte aligned: sequence b's
 *                    new rows are q[query_start_loc[b] .. query_start_loc[b+1]).
 *   query_start_loc  [num_seqs + 1] int32, device, non-decreasing, query_start_loc[num_seqs] <=
 *                    total_q; q_len_b = query_start_loc[b+1] - query_start_loc[b] <= max_q_len.
 *   context_lens     [num_seqs] int32, device: cached tokens including the q_len_b new ones (their
 *                    K/V are in the cache: paged_attn_append_kv); new row i sees
 *                    context_lens[b] - q_len_b + i + 1 tokens.
 *   out              [total_q, num_q_heads, head_dim] bf16, device: written for every packed row.
 *   max_q_len        host-side bound on q_len_b (sizes the grid); total_q the rows of q and out.
 * Other arguments as paged_attn_decode.  Limits: bf16 or E4M3 KV (E4M3: k_scale / v_scale
 * required; pages converted exactly to f16 in shared memory, products in f16 with Q rows
 * re-encoded as in paged_attn_verify), head_dim 64 or 128, block_size 16, num_q_heads /
 * num_kv_heads in {1, 2, 4, 8}, at most 65536 sequences.  Device-side: a sequence whose rows fall outside
 * [0, total_q) or exceed max_q_len is skipped and flagged; rows that see no token (context
 * shorter than the new rows) come out as zeros and are flagged (PA_ERR_DEVICE_BOUNDS from
 * paged_attn_check_device_errors).  Asynchronous on `stream`; its work list (4 bytes per
 * (sequence, tile) pair) comes from the library's stream-ordered pool.  Returns PA_OK (also for
 * num_seqs == 0 or total_q == 0), PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_NO_MEMORY or
 * PA_ERR_CUDA.
 */
int paged_attn_prefill(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* context_lens,
                       const int32_t* query_start_loc, int num_seqs, int total_q, int max_q_len,
                       int max_blocks_per_seq, int num_blocks, int max_context_len,
                       int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                       float scale, int kv_dtype, const float* k_scale, const float* v_scale,
                       void* out, void* stream);

/*
 * Sliding window with sinks: paged_attn_decode, paged_attn_verify and paged_attn_prefill in which a
 * row that would see the n first tokens sees token j < n only when j >= n - window (the window counts
 * the row's own token) or j < sinks (the first tokens, which take the softmax's surplus mass when the
 * middle of a long context is dropped).
 *   window >= 1; sinks >= 0; either may exceed the context, which then hides nothing.
 * Block-table entries of blocks that no row of the sequence sees are not read: a caller may give such
 * blocks back to its pool and leave any value there.  A token that no row of a (sequence, 128-row
 * tile) sees does not reach the output even as NaN; one that some row of the tile sees must be finite.
 * Work and scratch are those of the visible tokens.  Same arguments, errors and limits otherwise, but
 * max_context_len at most 2^30.  Kernels: the decode kernel (groups of 1, 2, 4 and 8), the rows kernel
 * (verify rows and other groups of decode, up to 32 rows per kv head, 16 over bf16 caches: mma.sync, a
 * row for each column of its n-tiles) and the prefill kernel (beyond, split like decode); the pages that are left are
 * numbered without the gap.
 */
int paged_attn_window_decode(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                             int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int window, int sinks, float scale, int kv_dtype, const float* k_scale,
                             const float* v_scale, void* out, void* stream);
int paged_attn_window_verify(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                             int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int window, int sinks, float scale, int kv_dtype, const float* k_scale,
                             const float* v_scale, void* out, void* stream);
int paged_attn_window_prefill(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* context_lens,
                              const int32_t* query_start_loc, int num_seqs, int total_q,
                              int max_q_len, int max_blocks_per_seq, int num_blocks,
                              int max_context_len, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, int window, int sinks, float scale, int kv_dtype,
                              const float* k_scale, const float* v_scale, void* out, void* stream);

/*
 * Bounds of the keys of cache blocks, what paged_attn_select_blocks reads in place of the keys: for each
 * (block, kv head) the largest and the smallest value of every dim over the block's tokens, as int8 codes
 * times one power of two.
 *   e            the smallest integer with max|k| 2^-e <= 127 over the block's tokens and dims (at least
 *                -126; 0 where every key is 0).
 *   bounds       [num_blocks, num_kv_heads, 2, head_dim] int8, device, 16-byte aligned: ceil(max 2^-e) of every
 *                dim, then floor(min 2^-e).
 *   bound_scale  [num_blocks, num_kv_heads] fp32, device: 2^e.
 * Both are written for every block that holds one of a sequence's last n tokens (context_lens counts them;
 * n past the context: all of its blocks), from all of the block's stored tokens; the others stay as they are.
 * A step calls it after paged_attn_append_kv with the same n, a prompt once with its length.  k_cache, kv_dtype and
 * k_scale as in paged_attn_decode (a block that several sequences share is written for each of them: they must hold the
 * same tokens of it); the key of a scaled cache is its fp32 value (code, times the 16-dim scale of
 * a 4-bit one, times k_scale: one rounding).  Keys must be finite: a NaN gives way to the block's other tokens, an
 * infinity to the largest code.  Out-of-range block ids and contexts past the table are skipped and flagged.
 * Asynchronous on `stream`; never allocates.  Returns PA_OK (also for num_seqs == 0 or n == 0),
 * PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED or PA_ERR_CUDA.
 */
int paged_attn_block_bounds(const void* k_cache, const int32_t* block_table,
                            const int32_t* context_lens, int num_seqs, int n,
                            int max_blocks_per_seq, int num_blocks, int num_kv_heads, int head_dim,
                            int block_size, int kv_dtype, const float* k_scale, int8_t* bounds,
                            float* bound_scale, void* stream);

/*
 * The blocks of each sequence that a step's queries should read, by what their keys can come to.  A query
 * row is rounded (to nearest even) to int8 codes c times 2^f by the rule of the bounds, f from the row's largest
 * |q|; block j's score for it is 2^f 2^e sum_i (c_i > 0 ? c_i hi_i : c_i lo_i), and its score for a kv head the
 * largest over the head's rows (every new token, every query head of the group).  It is an upper bound of the rounded
 * row's product with every key of the block; the row's own q . k may pass it by half a code of the row, 2^f / 2, times
 * sum_i |k_i|.  The sum is a whole number
 * below 2^22: the selection does not depend on the order of the arithmetic (while the products of the powers of
 * two and those sums stay between 2^-126 and 2^127).
 *   q            [num_seqs, q_len, num_q_heads, head_dim] bf16, device, 16-byte aligned, finite.
 *   bounds, bound_scale  as paged_attn_block_bounds writes them, for every block of the contexts.
 *   count        blocks to select: the first sink_blocks and the last recent_blocks (together at most count)
 *                whatever their scores, then the highest, ties to the lowest block.  The blocks that hold new
 *                tokens should be among the recent ones.
 *   blocks       [num_seqs, num_kv_heads, count] int32, device, written: columns of the block table, ascending, then -1
 *                where the context has fewer.
 * Limits: q_len * (num_q_heads / num_kv_heads) at most 32, head_dim 64 or 128, block_size 16.  A block id out of range is
 * flagged and comes behind every other.  Scratch: 4 bytes per (block, kv head) of max_context_len where that exceeds
 * 65536, or 16384 with more (sequence, kv head) pairs than SMs, else none.  Asynchronous on `stream`.  Returns PA_OK (also for num_seqs == 0), PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_NO_MEMORY
 * or PA_ERR_CUDA.
 */
int paged_attn_select_blocks(const void* q, const int8_t* bounds, const float* bound_scale,
                             const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                             int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int count, int sink_blocks, int recent_blocks, int32_t* blocks,
                             void* stream);

/*
 * Sparse attention over listed blocks: paged_attn_decode and paged_attn_verify in which a row of kv head g sees,
 * of the tokens that it would see, those of the blocks that blocks[b][g] lists.
 *   blocks       [num_seqs, num_kv_heads, num_listed] int32, device: columns of the block table in any order, each at
 *                most once (a column listed twice counts twice); negative entries are unused.  A column past
 *                the context is skipped and flagged (PA_ERR_DEVICE_BOUNDS).
 * Blocks that are not listed are neither looked up nor read.  A row whose list holds nothing that it sees comes out as
 * zeros.  Same arguments and errors otherwise; limits: q_len * (num_q_heads / num_kv_heads) at most 32,
 * num_listed in [1, 2^26], max_context_len at most 2^30.  Kernels: the decode kernel (decode, groups of 1, 2, 4 and 8, bf16 and
 * E4M3) and the rows kernel, split over the list.
 */
int paged_attn_sparse_decode(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens,
                             const int32_t* blocks, int num_seqs, int max_blocks_per_seq,
                             int num_blocks, int max_context_len, int q_len, int num_listed,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             float scale, int kv_dtype, const float* k_scale, const float* v_scale,
                             void* out, void* stream);
int paged_attn_sparse_verify(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens,
                             const int32_t* blocks, int num_seqs, int max_blocks_per_seq,
                             int num_blocks, int max_context_len, int q_len, int num_listed,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             float scale, int kv_dtype, const float* k_scale, const float* v_scale,
                             void* out, void* stream);

/*
 * Attention of a batch whose sequences share prefixes (prefix caching: one system prompt, one document, in
 * the same blocks for many sequences): the results of paged_attn_decode and paged_attn_verify, with the keys
 * and values of a shared prefix read once for all of its sequences.
 *   group_starts   [num_groups + 1] int32, device, non-decreasing: sequences group_starts[i] .. group_starts[i + 1]
 *                  - 1 share a prefix.  Sequences outside every group share nothing.
 *   prefix_lens    [num_groups] int32, device: tokens that group i shares, rounded down to whole blocks (what is left
 *                  is read from each sequence's own row).  Those blocks are looked up in the row of the group's first
 *                  sequence; the other rows' entries for them are not read.
 *   max_prefix_len host-side bound of prefix_lens, at most max_blocks_per_seq * 16.
 *   max_own_len    host-side bound of what a sequence has behind its prefix (context_lens[b] - prefix).  Both size grids
 *                  and scratch only.
 * The new tokens lie behind the prefix: a sequence with context_lens[b] < prefix + q_len, or with more of its own
 * than max_own_len, comes out as zeros and is flagged (PA_ERR_DEVICE_BOUNDS).  Where a group that has sequences shares
 * whole blocks past the bound (or past max_context_len), its prefix is cut to the bound and flagged (a bound below 16
 * shares nothing, and the groups are not read); group offsets that do not fit are
 * flagged and their group shares nothing, but where offsets decrease so that two groups claim a sequence, the
 * outputs of both groups and of those behind them are undefined.  Same arguments and errors otherwise; limits: max_context_len at
 * most 2^30, and the 128-row tiles of all groups (num_seqs * q_len rows of 128 / group tokens, one more a group) at most 65535.
 * Kernels: the tile kernel of paged_attn_prefill over the rows of all of a group's sequences (the prefix, split into
 * partitions), the window forms' kernels over the own tokens, one merge.  Precision: that of paged_attn_decode, but for
 * E4M3 caches of head_dim 128: the scores of the prefix, and of the own tokens of more than 32 rows per kv head, take
 * the query as two E4M3 terms, off by at most 2^-8 of it, as in paged_attn_verify and paged_attn_prefill.
 */
int paged_attn_prefix_decode(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens,
                             const int32_t* group_starts, const int32_t* prefix_lens, int num_seqs,
                             int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                             int num_groups, int max_prefix_len, int max_own_len, int num_q_heads,
                             int num_kv_heads, int head_dim, int block_size, float scale,
                             int kv_dtype, const float* k_scale, const float* v_scale, void* out,
                             void* stream);
int paged_attn_prefix_verify(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* context_lens,
                             const int32_t* group_starts, const int32_t* prefix_lens, int num_seqs,
                             int max_blocks_per_seq, int num_blocks, int max_context_len, int q_len,
                             int num_groups, int max_prefix_len, int max_own_len, int num_q_heads,
                             int num_kv_heads, int head_dim, int block_size, float scale,
                             int kv_dtype, const float* k_scale, const float* v_scale, void* out,
                             void* stream);

/*
 * Decode that also keeps the attention weight each cached token has received: paged_attn_decode, and
 *   weights[block, g, slot] = decay * weights[block, g, slot] + sum_h softmax(s_h)_j
 * for every token j of every sequence, h over the query heads of kv head g; the step's own token, j =
 * context_lens[b] - 1, has no sum yet and its slot is set to its weight.
 *   weights      [num_blocks, num_kv_heads, 16] fp32, device, 16-byte aligned: caller-owned, laid out as the cache
 *                (the sums of a prompt's tokens start at what the caller stores, zeros for instance).  Slots past a context are not touched.
 *   decay        finite; 0 overwrites without reading, 1 adds, less than 1 forgets.
 * Blocks that two sequences of the call share would get both sums in an undefined order: their sums are undefined.
 * Same arguments and errors otherwise; limits: num_q_heads / num_kv_heads at most 32, max_context_len at most 2^30.
 * Scratch: where the scores of max_context_len tokens do not fit in the shared memory of a cluster, 4 bytes per (query
 * head, token) of num_seqs * max_context_len beside the split's.
 */
int paged_attn_weighted_decode(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* context_lens,
                               float* weights, int num_seqs, int max_blocks_per_seq, int num_blocks,
                               int max_context_len, int q_len, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, float decay, float scale, int kv_dtype,
                               const float* k_scale, const float* v_scale, void* out, void* stream);

/*
 * Eviction by accumulated attention weight: each (sequence, kv head) keeps min(context_lens[b], keep) tokens -- the first
 * `sinks`, the last `recent` (together at most keep) and the others of the largest sums, ties to the earliest, a NaN
 * below everything -- and they move in their order, with their sums, to the blocks of new_table.
 *   k_cache, v_cache, k_scale, v_scale, kv_dtype, block_table, context_lens, max_context_len as in paged_attn_decode
 *                (4-bit caches: the scales are not used and may be NULL).
 *   weights      [num_blocks, num_kv_heads, 16] fp32, device, 16-byte aligned, as paged_attn_weighted_decode keeps
 *                them.
 *   new_table    [num_seqs, new_blocks_per_seq] int32, device, new_blocks_per_seq * 16 >= keep: blocks that hold no
 *                token of any of the call's sequences, each once.  Blocks past the kept tokens are not touched.
 *   new_lens     [num_seqs] int32, device, written: the new context lengths; not the memory of context_lens.
 * The old blocks are only read, so they may be shared, and the caller gives them back afterwards.  bf16 and 4-bit rows move as they
 * are; E4M3 pages get the scale amax / 448 of their tokens and are re-encoded as paged_attn_append_kv does.  Different
 * heads keep different tokens: a slot no longer stands for one position, so attention over what is left uses keys
 * rotated before (the caller counts positions on its own).  Out-of-range ids are flagged: a token that cannot be read
 * counts as sum 0 and becomes zeros, a page that cannot be written is left out.  Scratch: 4 bytes per (kept token, kv
 * head), and 4 per (token, kv head) where max_context_len exceeds 98304.  Asynchronous on `stream`.  Returns PA_OK
 * (also for num_seqs == 0), PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_NO_MEMORY or PA_ERR_CUDA.
 */
int paged_attn_evict(void* k_cache, void* v_cache, float* weights, const int32_t* block_table,
                     const int32_t* context_lens, const int32_t* new_table, int num_seqs,
                     int max_blocks_per_seq, int new_blocks_per_seq, int num_blocks,
                     int max_context_len, int num_kv_heads, int head_dim, int block_size,
                     int kv_dtype, float* k_scale, float* v_scale, int keep, int sinks, int recent,
                     int32_t* new_lens, void* stream);

/*
 * KV append: store the new tokens' K and V in the paged cache, the step that precedes the
 * attention call of each decode or verify step (studybook fde-roadmap ch.10, sections 10.2.2
 * and 10.3.2: the step's K/V join the cache; section 10.12.2 and aegloslab servingai 5.3.7:
 * position j lives in slot j % block_size of block block_table[b][j / block_size]).
 *   k_new, v_new [num_seqs, n_new, num_kv_heads, head_dim] bf16, device, 16-byte aligned.
 *   k_cache, v_cache, block_table, as in paged_attn_decode; written in place.
 *   context_lens [num_seqs] int32, device: lengths AFTER the append; sequence b's new tokens
 *     take positions [context_lens[b] - n_new, context_lens[b]).
 *   kv_dtype PA_KV_BF16: the rows are stored unchanged.
 *   kv_dtype PA_KV_FP4_E2M1: each 16 dims get scale = e4m3(min(amax / (6 s), 448)), s = k_scale[g]
 *     (v_scale[g]), read only, and codes e2m1(x / (scale * s)); both roundings to nearest even, fp32
 *     arithmetic (6 s and scale * s rounded first).  A zero scale stores zeros; infinities store the
 *     largest magnitude, NaNs +6 * scale * s.  Stored tokens do not change.
 *   kv_dtype PA_KV_FP8_E4M3: k_scale / v_scale [num_blocks, num_kv_heads] fp32, device, read
 *     and written.  Each touched (block, head) gets the scale amax / 448 over its valid tokens
 *     (1 if all are zero) -- symmetric per-block scale quantisation (studybook section 10.8.2);
 *     the older tokens of the block are re-encoded when the scale changes.  All arithmetic is
 *     fp32; E4M3 rounding is to nearest even, saturating at +-448.
 * Slots past each sequence's last token are not touched.  Blocks written must belong to their
 * sequence alone (copy a shared block before appending to it).  Sequences whose context is
 * shorter than n_new, and out-of-range block ids, are skipped and flagged in the error word
 * (PA_ERR_DEVICE_BOUNDS from paged_attn_check_device_errors).  Asynchronous on `stream`; never
 * allocates.  Returns PA_OK (also for num_seqs == 0 or n_new == 0: nothing is launched),
 * PA_ERR_INVALID_ARG (NULL pointer, negative size, misaligned row pointer, n_new above the
 * table's capacity), PA_ERR_UNSUPPORTED (block_size != 16, head_dim not 64 or 128) or
 * PA_ERR_CUDA.
 */
int paged_attn_append_kv(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         const int32_t* block_table, const int32_t* context_lens, int num_seqs,
                         int n_new, int max_blocks_per_seq, int num_blocks, int num_kv_heads,
                         int head_dim, int block_size, int kv_dtype, float* k_scale,
                         float* v_scale, void* stream);

/*
 * Read stored tokens back as bf16: the inverse of paged_attn_append_kv.  For every sequence the rows
 * of its last n tokens, positions [context_lens[b] - n, context_lens[b]), are gathered through the
 * block table, turned into the values that they stand for and rounded to bf16 once.
 *   caches, block_table, context_lens, kv_dtype, k_scale, v_scale as in paged_attn_decode (E4M3:
 *   scales [num_blocks, num_kv_heads]; E2M1: [num_kv_heads] or NULL).
 *   k_out, v_out [num_seqs, n, num_kv_heads, head_dim] bf16, device, 16-byte aligned, written.
 * Tokens before a sequence's first, and tokens in out-of-range blocks, come out as zeros and are
 * flagged (PA_ERR_DEVICE_BOUNDS from paged_attn_check_device_errors).  Asynchronous on `stream`;
 * never allocates.  Returns as paged_attn_append_kv.
 */
int paged_attn_read_kv(const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int32_t* context_lens, int num_seqs, int n, int max_blocks_per_seq,
                       int num_blocks, int num_kv_heads, int head_dim, int block_size, int kv_dtype,
                       const float* k_scale, const float* v_scale, void* k_out, void* v_out,
                       void* stream);

/*
 * Norm and rotation of queries and keys, the step before paged_attn_append_kv, in one pass.  Each
 * head row x of q and k becomes y = x / sqrt(mean(x^2) + eps) * weight; then the first rotary_dim
 * dims are rotated in pairs by the angles of the token's position:
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin),
 * pair i being dims (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved != 0.  fp32 arithmetic,
 * one rounding to bf16.
 *   q, k         [num_tokens, num_q_heads (num_kv_heads), head_dim] bf16, device, 16-byte aligned;
 *                q_stride and k_stride are the elements from one token to the next (multiples of 8, at
 *                least heads * head_dim), so both may be slices of one packed projection.
 *   q_weight,
 *   k_weight     [head_dim] bf16, device, 16-byte aligned.
 *   cos_sin      [max_position, rotary_dim] fp32, device, 16-byte aligned: row p holds the rotary_dim
 *                / 2 cosines, then the sines, of position p.
 *   positions    [num_tokens] int32, device.  A position outside [0, max_position) makes its token's
 *                rows zeros and is flagged (PA_ERR_DEVICE_BOUNDS).
 *   q_out, k_out as q and k with strides of their own; each may be its input with the same stride
 *                (in place) and otherwise must not overlap q or k.
 * Limits: head_dim 64 or 128, rotary_dim a multiple of 16 in [16, head_dim].  Asynchronous on
 * `stream`; never allocates.  Returns PA_OK (also for num_tokens == 0), PA_ERR_INVALID_ARG (NULL
 * pointer, negative size, misalignment, a stride too short, eps negative or not finite),
 * PA_ERR_UNSUPPORTED or PA_ERR_CUDA.
 */
int paged_attn_qk_norm_rope(const void* q, const void* k, const void* q_weight,
                            const void* k_weight, const float* cos_sin, const int32_t* positions,
                            int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int rotary_dim, int interleaved, int max_position, float eps,
                            int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                            int64_t k_out_stride, void* q_out, void* k_out, void* stream);

/*
 * Speculative acceptance, the step after paged_attn_verify: decide which of the K drafted tokens
 * a round keeps and draw the token that ends the round (speculative sampling: studybook
 * fde-roadmap ch.10, section 10.6.2; aegloslab servingai 5.3.10; sirzzang "Speculative
 * Decoding", verification).  Per sequence, left to right, draft i is accepted when
 * p_i(x_i) >= q_i(x_i), else when u_accept[i] < p_i(x_i) / q_i(x_i) (IEEE fp32 division); the
 * first rejection at i ends the round with a token drawn from norm(max(0, p_i - q_i)) (from p_i
 * if that residual has no mass); if all K are accepted a bonus token is drawn from p_K.  A draw
 * from weights r uses the sequence's 32-bit word: w(x) = floor(min(max(r, 0), 1) * 2^40),
 * Z = sum w, T = floor(Z * word / 2^32), token = smallest x whose inclusive prefix of w exceeds T
 * (integer sums: the result does not depend on the order of summation).
 *   p            [num_seqs, num_draft + 1, vocab_size] fp32, device: target probabilities at the
 *                K + 1 verified positions (softmax of the verify forward's logits).
 *   q            [num_seqs, num_draft, vocab_size] fp32, device: draft probabilities at the K
 *                drafted positions.  May be NULL when num_draft == 0.
 *   draft_tokens [num_seqs, num_draft] int32, device.
 *   u_accept     [num_seqs, num_draft] fp32 in [0, 1), device: one uniform per draft.
 *   u_sample     [num_seqs] uint32, device: one uniform word per round.
 *   out_tokens   [num_seqs, num_draft + 1] int32, device, written: the accepted drafts, then the
 *                replacement or bonus token, then -1.
 *   num_accepted [num_seqs] int32, device, written: accepted drafts (the round emits this + 1).
 * A draft token outside [0, vocab_size) makes that sequence emit nothing (num_accepted -1, all
 * tokens -1) and sets the error word (PA_ERR_DEVICE_BOUNDS from paged_attn_check_device_errors);
 * so does a draw whose weights are all zero (token -1).  Scratch (8 bytes per 4096 vocabulary
 * entries per sequence) comes from the library's stream-ordered pool.  Asynchronous on
 * `stream`.  Returns PA_OK (also for num_seqs == 0), PA_ERR_INVALID_ARG (NULL pointer, negative
 * size), PA_ERR_UNSUPPORTED (num_draft > 31, vocab_size > 2^21, num_seqs > 65535),
 * PA_ERR_NO_MEMORY or PA_ERR_CUDA.
 */
int paged_attn_spec_accept(const float* p, const float* q, const int32_t* draft_tokens,
                           const float* u_accept, const uint32_t* u_sample, int num_seqs,
                           int num_draft, int vocab_size, int32_t* out_tokens,
                           int32_t* num_accepted, void* stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error word.  Returns
 * PA_OK, PA_ERR_DEVICE_BOUNDS or PA_ERR_DEVICE_TIMEOUT (bounds wins when both are set), or
 * PA_ERR_CUDA.  Not from the pages: a diagnostic of this library.
 */
int paged_attn_check_device_errors(void* stream);

/*
 * Failure-detection self-test (not from the pages: a diagnostic of this library).  Launches one
 * warp on `stream` whose first thread waits on a shared-memory mbarrier that nothing ever
 * arrives at, through the same bounded wait the kernels use, cut off after `polls` polls:
 * helper 0 = the decode kernels' wait, helper 1 = the tcgen05 kernels' wait (which also
 * raises the CTA's abort flag), both made of suspending mbarrier.try_wait polls; helper 2 = a
 * loop of non-suspending mbarrier.test_wait probes, the form of the tensor-core issuers' idle
 * loops.  The wait gives up, the error word records a timeout (PA_ERR_DEVICE_TIMEOUT from
 * paged_attn_check_device_errors) and the kernel returns normally, so the context stays usable.
 * The kernels cut suspending waits off after PA_WAIT_LIMIT polls and idle loops after
 * PA_SPIN_LIMIT iterations; elapsed_ns / polls gives the time of one poll, hence of a full wait.
 *   polls       in [1, PA_WAIT_LIMIT] for helpers 0 and 1, [1, PA_SPIN_LIMIT] for helper 2;
 *   elapsed_ns  one uint64, device, 8-byte aligned, written: wall time of the wait (globaltimer).
 * Returns PA_OK (launched), PA_ERR_INVALID_ARG (helper not 0, 1 or 2, polls out of range, NULL
 * or misaligned elapsed_ns) or PA_ERR_CUDA.
 */
#define PA_WAIT_LIMIT (1u << 18)
#define PA_SPIN_LIMIT (1u << 22)
int paged_attn_selftest_wait(int helper, unsigned int polls, unsigned long long* elapsed_ns,
                             void* stream);

/* Static description of a status code (never NULL). */
const char* paged_attn_status_string(int status);

/*
 * Split-KV planning of paged_attn_decode.  A sequence's pages are cut into partitions of
 * pages_per_partition pages; each (sequence, kv head, partition) is one CTA and a log-sum-exp
 * merge combines the partitions.  paged_attn_set_max_partitions(p > 0) forces at most p
 * partitions per sequence (p = 1 disables splitting); p = 0 restores the automatic choice.
 * Process-wide setting.  Returns PA_OK or PA_ERR_INVALID_ARG (p < 0 or p > 4096).
 * (paged_attn_verify balances its work on the device instead: the pages of all sequences and kv
 * heads are laid end to end and cut into equal ranges, one per resident CTA, with the pieces of a
 * sequence merged by the same log-sum-exp rule; this setting does not affect it.)
 */
int paged_attn_set_max_partitions(int p);

/*
 * The split the library would choose for paged_attn_decode, as a pure function of the shape (no
 * CUDA call): writes pages_per_partition and the partition count of the longest sequence.  The
 * automatic plan aims at 8 CTAs per SM for bf16 pages and 4 for E4M3 pages (half the bytes per
 * CTA), with partitions of at most 64 (bf16) or 256 (E4M3) pages where 64 partitions allow; for 4-bit
 * pages at sqrt(pages * resident CTAs / (38 * num_seqs * num_kv_heads)) partitions, the resident CTAs
 * those of groups of up to 8.  num_sms is the device's SM count (152 on GB300).  Returns PA_OK,
 * PA_ERR_INVALID_ARG, or PA_ERR_UNSUPPORTED for 4-bit pages with q_len other than 1: verify then splits by its
 * rows per kv head, which are no argument.
 */
int paged_attn_plan(int num_sms, int num_seqs, int num_kv_heads, int max_context_len,
                    int block_size, int q_len, int kv_dtype, int* pages_per_partition,
                    int* max_partitions);

/*
 * Decode that allocates nothing (no counterpart on the pages: a service of this library).
 *
 * For callers that cannot allocate device memory while they serve -- a host framework whose
 * memory manager reserved the GPU's memory up front, or a real-time loop that forbids
 * allocation after start-up.  Same arguments and limits as paged_attn_decode except that the
 * group (num_q_heads / num_kv_heads) must be 1, 2, 4 or 8 (else PA_ERR_UNSUPPORTED), and the same
 * results within its tolerances (it runs the library's CUDA-core decode kernel, fp32 FMAs), but
 * the split-KV partials live in a fixed array in the library's device image
 * (paged_attn_static_scratch_bytes() bytes, 32 MiB, held on every GPU that loads the library
 * until the process exits) instead of stream-ordered pool memory.  The call makes no
 * cudaMalloc, cudaMallocAsync, cudaFree or other allocating call.
 *   - The first call on a device looks up the array's device address (with that device
 *     current); make that first call before capturing any stream.
 *   - Every call shares the one array: calls whose kernels overlap on the GPU (different
 *     streams, or several host threads) race on it.  Serialise them, e.g. on one stream.
 *   - A shape whose partials need more than the array returns PA_ERR_SCRATCH_LIMIT and
 *     launches nothing: partials take num_seqs * q_len * num_q_heads * P * (head_dim + 1) * 4
 *     bytes when the plan splits into P > 1 partitions (paged_attn_plan), none when P = 1.
 *   - On PA_ERR_CUDA the contents of `out` are undefined: a launch may have failed after an
 *     earlier one of the same call had already written some rows.
 */
int paged_attn_decode_static_scratch(const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_table, const int32_t* context_lens,
                                     int num_seqs, int max_blocks_per_seq, int num_blocks,
                                     int max_context_len, int q_len, int num_q_heads,
                                     int num_kv_heads, int head_dim, int block_size, float scale,
                                     int kv_dtype, const float* k_scale, const float* v_scale,
                                     void* out, void* stream);

/* Size in bytes of the fixed array paged_attn_decode_static_scratch uses. */
size_t paged_attn_static_scratch_bytes(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int paged_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_H_ */
