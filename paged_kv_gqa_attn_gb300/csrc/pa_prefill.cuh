// Paged chunked-prefill attention on 5th-generation tensor cores (tcgen05), sm_103a.
//
// Chunked prefill splits a long prompt into chunks and runs each chunk as one forward next to the
// running decodes (aegloslab servingai 5.3.15, Sarathi-style chunking with piggybacked decode):
// the chunk's tokens attend to everything already in the paged cache and causally to each other.
// Queries are packed per sequence (varlen): sequence b owns rows [qsl[b], qsl[b+1]) of q, with
// q_len_b of them, and its context_lens[b] counts them (their K/V are in the cache already), so
// new token i sees n = L - q_len_b + i + 1 tokens -- decode (q_len 1), verify (K + 1) and a
// prefill chunk in one call.
//
// Tile: the G query heads of a kv head share every K/V page, so one CTA takes 128 / G new tokens
// of one (sequence, kv head) as 128 rows r = token * G + head (a full M = 128 MMA tile) and walks
// the context in 64-token steps (FlashAttention tiling with an online softmax, studybook
// fde-roadmap ch.10, section 10.1.2):
//   S[128 x 64]  = Q[128 x d] . K_step^T              (tcgen05.mma, operands in shared memory)
//   O[128 x d]  += P[128 x 64] . V_step[64 x d]        (P from tensor memory, V from shared)
// Tensor memory: two S buffers (columns 0-63, 64-127; P overwrites its S as bf16 pairs) and O
// (columns 128..128+d): QK of step k+1 runs while the softmax of step k works.  Shared memory
// (~97 KB: Q, 2-stage K and V rings) lets two CTAs share an SM, so one's softmax overlaps the
// other's products.  Warps: 0-3 softmax (thread r = row r = TMEM lane r), 4 K producer, 5 V
// producer (2-D TMA boxes of 16 tokens x 64 dims, 128-byte swizzle), 6 MMA issuer.
// Grid: x = rank * Hkv + kv head, the rank of the (sequence, tile) pair in the planner's work
// list, which orders the pairs by their number of steps, largest first.
// E4M3 caches (FP8), as in the verify kernel (study book ch.10, section 10.8.2: one symmetric
// scale per (block, kv head)): with head_dim 128, Q.K^T runs on the E4M3 codes of K
// (kind::f8f6f4; K pages copied as swizzled 2-D boxes, Q as two E4M3 terms after a power-of-two
// row scale) and each page's K scale multiplies its scores; the V pages are bulk-copied into the
// upper half of the step's f16 tile and both producer warps convert half of its rows in place to
// f16 (exact), zeroing pages without a block and tokens past the tile's last row; P.V runs on f16
// with P carrying each page's V scale.  With head_dim 64 K is converted the same way and Q.K^T
// runs on f16 (Q re-encoded after the row scale).
// 4-bit caches: an eighth warp stages a step's pages (codes and scales) ahead, warp 4 turns K and warp 5 V into
// the f16 tiles (code * scale is exact in f16).  No scale belongs to a page: the head's K scale is part of
// the row's score factor and its V scale of the epilogue's, so the softmax runs the bf16 form's raw-score
// path.  2 x 1024 new tokens behind up to 16384: 614 us (bf16 pages 416): the conversions' stores and the
// products' operand reads fill most of the shared memory's cycles, and the converting warps slow the softmax
// warps of their sub-partitions.
// Sliding window with sinks (WIN): the tile's pages are the sinks' and those from its first row's
// window on, numbered without the gap between (page_span; both edges on whole steps, so that a step
// never straddles the gap); pages of a step that no row of the tile sees are neither looked up nor
// copied, and each row masks the tokens between its sinks and its window.
// Shared prefix (kFormPrefix, split): the rows are those of all of a group's sequences, which are neighbours in q,
// 128 / G tokens a tile; every row sees the whole prefix, read through the first sequence's table, once for each
// tile.  The rows' own tokens (kFormOwn, split) are the window form's with the window's begin where the prefix ends;
// both leave partials.
// bf16 weights of both are a high part and the rounded remainder, 16 significant bits as in the decode kernel, whose
// results a call that names its prefixes should have: the remainder takes the other half of the step's S columns and
// a second P.V.  64 sequences behind 8192 tokens in 5 partitions: 43.6 -> 45.6 us a call, with cut instead of rounded high
// parts the same; 32 sequences of 5 rows, groups of 8, 100 to 1500 own tokens: 72.0 -> 75.3 us for the own tokens' pairs;
// root mean square error of 16 sequences behind 1024: 8.43e-5 as decode's, with the high part alone 1.16e-4.  E4M3 scores at head_dim 128 stay on two E4M3 terms of Q, off by 2^-8 of it at most: a third would take
// shared memory from the own tokens' CTAs beside the tile's.
#pragma once

#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_stage_ring.h"
#include "pa_tc.cuh"
#include "pa_work_item.h"

namespace pa {
namespace {

template <int D>
struct PfTraits {
  static constexpr int kBS = 16;
  static constexpr int kTP = 4;                          // pages per step
  static constexpr int kStepTokens = kTP * kBS;          // 64
  static constexpr int kHalves = D / 64;                 // 64-dim swizzle atoms across d
  static constexpr int kRegion = kStepTokens * 128;      // one half of a step tile
  static constexpr int kBoxBytes = kBS * 128;            // one half of one page
  static constexpr int kTile = kHalves * kRegion;        // K or V tile of one step
  static constexpr int kRows = 128;
  static constexpr int kQHalf = kRows * 128;
  static constexpr int kQBytes = kHalves * kQHalf;
  static constexpr int kOffK = 0;                        // K stages 0, 1
  static constexpr int kOffV = kOffK + 2 * kTile;        // V stages 0, 1
  static constexpr int kOffQ = kOffV + 2 * kTile;
  static constexpr int kOffBar = kOffQ + kQBytes;
  // kfull[2], vfull[2], kempty[2], o_done[2], s_ready[2], p_ready[2], q_ready, final, and for
  // E4M3 and 4-bit caches kready[2], vready[2] (tile converted to f16), and the staging ring's (4-bit:
  // staged pages landed, and read); an even number keeps kOffRaw 16-byte aligned
  static constexpr int kNumBars = (18 + StageRing::kFullBars + StageRing::kEmptyBars + 1) / 2 * 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem base, abort flag
  static constexpr int kOffRaw = kOffMisc + 16;            // 4-bit: slots for a step's K or V pages as they came
  static_assert(kOffRaw % 16 == 0, "bulk copies land on 16-byte boundaries");
  static constexpr int smem(int kv) {                      // + slack for 1024-byte alignment
    return kOffRaw + (kv == kKvFp4 ? StageRing::kSlots * kTP * Fp4Page<D>::kBytes : 0) + 1024;
  }
  static constexpr int kSCol = 0;                          // S/P buffer j: columns 64 j ..
  static constexpr int kOCol = 128;
  static constexpr int kTmemCols = 256;
  static constexpr int threads(int kv) { return kv == kKvFp4 ? 256 : 224; }
  // kind::f16: D fp32 (bit 4), A bf16 (7-9), B bf16 (10-12), B MN-major (16), N >> 3 (17), M >> 4 (24)
  static constexpr uint32_t kIdescQK =
      (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kStepTokens >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  static constexpr uint32_t kIdescPV =
      (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  // E4M3 caches: f16 operands (A and B type 0)
  static constexpr uint32_t kIdescQK16 = kIdescQK & ~((1u << 7) | (1u << 10));
  static constexpr uint32_t kIdescPV16 = kIdescPV & ~((1u << 7) | (1u << 10));
};

#ifdef PA_TIMELINE
// Instrumented build only (-DPA_TIMELINE, a separate library; the product build has none of
// it): per CTA of the last (non-split) prefill launch, by blockIdx.x, read by
// paged_attn_timeline_read_prefill.  Slots: 0 entry, 1 exit (%globaltimer), 2 SM id, 3 steps,
// and sums over the steps s >= 2 of thread 0 of the softmax and of the MMA issuer (SM cycles,
// clock64): 4 softmax busy (S(s) seen -> P(s) arrived), 5 softmax waiting for S(s) (P(s-1)
// arrived -> S(s) seen), 6 handoff (last softmax warp's P(s) arrival -> PV(s) issued), 7 chain
// (PV(s-2) issued -> S(s) seen), 8 QK lag (PV(s-2) issued -> QK(s) issued), 9 steps summed,
// 10-13 the softmax step's phases (S loaded from tensor memory; row max and rescale; weights;
// P stored to tensor memory), 14 skew of the four softmax warps' P(s) arrivals (last - first).
constexpr int kPfTlCtas = 8192, kPfTlSlots = 16;
__device__ unsigned long long g_prefill_timeline[kPfTlCtas * kPfTlSlots];
__device__ __forceinline__ unsigned long long pf_gtime() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ unsigned long long pf_clock() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%clock64;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void pf_tl_put(int slot, unsigned long long v) {
  if (blockIdx.x < kPfTlCtas && gridDim.y == 1) g_prefill_timeline[blockIdx.x * kPfTlSlots + slot] = v;
}
#endif

// SPLIT = false: packed variable-length rows, one CTA per (kv head, (sequence, tile) pair) in the
// planner's order.  SPLIT = true (verify rows that exceed the verify kernel's 64: every sequence
// q_len rows, G * q_len <= 128, one tile): grid (partition, kv head, sequence) over the split-KV
// plan of decode -- the CTA walks the pages [part * ppp, part * ppp + ppp) of its sequence and,
// when the sequence has several partitions, writes the normalised partial rows and their
// log2-sum-exp for the log-sum-exp merge kernel; p.tree_mask, when set, replaces the causal mask.
template <int D, bool SPLIT, int KV, int FORM>
__global__ void __launch_bounds__(PfTraits<D>::threads(KV), 2) prefill_tc_kernel(const AttnParams p, const int32_t* tiles,
                                                            const __grid_constant__ CUtensorMap tmk,
                                                            const __grid_constant__ CUtensorMap tmv) {
  using T = PfTraits<D>;
  constexpr bool FP8 = KV == kKvE4m3, FP4 = KV == kKvFp4;
  constexpr bool PREFIX = FORM == kFormPrefix, OWN = FORM == kFormOwn;
  constexpr bool WIN = FORM == kFormWindow || OWN;  // pages numbered with a gap
  static_assert(SPLIT || !(PREFIX || OWN), "both leave partials");
  constexpr bool kConv = FP8 || FP4;  // operands converted to f16 in shared memory
  // E4M3 with head_dim 128: Q.K^T on the E4M3 codes of K (kind::f8f6f4, Q split into two E4M3
  // terms), P.V on f16; head_dim 64: both products on f16 (K and V converted)
  constexpr bool kKDirect = FP8 && D == 128;
  constexpr bool kPair = (PREFIX || OWN) && KV == kKvBf16;  // weights as high part and remainder
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, G = Hq / Hkv;
  const int Tt = T::kRows / G;  // new tokens per tile
  int g, b, tile, qs, QL, part = 0, prefix = 0;
  if constexpr (PREFIX) {  // tile blockIdx.z of the groups' tiles, laid end to end
    part = (int)blockIdx.x;
    g = (int)blockIdx.y;
    const int lane = threadIdx.x & 31, z = (int)blockIdx.z;
    b = -1;
    tile = QL = 0;
    int before = 0;
    const bool checks = z == 0 && g == 0 && part == 0;  // this CTA looks at every group
    for (int i0 = 0; i0 < p.num_groups && (b < 0 || checks); i0 += 32) {
      PrefixGroup r = {0, 0, 0};
      unsigned wrong = 0;
      if (i0 + lane < p.num_groups) r = prefix_group(p, i0 + lane, wrong);
      if (wrong && checks && threadIdx.x < 32) record_error(p.err, wrong);
      if (b >= 0) continue;  // (its tile is found)
      const int tiles_here = r.tokens > 0 ? ((r.last - r.first) * p.q_len + Tt - 1) / Tt : 0;
      int upto = tiles_here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, z < before + upto);
      const int at = past ? __ffs(past) - 1 : 31;
      if (past) {
        b = __shfl_sync(0xffffffffu, r.first, at);
        QL = (__shfl_sync(0xffffffffu, r.last, at) - b) * p.q_len;
        prefix = __shfl_sync(0xffffffffu, r.tokens, at);
        tile = z - before - __shfl_sync(0xffffffffu, upto - tiles_here, at);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    qs = b * p.q_len;
  } else if constexpr (SPLIT) {
    part = (int)blockIdx.x;
    g = (int)blockIdx.y;
    b = (int)blockIdx.z;
    tile = 0;
    QL = p.q_len;
    qs = b * QL;
  } else {
    g = (int)(blockIdx.x % (unsigned)Hkv);
    const int rank = (int)(blockIdx.x / (unsigned)Hkv);
    // The work list comes from the planner.  (No __restrict__: a read-only pointer's loads may move above the wait.)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (rank >= tiles[0]) return;                       // fewer tiles than the grid's bound (uniform)
    const int32_t item = tiles[1 + rank];
    b = work_seq(item);
    tile = work_tile(item);
    qs = p.query_start_loc[b];
    QL = p.query_start_loc[b + 1] - qs;
  }
  // the grid over the own tokens may take the room that this one leaves
  if constexpr (PREFIX) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (PREFIX && b < 0) return;  // fewer tiles than the grid's bound

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
  const uint32_t sK = base + T::kOffK, sV = base + T::kOffV, sQ = base + T::kOffQ;
  const uint32_t bar_kfull = base + T::kOffBar;  // + 8 * stage
  const uint32_t bar_vfull = bar_kfull + 16;
  const uint32_t bar_kempty = bar_vfull + 16;    // QK of a step done: K stage reusable
  const uint32_t bar_o_done = bar_kempty + 16;   // PV of a step done: V stage and S/P buffer reusable
  const uint32_t bar_s_ready = bar_o_done + 16;  // S of a step in tensor memory
  const uint32_t bar_p_ready = bar_s_ready + 16; // P of a step in tensor memory (4 warps)
  const uint32_t bar_q_ready = bar_p_ready + 16; // Q written (4 warps)
  const uint32_t bar_final = bar_q_ready + 8;    // every MMA issued has completed
  const uint32_t bar_kready = bar_final + 8;     // E4M3: + 8 * stage: K tile converted to f16
  const uint32_t bar_vready = bar_kready + 16;   // E4M3: + 8 * stage: V tile converted to f16
  const uint32_t bar_raw_full = bar_vready + 16;     // 4-bit: + 8 * full_bar(use): a step's K or V pages staged
  const uint32_t bar_raw_empty = bar_raw_full + 8 * StageRing::kFullBars;  // + 8 * empty_bar(use): and read
  uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + T::kOffMisc);
  volatile uint32_t* abort_flag = misc + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#ifdef PA_TIMELINE
  // stamps handed between the softmax and the issuer: P(s) arrived, PV(s) issued (by s % 2)
  __shared__ volatile unsigned long long tl_pdone[2], tl_pvissue[2], tl_pwarp[2][4];
  if (threadIdx.x == 0) {
    unsigned smid;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
    pf_tl_put(0, pf_gtime());
    pf_tl_put(2, smid);
    for (int i = 3; i < kPfTlSlots; ++i) pf_tl_put(i, 0ull);
  }
  unsigned long long tl_a = 0, tl_b = 0, tl_c = 0, tl_d = 0;  // the role's sums
  unsigned long long tl_ph[4] = {0ull, 0ull, 0ull, 0ull}, tl_mark = 0;
#endif

  // a longer context is flagged by the planner (split: by partition 0 of kv head 0)
  int L = PREFIX  ? prefix
          : SPLIT ? context_len(p, b, part == 0 && g == 0 && threadIdx.x == 0)
                  : max(min(p.context_lens[b], p.max_context_len), 0);
  if constexpr (OWN) {
    prefix = prefix_of(p, b);
    if (!own_tokens_fit(p, L, prefix)) L = 0;
  }
  const int t0 = tile * Tt;
  const int first_new = L - QL;                       // cache position of new token 0
  const int n_max = PREFIX ? L : first_new + min(t0 + Tt, QL);  // tokens the tile's last row sees
  const int npages = n_max > 0 ? (n_max + T::kBS - 1) / T::kBS : 0;
  // window: the first position the tile's first row sees past the sinks, and the pages in between left out
  const int win_lo = OWN ? prefix : WIN ? max(0, first_new + t0 + 1 - p.window) : 0;
  const int lo_page = win_lo / T::kBS;
  const int sink_pages = WIN ? (p.sinks + T::kBS - 1) / T::kBS : 0;
  PageSpan span = {npages, 0, npages};
  if constexpr (WIN) span = page_span(npages, win_lo, p.sinks, T::kTP);
  // the CTA's pages [pfirst, plast): all of them, or its partition (a whole number of steps)
  const int ppp = PREFIX ? p.prefix_ppp : SPLIT ? p.pages_per_partition : 0;
  const int pfirst = SPLIT ? part * ppp : 0;
  const int plast = SPLIT ? min(span.count, pfirst + ppp) : span.count;
  const int nparts = SPLIT ? (span.count + ppp - 1) / ppp + (OWN && prefix > 0 ? 1 : 0) : 1;
  const int nsteps = plast > pfirst ? (plast - pfirst + T::kTP - 1) / T::kTP : 0;
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  // block-table column of the CTA's page v; false: past its range, or seen by no row of the tile
  auto column = [&](int v, int& page) {
    page = v;
    if constexpr (WIN) {
      page = span.real(v);
      return v < plast && (page < sink_pages || page >= lo_page);
    }
    return v < plast;
  };
  // first token of step s (a step lies on one side of the window's gap)
  auto step_token = [&](int s) { return (WIN ? span.real(pfirst + s * T::kTP) : pfirst + s * T::kTP) * T::kBS; };

  if (!PREFIX && first_new + t0 + 1 <= 0 && part == 0) {
    // the tile's first row sees no token (context shorter than the new tokens): its rows that see
    // nothing come out as zeros
    if (threadIdx.x == 0) record_error(p.err, kErrShortContext);
  }
  if (SPLIT && npages > 0 && nsteps == 0) return;  // a partition past the sequence's pages
  if (nsteps == 0) {
    if (part != 0) return;
    for (int r = threadIdx.x; r < T::kRows; r += blockDim.x) {
      const int t = t0 + r / G;
      if (t >= QL) continue;
      __nv_bfloat16* dst = p.out + ((size_t)(qs + t) * Hq + g * G + r % G) * D;
      for (int c = 0; c < D; ++c) dst[c] = __float2bfloat16(0.f);
    }
    if constexpr (OWN) after_prefixes();
    return;
  }

  // ---- set-up: barriers, tensor memory -------------------------------------------------------
  if (threadIdx.x == 128) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_kfull + 8 * s, 1);
      mbar_init(bar_vfull + 8 * s, 1);
      mbar_init(bar_kempty + 8 * s, 1);
      mbar_init(bar_o_done + 8 * s, 1);
      mbar_init(bar_s_ready + 8 * s, 1);
      mbar_init(bar_p_ready + 8 * s, 4);
      mbar_init(bar_kready + 8 * s, 1);
      mbar_init(bar_vready + 8 * s, kKDirect ? 2 : 1);  // head_dim 128: both producer warps convert V
    }
    if constexpr (FP4) {
      for (int s = 0; s < StageRing::kFullBars; ++s) mbar_init(bar_raw_full + 8 * s, 1);
      for (int s = 0; s < StageRing::kEmptyBars; ++s) mbar_init(bar_raw_empty + 8 * s, 1);
    }
    mbar_init(bar_q_ready, 4);
    mbar_init(bar_final, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    if constexpr (!kConv || kKDirect) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    if constexpr (!kConv) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
  }
  if (warp == 6) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + T::kOffMisc),
                 "r"(T::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint32_t tO = tmem + T::kOCol;

  if ((warp == 4 || warp == 5) && FP8) {
    // ======== E4M3 producers: warp 4 copies the K ring, warp 5 the V ring (2 stages each).  A bulk
    // copy lands each fp8 page of a step in the upper half of the step's f16 tile; once it has
    // landed a warp reads its rows of the step into registers and writes them back in place as f16
    // (exact) in the 128-byte-swizzled layout the MMAs read -- zeroing pages without a block and
    // tokens past the tile's last row -- and marks the tile converted.  With head_dim 128 the K
    // pages need no conversion (Q.K^T runs on the E4M3 codes, kind::f8f6f4): warp 4 copies them as
    // 2-D boxes in the swizzled layout the MMA reads and converts token rows 0-31 of every V tile,
    // while warp 5 copies the V pages and converts rows 32-63.  Copies run up to the ring ahead of
    // the conversions: a warp polls both sides, so neither waits behind the other.
    const bool is_k = warp == 4;
    const uint32_t ring = is_k ? sK : sV;
    const uint32_t bar_full = is_k ? bar_kfull : bar_vfull;    // fp8 bytes landed
    const uint32_t bar_free = is_k ? bar_kempty : bar_o_done;  // QK / PV of the step two before done
    const uint8_t* cache = is_k ? p.k_cache : p.v_cache;
    // the ring this warp converts and its token rows [c_row0, c_row0 + kCRows)
    const bool conv_v = kKDirect || !is_k;
    const uint32_t c_ring = conv_v ? sV : sK;
    const uint32_t c_full = conv_v ? bar_vfull : bar_kfull;
    const uint32_t c_ready = conv_v ? bar_vready : bar_kready;
    const int c_row0 = kKDirect && !is_k ? 32 : 0;
    constexpr int kCRows = kKDirect ? 32 : T::kStepTokens;
    constexpr int kPageFp8 = T::kBS * D;              // bytes of one fp8 page
    constexpr int kStageFp8 = T::kTP * kPageFp8;      // one step: half the f16 tile
    constexpr int kCPR = D / 16;                      // 16-code chunks per token row
    constexpr int kPer = kCRows * kCPR / 32;          // chunks per lane per step
    static_assert(2 * kStageFp8 == T::kTile, "fp8 step in the upper half of its f16 tile");
    // block id of page pfirst + s * kTP + (lane & 3) for lanes 0-3 (-1: none, or outside the pool)
    auto step_id = [&](int s, bool flag) {
      int v = -1, page;
      if (column(pfirst + s * T::kTP + (lane & 3), page) && lane < T::kTP) {
        v = bt[page];
        if (v < 0 || v >= p.num_blocks) {
          if (flag) record_error(p.err, kErrBlockId);
          v = -1;
        }
      }
      return v;
    };
    // with head_dim 128 warp 4's copies (K) and conversions (V) are independent
    const bool own_conv = !(kKDirect && is_k);
    int gi = 0, gc = 0;  // steps copied, steps converted
    uint32_t idle = 0;
    while (gc < nsteps || gi < nsteps) {
      bool progressed = false;
      // (a) copy the next step's pages once its stage is free
      if (gi < nsteps && (gi < gc + 2 || !own_conv)) {
        bool free_ok = gi < 2;
        if (!free_ok && lane == 0) free_ok = mbar_test_wait(bar_free + 8 * (gi & 1), ((gi - 2) >> 1) & 1);
        if (__shfl_sync(0xffffffffu, free_ok, 0)) {
          const int v = step_id(gi, is_k);
          int pbs[T::kTP];
#pragma unroll
          for (int pg = 0; pg < T::kTP; ++pg) pbs[pg] = __shfl_sync(0xffffffffu, v, pg);
          if (lane == 0) {
            const uint32_t bar = bar_full + 8 * (gi & 1);
            int npg = 0;
#pragma unroll
            for (int pg = 0; pg < T::kTP; ++pg) npg += pbs[pg] >= 0;
            if (npg == 0) {
              mbar_arrive(bar);
            } else if (!own_conv) {
              // E4M3 K pages as 16 x 128-byte boxes, 128-byte swizzle: the MMA's K-major layout
              const uint32_t dst = ring + (gi & 1) * T::kTile;
              mbar_arrive_expect_tx(bar, npg * kPageFp8);
#pragma unroll
              for (int pg = 0; pg < T::kTP; ++pg)
                if (pbs[pg] >= 0) tma_load_2d(dst + pg * kPageFp8, &tmk, 0, (pbs[pg] * Hkv + g) * T::kBS, bar);
            } else {
              const uint32_t dst = ring + (gi & 1) * T::kTile + kStageFp8;
              mbar_arrive_expect_tx(bar, npg * kPageFp8);
#pragma unroll
              for (int pg = 0; pg < T::kTP; ++pg)
                if (pbs[pg] >= 0)
                  bulk_copy_g2s(dst + pg * kPageFp8, cache + ((size_t)pbs[pg] * Hkv + g) * kPageFp8, kPageFp8, bar);
            }
          }
          ++gi;
          progressed = true;
        }
      }
      // (b) convert this warp's rows of the oldest unconverted step once its bytes have landed (a
      // V step that warp 5 copied has landed once its full barrier's phase completed: warp 5
      // cannot copy into that stage again before this warp has converted it)
      if (gc < nsteps && (gc < gi || !own_conv)) {
        bool landed = false;
        if (lane == 0) landed = mbar_test_wait(c_full + 8 * (gc & 1), (gc >> 1) & 1);
        if (__shfl_sync(0xffffffffu, landed, 0)) {
          const uint32_t tile = c_ring + (gc & 1) * T::kTile;
          const uint32_t src = tile + kStageFp8;
          const unsigned okm = __ballot_sync(0xffffffffu, step_id(gc, false) >= 0) & ((1u << T::kTP) - 1u);
          const int tok = step_token(gc);
          // token rows [0, rows_ok), but for those between the sinks and the window
          const int ps = pfirst + gc * T::kTP;  // (tok is ps's first token but for a window's gap)
          const int rows_ok = min(n_max - tok + ps * T::kBS, min(ps + T::kTP, plast) * T::kBS) - ps * T::kBS;
          // batches of 32 * kBatch chunks: a batch holds whole token rows, and the f16 write of
          // row t lands on the E4M3 bytes of row t only, so reading the batch before writing it
          // (the warp-wide barrier below) keeps every later batch's bytes intact
          constexpr int kBatch = kPer >= 4 ? kPer / 4 : 1;
#pragma unroll 1
          for (int i0 = 0; i0 < kPer; i0 += kBatch) {
            uint4 code[kBatch];
#pragma unroll
            for (int ii = 0; ii < kBatch; ++ii) {
              const int q = lane + 32 * (i0 + ii), tr = c_row0 + q / kCPR, dc = q % kCPR;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(code[ii].x), "=r"(code[ii].y), "=r"(code[ii].z), "=r"(code[ii].w)
                           : "r"(src + tr * D + dc * 16)
                           : "memory");
            }
            __syncwarp();  // the batch's rows are in registers before any f16 row overwrites them
#pragma unroll
            for (int ii = 0; ii < kBatch; ++ii) {
              const int q = lane + 32 * (i0 + ii), tr = c_row0 + q / kCPR, dc = q % kCPR;
              const bool keep = ((okm >> (tr / T::kBS)) & 1u) && tr < rows_ok &&
                                (!WIN || tok + tr >= win_lo || tok + tr < p.sinks);
              const uint32_t c4[4] = {keep ? code[ii].x : 0u, keep ? code[ii].y : 0u, keep ? code[ii].z : 0u,
                                      keep ? code[ii].w : 0u};
              uint32_t h[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                h[2 * j] = e4m3x2_to_f16x2(c4[j]);
                h[2 * j + 1] = e4m3x2_to_f16x2(c4[j] >> 16);
              }
              // dims [16 dc, 16 dc + 16): half dc / 4, 16-byte chunks 2 (dc % 4) and the next
              const uint32_t row = tile + (dc >> 2) * T::kRegion + tr * 128;
              const int c8 = (dc & 3) * 2;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((c8 ^ (tr & 7)) << 4)), "r"(h[0]),
                           "r"(h[1]), "r"(h[2]), "r"(h[3])
                           : "memory");
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((c8 + 1) ^ (tr & 7)) << 4)),
                           "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                           : "memory");
            }
            __syncwarp();
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(c_ready + 8 * (gc & 1));
          ++gc;
          progressed = true;
        }
      }
      if (progressed) {
        idle = 0;
      } else if (++idle >= kSpinLimit || ((idle & 1023u) == 0 && *abort_flag)) {
        if (lane == 0) {
          if (!*abort_flag) record_error(p.err, kErrTimeout);
          *abort_flag = 1u;
        }
        break;
      }
    }
    // every copy started has landed before the CTA's shared memory can go away (a copy is started
    // only once the copy two steps before it was consumed, so only the last two can be in flight)
    if (lane == 0)
      for (int k = max(0, gi - 2); k < gi; ++k) mbar_wait(bar_full + 8 * (k & 1), (k >> 1) & 1);
    __syncwarp();
  } else if (FP4 && warp != 6 && warp >= 4) {
    // ======== 4-bit producers.  Warp 7 stages a step's K pages, then its V pages, by bulk copies into a ring
    // of three such slots (StageRing), so copies run ahead of warp 4, which converts K, and warp 5, which converts
    // V: each writes the f16 tile once QK (PV) of the step two before is done, and gives the slot back.  (Staged in the tile's own space, or one step ahead only,
    // the copies' latency was in every step: 651-840 us where this takes 614.)
    using P = Fp4Page<D>;
    constexpr uint32_t kSlot = T::kTP * P::kBytes;
    const uint32_t staging = base + T::kOffRaw;
    // block ids of 32 pages (8 steps) in the lanes; -1: no page, or outside the pool
    auto load_ids = [&](int v0) {
      int v = -1, page;
      if (column(v0 + lane, page)) {
        v = bt[page];
        if (v < 0 || v >= p.num_blocks) {
          if (warp == 7) record_error(p.err, kErrBlockId);
          v = -1;
        }
      }
      return v;
    };
    int ids = -1;
    if (warp == 7) {
      int u = 0;  // slots filled: K of step 0, V of step 0, K of step 1, ...
      bool go = true;
      for (int s = 0; s < nsteps && go; ++s) {
        if (s % 8 == 0) ids = load_ids(pfirst + s * T::kTP);
        int pbs[T::kTP];
        int npg = 0;
#pragma unroll
        for (int pg = 0; pg < T::kTP; ++pg) {
          pbs[pg] = __shfl_sync(0xffffffffu, ids, (s % 8) * T::kTP + pg);
          npg += pbs[pg] >= 0;
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (lane == 0 && go) {
            const int slot = StageRing::slot(u);
            const uint32_t bar = bar_raw_full + 8 * StageRing::full_bar(u);
            if (u >= StageRing::kSlots)
              go = wait_or_abort(bar_raw_empty + 8 * StageRing::empty_bar(u), StageRing::empty_parity(u), abort_flag,
                                 p.err);
            if (go) {
              if (npg == 0) {
                mbar_arrive(bar);
              } else {
                mbar_arrive_expect_tx(bar, npg * P::kBytes);
                const uint8_t* cache = kv == 0 ? p.k_cache : p.v_cache;
#pragma unroll
                for (int pg = 0; pg < T::kTP; ++pg)
                  if (pbs[pg] >= 0)
                    bulk_copy_g2s(staging + slot * kSlot + pg * P::kBytes,
                                  cache + ((size_t)pbs[pg] * Hkv + g) * P::kBytes, P::kBytes, bar);
              }
              ++u;
            }
          }
        }
        go = __shfl_sync(0xffffffffu, go, 0);
      }
      // every copy started has landed before the CTA's shared memory can go away
      if (lane == 0)
        for (int k = max(0, u - StageRing::kSlots); k < u; ++k)
          mbar_wait(bar_raw_full + 8 * StageRing::full_bar(k), StageRing::full_parity(k));
    } else {
      const bool is_k = warp == 4;
      const uint32_t ring = is_k ? sK : sV;
      const uint32_t bar_ready = is_k ? bar_kready : bar_vready;
      const uint32_t bar_free = is_k ? bar_kempty : bar_o_done;
      constexpr int kUnitsRow = D / 32;                  // 32 dims: 16 code bytes, 2 scales
      constexpr int kPerPage = T::kBS * kUnitsRow / 32;  // of them per lane and page
      // The lane's 32-dim columns and rows: the eight lanes of a 16-byte access meet eight different bank
      // groups both reading the codes (rows of d / 2 bytes) and writing the swizzled f16 rows.  d = 128: lanes
      // of columns 0, 1 and of columns 2, 3 take different row pairs of the same four rows.
      const int dq = lane % kUnitsRow;
      const int row_in = D == 128 ? ((lane >> 2) & 1) + 2 * (((lane >> 3) & 1) ^ (dq >> 1)) + 4 * (lane >> 4) : lane >> 1;
      constexpr int kRowsPer = 32 / kUnitsRow;  // token rows of one unit of all lanes
      for (int s = 0; s < nsteps; ++s) {
        if (s % 8 == 0) ids = load_ids(pfirst + s * T::kTP);
        const int u = StageRing::use(s, !is_k), slot = StageRing::slot(u);
        bool go = true;
        if (lane == 0)
          go = wait_or_abort(bar_raw_full + 8 * StageRing::full_bar(u), StageRing::full_parity(u), abort_flag, p.err);
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        if (lane == 0 && s >= 2) go = wait_or_abort(bar_free + 8 * (s & 1), ((s - 2) >> 1) & 1, abort_flag, p.err);
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        const uint32_t tile = ring + (s & 1) * T::kTile;
        const int tok = step_token(s);
        // pages that hold data; token rows [0, rows_ok), but for those between the sinks and the window
        const unsigned okm = (__ballot_sync(0xffffffffu, ids >= 0) >> ((s % 8) * T::kTP)) & ((1u << T::kTP) - 1u);
        const int rows_ok = min(n_max - tok, min(T::kTP, plast - pfirst - s * T::kTP) * T::kBS);
        const bool all = okm == (1u << T::kTP) - 1u && rows_ok >= T::kStepTokens &&
                         (!WIN || tok >= win_lo || tok + T::kStepTokens <= p.sinks);
        // a page at a time, the next one's codes loaded before this one's are written: a small loop (unrolled
        // over the step, its instructions were fetched again and again between the softmax's)
        uint4 code[2][kPerPage];
        uint16_t scl[2][kPerPage];
        auto load_page = [&](int pg, uint4 (&c)[kPerPage], uint16_t (&sc)[kPerPage]) {
          const uint32_t page = staging + slot * kSlot + pg * P::kBytes;
#pragma unroll
          for (int i = 0; i < kPerPage; ++i) {
            const int tr = row_in + kRowsPer * i;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(c[i].x), "=r"(c[i].y), "=r"(c[i].z), "=r"(c[i].w)
                         : "r"(page + tr * P::kCodeRow + dq * 16)
                         : "memory");
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(sc[i])
                         : "r"(page + P::kCodeBytes + tr * P::kScaleRow + dq * 2)
                         : "memory");
          }
        };
        load_page(0, code[0], scl[0]);
#pragma unroll 1
        for (int pg = 0; pg < T::kTP; ++pg) {
          if (pg + 1 < T::kTP) load_page(pg + 1, code[1], scl[1]);
#pragma unroll
          for (int i = 0; i < kPerPage; ++i) {
            const int tr = pg * T::kBS + row_in + kRowsPer * i;
            // a token without data becomes zeros (its scale too: a stray one may be a NaN)
            if (!all && (!((okm >> pg) & 1u) || tr >= rows_ok || (WIN && tok + tr < win_lo && tok + tr >= p.sinks))) {
              code[0][i] = make_uint4(0u, 0u, 0u, 0u);
              scl[0][i] = 0;
            }
            const uint32_t c4[4] = {code[0][i].x, code[0][i].y, code[0][i].z, code[0][i].w};
            const uint32_t s2 = e4m3x2_to_f16x2(scl[0][i]);
            const uint32_t row = tile + (dq >> 1) * T::kRegion + tr * 128;
            const int c8 = (dq & 1) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // eight dims: one 16-byte chunk of the swizzled f16 row
              const uint32_t sp = __byte_perm(s2, s2, j < 2 ? 0x1010 : 0x3232);
              uint32_t h[4];
              e2m1x8_to_f16x2(c4[j], h);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = mul_f16x2(h[e], sp);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((c8 + j) ^ (tr & 7)) << 4)), "r"(h[0]),
                           "r"(h[1]), "r"(h[2]), "r"(h[3])
                           : "memory");
            }
            code[0][i] = code[1][i];
            scl[0][i] = scl[1][i];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_ready + 8 * (s & 1));
          mbar_arrive(bar_raw_empty + 8 * StageRing::empty_bar(u));
        }
      }
    }
    __syncwarp();
  } else if (warp == 4 || warp == 5) {
    // ======== TMA producers: warp 4 fills the K ring, warp 5 the V ring (2 stages each) ========
    const bool is_k = warp == 4;
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    const uint32_t ring = is_k ? sK : sV;
    const uint32_t bar_full = is_k ? bar_kfull : bar_vfull;
    const uint32_t bar_free = is_k ? bar_kempty : bar_o_done;
    auto load_ids = [&](int pbase) {
      int v = -1, pg;
      if (column(pbase + lane, pg)) {
        v = bt[pg];
        if (v < 0 || v >= p.num_blocks) {
          if (is_k) record_error(p.err, kErrBlockId);
          v = -1;
        }
      }
      return v;
    };
    int cbase = pfirst;
    int cur = load_ids(cbase);
    int s = 0;
    for (; s < nsteps; ++s) {
      const int pstep = pfirst + s * T::kTP;
      if (pstep >= cbase + 32) {
        cbase += 32;
        cur = load_ids(cbase);
      }
      int pbs[T::kTP];
      int npg = 0;
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) {
        pbs[pg] = __shfl_sync(0xffffffffu, cur, (pstep - cbase + pg) & 31);
        npg += pbs[pg] >= 0;
      }
      bool ready = true;
      if (lane == 0) {
        if (s >= 2) ready = wait_or_abort(bar_free + 8 * (s & 1), ((s - 2) >> 1) & 1, abort_flag, p.err);
        if (ready) {
          const uint32_t region = ring + (s & 1) * T::kTile;
          const uint32_t bar = bar_full + 8 * (s & 1);
          if (npg == 0) {
            mbar_arrive(bar);
          } else {
            mbar_arrive_expect_tx(bar, npg * T::kHalves * T::kBoxBytes);
#pragma unroll
            for (int pg = 0; pg < T::kTP; ++pg) {
              if (pbs[pg] < 0) continue;
              const int row = (pbs[pg] * Hkv + g) * T::kBS;
#pragma unroll
              for (int hh = 0; hh < T::kHalves; ++hh)
                tma_load_2d(region + hh * T::kRegion + pg * T::kBoxBytes, map, hh * 64, row, bar);
            }
          }
        }
      }
      ready = __shfl_sync(0xffffffffu, ready, 0);
      if (!ready) break;
    }
    // every copy started has landed before the CTA's shared memory can go away
    if (lane == 0)
      for (int k = max(0, s - 2); k < s; ++k) mbar_wait(bar_full + 8 * (k & 1), (k >> 1) & 1);
    __syncwarp();
  } else if (warp == 6) {
    // ======================= MMA issuer ========================================================
    if (lane == 0) {
      auto mma_qk = [&](int s) {
        const uint32_t kreg = sK + (s & 1) * T::kTile;
        const uint32_t tS = tmem + T::kSCol + (s & 1) * 64;
        if constexpr (kKDirect) {
          // S = Q_hi . K^T + Q_lo . K^T on E4M3 operands: each token row of K is one 128-byte
          // swizzled row (128 codes), 32 codes per instruction; Q_hi and Q_lo are 128-row E4M3
          // tiles one Q half apart
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8(tS, smem_desc(sQ + term * T::kQHalf + kk * 32, 16, 1024), smem_desc(kreg + kk * 32, 16, 1024),
                      T::kIdescQK16, (term > 0 || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = (kk >> 2) * T::kRegion + (kk & 3) * 32;
            const uint32_t qoff = (kk >> 2) * T::kQHalf + (kk & 3) * 32;
            umma_bf16(tS, smem_desc(sQ + qoff, 16, 1024), smem_desc(kreg + koff, 16, 1024),
                      kConv ? T::kIdescQK16 : T::kIdescQK, kk > 0 ? 1u : 0u);
          }
        }
        umma_commit(bar_s_ready + 8 * (s & 1));
        umma_commit(bar_kempty + 8 * (s & 1));
      };
      auto mma_pv = [&](int s) {
        const uint32_t vreg = sV + (s & 1) * T::kTile;
        const uint32_t tP = tmem + T::kSCol + (s & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < T::kStepTokens / 16; ++kk) {
          // A = P in tensor memory (16 tokens = 8 columns of bf16 pairs); B = V MN-major
          umma_bf16_tmem_a(tO, tP + kk * 8, smem_desc(vreg + kk * 2048, T::kRegion, 1024),
                           kConv ? T::kIdescPV16 : T::kIdescPV, (s > 0 || kk > 0) ? 1u : 0u);
          if constexpr (kPair)
            umma_bf16_tmem_a(tO, tP + 32 + kk * 8, smem_desc(vreg + kk * 2048, T::kRegion, 1024), T::kIdescPV, 1u);
        }
        umma_commit(bar_o_done + 8 * (s & 1));
      };
      int gq = 0, gp = 0;
      uint32_t idle = 0;
      while (gp < nsteps) {
        bool progressed = false;
        if (gq < nsteps && mbar_test_wait((kConv && !kKDirect ? bar_kready : bar_kfull) + 8 * (gq & 1), (gq >> 1) & 1) &&
            (gq < 2 || mbar_test_wait(bar_o_done + 8 * (gq & 1), ((gq - 2) >> 1) & 1)) &&
            (gq > 0 || mbar_test_wait(bar_q_ready, 0))) {
          tc_fence_after();
#ifdef PA_TIMELINE
          if (gq >= 2) tl_b += pf_clock() - tl_pvissue[gq & 1];
#endif
          mma_qk(gq);
          ++gq;
          progressed = true;
        }
        if (gp < gq && mbar_test_wait(bar_p_ready + 8 * (gp & 1), (gp >> 1) & 1) &&
            mbar_test_wait((kConv ? bar_vready : bar_vfull) + 8 * (gp & 1), (gp >> 1) & 1)) {
          tc_fence_after();
#ifdef PA_TIMELINE
          {
            const unsigned long long now = pf_clock();
            if (gp >= 2) {
              unsigned long long lo = tl_pwarp[gp & 1][0], hi = lo;
              for (int w = 1; w < 4; ++w) {
                lo = min(lo, (unsigned long long)tl_pwarp[gp & 1][w]);
                hi = max(hi, (unsigned long long)tl_pwarp[gp & 1][w]);
              }
              tl_a += now - hi;
              tl_d += hi - lo;
            }
            tl_pvissue[gp & 1] = now;
          }
#endif
          mma_pv(gp);
          ++gp;
          progressed = true;
        }
        if (progressed) {
          idle = 0;
        } else if (++idle >= kSpinLimit || ((idle & 1023u) == 0 && *abort_flag)) {
          if (!*abort_flag) record_error(p.err, kErrTimeout);
          *abort_flag = 1u;
          break;
        }
      }
      // every MMA this thread issued has completed before tensor memory is released
      umma_commit(bar_final);
      mbar_wait(bar_final, 0);
#ifdef PA_TIMELINE
      pf_tl_put(6, tl_a);
      pf_tl_put(8, tl_b);
      pf_tl_put(14, tl_d);
#endif
    }
    __syncwarp();
  } else {
    // ======================= softmax: thread r owns row r ======================================
    const int r = threadIdx.x;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const int t = t0 + r / G;          // new-token index of this row
    const int h = g * G + r % G;       // its query head
    // (with a group that does not divide 128 the tile's last rows would be the next tile's first)
    const bool row_live = t < QL && (!PREFIX || r < Tt * G);
    const int n_r = !row_live ? 0 : PREFIX ? L : max(first_new + t + 1, 0);  // tokens this row sees
    // tree verify (split mode only): the new tokens the row sees are its ancestor bits; the chain
    // mask (bits 0 .. t) gives the causal row exactly
    const bool tree = SPLIT && !PREFIX && p.tree_mask != nullptr;
    const uint32_t anc = (tree && row_live) ? p.tree_mask[(size_t)b * QL + t] : 0u;
    // Q row r: bf16, K-major 128-byte swizzle (halves of 64 dims, 8-row groups 1024 B apart).
    // E4M3: the row scaled by a power of two 2^k first (exact, no overflow for any bf16 q) and its
    // scores by qdiv = 2^-k; head_dim 128: two E4M3 terms hi = e4m3(q 2^k), lo = e4m3(q 2^k - hi)
    // (e4m3_prescale_exp), each a 128-byte row of codes, one Q half apart; head_dim 64: f16
    // (f16_prescale_exp).
    float qdiv = 1.f;
    {
      const __nv_bfloat16* qrow = row_live ? p.q + ((size_t)(qs + t) * Hq + h) * D : nullptr;
      float up = 1.f;
      if constexpr (kConv) {
        uint32_t emax = 0;
        if (qrow)
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) emax = max(emax, bf16x8_max_exp(*reinterpret_cast<const uint4*>(qrow + c * 8)));
        const int kq = kKDirect ? e4m3_prescale_exp(emax) : f16_prescale_exp(emax);
        up = exp2_int(kq);
        qdiv = exp2_int(-kq);
      }
      if constexpr (kKDirect) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b2 = a;
          if (qrow) {
            a = *reinterpret_cast<const uint4*>(qrow + c * 16);
            b2 = *reinterpret_cast<const uint4*>(qrow + c * 16 + 8);
          }
          const uint32_t wq[8] = {a.x, a.y, a.z, a.w, b2.x, b2.y, b2.z, b2.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x0 = bf16x2_to_f2(wq[2 * j]), x1 = bf16x2_to_f2(wq[2 * j + 1]);
            const float v0 = x0.x * up, v1 = x0.y * up, v2 = x1.x * up, v3 = x1.y * up;
            const uint32_t h01 = f32x2_to_e4m3x2(v0, v1), h23 = f32x2_to_e4m3x2(v2, v3);
            const float2 d01 = e4m3x2_to_f2((uint16_t)h01), d23 = e4m3x2_to_f2((uint16_t)h23);
            const uint32_t l01 = f32x2_to_e4m3x2(v0 - d01.x, v1 - d01.y), l23 = f32x2_to_e4m3x2(v2 - d23.x, v3 - d23.y);
            hi[j] = h01 | (h23 << 16);
            lo[j] = l01 | (l23 << 16);
          }
          const uint32_t off = r * 128 + (((uint32_t)c ^ (r & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sQ + off), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]),
                       "r"(hi[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sQ + T::kQHalf + off), "r"(lo[0]), "r"(lo[1]),
                       "r"(lo[2]), "r"(lo[3])
                       : "memory");
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (qrow) v = *reinterpret_cast<const uint4*>(qrow + c * 8);
          if constexpr (kConv) {
            const float2 a = bf16x2_to_f2(v.x), b2 = bf16x2_to_f2(v.y), c2 = bf16x2_to_f2(v.z), d2 = bf16x2_to_f2(v.w);
            v = make_uint4(pack_f16(a.x * up, a.y * up), pack_f16(b2.x * up, b2.y * up), pack_f16(c2.x * up, c2.y * up),
                           pack_f16(d2.x * up, d2.y * up));
          }
          const uint32_t dst = sQ + (c >> 3) * T::kQHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q_ready);
    }
    // the row's factor from raw scores to base-2 scaled ones (E4M3: times each page's K scale below)
    const float rowmul = FP4 ? p.scale_log2 * qdiv * (p.k_scale ? p.k_scale[g] : 1.f) : p.scale_log2;
    const float v_head = FP4 && p.v_scale ? p.v_scale[g] : 1.f;
    // bf16 and 4-bit: pages of a step that hold usable data (bit per page)
    auto pages_ok = [&](int s, float (&ksc)[T::kTP], float (&vsc)[T::kTP]) {
      unsigned okp = 0;
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) {
        ksc[pg] = 0.f;
        vsc[pg] = 0.f;
        int page;
        if (column(pfirst + s * T::kTP + pg, page)) {
          const int pb = bt[page];
          if (pb >= 0 && pb < p.num_blocks) okp |= 1u << pg;
        }
      }
      return okp;
    };
    // bf16: one check of every block id of the tile's range by the 128 softmax threads (named
    // barrier 1); with a valid table the steps need no per-page lookups
    bool all_ok = false;
    if constexpr (!FP8) {
      unsigned bad = 0;
      for (int pg = pfirst + r; pg < plast; pg += T::kRows) {
        int col;
        if (!column(pg, col)) continue;
        const int pb = bt[col];
        bad |= (pb < 0 || pb >= p.num_blocks) ? 1u : 0u;
      }
      unsigned anybad;
      asm volatile(
          "{\n\t.reg .pred pb, pr;\n\tsetp.ne.u32 pb, %1, 0;\n\tbar.red.or.pred pr, 1, 128, pb;\n\tselp.u32 %0, 1, 0, pr;\n\t}"
          : "=r"(anybad)
          : "r"(bad)
          : "memory");
      all_ok = anybad == 0;
    }
    // pages of step s that lie in the tile's range (valid table)
    auto pages_in = [&](int s) {
      const int left = plast - (pfirst + s * T::kTP);
      const unsigned in = left >= T::kTP ? (1u << T::kTP) - 1u : (left > 0 ? (1u << left) - 1u : 0u);
      if constexpr (WIN) {  // and that some row sees
        const int r0 = span.real(pfirst + s * T::kTP);
        return in & (unsigned)(low_bits64(sink_pages - r0) | ~low_bits64(lo_page - r0));
      }
      return in;
    };
    // E4M3: the block ids of step s + 2 are loaded during step s, and the K and V scales of step
    // s + 1 from them (at clamped addresses, no branch on a loaded value), so neither dependent
    // round trip waits inside a step
    int ids_next[T::kTP];  // block ids of the step after the next one (-1: past the range)
    auto load_ids = [&](int s, int (&ids)[T::kTP]) {
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) {
        int page;
        ids[pg] = column(pfirst + s * T::kTP + pg, page) ? bt[page] : -1;
      }
    };
    auto scales_of = [&](const int (&ids)[T::kTP], float (&ksc)[T::kTP], float (&vsc)[T::kTP]) {
      unsigned okp = 0;
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) {
        const bool v = ids[pg] >= 0 && ids[pg] < p.num_blocks;
        okp |= (v ? 1u : 0u) << pg;
        const size_t at = (size_t)(v ? ids[pg] : 0) * Hkv + g;
        ksc[pg] = p.k_scale[at];
        // a page that is not there must not lend a weight of 0 the scale of whatever lies in block 0, which may
        // be a NaN, nor the outputs' unit its size (K's scale only meets scores that the mask replaces)
        const float vs = p.v_scale[at];
        vsc[pg] = v ? vs : 0.f;
      }
      return okp;
    };
    bool ok = true;
    float m_used = -INFINITY, l = 0.f;
    float ks_next[T::kTP], vs_next[T::kTP];
    unsigned pok_next;
    // E4M3: O is summed in units of v_unit = 2^v_exp (v_unit_exp); chosen in the first step
    float v_unit = 0.f, v_exp = 0.f;
    if constexpr (FP8) {
      load_ids(0, ids_next);
      pok_next = scales_of(ids_next, ks_next, vs_next);
      if (nsteps > 1) load_ids(1, ids_next);
    } else {
      pok_next = all_ok ? pages_in(0) : pages_ok(0, ks_next, vs_next);
    }
    for (int s = 0; s < nsteps; ++s) {
      const unsigned pok = pok_next;
      float ksc[T::kTP], vsc[T::kTP];
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) {
        ksc[pg] = ks_next[pg];
        vsc[pg] = vs_next[pg];
      }
      const uint32_t tS = tmem + T::kSCol + (s & 1) * 64 + lane_off;
      if (!(ok = wait_or_abort(bar_s_ready + 8 * (s & 1), (s >> 1) & 1, abort_flag, p.err))) break;
      tc_fence_after();
#ifdef PA_TIMELINE
      unsigned long long tl_s = 0;
      if (r == 0) {
        tl_s = pf_clock();
        if (s >= 2) {
          tl_b += tl_s - tl_pdone[(s - 1) & 1];
          tl_c += tl_s - tl_pvissue[s & 1];
        }
      }
#endif
      float sc[T::kStepTokens];
      {
        uint32_t raw64[64];
        tmem_ld_x64(tS, raw64);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 64; ++c) sc[c] = __uint_as_float(raw64[c]);
      }
#ifdef PA_TIMELINE
      if (r == 0 && s >= 2) {
        tl_mark = pf_clock();
        tl_ph[0] += tl_mark - tl_s;
      }
#endif
      if (s + 1 < nsteps) {
        if constexpr (FP8) {
          pok_next = scales_of(ids_next, ks_next, vs_next);
          if (s + 2 < nsteps) load_ids(s + 2, ids_next);
        } else {
          pok_next = all_ok ? pages_in(s + 1) : pages_ok(s + 1, ks_next, vs_next);
        }
      }
      const int tok0 = step_token(s);
      // visibility of the step's 64 tokens for this row: causal limit (or, for a tree, the whole
      // prefix and the ancestor bits of the new tokens) and pages holding data
      uint64_t vis;
      if (tree) {
        const int sh = first_new - tok0;  // bit of new token 0 within the step
        const uint64_t a = row_live ? (uint64_t)anc : 0ull;
        const uint64_t nb = sh >= 64 ? 0ull : sh >= 0 ? (a << sh) : (-sh >= 64 ? 0ull : (a >> -sh));
        vis = (row_live ? low_bits64(first_new - tok0) : 0ull) | nb;
      } else {
        vis = low_bits64(n_r - tok0);
        // without what lies between the sinks and the row's window
        if constexpr (WIN) vis &= low_bits64(p.sinks - tok0) | ~low_bits64(n_r - p.window - tok0);
      }
      {
        uint64_t pm = 0;
#pragma unroll
        for (int pg = 0; pg < T::kTP; ++pg)
          if ((pok >> pg) & 1u) pm |= 0xffffull << (16 * pg);
        vis &= pm;
      }
      // Full steps with a positive scale stay in raw scores: the row max of raw scores times the
      // scale is the max of the scaled ones, and each weight is ex2(s * scale - m) with the
      // scale folded into one packed FMA per pair.  Masked steps (the diagonal, block tails)
      // scale first and mask with -inf.
      const bool raw = !FP8 && vis == ~0ull && rowmul > 0.f;
      // E4M3: each page's scores carry its K scale
      float kmul[T::kTP];
#pragma unroll
      for (int pg = 0; pg < T::kTP; ++pg) kmul[pg] = FP8 ? ksc[pg] * qdiv * p.scale_log2 : rowmul;
      // E4M3: the outputs' unit, grown (the same for every row) when a scale passes it
      float v_shrink = 1.f;
      if constexpr (FP8) {
        const float top = max_abs(vsc);
        if (top >= v_unit * kVUnitTop) {
          const int e = v_unit_exp(top);
          if (s > 0) v_shrink = exp2_int(max(-126, (int)v_exp - e));
          v_exp = (float)e;
          v_unit = exp2_int(e);
        }
      }
      // E4M3 full steps with positive scales stay in raw scores too: the page's max of raw scores
      // times its K multiplier is its scaled max, and each weight is ex2(s * kmul - m + log2
      // vscale), the V scale folded into the exponent's packed FMA, the row sum recovered per page
      // by the same power.  The V scales must be at least 2^-60 units: a folded weight then drops
      // below the smallest normal float (and out of the row sum) only where the weight itself is
      // under 2^-66; a smaller scale would lose the page's weights from the row sum.
      const bool fraw = FP8 && vis == ~0ull && p.scale_log2 > 0.f &&
                        fminf(fminf(ksc[0], ksc[1]), fminf(ksc[2], ksc[3])) > 0.f &&
                        fminf(fminf(vsc[0], vsc[1]), fminf(vsc[2], vsc[3])) >= fmaxf(v_unit * 0x1p-60f, 0x1p-126f);
      float mxs[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) mxs[j] = -INFINITY;
      if (raw) {
#pragma unroll
        for (int c = 0; c < T::kStepTokens; ++c) mxs[c & 7] = fmaxf(mxs[c & 7], sc[c]);
      } else if (fraw) {
#pragma unroll
        for (int c = 0; c < T::kStepTokens; ++c) mxs[(c / T::kBS) * 2 + (c & 1)] = fmaxf(mxs[(c / T::kBS) * 2 + (c & 1)], sc[c]);
#pragma unroll
        for (int pg = 0; pg < T::kTP; ++pg) {
          mxs[2 * pg] = fmaxf(mxs[2 * pg], mxs[2 * pg + 1]) * kmul[pg];
          mxs[2 * pg + 1] = -INFINITY;
        }
      } else {
        const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
        for (int c = 0; c < T::kStepTokens; ++c) {
          const bool v = (((c < 32 ? v0 : v1) >> (c & 31)) & 1u) != 0;
          sc[c] = v ? sc[c] * kmul[c / T::kBS] : -INFINITY;
          mxs[c & 7] = fmaxf(mxs[c & 7], sc[c]);
        }
      }
      float mx = fmaxf(fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])),
                       fmaxf(fmaxf(mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7])));
      if (raw) mx *= rowmul;
      const float m_new = fmaxf(m_used, mx);
      const bool need = (m_used != -INFINITY) && (m_new > m_used + 8.f);
      if (__any_sync(0xffffffffu, need) || (FP8 && v_shrink != 1.f)) {
        // the O row is rescaled only once PV(s - 1) has landed in it
        if (!(ok = wait_or_abort(bar_o_done + 8 * ((s - 1) & 1), ((s - 1) >> 1) & 1, abort_flag, p.err))) break;
        tc_fence_after();
        const float alpha = need ? fast_exp2(m_used - m_new) : 1.f, o_alpha = FP8 ? alpha * v_shrink : alpha;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t rw[32];
          tmem_ld_x32(tO + lane_off + c0, rw);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) rw[c] = __float_as_uint(__uint_as_float(rw[c]) * o_alpha);
          tmem_st_x32(tO + lane_off + c0, rw);
        }
        tmem_wait_st();
        l *= alpha;
      }
      if (need || m_used == -INFINITY) m_used = m_new;
      const float basev = m_used == -INFINITY ? 0.f : m_used;
#ifdef PA_TIMELINE
      if (r == 0 && s >= 2) {
        const unsigned long long now = pf_clock();
        tl_ph[1] += now - tl_mark;
        tl_mark = now;
      }
#endif

      // zero the V rows of tokens that hold no data (past the tile's range, or pages without a
      // block): P is 0 there, but 0 * NaN would still poison the product.  Thread r < 64 takes
      // token r of the step, after the step's V tile has landed; with a valid table only the last
      // step can hold such tokens.  (E4M3 tiles come zeroed from the conversion.)
      if (!kConv && warp < 2 &&
          (!all_ok || tok0 + T::kStepTokens > n_max || (WIN && tok0 < win_lo && tok0 + T::kStepTokens > p.sinks))) {
        const int tok = tok0 + r;
        const bool tok_ok =
            ((pok >> (r >> 4)) & 1u) && tok < n_max && (!WIN || tok >= win_lo || tok < p.sinks);
        if (__any_sync(0xffffffffu, !tok_ok)) {
          if (!(ok = wait_or_abort(bar_vfull + 8 * (s & 1), (s >> 1) & 1, abort_flag, p.err))) break;
          if (!tok_ok) {
            const uint32_t vrow = sV + (s & 1) * T::kTile + r * 128;
#pragma unroll
            for (int hh = 0; hh < T::kHalves; ++hh)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vrow + hh * T::kRegion + c * 16),
                             "r"(0u)
                             : "memory");
          }
          fence_proxy_async_smem();
        }
      }
      // P row r as bf16 pairs over the first 32 columns of this step's S buffer
      uint32_t w[32];
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 one2 = make_float2(1.f, 1.f);
      const float2 sc2 = raw ? make_float2(rowmul, rowmul) : one2;
      const float2 nb2 = make_float2(-basev, -basev);
      float lstep = 0.f;
      if (FP8 && fraw) {
        const float unit_basev = basev + v_exp;
        // pair c lies in page c / 8; acc[page] sums the weights times the page's V scale
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int pg = c / (T::kBS / 2);
          const float bias = __log2f(vsc[pg]) - unit_basev;
          const float2 x = ffma2(make_float2(sc[2 * c], sc[2 * c + 1]), make_float2(kmul[pg], kmul[pg]),
                                 make_float2(bias, bias));
          const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          acc[pg] = ffma2(e, one2, acc[pg]);
          w[c] = pack_f16(e.x, e.y);
        }
#pragma unroll
        for (int pg = 0; pg < T::kTP; ++pg) lstep = fmaf(acc[pg].x + acc[pg].y, fast_exp2(-__log2f(vsc[pg])), lstep);
        lstep *= v_unit;
      } else {
        if constexpr (FP8) {
          const float down = 1.f / v_unit;
#pragma unroll
          for (int pg = 0; pg < T::kTP; ++pg) vsc[pg] *= down;
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 x = ffma2(make_float2(sc[2 * c], sc[2 * c + 1]), sc2, nb2);
          const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          if constexpr (FP8) {  // f16 P carries each page's V scale; l sums the plain weights
            acc[c & 3] = ffma2(e, one2, acc[c & 3]);
            const float vm = vsc[(2 * c) / T::kBS];
            w[c] = pack_f16(e.x * vm, e.y * vm);
          } else if constexpr (FP4) {  // f16 P (2^-11 a weight); l sums the weights before that rounding
            acc[c & 3] = ffma2(e, one2, acc[c & 3]);
            w[c] = pack_f16(e.x, e.y);
          } else if constexpr (kPair) {  // the high part; the remainder below
            acc[c & 3] = ffma2(e, one2, acc[c & 3]);
            w[c] = pack_bf16(e.x, e.y);
            const float2 high = bf16x2_to_f2(w[c]);
            sc[2 * c] = e.x - high.x;
            sc[2 * c + 1] = e.y - high.y;
          } else {
            // l sums the bf16-rounded weights that P.V multiplies (normalised by its own weights)
            w[c] = pack_bf16(e.x, e.y);
            acc[c & 3] = add_bf16x2_f2(w[c], acc[c & 3]);
          }
        }
        lstep = ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) + ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
      }
#ifdef PA_TIMELINE
      if (r == 0 && s >= 2) {
        const unsigned long long now = pf_clock();
        tl_ph[2] += now - tl_mark;
        tl_mark = now;
      }
#endif
      tmem_st_x32(tS, w);
      if constexpr (kPair) {  // the remainders over the other 32 columns
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pack_bf16(sc[2 * c], sc[2 * c + 1]);
        tmem_st_x32(tS + 32, w);
      }
      tmem_wait_st();
#ifdef PA_TIMELINE
      if (r == 0 && s >= 2) tl_ph[3] += pf_clock() - tl_mark;
#endif
      l += lstep;
      tc_fence_before();
      __syncwarp();
#ifdef PA_TIMELINE
      if (r == 0) {
        const unsigned long long now = pf_clock();
        if (s >= 2) tl_a += now - tl_s;
        tl_pdone[s & 1] = now;
      }
      if (lane == 0) tl_pwarp[s & 1][warp] = pf_clock();
#endif
      if (lane == 0) mbar_arrive(bar_p_ready + 8 * (s & 1));
    }
#ifdef PA_TIMELINE
    if (r == 0) {
      pf_tl_put(3, (unsigned long long)nsteps);
      pf_tl_put(4, tl_a);
      pf_tl_put(5, tl_b);
      pf_tl_put(7, tl_c);
      pf_tl_put(9, (unsigned long long)(nsteps > 2 ? nsteps - 2 : 0));
      for (int i = 0; i < 4; ++i) pf_tl_put(10 + i, tl_ph[i]);
    }
#endif
    if (ok) {
      // ---- epilogue: O row / l -> bf16 ------------------------------------------------------
      const int gl = nsteps - 1;
      ok = wait_or_abort(bar_o_done + 8 * (gl & 1), (gl >> 1) & 1, abort_flag, p.err);
      if (ok) {
        tc_fence_after();
        const float inv = l > 0.f ? (FP4 ? v_head : FP8 ? v_unit : 1.f) / l : 0.f;
        __nv_bfloat16* dst = p.out + ((size_t)(qs + t) * Hq + h) * D;
        // split sequence: the partition's normalised rows and log2-sum-exp for the merge kernel
        const bool partial = PREFIX || (SPLIT && nparts > 1);
        const size_t prow = ((size_t)(qs + t) * Hq + h) * p.max_partitions + (PREFIX ? p.own_partitions : 0) + part;
        if (partial && row_live) p.part_lse[prow] = l > 0.f ? m_used + __log2f(l) : -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t raw[32];
          tmem_ld_x32(tO + lane_off + c0, raw);
          tmem_wait_ld();
          if (!row_live) continue;
          if (partial) {
            float* pdst = p.part_o + prow * D + c0;
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<float4*>(pdst + c) =
                  make_float4(__uint_as_float(raw[c]) * inv, __uint_as_float(raw[c + 1]) * inv,
                              __uint_as_float(raw[c + 2]) * inv, __uint_as_float(raw[c + 3]) * inv);
            continue;
          }
          if constexpr (!PREFIX) {
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint4 v;
              v.x = pack_bf16(__uint_as_float(raw[c + 0]) * inv, __uint_as_float(raw[c + 1]) * inv);
              v.y = pack_bf16(__uint_as_float(raw[c + 2]) * inv, __uint_as_float(raw[c + 3]) * inv);
              v.z = pack_bf16(__uint_as_float(raw[c + 4]) * inv, __uint_as_float(raw[c + 5]) * inv);
              v.w = pack_bf16(__uint_as_float(raw[c + 6]) * inv, __uint_as_float(raw[c + 7]) * inv);
              *reinterpret_cast<uint4*>(dst + c0 + c) = v;
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::kTmemCols) : "memory");
  }
  if constexpr (OWN) after_prefixes();
#ifdef PA_TIMELINE
  if (threadIdx.x == 0) pf_tl_put(1, pf_gtime());
#endif
}

template <int D, int KV, int FORM>
cudaError_t prefill_tiles(const AttnParams& p, int max_q_len, int group, int32_t* tiles, const CUtensorMap& tk,
                          const CUtensorMap& tv, cudaStream_t st) {
  using T = PfTraits<D>;
  const void* fn = reinterpret_cast<const void*>(prefill_tc_kernel<D, false, KV, FORM>);
  cudaError_t e = set_smem_once(fn, T::smem(KV));
  if (e != cudaSuccess) return e;
  const int tt = T::kRows / group;
  e = launch_prefill_plan(p, tt, tiles, st);
  if (e != cudaSuccess) return e;
  const long long bound = (long long)p.num_seqs * ((max_q_len + tt - 1) / tt);
  AttnParams pp = p;
  const int32_t* ct = tiles;
  CUtensorMap k = tk, v = tv;
  void* args[] = {&pp, &ct, &k, &v};
  // x = rank * Hkv + kv head: the heaviest pairs, all heads of each, are dispatched first
  return launch_pdl(fn, dim3((unsigned)(bound * p.num_kv_heads)), dim3(T::threads(KV)), T::smem(KV), st, args);
}

template <int D, int KV, int FORM>
cudaError_t prefill_split(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using T = PfTraits<D>;
  const void* fn = reinterpret_cast<const void*>(prefill_tc_kernel<D, true, KV, FORM>);
  cudaError_t e = set_smem_once(fn, T::smem(KV));
  if (e != cudaSuccess) return e;
  dim3 grid(FORM == kFormOwn ? p.own_partitions : p.max_partitions, p.num_kv_heads, p.num_seqs);
  if constexpr (FORM == kFormPrefix) {
    grid.x = p.max_partitions - p.own_partitions;
    grid.z = prefix_tiles(p.num_seqs, p.q_len, p.num_q_heads / p.num_kv_heads, p.num_groups);
  }
  if (FORM == kFormOwn && p.max_partitions > p.own_partitions) {  // beside the prefixes
    AttnParams pp = p;
    const int32_t* none = nullptr;
    CUtensorMap k = tk, v = tv;
    void* args[] = {&pp, &none, &k, &v};
    return launch_pdl(fn, grid, dim3(T::threads(KV)), T::smem(KV), st, args);
  }
  prefill_tc_kernel<D, true, KV, FORM><<<grid, T::threads(KV), T::smem(KV), st>>>(p, nullptr, tk, tv);
  return cudaGetLastError();
}

// One head_dim of a launch, split (verify rows) or in the planner's tiles.
template <int D, int KV, int FORM>
cudaError_t prefill_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles, const CUtensorMap& tk,
                         const CUtensorMap& tv) {
  return tiles ? prefill_tiles<D, KV, FORM>(p, max_q_len, l.group, tiles, tk, tv, l.stream)
               : prefill_split<D, KV, FORM>(p, tk, tv, l.stream);
}

// One split form, for its cache type and head_dim.
template <int FORM>
cudaError_t split_any(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  const bool wide = l.head_dim == 128;
  if (!wide && l.head_dim != 64) return cudaErrorInvalidConfiguration;
  switch (l.kv) {
    case kKvBf16:
      return wide ? prefill_split<128, kKvBf16, FORM>(p, tk, tv, l.stream) : prefill_split<64, kKvBf16, FORM>(p, tk, tv, l.stream);
    case kKvE4m3:
      return wide ? prefill_split<128, kKvE4m3, FORM>(p, tk, tv, l.stream) : prefill_split<64, kKvE4m3, FORM>(p, tk, tv, l.stream);
    default:
      return wide ? prefill_split<128, kKvFp4, FORM>(p, tk, tv, l.stream) : prefill_split<64, kKvFp4, FORM>(p, tk, tv, l.stream);
  }
}

}  // namespace
}  // namespace pa
