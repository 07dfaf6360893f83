// Paged GQA attention of a few rows per kv head on the warp-level tensor-core instruction, sm_103a:
// 4-bit caches (decode and verify, with and without a window), and verify with a window over bf16 and
// E4M3 caches.
//
// The R = q_len * G rows of one kv head (row c is new token c / G, head c % G) are the columns of up to
// four 8-wide n-tiles; one page's work is the decode kernel's, widened:
//   S^T[16 tokens x R] = K[16 x d] . Q^T[d x R]          A = K, made once per page
//   O^T[d x R]        += V^T[d x 16] . P^T[16 x R]         A = V, made once per page
// Why here: turning 4-bit (or E4M3) pages into operands costs far more instructions than the products,
// and here it is paid once per page whatever R is, in registers; the 128-row tile kernel pays it through
// shared memory for 128 rows of which a verify step uses 20.
//
// 4-bit pages: a lane takes a quarter of each of its two K rows (16 bytes, a contiguous 512 bytes a warp)
// and an eighth of four V rows; E2M1 pairs become f16 pairs in one conversion a byte, V's bytes paired
// across two tokens by two logic operations a word; each pair is multiplied by its 16-dim scale in f16
// (exact: at most six significant bits).  Per 16-token page of d = 128 about 64 conversions, 64
// multiplications and 16 products an n-tile: near 260 warp instructions for 2304 bytes, about two
// thirds of what an SM issues while it receives them.  Measured (64 contexts of 1000 to 32768 tokens, 32 / 8
// heads of 128): 268 us, 70 % of the copy rate; with the arithmetic left out the same copies take 193 us, the
// copy rate.  The logic unit, which the conversions share at half rate, and the issue slots are each busy
// little more than half the time: 16 warps an SM do not cover their chains, and a fifth CTA would need
// fewer than 96 registers.  Pages go two to a step (301 -> 285 us), and move as 16-byte cp.async pieces of
// all lanes with no barrier to poll, nine instructions a step: the bulk-copy unit's uniform operands cost one
// lane near 60 instructions a page (285 -> 268 us).  At 20 rows (four drafts, groups of 4) the accumulators
// leave two CTAs an SM: 95 us for 32 contexts up to 8192 tokens, 25 %.
// f16 weights, q re-encoded as f16 after a power of two a row, and E4M3's folded page scales are as in
// the decode kernel; the head's K scale joins the row's score factor, its V scale the epilogue.
//
// Masks: a page that every row sees whole is the fast path; pages at the causal edge, at an edge of the
// window or of the sinks, and tree masks test each (row, token).  Tokens that no row sees have their V
// zeroed, whatever is stored there.
#pragma once

#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_mma.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

template <int D, int NT, int KV>
struct RowsTraits {
  static constexpr bool kBf16 = KV == kKvBf16, kFp8 = KV == kKvE4m3, kFp4 = KV == kKvFp4;
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBS = 16;
  static constexpr int kCols = 8 * NT;
  static constexpr int kRowBytes = kBf16 ? 2 * D : kFp8 ? D : D / 2;  // of codes
  static constexpr int kPageBytes = kFp4 ? Fp4Page<D>::kBytes : kBS * kRowBytes;
  static constexpr int kPP = kFp4 ? 2 : 1;       // pages per step of a warp
  static constexpr int kStageBytes = 2 * kPP * kPageBytes;  // K page then V page, for each page
  static constexpr int kStages = kBf16 ? 2 : kFp8 ? 3 : 4 / kPP;
  static constexpr int kMinBlocks = rows_resident_ctas(8 * NT);
  static constexpr int kBoxes = kRowBytes >= 128 ? kRowBytes / 128 : 1;  // TMA boxes per page (not 4-bit)
  static constexpr int kKSteps = D / 16;
  static constexpr int kMTiles = D / 16;
  static constexpr int kMerge = kWarps * kCols * (D + 2) * 4;  // per-warp outputs, maxima, sums
  static constexpr int kStageRegion = kWarps * kStages * kStageBytes;
  static constexpr int kDataRegion = kStageRegion > kMerge ? kStageRegion : kMerge;
  static constexpr int kBarRegion = kWarps * kStages * 8;  // (a multiple of 16: kWarps is even)
  static constexpr int kQRegion = NT * (kKSteps / 2) * 32 * 16;
  static constexpr int kSmem = 1024 + kDataRegion + kBarRegion + kQRegion;  // 1 KiB: alignment of the swizzle
  static_assert(kDataRegion % 16 == 0 && kBarRegion % 16 == 0, "barriers and Q fragments are aligned");
};

// First dim of a lane's four contraction dims in k-step st (the order of each row's words).
template <int D, int KV>
__device__ __forceinline__ int q_dim(int qi, int st) {
  if constexpr (KV == kKvFp4) return qi * (D / 4) + 4 * st;
  constexpr int RB = KV == kKvBf16 ? 2 * D : D;
  const int w = KV == kKvBf16 ? 2 * st : st;
  return (qk_chunk<RB>(qi, w >> 2) * 16 + (w & 3) * 4) / (KV == kKvBf16 ? 2 : 1);
}

// First of the two dims of row group gi in m-tile i.
template <int D, int KV>
__device__ __forceinline__ int o_dim(int gi, int i) {
  return KV == kKvBf16 ? 64 * (i >> 2) + 8 * gi + 2 * (i & 3) : (D / 8) * gi + 2 * i;
}

// A fragments of all k-steps of K: rows gi and gi + 8 of the page, the lane's quarter of each.
template <int D, int KV>
__device__ __forceinline__ void k_fragments(const uint8_t* kp, int gi, int qi, uint32_t (&a)[D / 16][4]) {
  if constexpr (KV == kKvFp4) {
    using P = Fp4Page<D>;
    constexpr int kWords = D / 32;  // 32-bit words of codes per lane and row
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = gi + 8 * half;
      uint32_t w[kWords], sc[2];  // f16 pairs (s, s) of the lane's one or two blocks
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(kp + r * P::kCodeRow + qi * 16);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        const uint32_t s2 =
            e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + P::kCodeBytes + r * P::kScaleRow + qi * 2));
        sc[0] = __byte_perm(s2, s2, 0x1010);
        sc[1] = __byte_perm(s2, s2, 0x3232);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(kp + r * P::kCodeRow + qi * 8);
        w[0] = x.x; w[1] = x.y;
        const uint32_t s2 = e4m3x2_to_f16x2(kp[P::kCodeBytes + r * P::kScaleRow + qi]);
        sc[0] = sc[1] = __byte_perm(s2, s2, 0x1010);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t h[4];
        e2m1x8_to_f16x2(w[i], h);
        const uint32_t s = sc[i / (kWords / 2)];
        a[2 * i][half] = mul_f16x2(h[0], s);
        a[2 * i][half + 2] = mul_f16x2(h[1], s);
        a[2 * i + 1][half] = mul_f16x2(h[2], s);
        a[2 * i + 1][half + 2] = mul_f16x2(h[3], s);
      }
    }
  } else {
    constexpr int RB = KV == kKvBf16 ? 2 * D : D;
    constexpr int kChunks = RB / 64;
    uint32_t k0[4 * kChunks], k1[4 * kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int ch = qk_chunk<RB>(qi, c);
      const uint4 x = *reinterpret_cast<const uint4*>(kp + chunk_off<RB>(gi, ch));
      const uint4 y = *reinterpret_cast<const uint4*>(kp + chunk_off<RB>(gi + 8, ch));
      k0[4 * c] = x.x; k0[4 * c + 1] = x.y; k0[4 * c + 2] = x.z; k0[4 * c + 3] = x.w;
      k1[4 * c] = y.x; k1[4 * c + 1] = y.y; k1[4 * c + 2] = y.z; k1[4 * c + 3] = y.w;
    }
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      if constexpr (KV == kKvBf16) {
        a[st][0] = k0[2 * st]; a[st][1] = k1[2 * st]; a[st][2] = k0[2 * st + 1]; a[st][3] = k1[2 * st + 1];
      } else {
        a[st][0] = e4m3x2_to_f16x2(k0[st]); a[st][1] = e4m3x2_to_f16x2(k1[st]);
        a[st][2] = e4m3x2_to_f16x2(k0[st] >> 16); a[st][3] = e4m3x2_to_f16x2(k1[st] >> 16);
      }
    }
  }
}

// The lane's words of V: an eighth (gi) of the rows of tokens 2qi, 2qi+1, 2qi+8, 2qi+9; tokens whose bit
// of `live` is clear become zeros.  4-bit: sc = the f16 scale pairs of the first and last two tokens.
template <int D, int KV>
__device__ __forceinline__ void v_words(const uint8_t* vp, int gi, int qi, uint32_t live,
                                        uint32_t (&v)[4][(KV == kKvBf16 ? 2 * D : KV == kKvE4m3 ? D : D / 2) / 32],
                                        uint32_t (&sc)[2]) {
  constexpr int RB = KV == kKvBf16 ? 2 * D : KV == kKvE4m3 ? D : D / 2;
  constexpr int kWords = RB / 32;
  uint32_t sb[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = 2 * qi + (r & 1) + 8 * (r >> 1);
    if constexpr (KV == kKvFp4) {
      using P = Fp4Page<D>;
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(vp + t * P::kCodeRow + gi * 8);
        v[r][0] = x.x; v[r][1] = x.y;
      } else {
        v[r][0] = *reinterpret_cast<const uint32_t*>(vp + t * P::kCodeRow + gi * 4);
      }
      sb[r] = vp[P::kCodeBytes + t * P::kScaleRow + (D == 128 ? gi : gi >> 1)];
    } else if constexpr (RB == 64) {
      const uint2 x = *reinterpret_cast<const uint2*>(vp + chunk_off<RB>(t, gi >> 1) + 8 * (gi & 1));
      v[r][0] = x.x; v[r][1] = x.y;
    } else {
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(vp + chunk_off<RB>(t, 8 * j + gi));
        v[r][4 * j] = x.x; v[r][4 * j + 1] = x.y; v[r][4 * j + 2] = x.z; v[r][4 * j + 3] = x.w;
      }
    }
  }
  if (live != 0xffffu) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 2 * qi + (r & 1) + 8 * (r >> 1);
      if (!((live >> t) & 1u)) {
        sb[r] = 0u;
#pragma unroll
        for (int w = 0; w < kWords; ++w) v[r][w] = 0u;
      }
    }
  }
  if constexpr (KV == kKvFp4) {
    sc[0] = e4m3x2_to_f16x2(sb[0] | (sb[1] << 8));
    sc[1] = e4m3x2_to_f16x2(sb[2] | (sb[3] << 8));
  }
}

// The row, head and visible tokens of column c.
struct RowsMask {
  const uint32_t* tree;  // the sequence's ancestor masks, or null
  int first_new, sinks, window;
  // whether row i (of the new tokens) sees the token at `pos`, a position below the context's end
  template <bool WIN>
  __device__ __forceinline__ bool sees(int i, int pos) const {
    if (tree) return pos < first_new || ((tree[i] >> (pos - first_new)) & 1u) != 0;
    const int own = first_new + i;
    return pos <= own && (!WIN || pos > own - window || pos < sinks);
  }
};

template <int D, int NT, int KV, bool WIN>
__global__ void __launch_bounds__((RowsTraits<D, NT, KV>::kThreads), (RowsTraits<D, NT, KV>::kMinBlocks))
    rows_mma_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv) {
  using T = RowsTraits<D, NT, KV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gi = lane >> 2, qi = lane & 3;
  const int part = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, G = Hq / Hkv;
  const int R = p.q_len * G;  // columns in use
  const int ppp = p.pages_per_partition;
  const int pbeg = part * ppp;
  // the warp's j-th page: steps of kPP consecutive pages, dealt to the warps in turn
  auto page_no = [&](int j) { return pbeg + (warp + T::kWarps * (j / T::kPP)) * T::kPP + j % T::kPP; };
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  // without a window the first block ids depend on the partition only: load them with the length
  const int row0 = page_no(lane), row1 = page_no(32 + lane);
  const int raw0 = !WIN && row0 < p.max_blocks_per_seq ? bt[row0] : -1;
  const int raw1 = !WIN && row1 < p.max_blocks_per_seq ? bt[row1] : -1;
  const int L = context_len(p, b, part == 0 && g == 0 && threadIdx.x == 0);
  const int first_new = L - p.q_len;

  if (first_new < 0 && part == 0 && threadIdx.x == 0) record_error(p.err, kErrShortContext);
  if (L <= 0) {  // no token to attend to: zeros
    if (part == 0)
      for (int idx = threadIdx.x; idx < R * D; idx += T::kThreads) {
        const int c = idx / D;
        p.out[(((size_t)b * p.q_len + c / G) * Hq + g * G + c % G) * D + idx % D] = __float2bfloat16(0.f);
      }
    return;
  }
  const int lo_first = WIN ? max(0, first_new + 1 - p.window) : 0;  // window begin of the first row
  const int lo_last = WIN ? max(0, L - p.window) : 0;               // and of the last
  PageSpan span = {0, 0, (L + T::kBS - 1) / T::kBS};
  if constexpr (WIN) span = page_span(span.count, lo_first, p.sinks, 1);
  const int npages = span.count;  // pages that some row sees
  if (pbeg >= npages) return;
  const int pend = min(npages, pbeg + ppp);
  const int nparts = (npages + ppp - 1) / ppp;
  RowsMask mask = {p.tree_mask ? p.tree_mask + (size_t)b * p.q_len : nullptr, first_new, p.sinks, p.window};

  if (!T::kFp4 && threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
  }
  uint8_t* stages = smem + warp * T::kStages * T::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kDataRegion) + warp * T::kStages;  // (not 4-bit)
  const int nsteps = (pend - pbeg + T::kPP - 1) / T::kPP;
  const int nk = warp < nsteps ? (nsteps - warp + T::kWarps - 1) / T::kWarps : 0;  // the warp's steps
  if (!T::kFp4 && lane == 0) {
#pragma unroll
    for (int s = 0; s < T::kStages; ++s) mbar_init(smem_addr(&bars[s]), 1);
    fence_mbar_init();
  }
  __syncwarp();

  // block ids (E4M3: and scales) of the warp's pages, two windows of 32 in lane registers
  auto load_window = [&](int jb) {
    const int v = page_no(jb + lane);
    return v < pend ? bt[WIN ? span.real(v) : v] : -1;
  };
  auto load_scale = [&](const float* sc, int id) {
    return (T::kFp8 && id >= 0 && id < p.num_blocks) ? sc[(size_t)id * Hkv + g] : 1.f;
  };
  int wb = 0;
  int idw0 = WIN ? load_window(0) : row0 < pend ? raw0 : -1;
  int idw1 = WIN ? load_window(32) : row1 < pend ? raw1 : -1;
  float ksw0 = load_scale(p.k_scale, idw0), vsw0 = load_scale(p.v_scale, idw0);
  float ksw1 = load_scale(p.k_scale, idw1), vsw1 = load_scale(p.v_scale, idw1);
  auto id_of = [&](int j) {  // j in [wb, wb + 64), warp-uniform
    const int o = j - wb;
    return o < 32 ? __shfl_sync(0xffffffffu, idw0, o) : __shfl_sync(0xffffffffu, idw1, o - 32);
  };
  const uint64_t kv_policy = l2_evict_first_policy();
  // 4-bit pages: lanes take 16-byte pieces, the codes of each page in whole-warp copies, then the scales of
  // all the step's pages in one (lane / kScalePieces of them: K, V of the first page, K, V of the second).
  constexpr int kScalePieces = D / 16;  // 16-byte pieces of a page's scales
  const bool scale_v = (lane / kScalePieces) & 1;
  const int scale_page = lane / (2 * kScalePieces);
  const unsigned block_bytes = (unsigned)Hkv * T::kPageBytes;  // at most 65535 * 1152
  const unsigned head = (unsigned)g * T::kPageBytes + lane * 16;
  auto issue = [&](int k) {  // whole warp: start the copies of the warp's k-th step
    int ids[T::kPP];
    bool ok[T::kPP];
#pragma unroll
    for (int pp = 0; pp < T::kPP; ++pp) {
      ids[pp] = id_of(k * T::kPP + pp);
      ok[pp] = (unsigned)ids[pp] < (unsigned)p.num_blocks;
      if (!ok[pp] && lane == 0 && page_no(k * T::kPP + pp) < pend) record_error(p.err, kErrBlockId);
    }
    const int s = k % T::kStages;
    const uint32_t stage = smem_addr(stages + s * T::kStageBytes);
    if constexpr (T::kFp4) {
      using P = Fp4Page<D>;
#pragma unroll
      for (int pp = 0; pp < T::kPP; ++pp) {
        if (!ok[pp]) continue;
        const uint64_t at = (uint64_t)(unsigned)ids[pp] * block_bytes + head;
        const uint32_t dst = stage + pp * 2 * T::kPageBytes + lane * 16;
#pragma unroll
        for (int i = 0; i < P::kCodeBytes; i += 512) {
          cp_async_16(dst + i, p.k_cache + at + i, kv_policy);
          cp_async_16(dst + T::kPageBytes + i, p.v_cache + at + i, kv_policy);
        }
      }
      static_assert(T::kPP <= 2 && 2 * 2 * kScalePieces <= 32, "a step's scales are one copy a lane");
      const int sid = scale_page == 0 ? ids[0] : ids[T::kPP - 1];
      if (scale_page < T::kPP && (unsigned)sid < (unsigned)p.num_blocks) {
        // piece lane % kScalePieces of that page's scales (head holds lane * 16 already)
        const int piece = P::kCodeBytes - (lane - lane % kScalePieces) * 16;
        cp_async_16(stage + (2 * scale_page + scale_v) * T::kPageBytes + piece + lane * 16,
                    (scale_v ? p.v_cache : p.k_cache) + ((uint64_t)(unsigned)sid * block_bytes + head) + piece, kv_policy);
      }
      return;
    }
    if (lane != 0) return;
    const uint32_t bar = smem_addr(&bars[s]);
    static_assert(T::kFp4 || T::kPP == 1, "one page a step");
    if (!ok[0]) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, 2 * T::kPageBytes);
    const int row = (int)(((int64_t)ids[0] * Hkv + g) * T::kBS);
#pragma unroll
    for (int j = 0; j < T::kBoxes; ++j) {
      const int x = j * (T::kBf16 ? 64 : 128);
      tma_load_2d_hint(stage + j * (16 * 128), &tmk, x, row, bar, kv_policy);
      tma_load_2d_hint(stage + T::kPageBytes + j * (16 * 128), &tmv, x, row, bar, kv_policy);
    }
  };
#pragma unroll
  for (int k = 0; k < T::kStages; ++k) {
    if (k < nk) issue(k);
    if constexpr (T::kFp4) cp_async_commit();  // one group a step, empty or not
  }

  // B fragments of Q^T (column gi of each n-tile), two k-steps a 16-byte piece, in shared memory: they are
  // the same for every warp, and registers hold the accumulators of more CTAs instead.  Byte caches: each
  // row scaled by a power of two before its f16 re-encoding; mul[nt][e] = what turns a raw score of column
  // 2qi + e into base-2 units.
  uint4* q_frag = reinterpret_cast<uint4*>(smem + T::kDataRegion + T::kBarRegion);
  float mul[NT][2];
  const float head_mul = p.scale_log2 * (T::kFp4 && p.k_scale ? p.k_scale[g] : 1.f);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = 8 * nt + gi;
    const bool real = c < R;
    const __nv_bfloat16* qrow = p.q + (((size_t)b * p.q_len + (real ? c / G : 0)) * Hq + g * G + (real ? c % G : 0)) * D;
    uint2 xs[T::kKSteps];
    uint32_t emax = 0;
#pragma unroll
    for (int st = 0; st < T::kKSteps; ++st) {
      xs[st] = real ? *reinterpret_cast<const uint2*>(qrow + q_dim<D, KV>(qi, st)) : make_uint2(0u, 0u);
      if constexpr (!T::kBf16) emax = max(emax, max(bf16x2_max_exp(xs[st].x), bf16x2_max_exp(xs[st].y)));
    }
    mul[nt][0] = mul[nt][1] = head_mul;
    if constexpr (!T::kBf16) {
      emax = max(emax, __shfl_xor_sync(0xffffffffu, emax, 1));
      emax = max(emax, __shfl_xor_sync(0xffffffffu, emax, 2));
      const int kq = f16_prescale_exp(emax);
      const float up = exp2_int(kq);
#pragma unroll
      for (int st = 0; st < T::kKSteps; ++st) {
        const float2 lo = bf16x2_to_f2(xs[st].x), hi = bf16x2_to_f2(xs[st].y);
        xs[st] = make_uint2(pack_f16(lo.x * up, lo.y * up), pack_f16(hi.x * up, hi.y * up));
      }
      // score column 2qi + e of the tile is the row whose exponent sits in the lanes of row 2qi + e
      mul[nt][0] *= exp2_int(-__shfl_sync(0xffffffffu, kq, (2 * qi) * 4));
      mul[nt][1] *= exp2_int(-__shfl_sync(0xffffffffu, kq, (2 * qi + 1) * 4));
    }
#pragma unroll
    for (int st = 0; st < T::kKSteps; st += 2)
      if (st / 2 % T::kWarps == warp)
        q_frag[(nt * (T::kKSteps / 2) + st / 2) * 32 + lane] = make_uint4(xs[st].x, xs[st].y, xs[st + 1].x, xs[st + 1].y);
  }
  __syncthreads();

  float o[NT][T::kMTiles][4];
  float m[NT][2], l[NT][2];  // running maximum and sum of columns 2qi, 2qi+1 (l: this thread's tokens)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < T::kMTiles; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }
  float lv_top = kVFoldMin;

  int k_done = 0;
  bool timed_out = false;
  for (int k = 0; k < nk; ++k) {
    const int s = k % T::kStages;
    if constexpr (T::kFp4) {
      cp_async_wait<T::kStages - 1>();  // this lane's pieces of the step; the others' by the warp barrier
      __syncwarp();
    } else {
      const bool landed = mbar_wait(smem_addr(&bars[s]), (k / T::kStages) & 1);
      if (__any_sync(0xffffffffu, !landed)) {
        timed_out = true;
        break;
      }
      k_done = k + 1;
    }
    if (k * T::kPP == wb + 32) {  // slide the windows (the issue below looks at most kStages ahead)
      wb += 32;
      idw0 = idw1;
      idw1 = load_window(wb + 32);
      if constexpr (T::kFp8) {
        ksw0 = ksw1;
        vsw0 = vsw1;
        ksw1 = load_scale(p.k_scale, idw1);
        vsw1 = load_scale(p.v_scale, idw1);
      }
    }
    // the step's pages: the tokens that some row sees (none where there is no page), and whether every row
    // sees every token
    int tok0[T::kPP];
    uint32_t live[T::kPP];
    bool whole = true, any_page = false;
#pragma unroll
    for (int pp = 0; pp < T::kPP; ++pp) {
      const int pb = id_of(k * T::kPP + pp);
      const bool ok = pb >= 0 && pb < p.num_blocks;
      const int v_at = page_no(k * T::kPP + pp);
      tok0[pp] = (WIN ? span.real(v_at) : v_at) * T::kBS;
      const bool all = ok && tok0[pp] + T::kBS <= first_new + (mask.tree ? 0 : 1) &&
                       (!WIN || tok0[pp] >= lo_last || tok0[pp] + T::kBS <= p.sinks);
      live[pp] = 0xffffu;
      if (!all) {
        uint64_t some = low_bits64(L - tok0[pp]);
        if constexpr (WIN) some &= low_bits64(p.sinks - tok0[pp]) | ~low_bits64(lo_first - tok0[pp]);
        live[pp] = ok ? (uint32_t)some & 0xffffu : 0u;
      }
      whole = whole && all;
      any_page = any_page || ok;
    }
    if (any_page) {
      const uint8_t* kp = stages + s * T::kStageBytes;

      // ---- S^T = K . Q^T ----
      float x[T::kPP][NT][4];
#pragma unroll
      for (int pp = 0; pp < T::kPP; ++pp) {
        uint32_t a[T::kKSteps][4];
        k_fragments<D, KV>(kp + pp * 2 * T::kPageBytes, gi, qi, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          x[pp][nt][0] = x[pp][nt][1] = x[pp][nt][2] = x[pp][nt][3] = 0.f;
#pragma unroll
          for (int st = 0; st < T::kKSteps; st += 2) {
            const uint4 qf = q_frag[(nt * (T::kKSteps / 2) + st / 2) * 32 + lane];
            mma_16816<T::kBf16>(x[pp][nt], a[st][0], a[st][1], a[st][2], a[st][3], qf.x, qf.y);
            mma_16816<T::kBf16>(x[pp][nt], a[st + 1][0], a[st + 1][1], a[st + 1][2], a[st + 1][3], qf.z, qf.w);
          }
        }
      }

      // ---- online softmax: x[..][0..1] = token gi, columns 2qi, 2qi+1; x[..][2..3] = token gi + 8 ----
      float ks = 1.f;
      VScaleFold vf = {0.f, 1.f, 0u};
      if constexpr (T::kFp8) {
        const int o32 = k - wb;
        ks = __shfl_sync(0xffffffffu, ksw0, o32);
        vf = fold_v_scale(__shfl_sync(0xffffffffu, vsw0, o32), lv_top);
      }
      bool need = false;
      float top[NT][2];  // the step's largest score of the thread's columns
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int pp = 0; pp < T::kPP; ++pp) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[pp][nt][e] = T::kFp8 ? fmaf(x[pp][nt][e], mul[nt][e & 1] * ks, vf.lv) : x[pp][nt][e] * mul[nt][e & 1];
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 8 * nt + 2 * qi + (e & 1), t = gi + 8 * (e >> 1);
              const bool see = ((live[pp] >> t) & 1u) && (c >= R || mask.template sees<WIN>(c / G, tok0[pp] + t));
              if (!see) x[pp][nt][e] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nt][e] = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
#pragma unroll
          for (int pp = 1; pp < T::kPP; ++pp) top[nt][e] = fmaxf(top[nt][e], fmaxf(x[pp][nt][e], x[pp][nt][e + 2]));
          need |= top[nt][e] > m[nt][e] + kTau;
        }
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float lm = top[nt][e];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) lm = fmaxf(lm, __shfl_xor_sync(0xffffffffu, lm, sh));
            const float n = fmaxf(m[nt][e], lm);
            const float al = n == -INFINITY ? 1.f : fast_exp2(m[nt][e] - n);
            if constexpr (T::kFp8)
              l[nt][e] = n == -INFINITY ? 0.f : scale_exp2(l[nt][e], m[nt][e] - n);
            else
              l[nt][e] *= al;
            m[nt][e] = n;
#pragma unroll
            for (int i = 0; i < T::kMTiles; ++i) {
              o[nt][i][e] *= al;
              o[nt][i][e + 2] *= al;
            }
          }
        }
      }
#pragma unroll
      for (int pp = 0; pp < T::kPP; ++pp) {
        // B fragments of P^T: b[nt][0] = tokens 2qi, 2qi+1 of column gi, b[nt][1] = tokens 2qi+8, 2qi+9
        uint32_t bf[NT][2], bl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = fast_exp2(x[pp][nt][e] - m[nt][e & 1]);
          if (!whole)  // a column that has seen nothing yet has no maximum
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = x[pp][nt][e] == -INFINITY ? 0.f : w[e];
          l[nt][0] += (w[0] + w[2]) * vf.rvs;
          l[nt][1] += (w[1] + w[3]) * vf.rvs;
          if constexpr (T::kBf16) {
            bf[nt][0] = movmatrix_trans(pack_bf16(w[0], w[1]));
            bf[nt][1] = movmatrix_trans(pack_bf16(w[2], w[3]));
            bl[nt][0] = movmatrix_trans(pack_bf16(bf16_rem(w[0]), bf16_rem(w[1])));
            bl[nt][1] = movmatrix_trans(pack_bf16(bf16_rem(w[2]), bf16_rem(w[3])));
          } else {
            bf[nt][0] = movmatrix_trans(pack_f16(w[0], w[1]) ^ vf.neg);
            bf[nt][1] = movmatrix_trans(pack_f16(w[2], w[3]) ^ vf.neg);
          }
        }

        // ---- O^T += V^T . P^T ----
        constexpr int kWords = T::kRowBytes / 32;
        uint32_t v[4][kWords], sc[2];
        v_words<D, KV>(kp + pp * 2 * T::kPageBytes + T::kPageBytes, gi, qi, live[pp], v, sc);
        auto pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816<T::kBf16>(o[nt][i], a0, a1, a2, a3, bf[nt][0], bf[nt][1]);
            if constexpr (T::kBf16) mma_16816<true>(o[nt][i], a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
          }
        };
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          if constexpr (T::kBf16) {
            pv(w, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
               __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632));
          } else if constexpr (T::kFp8) {
            const uint32_t xa = __byte_perm(v[0][w], v[1][w], 0x5140), ya = __byte_perm(v[0][w], v[1][w], 0x7362);
            const uint32_t xb = __byte_perm(v[2][w], v[3][w], 0x5140), yb = __byte_perm(v[2][w], v[3][w], 0x7362);
            pv(2 * w, e4m3x2_to_f16x2(xa), e4m3x2_to_f16x2(xa >> 16), e4m3x2_to_f16x2(xb), e4m3x2_to_f16x2(xb >> 16));
            pv(2 * w + 1, e4m3x2_to_f16x2(ya), e4m3x2_to_f16x2(ya >> 16), e4m3x2_to_f16x2(yb),
               e4m3x2_to_f16x2(yb >> 16));
          } else {
            // byte i of lo / hi: the low / high nibbles (dims 2i / 2i+1) of two tokens
            uint32_t lo[4], hi[4], lo8[4], hi8[4];
            e2m1x8_to_f16x2((v[0][w] & 0x0f0f0f0fu) | ((v[1][w] << 4) & 0xf0f0f0f0u), lo);
            e2m1x8_to_f16x2(((v[0][w] >> 4) & 0x0f0f0f0fu) | (v[1][w] & 0xf0f0f0f0u), hi);
            e2m1x8_to_f16x2((v[2][w] & 0x0f0f0f0fu) | ((v[3][w] << 4) & 0xf0f0f0f0u), lo8);
            e2m1x8_to_f16x2(((v[2][w] >> 4) & 0x0f0f0f0fu) | (v[3][w] & 0xf0f0f0f0u), hi8);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              pv(4 * w + i, mul_f16x2(lo[i], sc[0]), mul_f16x2(hi[i], sc[0]), mul_f16x2(lo8[i], sc[1]),
                 mul_f16x2(hi8[i], sc[1]));
          }
        }
      }
    }
    __syncwarp();
    if (k + T::kStages < nk) issue(k + T::kStages);
    if constexpr (T::kFp4) cp_async_commit();
  }
  if constexpr (T::kFp4) cp_async_wait<0>();
  if (timed_out) {
    // let every copy this warp started land (bounded) before its stages are reused
    if (lane == 0) {
      record_error(p.err, kErrTimeout);
      const int issued = min(nk, k_done + T::kStages);
      for (int k = k_done; k < issued; ++k) mbar_wait(smem_addr(&bars[k % T::kStages]), (k / T::kStages) & 1);
    }
    __syncwarp();
  }
  // the merge kernel (launched as a programmatic dependent) may start its prologue now
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  __syncthreads();  // every warp is done with its stages
  float* wacc = reinterpret_cast<float*>(smem);   // [kWarps][kCols][D]
  float* wm = wacc + T::kWarps * T::kCols * D;    // [kWarps][kCols]
  float* wl = wm + T::kWarps * T::kCols;          // [kWarps][kCols]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], sh);
      const int c = 8 * nt + 2 * qi + e;
      if (gi == 0) {
        wm[warp * T::kCols + c] = m[nt][e];
        wl[warp * T::kCols + c] = l[nt][e];
      }
#pragma unroll
      for (int i = 0; i < T::kMTiles; ++i)
        *reinterpret_cast<float2*>(wacc + (warp * T::kCols + c) * D + o_dim<D, KV>(gi, i)) =
            make_float2(o[nt][i][e], o[nt][i][e + 2]);
    }
  }
  __syncthreads();
  // combine the warps; store finished rows, or the partition's normalised rows and log2-sum-exps
  const float v_head = T::kFp4 && p.v_scale ? p.v_scale[g] : 1.f;
  for (int idx = threadIdx.x; idx < R * (D / 4); idx += T::kThreads) {
    const int c = idx / (D / 4), dd = (idx % (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < T::kWarps; ++w) M = fmaxf(M, wm[w * T::kCols + c]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < T::kWarps; ++w) {
        const float half = fast_exp2(0.5f * (wm[w * T::kCols + c] - M));  // (E4M3: as scale_exp2)
        const float f = T::kFp8 ? half * half : fast_exp2(wm[w * T::kCols + c] - M);
        const float4 v = *reinterpret_cast<const float4*>(wacc + (w * T::kCols + c) * D + dd);
        lsum += T::kFp8 ? half * (half * wl[w * T::kCols + c]) : f * wl[w * T::kCols + c];
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      const float inv = v_head / lsum;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    const size_t row = ((size_t)b * p.q_len + c / G) * Hq + g * G + c % G;
    if (nparts == 1) {
      *reinterpret_cast<uint2*>(p.out + row * D + dd) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    } else {
      const size_t at = row * p.max_partitions + part;
      *reinterpret_cast<float4*>(p.part_o + at * D + dd) = acc;
      if (dd == 0) p.part_lse[at] = M == -INFINITY ? -INFINITY : M + __log2f(lsum);
    }
  }
}

template <int D, int NT, int KV, bool WIN>
cudaError_t rows_launch(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using T = RowsTraits<D, NT, KV>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(rows_mma_kernel<D, NT, KV, WIN>), T::kSmem);
  if (e != cudaSuccess) return e;
  dim3 grid(p.max_partitions, p.num_kv_heads, p.num_seqs);
  rows_mma_kernel<D, NT, KV, WIN><<<grid, T::kThreads, T::kSmem, st>>>(p, tk, tv);
  return cudaGetLastError();
}

template <int D, int KV, bool WIN>
cudaError_t rows_tiles(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  const int nt = (l.group * p.q_len + 7) / 8;
  if (nt == 1) return rows_launch<D, 1, KV, WIN>(p, tk, tv, l.stream);
  if (nt == 2) return rows_launch<D, 2, KV, WIN>(p, tk, tv, l.stream);
  if constexpr (KV != kKvBf16) {  // (more bf16 rows run the tile kernel)
    if (nt == 3) return rows_launch<D, 3, KV, WIN>(p, tk, tv, l.stream);
    if (nt == 4) return rows_launch<D, 4, KV, WIN>(p, tk, tv, l.stream);
  }
  return cudaErrorInvalidConfiguration;
}

}  // namespace
}  // namespace pa
