// Device helpers shared by the paged-attention kernels (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

// Bits of the per-device error word.
constexpr unsigned kErrBlockId = 1u;       // a block-table entry outside [0, num_blocks)
constexpr unsigned kErrShortContext = 2u;  // a row that sees no token, or a context above the bound
constexpr unsigned kErrTimeout = 4u;       // an mbarrier wait hit its iteration limit
constexpr unsigned kErrBadInput = 8u;      // a token id outside the vocabulary, or a distribution with no mass

// Upper bounds before a wait gives up (a page copy lands in microseconds).  kWaitLimit counts
// mbarrier.try_wait polls, each of which suspends the thread for up to a hardware time limit
// while the phase is incomplete (3.8 us per poll measured on GB300): 2^18 polls is about one
// second.  kSpinLimit counts iterations of the issuer loops that probe several barriers with the
// non-suspending mbarrier.test_wait (tens of ns each): 2^22 iterations is a fraction of a second.
constexpr uint32_t kWaitLimit = 1u << 18;
constexpr uint32_t kSpinLimit = 1u << 22;

constexpr float kLog2e = 1.4426950408889634f;

// What an attention kernel reads of a sequence, and what it writes beside the rows (a template parameter, so
// that a form costs the others nothing).
constexpr int kFormAll = 0;     // every token
constexpr int kFormWindow = 1;  // a window of the last tokens, and the first ones
constexpr int kFormBlocks = 2;  // the blocks that a list names for each (sequence, kv head)
constexpr int kFormOwn = 3;     // what lies behind the prefix that a group of sequences shares
constexpr int kFormPrefix = 4;  // the shared prefix, for the rows of all of its group's sequences (tile kernel)
constexpr int kFormScores = 5;  // every token; the scores are kept for the tokens' weights

// Arguments of every attention kernel.  Pointers are device pointers.
struct AttnParams {
  const __nv_bfloat16* q;       // [B, q_len, Hq, d]
  const uint8_t* k_cache;       // [NB, Hkv, bs, d] (bf16 or E4M3 bytes)
  const uint8_t* v_cache;
  const int32_t* block_table;   // [B, max_blocks_per_seq]
  const int32_t* context_lens;  // [B]
  const float* k_scale;         // [NB, Hkv] (fp8 only)
  const float* v_scale;
  __nv_bfloat16* out;           // [B, q_len, Hq, d]
  float* part_o;                // [B, q_len, Hq, P, d]  normalised partial outputs
  float* part_lse;              // [B, q_len, Hq, P]     log2 of each partition's softmax mass
  const uint32_t* tree_mask;    // [B, q_len] ancestor bitmasks over the new tokens, or null (causal)
  const int32_t* query_start_loc;  // [B + 1] packed query rows per sequence (prefill), or null
  unsigned* err;                // per-device error word
  int num_seqs;
  int max_blocks_per_seq;
  int num_blocks;
  int q_len;
  int num_q_heads;
  int num_kv_heads;
  int pages_per_partition;
  int max_partitions;
  int max_context_len;          // host-side bound; longer contexts are clamped and flagged
  int total_q;                  // rows of the packed q / out (prefill)
  float scale_log2;             // scale * log2(e): scores are kept in base-2 units
  int window;                   // tokens a row sees up to its own, past the sinks; 0: all
  int sinks;                    // first tokens that stay visible (with a window)
  int page_align;               // window: pages that page_span rounds its edges to (see there)
  const int32_t* blocks;        // kFormBlocks: [B, Hkv, num_listed] block-table columns
  int num_listed;
  const int32_t* group_starts;  // kFormOwn, kFormPrefix: [num_groups + 1] first sequence of each group
  const int32_t* prefix_lens;   // [num_groups] tokens that the sequences of a group share
  int num_groups;
  int max_prefix_len;           // host-side bounds; longer ones are clamped (prefix) or refused (own), and flagged
  int max_own_len;
  int own_partitions;           // partial slots [0, own_partitions) of a row: its own tokens; the rest: the prefix
  int prefix_ppp;               // pages per partition of the prefix
  float* scores;                // kFormScores: [B, Hkv, max_context_len, G] base-2 scores
  float* lse;                   // [B, Hq] log2 of each row's softmax mass
  float* weights;               // kFormScores, joined: [NB, Hkv, 16] sums of the tokens' weights
  float decay;
};

constexpr int kJoinMax = 8;  // partitions of a cluster at most
constexpr int kNoBlock = -0x7fffffff - 1;  // kFormBlocks: an unused entry of the list, in place of a block id

// The group of sequences [first, last) that share `tokens` prefix tokens, a whole number of blocks.
struct PrefixGroup {
  int first, last, tokens;
};
// Group i, with every bound checked: offsets that do not fit leave it empty.  Flags what it finds wrong when asked.
__device__ __forceinline__ PrefixGroup prefix_group(const AttnParams& p, int i, unsigned& wrong) {
  PrefixGroup r = {p.group_starts[i], p.group_starts[i + 1], p.prefix_lens[i]};
  if (r.first < 0 || r.last < r.first || r.last > p.num_seqs) {
    wrong |= kErrBadInput;
    r.first = r.last = 0;
  }
  r.tokens = max(r.tokens, 0) / 16 * 16;
  if (r.tokens > p.max_prefix_len) {
    if (r.last > r.first) wrong |= kErrShortContext;  // (a group of no sequences shares nothing)
    r.tokens = p.max_prefix_len / 16 * 16;
  }
  return r;
}
// The grid over the own tokens is a programmatic dependent of the one over the prefixes, which it does not read from: they
// share the SMs.  Its first CTA ends after that grid, so that what waits for this one (the merge) has both.  Called
// on every way out of a kernel's first CTA.
__device__ __forceinline__ void after_prefixes() {
  if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Whether a sequence's new rows all lie behind its prefix, and no more than the bound does.
__device__ __forceinline__ bool own_tokens_fit(const AttnParams& p, int L, int prefix) {
  return (prefix == 0 || L - p.q_len >= prefix) && L - prefix <= p.max_own_len;
}
// Prefix tokens of sequence b: those of the first group that holds it, or 0.  Whole warp.
__device__ __forceinline__ int prefix_of(const AttnParams& p, int b) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < p.num_groups; i0 += 32) {
    PrefixGroup r = {0, 0, 0};
    unsigned wrong = 0;
    if (i0 + lane < p.num_groups) r = prefix_group(p, i0 + lane, wrong);
    const unsigned in = __ballot_sync(0xffffffffu, b >= r.first && b < r.last);
    if (in) return __shfl_sync(0xffffffffu, r.tokens, __ffs(in) - 1);
  }
  return 0;
}

// The pages of a sequence (or tile) that a window with sinks leaves, numbered without the gap: page v
// of [0, count) is column v of the block table before `head` and column v + gap from there on.  With
// align > 1 both edges of the gap are whole multiples of it (a few unseen pages count too).
struct PageSpan {
  int head, gap, count;
  __device__ __forceinline__ int real(int v) const { return v < head ? v : v + gap; }
};
__device__ __forceinline__ PageSpan page_span(int npages, int win_lo, int sinks, int align) {
  const int head = ((sinks + 15) / 16 + align - 1) / align * align;
  const int first = win_lo / 16 / align * align;
  const int gap = max(0, first - head);
  return {head, gap, npages - gap};
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarrier + bulk asynchronous copy (TMA unit) -------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Non-blocking probe of one phase (never suspends the thread: for loops that poll several
// barriers, where a suspended probe of one would miss another one completing).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait on one phase of an mbarrier.  Returns false when `limit` polls did not see it.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t limit = kWaitLimit) {
  for (uint32_t it = 0; it < limit; ++it)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// One contiguous global -> shared copy through the TMA unit, completing on `bar`.
// dst, src 16-byte aligned; bytes a multiple of 16.
__device__ __forceinline__ void bulk_copy_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 16 bytes global -> shared per thread, without a barrier: completion by commit / wait groups of the
// issuing thread.  For copies too small to be worth the bulk-copy unit's uniform operands.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of the thread's latest groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- arithmetic ------------------------------------------------------------------------------

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// l * 2^x for x down to -252: a row sum whose maximum moved by more than a float's exponents (E4M3 page scales
// are part of the maximum, but not of the sum).
__device__ __forceinline__ float scale_exp2(float l, float x) {
  const float h = fast_exp2(0.5f * x);
  return l * h * h;
}

union F2U {
  float2 f;
  unsigned long long u;
};

// d = a * b + c on a pair of fp32 lanes (one sm_100-family FFMA2 instruction).
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  F2U ua, ub, uc, ud;
  ua.f = a;
  ub.f = b;
  uc.f = c;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(ud.u) : "l"(ua.u), "l"(ub.u), "l"(uc.u));
  return ud.f;
}

// Two packed bf16 -> two fp32 (a bf16 is the upper half of a binary32: exact).
__device__ __forceinline__ float2 bf16x2_to_f2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// acc.x += low bf16 of w, acc.y += high bf16 of w, in fp32: the sm_100-family mixed-precision add
// (the bf16 operand widens exactly, one rounding of the sum), bit for bit
// ffma2(bf16x2_to_f2(w), {1, 1}, acc) without the two unpacking instructions.
__device__ __forceinline__ float2 add_bf16x2_f2(uint32_t w, float2 acc) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(w));
  return acc;
}

// Two packed E4M3 bytes (low byte first) -> two fp32, through the hardware e4m3x2 -> f16x2
// conversion (exact: every E4M3 value is an fp16 value).
__device__ __forceinline__ float2 e4m3x2_to_f2(uint16_t w) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(w));
  __half2 h = *reinterpret_cast<__half2*>(&h2);
  return __half22float2(h);
}

// The scale of an E4M3 page whose largest magnitude is amax (not below the smallest fp32 number: a quotient that underflows to
// zero would make NaNs of the codes).
__device__ __forceinline__ float e4m3_page_scale(float amax) {
  return amax > 0.f ? fmaxf(amax / 448.f, 0x1p-149f) : 1.f;
}

__device__ __forceinline__ void record_error(unsigned* err, unsigned bit) {
  if (err) atomicOr(err, bit);
}

// Whether a context of L tokens has its last n and ends within its block-table row.  L may be any int: nothing
// here overflows.
__device__ __forceinline__ bool context_holds(int L, int n, int max_blocks) {
  return L >= n && L >= 0 && (L >> 4) + ((L & 15) != 0 ? 1 : 0) <= max_blocks;
}

// context_lens[b], clamped to the host-side bound the grid and scratch were sized for (a longer
// context would index past its block-table row); thread 0 of partition 0 flags the clamp.  A negative
// length, however large, is no token: differences of it would wrap round.
__device__ __forceinline__ int context_len(const AttnParams& p, int b, bool flag) {
  int L = p.context_lens[b];
  if (L > p.max_context_len) {
    if (flag) record_error(p.err, kErrShortContext);
    L = p.max_context_len;
  }
  return max(L, 0);
}

// ---- partitions of a row as one cluster ---------------------------------------------------------

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of a CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// A row's softmax mass: sum * 2^top.  (Kept apart: a log2-sum-exp of large sums loses more than the fp32 sum does.)
struct Mass {
  float top, sum;
};

// The cluster's CTAs are the partitions of `rows` rows; each has left its normalised rows [rows][D] and their masses
// [rows] in shared memory (the same offsets in all).  Each joins a share of the outputs and stores them, out_row(r) being
// row r's place, and, with ROWS, every row's (top, 1 / sum) in joined[r].  Ends with the CTA's arrival: it may not
// leave before cluster_wait().  All threads; a barrier of the CTA must follow before `joined` is read.
template <int D, bool ROWS, class OutRow>
__device__ __forceinline__ void join_partitions(const float* part_o, const Mass* part_mass, int rows, Mass* joined,
                                                OutRow out_row) {
  const int parts = gridDim.x, rank = blockIdx.x;
  const uint32_t o_at = smem_addr(part_o), m_at = smem_addr(part_mass);
  cluster_arrive();
  cluster_wait();
  for (int i = rank * blockDim.x + threadIdx.x; i < rows * (D / 4); i += parts * blockDim.x) {
    const int r = i / (D / 4), dd = i % (D / 4) * 4;
    float m[kJoinMax], l[kJoinMax], M = -INFINITY;
    float4 o[kJoinMax];
#pragma unroll
    for (int q = 0; q < kJoinMax; ++q) {  // all loads in flight together
      m[q] = -INFINITY;
      if (q < parts) {
        m[q] = cluster_ld(cluster_addr(m_at + r * 8, q));
        l[q] = cluster_ld(cluster_addr(m_at + r * 8 + 4, q));
        o[q] = cluster_ld4(cluster_addr(o_at + (r * D + dd) * 4, q));
      }
    }
#pragma unroll
    for (int q = 0; q < kJoinMax; ++q) M = fmaxf(M, m[q]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kJoinMax; ++q) {
      if (q >= parts || m[q] == -INFINITY) continue;
      const float w = scale_exp2(l[q], m[q] - M);
      sum += w;
      acc.x += w * o[q].x;
      acc.y += w * o[q].y;
      acc.z += w * o[q].z;
      acc.w += w * o[q].w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;  // (nothing seen: zeros)
    __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(out_row(r) + dd) =
        make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&c));
  }
  if constexpr (ROWS) {
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
      float M = -INFINITY, sum = 0.f;
      for (int q = 0; q < parts; ++q) M = fmaxf(M, cluster_ld(cluster_addr(m_at + r * 8, q)));
      for (int q = 0; q < parts; ++q)
        sum += scale_exp2(cluster_ld(cluster_addr(m_at + r * 8 + 4, q)), cluster_ld(cluster_addr(m_at + r * 8, q)) - M);
      joined[r] = {M, 1.f / sum};
    }
  }
  cluster_arrive();
}

// The step's weights of the CTA's tokens [t0, t1) of (b, g), from their scores [t1 - t0][G] and the rows' (top, 1 / sum),
// both in shared memory, folded into the sums (L: the context's length; t0 a block's first token).  A thread takes a quarter
// of a block's tokens at a time, two of them in flight.
__device__ __forceinline__ void fold_weights(const AttnParams& p, int b, int g, int G, int t0, int t1, int L,
                                             const float* scores, const Mass* rows) {
  constexpr int kFlight = 2;
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  const int step = 4 * blockDim.x;
  for (int u = t0 + 4 * threadIdx.x; u < t1; u += kFlight * step) {
    int pb[kFlight];
    float4 old[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) pb[f] = u + f * step < t1 ? bt[(u + f * step) / 16] : -1;
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (pb[f] >= p.num_blocks) pb[f] = -1;  // (flagged by the attention)
      old[f] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (pb[f] >= 0 && p.decay != 0.f)
        old[f] = *reinterpret_cast<const float4*>(p.weights + ((size_t)pb[f] * p.num_kv_heads + g) * 16 + (u + f * step) % 16);
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int t = u + f * step;
      if (t >= t1 || pb[f] < 0) continue;
      const float o4[4] = {old[f].x, old[f].y, old[f].z, old[f].w};
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = 0.f;
        const float* x = scores + (t + i - t0) * G;
        if (t + i < t1)
          for (int h = 0; h < G; ++h) w[i] += fast_exp2(x[h] - rows[h].top) * rows[h].sum;
        if (t + i < L - 1 && p.decay != 0.f) w[i] += o4[i] * p.decay;  // (one rounding at the size of the sum)
      }
      float* dst = p.weights + ((size_t)pb[f] * p.num_kv_heads + g) * 16 + t % 16;
      if (t + 4 <= t1) {
        *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i < t1) dst[i] = w[i];
      }
    }
  }
}

// Last step of a split-KV partition: combine the per-warp online-softmax states that the CTA's
// warps left in shared memory (wacc [W][G][D] unnormalised outputs, wm [W][G] running maxima and
// wl [W][G] sums, base 2) and store either the finished bf16 rows (the sequence has one
// partition) or the normalised partial output and its log2-sum-exp for the merge kernel.
// JOIN: the partial goes to shared memory for join_partitions, whatever nparts is.
template <int G, int D, int W, bool E4M3 = false, int FORM = kFormAll, bool JOIN = false>
__device__ __forceinline__ void store_partition(const AttnParams& p, const float* wacc, const float* wm,
                                                const float* wl, int b, int g, int part, int nparts,
                                                float* join_o = nullptr, Mass* join_mass = nullptr) {
  const int Hq = p.num_q_heads;
  for (int idx = threadIdx.x; idx < G * D; idx += blockDim.x) {
    const int h = idx / D;
    const int dd = idx - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, wm[w * G + h]);
    float o = 0.f, lsum = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if constexpr (E4M3) {  // as scale_exp2
          const float half = fast_exp2(0.5f * (wm[w * G + h] - M));
          lsum += half * (half * wl[w * G + h]);
          o += half * (half * wacc[(w * G + h) * D + dd]);
        } else {
          const float f = fast_exp2(wm[w * G + h] - M);
          lsum += f * wl[w * G + h];
          o += f * wacc[(w * G + h) * D + dd];
        }
      }
      o = o / lsum;
    }
    const int qh = g * G + h;
    if constexpr (JOIN) {
      join_o[idx] = o;
      if (dd == 0) join_mass[h] = {M, lsum};
      continue;
    }
    if (nparts == 1) {
      p.out[((size_t)b * Hq + qh) * D + dd] = __float2bfloat16(o);
      if (FORM == kFormScores && dd == 0) p.lse[(size_t)b * Hq + qh] = M + __log2f(lsum);
    } else {
      const size_t row = ((size_t)b * Hq + qh) * p.max_partitions + part;
      p.part_o[row * D + dd] = o;
      if (dd == 0) p.part_lse[row] = (M == -INFINITY) ? -INFINITY : M + __log2f(lsum);
    }
  }
}

}  // namespace pa
