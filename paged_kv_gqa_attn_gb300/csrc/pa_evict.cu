// Eviction from the cache by accumulated attention weight.
//
// Each (sequence, kv head) keeps the first `sinks` tokens, the last `recent` ones and, up to `keep` in all, those
// whose sums (pa_weights.cu) are the largest, ties to the earliest.  The kept tokens move in order to the blocks
// of another table; the old blocks are only read, so blocks that other sequences share stay whole, every row moves
// independently of the others, and the caller gives the old ones back afterwards.
//
// Contexts of up to 98304 tokens are selected by a cluster of up to eight CTAs for each (sequence, kv head), a share of
// the sums in each one's shared memory as keys.  The k-th largest is found digit by digit (as in pa_topk.cuh),
// each CTA adding its counters to everybody's, and the kept positions go to scratch.  A second kernel moves the rows, its
// warps spread over the device.  Measured with 16 contexts of up to 32768 tokens, 8 heads, 4096 kept: 111 us (116 while
// the selection moved the sums; selected by one CTA each 120; with the second kernel's CTAs started early, to wait on
// the SMs for the first's, 131).  Moved by the selecting clusters instead, after a barrier, over contexts of 2048 to 32768
// tokens and 512 to 4096 kept: 8 (sequence, head) pairs 1.06 to 1.46 times as long (bf16; E4M3 1.0 to 1.83, 4-bit 0.99 to
// 1.33), 16 pairs 1.13 to 1.25 (1.03 to 1.44, 0.99 to 1.18), 32 0.99 to 1.06 (0.95 to 1.03, 0.96 to 1.01), 38 to 128 1.09 to
// 1.47 (1.09 to 1.64, 0.92 to 1.27): few clusters leave most of the device idle, many select, then move, all at once.  Longer
// contexts are selected by one CTA each, with the keys in scratch.  A page and its sums are moved by a warp with all of
// its loads in flight.
//
// bf16 rows and 4-bit rows (codes and their scales belong to the token) move as they are; E4M3 pages get the scale
// amax / 448 of their new tokens, values times the old scales re-encoded in fp32 to nearest even as the append
// does.  Bound by the kept rows' bytes, read and written once.
#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_tc.cuh"
#include "pa_topk.cuh"

namespace pa {
namespace {

constexpr int kMoveWarps = 4;

// The sequence's length inside its table row.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  return max(0, min(p.context_lens[b], p.max_context_len));
}

// Contexts past the cluster's shared memory: one CTA per (kv head, sequence), all_keys [B, Hkv, max_context_len].
__global__ void __launch_bounds__(1024) evict_pick_kernel(const EvictParams p, uint32_t* all_keys) {
  __shared__ TopkShared sh;
  const int g = blockIdx.x, b = blockIdx.y;
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  const int L = evict_len(p, b), k = min(L, p.keep);
  const size_t unit = (size_t)b * p.num_kv_heads + g;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0 && g == 0) {
    p.new_lens[b] = k;
    if (p.context_lens[b] > p.max_context_len) record_error(p.err, kErrShortContext);
  }
  int32_t* kept = p.kept + unit * p.keep;
  const int threads = blockDim.x;
  if (L <= p.keep) {
    for (int i = threadIdx.x; i < L; i += threads) kept[i] = i;
    return;
  }
  uint32_t* keys = all_keys + unit * p.max_context_len;
  // the sums, kBatch of a thread in flight at once (their addresses wait for the table)
  constexpr int kBatch = 8;
  for (int i0 = threadIdx.x; i0 < L; i0 += kBatch * threads) {
    int pb[kBatch];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) pb[j] = i0 + j * threads < L ? bt[(i0 + j * threads) / 16] : 0;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * threads;
      const bool there = pb[j] >= 0 && pb[j] < p.num_blocks;
      if (!there) record_error(p.err, kErrBlockId);
      w[j] = there && i < L ? p.weights[((size_t)pb[j] * p.num_kv_heads + g) * 16 + i % 16] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * threads;
      if (i < L) keys[i] = i < p.sinks || i >= L - p.recent ? kKeyAlways : order_key(w[j]);
    }
  }
  __syncthreads();
  topk_in_order(keys, L, k, sh, [&](int at, int i) { kept[at] = i; });
}

// A warp moves the page (new block, head), rows and sums: lane t < 16 knows where token t comes from.
template <int D, int KV>
__device__ __forceinline__ void move_page(const EvictParams& p, int b, int g, int page, int k) {
  constexpr int kRowBytes = KV == kKvBf16 ? 2 * D : KV == kKvE4m3 ? D : D / 2;  // of codes
  constexpr int kPageBytes = KV == kKvFp4 ? Fp4Page<D>::kBytes : 16 * kRowBytes;
  constexpr int kPieces = kRowBytes / 16;           // 16-byte pieces of a row
  constexpr int kRowsAtOnce = 32 / kPieces, kLoads = 16 / kRowsAtOnce;
  const int lane = threadIdx.x & 31;
  const int valid = min(16, k - page * 16);
  const int nb = p.new_table[(size_t)b * p.new_blocks + page];
  if (nb < 0 || nb >= p.num_blocks) {
    if (lane == 0) record_error(p.err, kErrBlockId);
    return;
  }
  const size_t dst_page = (size_t)nb * p.num_kv_heads + g;
  int src_block = -1, src_slot = 0;
  if (lane < valid) {
    const int at = p.kept[((size_t)b * p.num_kv_heads + g) * p.keep + page * 16 + lane];
    src_block = p.block_table[(size_t)b * p.max_blocks_per_seq + at / 16];
    src_slot = at % 16;
    if (src_block < 0 || src_block >= p.num_blocks) {  // its row and its sum become zeros
      src_block = -1;
      record_error(p.err, kErrBlockId);
    }
  }
  float sum = 0.f;
  if (src_block >= 0) sum = p.weights[((size_t)src_block * p.num_kv_heads + g) * 16 + src_slot];
  const int piece = lane % kPieces, row0 = lane / kPieces;
  uint4 x[2][kLoads];
  float s[2][kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = row0 + i * kRowsAtOnce;
    const int blk = __shfl_sync(0xffffffffu, src_block, r), slot = __shfl_sync(0xffffffffu, src_slot, r);
    const size_t src_page = (size_t)max(blk, 0) * p.num_kv_heads + g;
    const size_t off = src_page * kPageBytes + slot * kRowBytes + piece * 16;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      x[kv][i] = make_uint4(0u, 0u, 0u, 0u);
      s[kv][i] = 0.f;
      if (blk >= 0) {
        x[kv][i] = *reinterpret_cast<const uint4*>((kv ? p.v_cache : p.k_cache) + off);
        if constexpr (KV == kKvE4m3) s[kv][i] = (kv ? p.v_scale : p.k_scale)[src_page];
      }
    }
  }
  if (lane < valid) p.weights[dst_page * 16 + lane] = sum;
  if constexpr (KV == kKvFp4) {  // lanes 0-15: a token's K scales, lanes 16-31: its V scales
    using P = Fp4Page<D>;
    const int t = lane & 15, kv = lane >> 4;
    const int blk = __shfl_sync(0xffffffffu, src_block, t), slot = __shfl_sync(0xffffffffu, src_slot, t);
    if (t < valid) {
      uint32_t w[P::kScaleRow / 4];
      const uint8_t* src = (kv ? p.v_cache : p.k_cache) + ((size_t)max(blk, 0) * p.num_kv_heads + g) * kPageBytes +
                           P::kCodeBytes + slot * P::kScaleRow;
      uint8_t* dst = (kv ? p.v_cache : p.k_cache) + dst_page * kPageBytes + P::kCodeBytes + t * P::kScaleRow;
#pragma unroll
      for (int j = 0; j < P::kScaleRow / 4; ++j) w[j] = blk >= 0 ? reinterpret_cast<const uint32_t*>(src)[j] : 0u;
#pragma unroll
      for (int j = 0; j < P::kScaleRow / 4; ++j) reinterpret_cast<uint32_t*>(dst)[j] = w[j];
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* dst = (kv ? p.v_cache : p.k_cache) + dst_page * kPageBytes + piece * 16;
    if constexpr (KV != kKvE4m3) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = row0 + i * kRowsAtOnce;
        if (r < valid) *reinterpret_cast<uint4*>(dst + r * kRowBytes) = x[kv][i];
      }
    } else {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w[4] = {x[kv][i].x, x[kv][i].y, x[kv][i].z, x[kv][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = e4m3x2_to_f2((uint16_t)w[j]), c = e4m3x2_to_f2((uint16_t)(w[j] >> 16));
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x * s[kv][i]), fabsf(a.y * s[kv][i])),
                                   fmaxf(fabsf(c.x * s[kv][i]), fabsf(c.y * s[kv][i]))));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = e4m3_page_scale(amax);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = row0 + i * kRowsAtOnce;
        const uint32_t w[4] = {x[kv][i].x, x[kv][i].y, x[kv][i].z, x[kv][i].w};
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = e4m3x2_to_f2((uint16_t)w[j]), c = e4m3x2_to_f2((uint16_t)(w[j] >> 16));
          const float f = s[kv][i];
          out[j] = f32x2_to_e4m3x2(a.x * f / scale, a.y * f / scale) |
                   (f32x2_to_e4m3x2(c.x * f / scale, c.y * f / scale) << 16);
        }
        if (r < valid) *reinterpret_cast<uint4*>(dst + r * kRowBytes) = make_uint4(out[0], out[1], out[2], out[3]);
      }
      if (lane == 0) (kv ? p.v_scale : p.k_scale)[dst_page] = scale;
    }
  }
}

template <int D, int KV>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p) {
  const int page = blockIdx.x, b = blockIdx.y, g = blockIdx.z * kMoveWarps + (threadIdx.x >> 5);
  const int k = min(evict_len(p, b), p.keep);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (g < p.num_kv_heads && page * 16 < k) move_page<D, KV>(p, b, g, page, k);
}

constexpr int kEvictCtas = 8, kEvictThreads = 256;  // CTAs of a cluster at most
constexpr int kEvictKeys = 12288;  // keys of a CTA at most

struct EvictShared {
  alignas(16) int hist[256 * 4];  // this CTA's counters, four a digit
  int total[2][256];              // the cluster's: every CTA adds its own to all of them; of every other digit
  uint32_t top, bottom;           // of the cluster's keys that are not forced, and how many are
  int always;
  int digit, above, at;
  int gt[kEvictCtas], eq[kEvictCtas];  // of the CTAs
  int warp_gt[kEvictThreads / 32], warp_eq[kEvictThreads / 32];
};

__device__ __forceinline__ void cluster_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// One cluster per (sequence, kv head).  CTA r has the keys of tokens [r * share, r * share + share).
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ EvictShared sh;
  const int ctas = gridDim.x, rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  const int L = evict_len(p, b), k = min(L, p.keep);
  const size_t unit = (size_t)b * p.num_kv_heads + g;
  int32_t* kept = p.kept + unit * p.keep;
  if (rank == 0 && g == 0 && tid == 0) {
    p.new_lens[b] = k;
    if (p.context_lens[b] > p.max_context_len) record_error(p.err, kErrShortContext);
  }
  const int share = (L + ctas * 16 - 1) / (ctas * 16) * 16;
  const int begin = min(rank * share, L), n = min(share, L - begin);
  if (L <= p.keep) {  // (the whole cluster) every token
    for (int i = tid; i < n; i += kEvictThreads) kept[begin + i] = begin + i;
  } else {
    static_assert(kEvictThreads == 256, "a thread a digit");
    sh.total[0][tid] = sh.total[1][tid] = 0;
    if (tid == 0) {
      sh.top = 0u;
      sh.bottom = kKeyAlways;
      sh.always = 0;
    }
    cluster_arrive();
    const uint32_t here = smem_addr(&sh);
    auto in_cta = [&](int r, const void* member) { return cluster_addr(here, r) + (smem_addr(member) - here); };
    // the keys, a quarter of a block's of a thread at a time, kQuads in flight
    constexpr int kQuads = 4;
    uint32_t top = 0u, bottom = kKeyAlways;
    int always = 0;
    for (int i0 = 4 * tid; i0 < n; i0 += kQuads * 4 * kEvictThreads) {
      int pb[kQuads];
      float4 w[kQuads];
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const int i = i0 + j * 4 * kEvictThreads;
        pb[j] = i < n ? bt[(begin + i) / 16] : 0;
      }
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const int i = i0 + j * 4 * kEvictThreads;
        const bool there = pb[j] >= 0 && pb[j] < p.num_blocks;
        if (!there) record_error(p.err, kErrBlockId);
        w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there && i < n)
          w[j] = *reinterpret_cast<const float4*>(p.weights + ((size_t)pb[j] * p.num_kv_heads + g) * 16 + (begin + i) % 16);
      }
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const float w4[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        const int i = i0 + j * 4 * kEvictThreads, from = begin + i;
        if (i >= n) break;
        uint32_t x4[4];
        const bool inner = from >= p.sinks && from + 4 <= L - p.recent && i + 4 <= n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (past the share's end a key that no digit counts; the room is there, shares are multiples of 16)
          const bool forced = !inner && (from + e < p.sinks || from + e >= L - p.recent || i + e >= n);
          x4[e] = forced ? kKeyAlways : order_key(w4[e]);
          always += forced && i + e < n;
          top = max(top, forced ? 0u : x4[e]);
          bottom = min(bottom, x4[e]);
        }
        *reinterpret_cast<uint4*>(keys + i) = make_uint4(x4[0], x4[1], x4[2], x4[3]);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bottom = __reduce_min_sync(0xffffffffu, bottom);
    always = __reduce_add_sync(0xffffffffu, always);
    cluster_wait();  // every CTA runs, and its counters are clear
    if (lane < ctas) {  // (a lane a CTA)
      asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(in_cta(lane, &sh.top)), "r"(top) : "memory");
      asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(in_cta(lane, &sh.bottom)), "r"(bottom)
                   : "memory");
      if (always) cluster_add(in_cta(lane, &sh.always), always);
    }
    cluster_sync();
    int need = k - sh.always;  // keys to take among the candidates: those that agree with low in the known bits
    const int differ = 32 - __clz(sh.top ^ sh.bottom);
    uint32_t known = differ >= 32 ? 0u : ~0u << differ, low = sh.top & known;
    bool exact = need <= 0;  // all candidates are taken
    if (exact) low = kKeyAlways;
    for (int shift = differ, turn = 0; shift > 0 && !exact; turn ^= 1) {  // (the same in every CTA)
      shift = max(shift - 8, 0);
      for (int i = tid; i < 256; i += kEvictThreads) *reinterpret_cast<int4*>(&sh.hist[4 * i]) = make_int4(0, 0, 0, 0);
      __syncthreads();
      for (int i = 4 * tid; i < n; i += 4 * kEvictThreads) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t xs[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((xs[e] & known) == low && xs[e] != kKeyAlways)
            atomicAdd(&sh.hist[((xs[e] & ~known) >> shift) * 4 + (lane & 3)], 1);
      }
      __syncthreads();
      const int4 c = *reinterpret_cast<const int4*>(&sh.hist[4 * tid]);
      const int mine = (c.x + c.y) + (c.z + c.w);
      if (mine)
        for (int r = 0; r < ctas; ++r) cluster_add(in_cta(r, &sh.total[turn][tid]), mine);
      cluster_sync();
      if (warp == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
        int count[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          count[j] = sh.total[turn][255 - 8 * lane - j];
          sh.total[turn][255 - 8 * lane - j] = 0;  // for the digit after the next, a barrier of the cluster away
          sum += count[j];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const unsigned reached = __ballot_sync(0xffffffffu, upto >= need);  // (never empty: need candidates are there)
        if (lane == __ffs(reached) - 1) {
          int above = upto - sum;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above + count[j] >= need) {
              sh.digit = 255 - 8 * lane - j;
              sh.above = above;
              sh.at = count[j];
              break;
            }
            above += count[j];
          }
        }
      }
      __syncthreads();
      low |= (uint32_t)sh.digit << shift;
      known = ~0u << shift;
      need -= sh.above;
      exact = sh.at == need;  // (what is not known of low is zeros)
    }
    // which keys are taken: each warp a run of them, 32 at a time; how many before it, in the CTAs before and in this one
    const int per = (n + kEvictThreads - 1) / kEvictThreads * 32;
    const int from = min(n, warp * per), till = min(n, from + per);
    auto above_at = [&](int i, bool& above, bool& at) {
      const uint32_t x = i < till ? keys[i] : 0u;
      above = i < till && (exact ? x >= low : x > low);
      at = i < till && !exact && x == low;
    };
    int gt = 0, eq = 0;
    for (int i0 = from; i0 < till; i0 += 32) {
      bool above, at;
      above_at(i0 + lane, above, at);
      gt += __popc(__ballot_sync(0xffffffffu, above));
      eq += __popc(__ballot_sync(0xffffffffu, at));
    }
    if (lane == 0) {
      sh.warp_gt[warp] = gt;
      sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    int gt_before = 0, eq_before = 0, gt_cta = 0, eq_cta = 0;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
      gt_cta += sh.warp_gt[w];
      eq_cta += sh.warp_eq[w];
      if (w < warp) {
        gt_before += sh.warp_gt[w];
        eq_before += sh.warp_eq[w];
      }
    }
    if (tid < ctas) {  // to every CTA
      const uint32_t there = cluster_addr(smem_addr(&sh), tid) - smem_addr(&sh);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there + smem_addr(&sh.gt[rank])), "r"(gt_cta) : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there + smem_addr(&sh.eq[rank])), "r"(eq_cta) : "memory");
    }
    cluster_sync();
    int gt_all = 0;
    for (int r = 0; r < ctas; ++r) {
      gt_all += sh.gt[r];
      if (r < rank) {
        gt_before += sh.gt[r];
        eq_before += sh.eq[r];
      }
    }
    const int room = k - gt_all;  // keys equal to low that are taken, the earliest
    const unsigned before = (1u << lane) - 1u;
    for (int i0 = from; i0 < till; i0 += 32) {
      bool above, at;
      above_at(i0 + lane, above, at);
      const unsigned ga = __ballot_sync(0xffffffffu, above), ea = __ballot_sync(0xffffffffu, at);
      const int my_gt = gt_before + __popc(ga & before), my_eq = eq_before + __popc(ea & before);
      if (above || (at && my_eq < room)) kept[my_gt + min(my_eq, room)] = begin + i0 + lane;
      gt_before += __popc(ga);
      eq_before += __popc(ea);
    }
  }
}

template <int D>
const void* move_kernel(int kv) {
  return kv == kKvBf16   ? reinterpret_cast<const void*>(evict_move_kernel<D, kKvBf16>)
         : kv == kKvE4m3 ? reinterpret_cast<const void*>(evict_move_kernel<D, kKvE4m3>)
                         : reinterpret_cast<const void*>(evict_move_kernel<D, kKvFp4>);
}

}  // namespace

// The kept positions, then (contexts too long for shared memory) the keys.
size_t evict_scratch_bytes(int num_seqs, int num_kv_heads, int keep, int max_context_len) {
  const size_t units = (size_t)num_seqs * num_kv_heads;
  const bool two = max_context_len > kEvictCtas * kEvictKeys;
  return units * keep * sizeof(int32_t) + (two ? units * max_context_len * sizeof(uint32_t) : 0);
}

cudaError_t launch_evict(const EvictParams& p, int head_dim, int kv_dtype, int num_sms, cudaStream_t st) {
  if (head_dim != 128 && head_dim != 64) return cudaErrorInvalidConfiguration;
  EvictParams pp = p;
  void* args[] = {&pp};
  if (p.max_context_len <= kEvictCtas * kEvictKeys) {
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads;
    int ctas = kEvictCtas;  // one wave of four CTAs an SM where the keys fit
    while (ctas > 1 && units * ctas > 4 * (int64_t)num_sms && (ctas / 2) * kEvictKeys >= p.max_context_len) ctas /= 2;
    const void* fn = reinterpret_cast<const void*>(evict_kernel);
    cudaError_t e = set_smem_once(fn, kEvictKeys * 4);
    if (e != cudaSuccess) return e;
    const int share = (p.max_context_len + ctas * 16 - 1) / (ctas * 16) * 16;
    e = launch_clusters(fn, dim3(ctas, p.num_kv_heads, p.num_seqs), dim3(kEvictThreads), share * 4, ctas, st, args);
    if (e != cudaSuccess) return e;
  } else {
    uint32_t* keys = reinterpret_cast<uint32_t*>(p.kept + (size_t)p.num_seqs * p.num_kv_heads * p.keep);
    evict_pick_kernel<<<dim3(p.num_kv_heads, p.num_seqs), 1024, 0, st>>>(p, keys);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int pages = (min(p.keep, p.max_context_len) + 15) / 16;
  if (pages == 0) return cudaSuccess;
  const dim3 grid(pages, p.num_seqs, (p.num_kv_heads + kMoveWarps - 1) / kMoveWarps);
  return launch_dependent(head_dim == 128 ? move_kernel<128>(kv_dtype) : move_kernel<64>(kv_dtype), grid,
                          dim3(kMoveWarps * 32), 0, st, args);
}

}  // namespace pa
