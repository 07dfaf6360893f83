// Eviction from the cache by accumulated attention weight.
//
// Each (sequence, kv head) keeps the first `sinks` tokens, the last `recent` ones and, up to `keep` in all, those whose
// sums (pa_weights.cu) are the largest, ties to the earliest.  The kept tokens move in order to the blocks of another
// table; the old blocks are only read, so blocks that other sequences share stay whole, every row moves
// independently of the others, and the caller gives the old ones back afterwards.
//
// Two kernels.  The first finds the kept positions: one CTA per (kv head, sequence), the sums as keys in shared memory
// (pa_topk.cuh), and moves the sums.  The second moves rows: a warp for each new (block, head) page, all of a page's K and
// V loads in flight at once.  bf16 rows and 4-bit rows (codes and their scales belong to the token) move as they
// are; E4M3 pages get the scale amax / 448 of their new tokens, values times the old scales re-encoded in fp32 to
// nearest even as the append does.  Bound by the kept rows' bytes, read and written once.
#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_tc.cuh"
#include "pa_topk.cuh"

namespace pa {
namespace {

constexpr int kKeySmem = 50000;  // sums that are kept in shared memory
constexpr int kMoveWarps = 4;

// The sequence's length inside its table row.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  return max(0, min(p.context_lens[b], p.max_context_len));
}

// keys_global: [B, Hkv, max_context_len] where the sums do not fit in shared memory, else null.
__global__ void __launch_bounds__(1024) evict_pick_kernel(const EvictParams p, uint32_t* keys_global) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ TopkShared sh;
  const int g = blockIdx.x, b = blockIdx.y;
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  const int32_t* to = p.new_table + (size_t)b * p.new_blocks;
  const int L = evict_len(p, b), k = min(L, p.keep);
  const size_t unit = (size_t)b * p.num_kv_heads + g;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0 && g == 0) {
    p.new_lens[b] = k;
    if (p.context_lens[b] > p.max_context_len) record_error(p.err, kErrShortContext);
  }
  int32_t* kept = p.kept + unit * p.keep;
  // the sums of k kept positions (pos(at) ascending) go to the new blocks, kMoves of a thread in flight at once
  constexpr int kMoves = 4;
  const int threads = blockDim.x;
  auto move_sums = [&](auto pos) {
    for (int a0 = threadIdx.x; a0 < k; a0 += kMoves * threads) {
      int from[kMoves], i[kMoves];
      float w[kMoves];
#pragma unroll
      for (int j = 0; j < kMoves; ++j) i[j] = a0 + j * threads < k ? pos(a0 + j * threads) : 0;
#pragma unroll
      for (int j = 0; j < kMoves; ++j) from[j] = bt[i[j] / 16];
#pragma unroll
      for (int j = 0; j < kMoves; ++j) {
        const bool there = from[j] >= 0 && from[j] < p.num_blocks;
        if (!there) record_error(p.err, kErrBlockId);
        w[j] = there ? p.weights[((size_t)from[j] * p.num_kv_heads + g) * 16 + i[j] % 16] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kMoves; ++j) {
        const int at = a0 + j * threads;
        if (at >= k) continue;
        const int pb = to[at / 16];
        if (pb >= 0 && pb < p.num_blocks)  // (out of range: flagged by the kernel that moves the rows)
          p.weights[((size_t)pb * p.num_kv_heads + g) * 16 + at % 16] = w[j];
      }
    }
  };
  if (L <= p.keep) {
    for (int i = threadIdx.x; i < L; i += threads) kept[i] = i;
    move_sums([](int at) { return at; });
    return;
  }
  uint32_t* keys = keys_global ? keys_global + unit * p.max_context_len : smem_keys;
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
  __syncthreads();  // (the CTA's own writes)
  move_sums([&](int at) { return kept[at]; });
}

// A warp moves the page (new block, head): lane t < 16 knows where token t comes from.
template <int D, int KV>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p) {
  constexpr int kRowBytes = KV == kKvBf16 ? 2 * D : KV == kKvE4m3 ? D : D / 2;  // of codes
  constexpr int kPageBytes = KV == kKvFp4 ? Fp4Page<D>::kBytes : 16 * kRowBytes;
  constexpr int kPieces = kRowBytes / 16;           // 16-byte pieces of a row
  constexpr int kRowsAtOnce = 32 / kPieces, kLoads = 16 / kRowsAtOnce;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = blockIdx.x, b = blockIdx.y;
  const int g = blockIdx.z * kMoveWarps + warp;
  const int k = min(evict_len(p, b), p.keep);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (g >= p.num_kv_heads || page * 16 >= k) return;
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
    if (src_block < 0 || src_block >= p.num_blocks) src_block = -1;  // its row becomes zeros (flagged with its sum)
  }
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
      const float scale = amax > 0.f ? amax / 448.f : 1.f;
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
  return units * keep * sizeof(int32_t) + (max_context_len > kKeySmem ? units * max_context_len * sizeof(uint32_t) : 0);
}

cudaError_t launch_evict(const EvictParams& p, int head_dim, int kv_dtype, cudaStream_t st) {
  const bool in_smem = p.max_context_len <= kKeySmem;
  const void* pick = reinterpret_cast<const void*>(evict_pick_kernel);
  cudaError_t e = set_smem_once(pick, kKeySmem * 4);
  if (e != cudaSuccess) return e;
  const int threads = p.max_context_len <= 2048 ? 256 : p.max_context_len <= 4096 ? 512 : 1024;
  uint32_t* keys = in_smem ? nullptr : reinterpret_cast<uint32_t*>(p.kept + (size_t)p.num_seqs * p.num_kv_heads * p.keep);
  evict_pick_kernel<<<dim3(p.num_kv_heads, p.num_seqs), threads, in_smem ? p.max_context_len * 4 : 0, st>>>(p, keys);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int pages = (min(p.keep, p.max_context_len) + 15) / 16;
  if (pages == 0) return cudaSuccess;
  EvictParams pp = p;
  void* args[] = {&pp};
  const dim3 grid(pages, p.num_seqs, (p.num_kv_heads + kMoveWarps - 1) / kMoveWarps);
  if (head_dim != 128 && head_dim != 64) return cudaErrorInvalidConfiguration;
  return launch_dependent(head_dim == 128 ? move_kernel<128>(kv_dtype) : move_kernel<64>(kv_dtype), grid,
                          dim3(kMoveWarps * 32), 0, st, args);
}

}  // namespace pa
