// Bounds of the keys of cache blocks: what the selection of blocks reads in place of their keys.
//
// For each (block, kv head) the largest and the smallest value of every dim over the block's tokens, as int8 codes times
// one power of two 2^e: the smallest e with amax 2^-e <= 127, upper codes rounded up and lower ones down, so that
// q . k <= sum_i max(q_i hi_i, q_i lo_i) holds for every token.  Scaling by a power of two is exact, so the codes do
// not depend on how they are computed.  2 d + 4 bytes stand for the 32 d of a bf16 block's keys.
//
// A pass over the keys bound by their bytes: one warp takes the page of one (block, head), all of its loads in flight
// at once (bf16, d = 128: eight 16-byte pieces a lane), and folds rows in packed 16-bit maxima and minima: E4M3 codes and
// 4-bit codes times their scales are exact in f16, and the page's (head's) fp32 scale is applied once, at the end, as
// rounding a product is monotone in its factor.  The lanes that hold the same dims of different rows then halve the dims
// between them at every exchange, so that each ends with d / 32 dims of its own to round (all of them ending with all dims
// cost 700 instructions a page where this takes 300, and more than half the time).
#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kBoundsWarps = 4;
constexpr int kBoundsCols = 4;  // columns of a CTA at most

// Folds of 16-bit pairs; a NaN gives way to the other operand.
template <bool BF16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int D, int KV>
struct BoundsTraits {
  static constexpr bool kBf16 = KV == kKvBf16;
  static constexpr int kRowBytes = kBf16 ? 2 * D : KV == kKvE4m3 ? D : D / 2;  // of codes
  static constexpr int kPieces = kRowBytes / 16;   // 16-byte pieces of a row: a lane each
  static constexpr int kRowsAtOnce = 32 / kPieces;
  static constexpr int kLoads = 16 / kRowsAtOnce;
  static constexpr int kDims = D / kPieces;        // dims of a lane: 8, 16 or 32
  static constexpr int kPairs = kDims / 2;
  static constexpr int kPageBytes = KV == kKvFp4 ? Fp4Page<D>::kBytes : 16 * kRowBytes;
  static constexpr int kOwnPairs = D / 64;         // of a lane in the end
  static_assert(kPairs / kRowsAtOnce == kOwnPairs, "the lanes of a piece share its dims");
};

template <int D, int KV>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(const BoundsParams p, int cols) {
  using T = BoundsTraits<D, KV>;
  constexpr uint32_t kLowest = T::kBf16 ? 0xff80ff80u : 0xfc00fc00u, kHighest = T::kBf16 ? 0x7f807f80u : 0x7c007c00u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int L = p.context_lens[b];
  if (!context_holds(L, 0, p.max_blocks_per_seq)) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) record_error(p.err, kErrShortContext);
    return;
  }
  const int col0 = max(0, L - p.n) / 16 + blockIdx.x * cols;  // the CTA's columns [col0, col0 + count)
  const int count = min(cols, (L + 15) / 16 - col0);
  if (count <= 0) return;
  int ids[kBoundsCols];
#pragma unroll
  for (int c = 0; c < kBoundsCols; ++c) {
    ids[c] = c < count ? p.block_table[(size_t)b * p.max_blocks_per_seq + col0 + c] : 0;
    if (ids[c] < 0 || ids[c] >= p.num_blocks) {
      ids[c] = -1;
      if (blockIdx.z == 0 && threadIdx.x == 0) record_error(p.err, kErrBlockId);
    }
  }
  const int piece = lane % T::kPieces, row0 = lane / T::kPieces;
  // a page's loads: its codes (4-bit: and their scales)
  struct Page {
    uint4 x[T::kLoads];
    uint32_t sc[KV == kKvFp4 ? T::kLoads : 1];
    float s;
  };
  auto load = [&](Page& q, int c, int g) {
    const size_t page = (size_t)max(ids[c], 0) * p.num_kv_heads + g;
    const uint8_t* src = p.k_cache + page * T::kPageBytes;
    const int valid = ids[c] < 0 ? 0 : min(16, L - (col0 + c) * 16);
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      const int r = row0 + i * T::kRowsAtOnce;
      if (r < valid) {
        q.x[i] = *reinterpret_cast<const uint4*>(src + r * T::kRowBytes + piece * 16);
        if constexpr (KV == kKvFp4)
          q.sc[i] = *reinterpret_cast<const uint16_t*>(src + Fp4Page<D>::kCodeBytes + r * Fp4Page<D>::kScaleRow + piece * 2);
      }
    }
    q.s = 1.f;
    if constexpr (KV == kKvE4m3) q.s = p.k_scale[page];
    if constexpr (KV == kKvFp4) q.s = p.k_scale ? p.k_scale[g] : 1.f;
  };
  auto bounds_of = [&](const Page& q, int c, int g) {
    if (ids[c] < 0) return;
    const size_t page = (size_t)ids[c] * p.num_kv_heads + g;
    const int valid = min(16, L - (col0 + c) * 16);
    const float s = q.s;
    uint32_t hi[T::kPairs], lo[T::kPairs];
#pragma unroll
    for (int j = 0; j < T::kPairs; ++j) {
      hi[j] = kLowest;
      lo[j] = kHighest;
    }
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      if (row0 + i * T::kRowsAtOnce >= valid) continue;
      const uint32_t w[4] = {q.x[i].x, q.x[i].y, q.x[i].z, q.x[i].w};
      uint32_t v[T::kPairs];
      if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w[j];
      } else if constexpr (KV == kKvE4m3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = e4m3x2_to_f16x2(w[j]);
          v[2 * j + 1] = e4m3x2_to_f16x2(w[j] >> 16);
        }
      } else {
        const uint32_t s2 = e4m3x2_to_f16x2(q.sc[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[4];
          e2m1x8_to_f16x2(w[j], h);
          const uint32_t sp = __byte_perm(s2, s2, j < 2 ? 0x1010 : 0x3232);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * j + e] = mul_f16x2(h[e], sp);
        }
      }
#pragma unroll
      for (int j = 0; j < T::kPairs; ++j) {
        hi[j] = max_pair<T::kBf16>(hi[j], v[j]);
        lo[j] = min_pair<T::kBf16>(lo[j], v[j]);
      }
    }
    // lanes of the same piece, o apart: each keeps one half of the pairs it still has and gets the other's of it
    int kept = 0;  // first pair that the lane keeps
#pragma unroll
    for (int o = 16, left = T::kPairs / 2; o >= T::kPieces; o >>= 1, left >>= 1) {
      const bool top = (lane & o) != 0;
#pragma unroll
      for (int j = 0; j < left; ++j) {
        const uint32_t give_hi = top ? hi[j] : hi[left + j], give_lo = top ? lo[j] : lo[left + j];
        hi[j] = max_pair<T::kBf16>(top ? hi[left + j] : hi[j], __shfl_xor_sync(0xffffffffu, give_hi, o));
        lo[j] = min_pair<T::kBf16>(top ? lo[left + j] : lo[j], __shfl_xor_sync(0xffffffffu, give_lo, o));
      }
      if (top) kept += left;
    }
    // the lane's dims, times the fp32 scale; a negative scale turns the ends round
    float top[2 * T::kOwnPairs], bottom[2 * T::kOwnPairs];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < T::kOwnPairs; ++j) {
      float2 a, c;
      if constexpr (T::kBf16) {
        a = bf16x2_to_f2(hi[j]);
        c = bf16x2_to_f2(lo[j]);
      } else {
        a = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
        c = __half22float2(*reinterpret_cast<const __half2*>(&lo[j]));
        a = make_float2(a.x * s, a.y * s);
        c = make_float2(c.x * s, c.y * s);
      }
      top[2 * j] = fmaxf(a.x, c.x);
      top[2 * j + 1] = fmaxf(a.y, c.y);
      bottom[2 * j] = fminf(a.x, c.x);
      bottom[2 * j + 1] = fminf(a.y, c.y);
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(top[i]), fabsf(bottom[i])));
    }
    // (magnitudes in the order of their bits; an infinity: the widest bounds)
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(fminf(amax, 3.4028235e38f)));
    int e = (int)(bits >> 23) - 127 - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);  // above 127 / 64: one more
    e = bits == 0 ? 0 : max(e, -126);
    const float down = exp2_int(-e);
    uint32_t upper = 0u, lower = 0u;
#pragma unroll
    for (int i = 0; i < 2 * T::kOwnPairs; ++i) {
      upper |= (uint32_t)(max(-127, min(127, __float2int_ru(top[i] * down))) & 0xff) << (8 * i);
      lower |= (uint32_t)(max(-127, min(127, __float2int_rd(bottom[i] * down))) & 0xff) << (8 * i);
    }
    int8_t* dst = p.bounds + page * (2 * D) + piece * T::kDims + 2 * kept;
    if constexpr (T::kOwnPairs == 2) {
      *reinterpret_cast<uint32_t*>(dst) = upper;
      *reinterpret_cast<uint32_t*>(dst + D) = lower;
    } else {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)upper;
      *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)lower;
    }
    if (lane == 0) p.bound_scale[page] = exp2_int(e);
  };
  for (int g = blockIdx.z * kBoundsWarps + warp; g < p.num_kv_heads; g += gridDim.z * kBoundsWarps) {
    Page cur, next;
    load(cur, 0, g);
#pragma unroll
    for (int c = 0; c < kBoundsCols; ++c) {  // the next page's loads before this one's arithmetic
      if (c >= count) break;
      if (c + 1 < kBoundsCols && c + 1 < count) load(next, c + 1 < kBoundsCols ? c + 1 : 0, g);
      bounds_of(cur, c, g);
      cur = next;
    }
  }
}

template <int D>
cudaError_t launch_d(const BoundsParams& p, int kv, cudaStream_t st) {
  const int touched = min((p.n + 14) / 16 + 1, p.max_blocks_per_seq);  // columns that n tokens touch at most
  const int z = min((p.num_kv_heads + kBoundsWarps - 1) / kBoundsWarps, 64);
  // several columns a CTA where there are enough of them to fill the device all the same (152 SMs of six to eight CTAs)
  const int cols = (int64_t)touched * p.num_seqs * z >= 152 * 8 * kBoundsCols ? kBoundsCols : 1;
  const dim3 grid((touched + cols - 1) / cols, p.num_seqs, z);
  if (kv == kKvBf16)
    block_bounds_kernel<D, kKvBf16><<<grid, kBoundsWarps * 32, 0, st>>>(p, cols);
  else if (kv == kKvE4m3)
    block_bounds_kernel<D, kKvE4m3><<<grid, kBoundsWarps * 32, 0, st>>>(p, cols);
  else
    block_bounds_kernel<D, kKvFp4><<<grid, kBoundsWarps * 32, 0, st>>>(p, cols);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsParams& p, int head_dim, int kv_dtype, cudaStream_t st) {
  if (head_dim == 128) return launch_d<128>(p, kv_dtype, st);
  if (head_dim == 64) return launch_d<64>(p, kv_dtype, st);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
