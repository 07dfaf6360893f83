// Bounds of the keys of cache blocks: what the selection of blocks reads in place of their keys.
//
// For each (block, kv head) the largest and the smallest value of every dim over the block's tokens, as int8 codes
// times one power of two 2^e: the smallest e with amax 2^-e <= 127, upper codes rounded up and lower ones down, so
// that q . k <= sum_i max(q_i hi_i, q_i lo_i) holds for every token.  Scaling by a power of two is exact, so the
// codes do not depend on how they are computed.  2 d + 4 bytes stand for the 32 d of a bf16 block's keys.
//
// A pass over the keys bound by their bytes: one warp takes the page of one (block, head), all of its loads in
// flight at once, a row of 128 or 256 bytes in one load of all lanes, so that a lane holds the same dims of every
// row (narrower rows: of every second or fourth; the lanes that share dims then halve them between them, an
// exchange each).  Rows are folded in packed 16-bit maxima and minima: E4M3 codes and 4-bit codes times their
// scales are exact in f16, and the page's (head's) fp32 scale is applied once, at the end, as rounding a product
// is monotone in its factor.  Measured with 8 E4M3 contexts of 9000 to 32768 tokens (floor 29.6 us): 16-byte
// loads, the lanes of a piece exchanging their dims, 54 us with all dims in every lane and 43 with halves (the
// logic unit at three quarters of its rate), rounding without conversions 41; a lane's dims its own 37, with ten
// CTAs an SM and no page ahead (a page ahead takes registers: eight CTAs and 39 us; two ahead 48).
#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kBoundsWarps = 4;
constexpr int kBoundsCols = 4;  // columns of a CTA at most (one a lane)

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
  static constexpr int kPieceBytes = kRowBytes == 256 ? 8 : 4;  // of a row: a lane each
  static constexpr int kWords = kPieceBytes / 4;
  static constexpr int kPieces = kRowBytes / kPieceBytes;
  static constexpr int kRowsAtOnce = 32 / kPieces;
  static constexpr int kLoads = 16 / kRowsAtOnce;
  static constexpr int kDims = D / kPieces;        // dims of a lane: 2, 4 or 8
  static constexpr int kPairs = kDims / 2;
  static constexpr int kPageBytes = KV == kKvFp4 ? Fp4Page<D>::kBytes : 16 * kRowBytes;
  static constexpr int kMinCtas = kRowBytes == 256 ? 8 : 10;  // of an SM (a page in registers: 32 or 16 a thread)
  static constexpr int kOwnPairs = D / 64;         // of a lane in the end
  static_assert(kPairs / kRowsAtOnce == kOwnPairs, "the lanes of a piece share its dims");
};

template <int D, int KV>
__global__ void __launch_bounds__(kBoundsWarps * 32, (BoundsTraits<D, KV>::kMinCtas)) block_bounds_kernel(const BoundsParams p, int cols) {
  using T = BoundsTraits<D, KV>;
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
  int ids = lane < count ? p.block_table[(size_t)b * p.max_blocks_per_seq + col0 + lane] : 0;  // lane c: column c's block
  if (ids < 0 || ids >= p.num_blocks) {
    ids = -1;
    if (blockIdx.z == 0 && warp == 0) record_error(p.err, kErrBlockId);
  }
  const int piece = lane % T::kPieces, row0 = lane / T::kPieces;
  auto bounds_of = [&](int id, int col, int g) {
    const size_t page = (size_t)id * p.num_kv_heads + g;
    const uint8_t* src = p.k_cache + page * T::kPageBytes;
    const int last = min(16, L - col * 16) - 1;
    uint32_t x[T::kLoads][T::kWords], sc[KV == kKvFp4 ? T::kLoads : 1];  // codes (4-bit: and their scales)
    auto row = [&](int i, int r) {
      const uint8_t* at = src + r * T::kRowBytes + piece * T::kPieceBytes;
      if constexpr (T::kWords == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        x[i][0] = w.x;
        x[i][1] = w.y;
      } else {
        x[i][0] = *reinterpret_cast<const uint32_t*>(at);
      }
      if constexpr (KV == kKvFp4) sc[i] = src[Fp4Page<D>::kCodeBytes + r * Fp4Page<D>::kScaleRow + piece / 2];
    };
    if (last == 15) {
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) row(i, row0 + i * T::kRowsAtOnce);
    } else {  // rows past the last: it once more
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) row(i, min(row0 + i * T::kRowsAtOnce, last));
    }
    float s = 1.f;
    if constexpr (KV == kKvE4m3) s = p.k_scale[page];
    if constexpr (KV == kKvFp4) s = p.k_scale ? p.k_scale[g] : 1.f;
    uint32_t hi[T::kPairs], lo[T::kPairs];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      uint32_t v[T::kPairs];
      if constexpr (KV == kKvBf16) {
#pragma unroll
        for (int j = 0; j < T::kWords; ++j) v[j] = x[i][j];
      } else if constexpr (KV == kKvE4m3) {
        v[0] = e4m3x2_to_f16x2(x[i][0]);
        v[1] = e4m3x2_to_f16x2(x[i][0] >> 16);
      } else {
        const uint32_t s2 = e4m3x2_to_f16x2(sc[i]), sp = __byte_perm(s2, s2, 0x1010);
        e2m1x8_to_f16x2(x[i][0], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul_f16x2(v[j], sp);
      }
#pragma unroll
      for (int j = 0; j < T::kPairs; ++j) {
        hi[j] = i == 0 ? v[j] : max_pair<T::kBf16>(hi[j], v[j]);
        lo[j] = i == 0 ? v[j] : min_pair<T::kBf16>(lo[j], v[j]);
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
    const bool turned = !T::kBf16 && s < 0.f;
    float top[2 * T::kOwnPairs], bottom[2 * T::kOwnPairs];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < T::kOwnPairs; ++j) {
      const uint32_t above = turned ? lo[j] : hi[j], below = turned ? hi[j] : lo[j];
      float2 a, c;
      if constexpr (T::kBf16) {
        a = bf16x2_to_f2(above);
        c = bf16x2_to_f2(below);
      } else {
        a = __half22float2(*reinterpret_cast<const __half2*>(&above));
        c = __half22float2(*reinterpret_cast<const __half2*>(&below));
        a = make_float2(a.x * s, a.y * s);
        c = make_float2(c.x * s, c.y * s);
      }
      top[2 * j] = a.x;
      top[2 * j + 1] = a.y;
      bottom[2 * j] = c.x;
      bottom[2 * j + 1] = c.y;
      amax = fmaxf(fmaxf(amax, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(c.x), fabsf(c.y)));
    }
    // (magnitudes in the order of their bits)
    constexpr float kMax = 3.4028235e38f;
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(fminf(amax, kMax)));
    int e = (int)(bits >> 23) - 127 - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);  // above 127 / 64: one more
    e = bits == 0 ? 0 : max(e, -126);
    float down = exp2_int(-e);
    if (bits == __float_as_uint(kMax)) {  // perhaps an infinity: the largest code
#pragma unroll
      for (int i = 0; i < 2 * T::kOwnPairs; ++i) {
        top[i] = fmaxf(fminf(__fmul_ru(top[i], down), 127.f), -127.f);
        bottom[i] = fmaxf(fminf(__fmul_rd(bottom[i], down), 127.f), -127.f);
      }
      down = 1.f;
    }
    // rounded up and down to whole numbers by the addition of 1.5 2^23, whose low byte then is the code
    uint32_t up[2 * T::kOwnPairs], dn[2 * T::kOwnPairs];
#pragma unroll
    for (int i = 0; i < 2 * T::kOwnPairs; ++i) {
      up[i] = __float_as_uint(__fmaf_ru(top[i], down, 12582912.f));
      dn[i] = __float_as_uint(__fmaf_rd(bottom[i], down, 12582912.f));
    }
    int8_t* dst = p.bounds + page * (2 * D) + piece * T::kDims + 2 * kept;
    if constexpr (T::kOwnPairs == 2) {
      *reinterpret_cast<uint32_t*>(dst) = __byte_perm(__byte_perm(up[0], up[1], 0x0040), __byte_perm(up[2], up[3], 0x0040), 0x5410);
      *reinterpret_cast<uint32_t*>(dst + D) =
          __byte_perm(__byte_perm(dn[0], dn[1], 0x0040), __byte_perm(dn[2], dn[3], 0x0040), 0x5410);
    } else {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)__byte_perm(up[0], up[1], 0x0040);
      *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)__byte_perm(dn[0], dn[1], 0x0040);
    }
    if (lane == 0) p.bound_scale[page] = exp2_int(e);
  };
  for (int g = blockIdx.z * kBoundsWarps + warp; g < p.num_kv_heads; g += gridDim.z * kBoundsWarps) {
    for (int c = 0; c < count; ++c) {
      const int id = __shfl_sync(0xffffffffu, ids, c);
      if (id >= 0) bounds_of(id, col0 + c, g);
    }
  }
}

template <int D>
cudaError_t launch_d(const BoundsParams& p, int kv, int num_sms, cudaStream_t st) {
  const int touched = min((p.n + 14) / 16 + 1, p.max_blocks_per_seq);  // columns that n tokens touch at most
  const int z = min((p.num_kv_heads + kBoundsWarps - 1) / kBoundsWarps, 64);
  // several columns a CTA where there are enough of them to fill the device all the same (SMs of eight to ten CTAs)
  const int cols = (int64_t)touched * p.num_seqs * z >= (int64_t)num_sms * 8 * kBoundsCols ? kBoundsCols : 1;
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

cudaError_t launch_block_bounds(const BoundsParams& p, int head_dim, int kv_dtype, int num_sms, cudaStream_t st) {
  if (head_dim == 128) return launch_d<128>(p, kv_dtype, num_sms, st);
  if (head_dim == 64) return launch_d<64>(p, kv_dtype, num_sms, st);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
