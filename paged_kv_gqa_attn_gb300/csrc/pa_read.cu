// Read stored tokens back as bf16: the inverse of the append, for every cache type.
//
// The last n tokens of each sequence are gathered through the block table and written as contiguous
// rows: bf16 rows unchanged, E4M3 codes times their page's scale, E2M1 codes times their 16-dim
// block's E4M3 scale (exact in fp32: at most six significant bits) times the head's fp32 scale.
// A gather bound by bytes: a thread owns 16 dims of one row (32, 16 or 8 + 1 bytes read, 32 written).
#include "pa_fp4.cuh"
#include "pa_kernels.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

template <int D, int KV>
__global__ void __launch_bounds__(128) read_kv_kernel(const ReadParams p) {
  constexpr int kC = D / 16;  // 16-dim pieces per head row
  const int row = blockIdx.x;  // b * n + t
  const int b = row / p.n, t = row - b * p.n;
  const int per_side = p.num_kv_heads * kC;
  const int L = p.context_lens[b];
  const bool fits = context_holds(L, 0, p.max_blocks_per_seq);
  const int j = fits ? L - p.n + t : -1;
  int pb = -1;
  if (j < 0) {
    if (threadIdx.x == 0) record_error(p.err, kErrShortContext);
  } else {
    pb = p.block_table[(size_t)b * p.max_blocks_per_seq + j / 16];
    if (pb < 0 || pb >= p.num_blocks) {
      if (threadIdx.x == 0) record_error(p.err, kErrBlockId);
      pb = -1;
    }
  }
  for (int i = threadIdx.x; i < 2 * per_side; i += blockDim.x) {
    const bool is_v = i >= per_side;
    const int r = is_v ? i - per_side : i;
    const int g = r / kC, c = r - g * kC;
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};  // a token that is not there: zeros, flagged
    if (pb >= 0) {
      const size_t page = (size_t)pb * p.num_kv_heads + g;
      const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
      const float* scales = is_v ? p.v_scale : p.k_scale;
      const int slot = j & 15;
      if constexpr (KV == kKvBf16) {
        const uint4* src = reinterpret_cast<const uint4*>(cache + (page * 16 + slot) * D * 2) + 2 * c;
        const uint4 a = src[0], d = src[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = d.x; w[5] = d.y; w[6] = d.z; w[7] = d.w;
      } else if constexpr (KV == kKvE4m3) {
        const uint4 a = *(reinterpret_cast<const uint4*>(cache + (page * 16 + slot) * D) + c);
        const float s = scales[page];
        const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = e4m3x2_to_f2((uint16_t)q[k]), hi = e4m3x2_to_f2((uint16_t)(q[k] >> 16));
          w[2 * k] = pack_bf16(lo.x * s, lo.y * s);
          w[2 * k + 1] = pack_bf16(hi.x * s, hi.y * s);
        }
      } else {
        const uint8_t* base = cache + page * Fp4Page<D>::kBytes;
        const uint2 a = *reinterpret_cast<const uint2*>(base + slot * Fp4Page<D>::kCodeRow + c * 8);
        const uint8_t sc = base[Fp4Page<D>::kCodeBytes + slot * Fp4Page<D>::kScaleRow + c];
        const float step = e4m3x2_to_f2(sc).x, s = scales ? scales[g] : 1.f;
        const uint32_t q[2] = {a.x, a.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[4];
          e2m1x8_to_f16x2(q[k], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
            w[4 * k + e] = pack_bf16(f.x * step * s, f.y * step * s);
          }
        }
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(is_v ? p.v_out : p.k_out) + ((size_t)row * per_side + r) * 2;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D>
cudaError_t launch_d(const ReadParams& p, int kv, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.num_seqs * p.n);
  if (kv == kKvBf16)
    read_kv_kernel<D, kKvBf16><<<grid, 128, 0, st>>>(p);
  else if (kv == kKvE4m3)
    read_kv_kernel<D, kKvE4m3><<<grid, 128, 0, st>>>(p);
  else
    read_kv_kernel<D, kKvFp4><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_read_kv(const ReadParams& p, int head_dim, int kv_dtype, cudaStream_t st) {
  if (head_dim == 128) return launch_d<128>(p, kv_dtype, st);
  if (head_dim == 64) return launch_d<64>(p, kv_dtype, st);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
