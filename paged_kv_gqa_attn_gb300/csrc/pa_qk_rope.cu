// RMS norm of every query and key head row and the position rotation, in one pass: the step between
// the projection and the KV append.
//
//   y = x / sqrt(mean(x^2) + eps) * weight                       (per head row of d dims)
//   (a, b) -> (a cos - b sin, b cos + a sin)                     (pairs of the first `rotary` dims)
//
// A pair is (i, i + rotary / 2), or (2i, 2i + 1) when interleaved; cos and sin are row positions[t] of
// a table [max_position][rotary]: rotary / 2 cosines, then rotary / 2 sines, fp32.  All arithmetic is
// fp32, rounded to bf16 once at the store.
//
// Bound by bytes (2 d read and 2 d written a row, about 8 flops an element).  A group of d / 8 lanes
// owns one head row, 16 bytes a lane, so a warp moves two or four whole rows per instruction; a group
// keeps its token's cosines and sines in registers over kPer rows, whose loads are all in flight
// before the first is used.  The pair partner i + rotary / 2 of a lane's eight dims is eight dims of
// one other lane of the group (rotary is a multiple of 16): one shuffle per element.
#include "pa_kernels.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kPer = 5;  // rows a group has in flight: 40 heads of 128 dims are one round of a CTA

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = bf16x2_to_f2(w[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;                  // lanes per row
  constexpr int kGroups = kRopeThreads / kLanes;  // rows in flight per CTA and round
  const int t = blockIdx.x;
  const int grp = threadIdx.x / kLanes;
  const int li = threadIdx.x % kLanes;
  const int heads = p.num_q_heads + p.num_kv_heads;
  const int h_first = blockIdx.y * (kGroups * kPer) + grp;

  // the rows' loads first: they depend on nothing
  uint4 raw[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int h = h_first + j * kGroups;
    if (h < heads) {
      const bool is_q = h < p.num_q_heads;
      const __nv_bfloat16* src = is_q ? p.q + t * p.q_stride + (int64_t)h * D
                                      : p.k + t * p.k_stride + (int64_t)(h - p.num_q_heads) * D;
      raw[j] = *reinterpret_cast<const uint4*>(src + li * 8);
    }
  }
  const int pos = p.positions[t];
  const bool pos_ok = pos >= 0 && pos < p.max_position;
  if (!pos_ok && threadIdx.x == 0) record_error(p.err, kErrBadInput);
  const int half = p.rotary >> 1;
  // this lane's cosines and sines; dims past `rotary` turn by nothing
  float cs[8], sn[8];
  constexpr int kPairs = INTERLEAVED ? 4 : 8;
  const bool turns = li * 8 < p.rotary;
  const bool upper = !INTERLEAVED && li * 8 >= half;
  {
    const int at = INTERLEAVED ? li * 4 : (upper ? li * 8 - half : li * 8);
    const float* row = p.cos_sin + (int64_t)(pos_ok ? pos : 0) * p.rotary + at;
#pragma unroll
    for (int i = 0; i < kPairs; i += 4) {
      float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (turns) {
        c = *reinterpret_cast<const float4*>(row + i);
        s = *reinterpret_cast<const float4*>(row + half + i);
      }
      cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
      sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
    }
  }
  const uint4 qw = reinterpret_cast<const uint4*>(p.q_weight)[li];
  const uint4 kw = reinterpret_cast<const uint4*>(p.k_weight)[li];
  // the lane of this group that holds the partner dims (itself past `rotary`)
  const int base = (threadIdx.x & 31) - li;
  const int partner = base + (turns ? (upper ? li - half / 8 : li + half / 8) : li);

#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int h = h_first + j * kGroups;
    const bool live = h < heads;  // the same for every lane of the group; shuffles stay warp-wide
    const bool is_q = h < p.num_q_heads;
    float x[8], w[8];
    unpack8(live ? raw[j] : make_uint4(0u, 0u, 0u, 0u), x);
    unpack8(is_q ? qw : kw, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
    float y[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv * w[i];
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[2 * i] = y[2 * i] * cs[i] - y[2 * i + 1] * sn[i];
        z[2 * i + 1] = y[2 * i + 1] * cs[i] + y[2 * i] * sn[i];
      }
      if (!turns)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = y[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, y[i], partner);
        z[i] = turns ? y[i] * cs[i] + (upper ? o : -o) * sn[i] : y[i];
      }
    }
    if (live) {
      __nv_bfloat16* dst = is_q ? p.q_out + t * p.q_out_stride + (int64_t)h * D
                                : p.k_out + t * p.k_out_stride + (int64_t)(h - p.num_q_heads) * D;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);  // a position outside the table: zeros, flagged
      if (pos_ok) v = make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
      *reinterpret_cast<uint4*>(dst + li * 8) = v;
    }
  }
}

template <int D, bool INTERLEAVED>
cudaError_t launch_one(const RopeParams& p, cudaStream_t st) {
  constexpr int rows = kRopeThreads / (D / 8) * kPer;  // head rows per CTA
  const int heads = p.num_q_heads + p.num_kv_heads;
  qk_norm_rope_kernel<D, INTERLEAVED>
      <<<dim3((unsigned)p.num_tokens, (unsigned)((heads + rows - 1) / rows)), kRopeThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, bool interleaved, cudaStream_t st) {
  if (head_dim == 128) return interleaved ? launch_one<128, true>(p, st) : launch_one<128, false>(p, st);
  if (head_dim == 64) return interleaved ? launch_one<64, true>(p, st) : launch_one<64, false>(p, st);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
