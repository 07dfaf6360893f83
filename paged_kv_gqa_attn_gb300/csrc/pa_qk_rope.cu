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
// Bound by bytes (2 d read and 2 d written a row), next by instructions (issue slots 56 % busy at 68 %
// of the DRAM rate, a token's rows together).  A group of d / 8 lanes owns
// one head row, eight dims a lane.  What depends on the token alone is folded once and kept in registers
// over its rows: with c = weight cos and s = -+ partner's weight sin, a rotated dim is
// (x c + x' s) / sqrt(..), two packed products and sums a pair; x', the partner's eight dims, arrives as
// four shuffles of bf16 pairs (the partner i + rotary / 2 of a lane's dims is eight dims of one other lane,
// rotary being a multiple of 16).  The rows' loads are all in flight before the first is used.
// 16384 tokens of 32 + 8 heads of 128: 59.5 us.
#include "pa_kernels.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeCtas = 14;  // per SM (128 threads: 8 CTAs 63.2 us; 64: 14 61.8 us)

__device__ __forceinline__ void unpack8(const uint4 v, float2 (&f)[4]) {
  f[0] = bf16x2_to_f2(v.x);
  f[1] = bf16x2_to_f2(v.y);
  f[2] = bf16x2_to_f2(v.z);
  f[3] = bf16x2_to_f2(v.w);
}

// One lane's eight dims of a token: what to multiply its own and its partner's values by.
struct RopeTurn {
  float2 own[4], other[4];
};

// The group's rows h0 + grp, h0 + grp + groups, ... of one tensor of a token.
template <int D, int N>
__device__ __forceinline__ void rope_load(const __nv_bfloat16* src, int heads, int h0, int grp, int li, uint4 (&raw)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int h = h0 + j * (kRopeThreads / (D / 8)) + grp;
    raw[j] = h < heads ? *reinterpret_cast<const uint4*>(src + (int64_t)h * D + li * 8) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Norm and rotate the rows of one tensor of a token, N rows of a group in flight; `raw` holds the first N.
template <int D, int N, bool INTERLEAVED>
__device__ __forceinline__ void rope_rows(const __nv_bfloat16* src, __nv_bfloat16* dst, int heads, int grp, int li,
                                          int partner, const RopeTurn& w, float eps, bool zero, uint4 (&raw)[N]) {
  constexpr int kLanes = D / 8, kGroups = kRopeThreads / kLanes;
  for (int h0 = 0; h0 < heads; h0 += kGroups * N) {  // the same for every group: shuffles stay warp-wide
    if (h0 > 0) rope_load<D, N>(src, heads, h0, grp, li, raw);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (h0 + j * kGroups >= heads) break;
      const int h = h0 + j * kGroups + grp;
      float2 x[4];
      unpack8(raw[j], x);
      float2 sq = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = ffma2(x[i], x[i], sq);
      float ss = sq.x + sq.y;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss * (1.f / D) + eps);
      float2 y[4];
      if constexpr (INTERLEAVED) {  // partners are the two halves of each pair
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_float2(x[i].y, x[i].x);
      } else {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw[j].x, partner);
        o.y = __shfl_sync(0xffffffffu, raw[j].y, partner);
        o.z = __shfl_sync(0xffffffffu, raw[j].z, partner);
        o.w = __shfl_sync(0xffffffffu, raw[j].w, partner);
        unpack8(o, y);
      }
      uint32_t z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 zero2 = make_float2(0.f, 0.f);
        const float2 r = ffma2(y[i], w.other[i], ffma2(x[i], w.own[i], zero2));
        z[i] = zero ? 0u : pack_bf16(r.x * inv, r.y * inv);
      }
      if (h < heads)
        *reinterpret_cast<uint4*>(dst + (int64_t)h * D + li * 8) = make_uint4(z[0], z[1], z[2], z[3]);
    }
  }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8;  // lanes per row
  const int t = blockIdx.x;
  const int grp = threadIdx.x / kLanes;
  const int li = threadIdx.x % kLanes;
  // the rows first: they depend on nothing.  4 of q and 2 of k a group and round (of 128 dims: 16 and 8 heads)
  const __nv_bfloat16 *q = p.q + t * p.q_stride, *k = p.k + t * p.k_stride;
  uint4 q_raw[4], k_raw[2];
  rope_load<D, 4>(q, p.num_q_heads, 0, grp, li, q_raw);
  rope_load<D, 2>(k, p.num_kv_heads, 0, grp, li, k_raw);
  const int pos = p.positions[t];
  const bool pos_ok = pos >= 0 && pos < p.max_position;
  if (!pos_ok && threadIdx.x == 0) record_error(p.err, kErrBadInput);  // the token's rows become zeros
  const int half = p.rotary >> 1;
  const bool turns = li * 8 < p.rotary;  // dims past `rotary` turn by nothing
  const bool upper = !INTERLEAVED && li * 8 >= half;
  // the lane of this group that holds the partner dims (itself past `rotary`, and when interleaved)
  const int partner_li = INTERLEAVED || !turns ? li : upper ? li - half / 8 : li + half / 8;
  const int partner = (threadIdx.x & 31) - li + partner_li;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (turns) {
    const float* row = p.cos_sin + (int64_t)(pos_ok ? pos : 0) * p.rotary;
    if constexpr (INTERLEAVED) {  // four pairs
      const float4 c = *reinterpret_cast<const float4*>(row + li * 4);
      const float4 s = *reinterpret_cast<const float4*>(row + half + li * 4);
      cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
      sn[0] = -s.x; sn[1] = s.x; sn[2] = -s.y; sn[3] = s.y;
      sn[4] = -s.z; sn[5] = s.z; sn[6] = -s.w; sn[7] = s.w;
    } else {  // eight pairs, of which this lane has the first or the second dims
      const int at = upper ? li * 8 - half : li * 8;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 c = *reinterpret_cast<const float4*>(row + at + i);
        const float4 s = *reinterpret_cast<const float4*>(row + half + at + i);
        cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
        sn[i] = upper ? s.x : -s.x;
        sn[i + 1] = upper ? s.y : -s.y;
        sn[i + 2] = upper ? s.z : -s.z;
        sn[i + 3] = upper ? s.w : -s.w;
      }
    }
  }
  auto turn = [&](const __nv_bfloat16* weight) {
    float2 own[4], other[4];
    unpack8(reinterpret_cast<const uint4*>(weight)[li], own);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) other[i] = make_float2(own[i].y, own[i].x);
    } else {
      unpack8(reinterpret_cast<const uint4*>(weight)[partner_li], other);
    }
    RopeTurn w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.own[i] = make_float2(own[i].x * cs[2 * i], own[i].y * cs[2 * i + 1]);
      w.other[i] = make_float2(other[i].x * sn[2 * i], other[i].y * sn[2 * i + 1]);
    }
    return w;
  };
  rope_rows<D, 4, INTERLEAVED>(q, p.q_out + t * p.q_out_stride, p.num_q_heads, grp, li, partner, turn(p.q_weight),
                               p.eps, !pos_ok, q_raw);
  rope_rows<D, 2, INTERLEAVED>(k, p.k_out + t * p.k_out_stride, p.num_kv_heads, grp, li, partner, turn(p.k_weight),
                               p.eps, !pos_ok, k_raw);
}

template <int D, bool INTERLEAVED>
cudaError_t launch_one(const RopeParams& p, cudaStream_t st) {
  qk_norm_rope_kernel<D, INTERLEAVED><<<(unsigned)p.num_tokens, kRopeThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, bool interleaved, cudaStream_t st) {
  if (head_dim == 128) return interleaved ? launch_one<128, true>(p, st) : launch_one<128, false>(p, st);
  if (head_dim == 64) return interleaved ? launch_one<64, true>(p, st) : launch_one<64, false>(p, st);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
