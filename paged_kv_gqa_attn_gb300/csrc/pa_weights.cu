// The step's softmax weights, folded into the sums that are kept for every cached token.
//
// Attention with kept scores leaves the base-2 scores x of a token's G query heads and each row's log2-sum-exp;
// the token's weight is sum_h 2^(x_h - lse_h), and its sum becomes decay * sum + weight; the step's own token has
// no sum yet, so that its slot is set.  A pass bound by bytes (4 G read, 4 read and written a token): a second one
// over K in place of the kept scores would read 2 d bytes a token instead.
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kFoldTokens = 4;  // of a thread: a quarter of a block's (one a thread: 35 us where four take 22,
                                // 64 contexts of 1000 to 16384 tokens, groups of 4)

template <int G>  // 0: any group
__global__ void __launch_bounds__(256) fold_weights_kernel(const WeightParams p) {
  const int group = G > 0 ? G : p.group;
  // the sequences whose scores were written last come first: they are still in the L2
  const int g = blockIdx.y, b = gridDim.z - 1 - blockIdx.z;
  const int L = max(0, min(p.context_lens[b], p.max_context_len));
  const int t = (blockIdx.x * 256 + threadIdx.x) * kFoldTokens;
  int pb = -1;
  if (t < L) pb = p.block_table[(size_t)b * p.max_blocks_per_seq + t / 16];
  const bool there = pb >= 0 && pb < p.num_blocks;  // (an id out of range was flagged by the attention)
  const int n = min(kFoldTokens, L - t);
  float* dst = p.weights + ((size_t)(there ? pb : 0) * p.num_kv_heads + g) * 16 + t % 16;
  float old[kFoldTokens] = {0.f, 0.f, 0.f, 0.f};
  if (there && p.decay != 0.f) {  // (a quarter of a block's sums lies within the pool, whatever the context)
    const float4 v = *reinterpret_cast<const float4*>(dst);
    const float w4[kFoldTokens] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kFoldTokens; ++i)
      if (t + i < L - 1) old[i] = w4[i] * p.decay;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!there) return;
  const float* lse = p.lse + ((size_t)b * p.num_kv_heads + g) * group;
  const float* x = p.scores + (((size_t)b * p.num_kv_heads + g) * p.max_context_len + t) * group;
  float w[kFoldTokens] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (G >= 4) {
#pragma unroll
    for (int h = 0; h < G; h += 4) {
      const float4 l = *reinterpret_cast<const float4*>(lse + h);
      float4 s[kFoldTokens];
#pragma unroll
      for (int i = 0; i < kFoldTokens; ++i) s[i] = i < n ? *reinterpret_cast<const float4*>(x + i * G + h) : l;
#pragma unroll
      for (int i = 0; i < kFoldTokens; ++i)
        w[i] += (fast_exp2(s[i].x - l.x) + fast_exp2(s[i].y - l.y)) + (fast_exp2(s[i].z - l.z) + fast_exp2(s[i].w - l.w));
    }
  } else {
    for (int h = 0; h < group; ++h)
#pragma unroll
      for (int i = 0; i < kFoldTokens; ++i)
        if (i < n) w[i] += fast_exp2(x[i * group + h] - lse[h]);
  }
  if (n == kFoldTokens) {
    *reinterpret_cast<float4*>(dst) = make_float4(old[0] + w[0], old[1] + w[1], old[2] + w[2], old[3] + w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kFoldTokens; ++i)
    if (i < n) dst[i] = old[i] + w[i];
}

}  // namespace

cudaError_t launch_fold_weights(const WeightParams& p, cudaStream_t st) {
  if (p.max_context_len < 1) return cudaSuccess;
  const int per_cta = 256 * kFoldTokens;
  const dim3 grid((p.max_context_len + per_cta - 1) / per_cta, p.num_kv_heads, p.num_seqs);
  WeightParams pp = p;
  void* args[] = {&pp};
  const void* fn = p.group == 8   ? reinterpret_cast<const void*>(fold_weights_kernel<8>)
                   : p.group == 4 ? reinterpret_cast<const void*>(fold_weights_kernel<4>)
                                  : reinterpret_cast<const void*>(fold_weights_kernel<0>);
  return launch_dependent(fn, grid, dim3(256), 0, st, args);
}

}  // namespace pa
