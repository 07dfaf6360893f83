// The step's softmax weights, folded into the sums that are kept for every cached token.
//
// Attention with kept scores leaves the base-2 scores x of a token's G query heads and each row's log2-sum-exp; the
// token's weight is sum_h 2^(x_h - lse_h), and its sum becomes decay * sum + weight; the step's own token has no sum yet,
// so that its slot is set.  A pass bound by bytes (4 G read, 4 read and written a token): a second one over K in place
// of the kept scores would read 2 d bytes a token instead.
#include "pa_kernels.h"

namespace pa {
namespace {

template <int G>  // 0: any group
__global__ void __launch_bounds__(256) fold_weights_kernel(const WeightParams p) {
  const int group = G > 0 ? G : p.group;
  const int g = blockIdx.y, b = blockIdx.z;
  const int L = max(0, min(p.context_lens[b], p.max_context_len));
  const int t = blockIdx.x * 256 + threadIdx.x;
  int pb = -1;
  if (t < L) pb = p.block_table[(size_t)b * p.max_blocks_per_seq + t / 16];
  const bool there = pb >= 0 && pb < p.num_blocks;  // (an id out of range was flagged by the attention)
  float* dst = p.weights + ((size_t)(there ? pb : 0) * p.num_kv_heads + g) * 16 + t % 16;
  float old = 0.f;
  if (there && p.decay != 0.f && t != L - 1) old = *dst * p.decay;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!there) return;
  const float* lse = p.lse + ((size_t)b * p.num_kv_heads + g) * group;
  const float* x = p.scores + (((size_t)b * p.num_kv_heads + g) * p.max_context_len + t) * group;
  float w = 0.f;
  if constexpr (G >= 4) {
#pragma unroll
    for (int h = 0; h < G; h += 4) {
      const float4 s = *reinterpret_cast<const float4*>(x + h), l = *reinterpret_cast<const float4*>(lse + h);
      w += (fast_exp2(s.x - l.x) + fast_exp2(s.y - l.y)) + (fast_exp2(s.z - l.z) + fast_exp2(s.w - l.w));
    }
  } else {
    for (int h = 0; h < group; ++h) w += fast_exp2(x[h] - lse[h]);
  }
  *dst = old + w;
}

}  // namespace

cudaError_t launch_fold_weights(const WeightParams& p, cudaStream_t st) {
  if (p.max_context_len < 1) return cudaSuccess;
  const dim3 grid((p.max_context_len + 255) / 256, p.num_kv_heads, p.num_seqs);
  WeightParams pp = p;
  void* args[] = {&pp};
  const void* fn = p.group == 8   ? reinterpret_cast<const void*>(fold_weights_kernel<8>)
                   : p.group == 4 ? reinterpret_cast<const void*>(fold_weights_kernel<4>)
                                  : reinterpret_cast<const void*>(fold_weights_kernel<0>);
  return launch_dependent(fn, grid, dim3(256), 0, st, args);
}

}  // namespace pa
