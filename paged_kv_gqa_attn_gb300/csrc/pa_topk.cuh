// The k largest of n numbers by one CTA, in the order of their indices (sm_103a).
//
// Numbers become unsigned keys of the same order.  The k-th largest key is found from its top bits down, two a round:
// each round counts the keys at or above the three candidates that the next two bits allow, one reduction a warp and
// one atomic add for each count.  A candidate that exactly k keys reach ends it early, which scattered numbers bring
// about after a third to a half of the sixteen rounds; equal keys at the border run to the last bit and are then taken
// from the lowest index on.  Nothing depends on an order of atomics: counts are whole numbers.
#pragma once

#include <stdint.h>

namespace pa {

// Unsigned keys in the order of the floats (-0 as 0); a NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 0u : (u >> 31) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kKeyAlways = 0xffffffffu;  // above every number

struct TopkShared {
  int count[16][3];
  int warp_gt[32], warp_eq[32];
};

// keys[0, n) in shared or global memory, written before a barrier; every thread of the CTA (a multiple of 32, at most
// 1024) calls this with 0 < k < n.  Calls take(position, index) for each key taken, positions 0 .. k - 1 in
// the order of the indices.
template <class Take>
__device__ __forceinline__ void topk_in_order(const uint32_t* keys, int n, int k, TopkShared& sh, Take take) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (tid < 48) sh.count[tid / 3][tid % 3] = 0;
  __syncthreads();
  // keys >= low are at least k in number, keys >= high fewer (high: the next candidate above low)
  uint32_t low = 0u;
  bool exact = false;  // exactly k keys are >= low
  for (int round = 0; round < 16 && !exact; ++round) {
    const int shift = 30 - 2 * round;
    const uint32_t c1 = low | (1u << shift), c2 = low | (2u << shift), c3 = low | (3u << shift);
    int n1 = 0, n2 = 0, n3 = 0;
    for (int i = tid; i < n; i += threads) {
      const uint32_t x = keys[i];
      n1 += x >= c1;
      n2 += x >= c2;
      n3 += x >= c3;
    }
    n1 = __reduce_add_sync(0xffffffffu, n1);
    n2 = __reduce_add_sync(0xffffffffu, n2);
    n3 = __reduce_add_sync(0xffffffffu, n3);
    if (lane == 0) {
      atomicAdd(&sh.count[round][0], n1);
      atomicAdd(&sh.count[round][1], n2);
      atomicAdd(&sh.count[round][2], n3);
    }
    __syncthreads();
    const int m1 = sh.count[round][0], m2 = sh.count[round][1], m3 = sh.count[round][2];
    if (m3 >= k) {
      low = c3;
      exact = m3 == k;
    } else if (m2 >= k) {
      low = c2;
      exact = m2 == k;
    } else if (m1 >= k) {
      low = c1;
      exact = m1 == k;
    }
  }
  // each thread a run of keys (an odd number: no two lanes in one bank); how many lie above low, and at it, before it
  const int per = ((n + threads - 1) / threads) | 1;
  const int first = min(n, tid * per), last = min(n, first + per);
  int gt = 0, eq = 0;
  for (int i = first; i < last; ++i) {
    const uint32_t x = keys[i];
    gt += exact ? x >= low : x > low;
    eq += !exact && x == low;
  }
  int gt_inc = gt, eq_inc = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, gt_inc, o), b = __shfl_up_sync(0xffffffffu, eq_inc, o);
    if (lane >= o) {
      gt_inc += a;
      eq_inc += b;
    }
  }
  if (lane == 31) {
    sh.warp_gt[warp] = gt_inc;
    sh.warp_eq[warp] = eq_inc;
  }
  __syncthreads();
  int gt_before = gt_inc - gt, eq_before = eq_inc - eq, gt_all = 0;
  for (int w = 0; w < threads / 32; ++w) {
    gt_all += sh.warp_gt[w];
    if (w < warp) {
      gt_before += sh.warp_gt[w];
      eq_before += sh.warp_eq[w];
    }
  }
  const int room = k - gt_all;  // keys equal to low that are taken
  for (int i = first; i < last; ++i) {
    const uint32_t x = keys[i];
    const bool above = exact ? x >= low : x > low, at = !exact && x == low;
    if (above || (at && eq_before < room)) take(gt_before + min(eq_before, room), i);
    gt_before += above;
    eq_before += at;
  }
}

}  // namespace pa
