// The k largest of n numbers by one CTA, in the order of their indices (sm_103a).
//
// Numbers become unsigned keys of the same order.  The k-th largest key is found eight bits at a time, from the
// highest bit in which the keys differ (scores of one query have the same sign and nearly the same exponent: from
// bit 31 all of them would meet in one counter): a histogram of the next digit over the keys that agree with what
// is known so far, in shared memory with four counters a digit (a lane takes one by its number), and one warp's
// scan from the highest digit down.  A digit whose keys are all taken ends it early; equal keys at the border run
// to the last bit and are then taken from the lowest index on.  Counts are whole numbers: nothing depends on an
// order of atomics.
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
  alignas(16) int hist[256 * 4];
  int warp_gt[32], warp_eq[32];
  int digit, above, at;  // the digit of the k-th key, and how many candidates lie above it and at it
  uint32_t top, bottom;  // the largest and the smallest key that is not kKeyAlways, and how many are
  int always;
};

// keys[0, n) in shared or global memory, written before a barrier; every thread of the CTA (a multiple of 32, at most
// 1024) calls this with 0 < k < n, and at most k keys kKeyAlways.  Calls take(position, index) for each key taken, positions
// 0 .. k - 1 in the order of the indices.
template <class Take>
__device__ __forceinline__ void topk_in_order(const uint32_t* keys, int n, int k, TopkShared& sh, Take take) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (tid == 0) {
    sh.top = 0u;
    sh.bottom = kKeyAlways;
    sh.always = 0;
  }
  __syncthreads();
  {
    uint32_t top = 0u, bottom = kKeyAlways;
    int always = 0;
    for (int i = tid; i < n; i += threads) {
      const uint32_t x = keys[i];
      always += x == kKeyAlways;
      top = max(top, x == kKeyAlways ? 0u : x);
      bottom = min(bottom, x);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bottom = __reduce_min_sync(0xffffffffu, bottom);
    always = __reduce_add_sync(0xffffffffu, always);
    if (lane == 0) {
      atomicMax(&sh.top, top);
      atomicMin(&sh.bottom, bottom);
      atomicAdd(&sh.always, always);
    }
  }
  __syncthreads();
  int need = k - sh.always;  // keys to take among the candidates: those that agree with low in the known bits
  const int differ = 32 - __clz(sh.top ^ sh.bottom);  // bits from the highest that differs down
  uint32_t known = differ >= 32 ? 0u : ~0u << differ, low = sh.top & known;
  bool exact = false;  // all candidates are taken (those above low, and at it)
  if (need <= 0) {
    low = kKeyAlways;
    exact = true;
  }
  int shift = differ;
  while (shift > 0 && !exact) {
    shift = max(shift - 8, 0);
    for (int i = tid; i < 256 * 4; i += threads) sh.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += threads) {
      const uint32_t x = keys[i];
      if ((x & known) == low && x != kKeyAlways) atomicAdd(&sh.hist[((x & ~known) >> shift) * 4 + (lane & 3)], 1);
    }
    __syncthreads();
    if (warp == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
      int count[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int4 c = *reinterpret_cast<const int4*>(&sh.hist[(255 - 8 * lane - j) * 4]);
        count[j] = (c.x + c.y) + (c.z + c.w);
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
    exact = sh.at == need;  // (what is not known of low is zeros: every candidate is at or above it)
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
