// Order and barriers of the 4-bit tile kernel's staging ring: plain index arithmetic, the same on the host
// and on the device.
//
// One producer fills three slots in turn with the uses u = 0, 1, 2, ... = K of step 0, V of step 0, K of step
// 1, ...; one warp takes the K uses, another the V uses, and gives each slot back.  Consecutive uses of a slot
// belong to different warps, so a landed-barrier per slot would show each warp only every second of its
// phases: a warp that waits for a parity while the use before, the other warp's, is still in flight would pass
// at once, on the parity of the phase before that.  The landed-barriers are therefore numbered by u % 6, the
// period after which the same warp meets the same slot: each has one waiting warp, which sees every phase.
// The given-back barriers are waited for by the producer alone, which sees every phase of each slot's.
#pragma once

#ifdef __CUDACC__
#define PA_RING_FN __host__ __device__ __forceinline__
#else
#define PA_RING_FN inline
#endif

namespace pa {

struct StageRing {
  static constexpr int kSlots = 3;
  static constexpr int kFullBars = 2 * kSlots;  // a use's pages have landed
  static constexpr int kEmptyBars = kSlots;     // a slot has been read

  static PA_RING_FN int use(int step, bool is_v) { return 2 * step + (is_v ? 1 : 0); }
  static PA_RING_FN int slot(int u) { return u % kSlots; }
  // what the use's reader waits for, and the producer before it ends
  static PA_RING_FN int full_bar(int u) { return u % kFullBars; }
  static PA_RING_FN unsigned full_parity(int u) { return (unsigned)(u / kFullBars) & 1u; }
  // the use's reader arrives here; before it fills the slot again for use u >= kSlots the producer waits for
  // the phase of use u - kSlots
  static PA_RING_FN int empty_bar(int u) { return u % kSlots; }
  static PA_RING_FN unsigned empty_parity(int u) { return (unsigned)(u / kSlots - 1) & 1u; }
};

}  // namespace pa
