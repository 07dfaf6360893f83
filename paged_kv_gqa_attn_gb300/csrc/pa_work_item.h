// A prefill work item: one 128-row tile of one sequence in a 32-bit word, the sequence in the low half and the
// tile in the high half.  The host admits at most kWorkSeqs sequences and kWorkTiles tiles of one, so both
// halves are used whole: unsigned arithmetic, as a tile from 32768 on sets the word's sign bit.  Plain
// arithmetic, the same on the host and on the device.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_WORK_FN __host__ __device__ __forceinline__
#else
#define PA_WORK_FN inline
#endif

namespace pa {

constexpr int kWorkSeqs = 1 << 16, kWorkTiles = (1 << 16) - 1;

PA_WORK_FN int32_t work_item(int seq, int tile) { return (int32_t)((uint32_t)seq | ((uint32_t)tile << 16)); }
PA_WORK_FN int work_seq(int32_t item) { return (int)((uint32_t)item & 0xffffu); }
PA_WORK_FN int work_tile(int32_t item) { return (int)((uint32_t)item >> 16); }

}  // namespace pa
