// Fragment helpers of the kernels on the warp-level tensor-core instruction (mma.sync m16n8k16): page
// layouts in shared memory, the product itself, the transposition between its two uses.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr float kTau = 8.f;  // largest softmax weight, log2, before the running max is refreshed

// What an E4M3 page's V scale adds to its scores (lv = log2 |scale|), what takes it out of the row sum again (rvs
// = 2^-lv), and the sign of f16 weights.  `top` is the largest lv so far of this warp.  A smaller scale than 2^(top
// - 60), zero among them, counts as that: the page's weights stay in the fp32 range and in the row sum, and its
// values are off by 2^-60 of the largest.  (4 x 131072 tokens: 164.6 -> 165.5 us.)
struct VScaleFold {
  float lv, rvs;
  uint32_t neg;
};
__device__ __forceinline__ VScaleFold fold_v_scale(float vs, float& top) {
  VScaleFold f;
  f.lv = __log2f(fmaxf(fabsf(vs), 0x1p-100f));
  top = fmaxf(top, f.lv);
  f.lv = fmaxf(f.lv, top - 60.f);
  f.rvs = fast_exp2(-f.lv);
  f.neg = vs < 0.f ? 0x80008000u : 0u;
  return f;
}
constexpr float kVFoldMin = -100.f;  // of lv, where `top` starts

// Byte offset of 16-byte chunk `c` of row `r` of a page as the TMA unit writes it.  Rows of 128 B
// or more arrive as boxes of 128-byte rows with the 128-byte swizzle (chunk ^ row % 8), box j
// holding chunks 8j .. 8j+7 of every row; 64-byte rows use the 64-byte swizzle
// (chunk ^ (row / 2) % 4).  Pages are 1 KiB aligned.
template <int RB>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  if constexpr (RB == 64)
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return (c >> 3) * (16 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// The c-th K chunk of thread q: a quarter of the row, taken as chunk pairs 2q, 2q+1 of each
// 128-byte box (so that the 8 threads of a load phase hit 8 different bank groups), or chunk q
// of a 64-byte row.
template <int RB>
__device__ __forceinline__ int qk_chunk(int q, int c) {
  if constexpr (RB == 64)
    return q;
  else
    return 8 * (c >> 1) + 2 * q + (c & 1);
}

// D[16x8] += A[16x16] . B[16x8], f16 (or bf16) operands, fp32 accumulators (warp-collective).
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held as mma fragments (warp-collective).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// What bf16 rounding leaves of p (rounded to bf16 again, it carries p's next 8 significant bits).
__device__ __forceinline__ float bf16_rem(float p) { return p - __bfloat162float(__float2bfloat16_rn(p)); }

}  // namespace pa
