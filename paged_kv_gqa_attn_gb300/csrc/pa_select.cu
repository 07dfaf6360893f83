// Selection of the cache blocks that a step's queries should read: a cheap score for each block, the highest kept.
//
// A query row is rounded to int8 codes times a power of two 2^f, a block's bounds are int8 codes times 2^e
// (pa_bounds.cu), and its score for the row is 2^f 2^e sum_i max(c_i hi_i, c_i lo_i): with c+ = max(c, 0) and c- =
// min(c, 0) a product of [c+ | c-] with [hi | lo], 2 d long: a matrix product of 16 blocks by 8 rows on the tensor
// cores, whose partial sums are whole numbers below 2^22.  No rounding anywhere, so the selection does not depend
// on how it is computed: up to eight rows take the int8 form of the instruction, more the f16 form (codes are
// exact in f16, sums in fp32), as int8 runs at a small part of f16's rate here and its pipe was the bound (20 rows
// a head: 2 us a tile; a step with them 50 us in int8, 45 in f16), while turning bytes into f16 costs the few-row
// form more than it saves (151 us against 140, 64 contexts of up to 32768).  A block counts for a kv head with its
// best row.
//
// Scores: a warp takes 16 blocks of one (sequence, kv head) at a time, straight from global memory into A
// fragments (the contraction's order is free: a lane reads whole 16-byte pieces, and the rows' codes are laid out
// alike, once for the CTA's warps, in shared memory).  Bound by the bounds' bytes: a warp's next tile is loaded
// before this one's products.  (A ring of cp.async copies in shared memory, two tiles ahead, measured no faster:
// its room leaves fewer warps.)
//
// Selection (pa_topk.cuh): contexts of up to 1024 blocks, or up to 4096 of no more (sequence, kv head) pairs than
// there are SMs, take one kernel, a cluster of one to eight CTAs for each pair, whose scores meet as keys in the
// first CTA's shared memory: one launch, no scratch.  Else two: scores in scratch, then one CTA per pair.  In one
// kernel and in two, us: 4 contexts of 8 heads, up to 4096 / 16384 / 65536 tokens 10.3 and 11.8 / 12.3 and 14.7 /
// 20.6 and 22.0; 64 contexts 14.4 and 17.3 / 30.1 and 29.5 / 82 and 66; 256 contexts 28.7 and 35.3 / 73.5 and
// 80.8; 64 of 2 heads, 65536 33.4 and 35.1.  (Many long ones lose: a cluster's CTAs leave together, and its
// selection waits for the last of their scores.)
#include "pa_kernels.h"
#include "pa_mma.cuh"
#include "pa_tc.cuh"
#include "pa_topk.cuh"

namespace pa {
namespace {

constexpr int kScoreWarps = 4;

// D[16x8] += A[16x32] . B[32x8], int8 operands, int32 accumulators (warp-collective).
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four signed bytes -> two f16 pairs, exactly: biased by 128 they are the low bits of 1024 + x.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const uint32_t bias = 0x64806480u;  // 1024 + 128
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

// e of the int8 codes of numbers up to amax: the smallest with amax 2^-e <= 127, at least -126.
__device__ __forceinline__ int code_exp(float amax) {
  const uint32_t bits = __float_as_uint(fminf(amax, 3.4028235e38f));
  const int e = (int)(bits >> 23) - 127 - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return bits == 0 ? 0 : max(e, -126);
}

template <int D, int NT>
struct ScoreShared {
  static constexpr bool kInt8 = NT == 1;
  static constexpr int kChunks = D / 64;  // 16-byte pieces of a lane in each half ([hi] and [lo]) of a row
  // B fragments (for 16 codes one 16-byte piece in int8, two in f16): positive parts, then negative ones
  uint4 q_frag[NT][2 * kChunks][kInt8 ? 1 : 2][32];
  float q_up[8 * NT];  // 2^f of each row
};

// Scores of 16-block tiles first, first + stride, ... (at most `most` of them, below ncols blocks) of (b, g) by each warp of
// a CTA: sink(column, score) for every block.  Blocks that are not there score -infinity and are flagged.  WARP: the warp
// alone works on (b, g), and sh is its own.
template <int D, int NT, bool WARP, class Sink>
__device__ __forceinline__ void score_tiles(const SelectParams& p, int b, int g, int ncols, int first, int stride, int most,
                                            ScoreShared<D, NT>& sh, Sink sink) {
  using S = ScoreShared<D, NT>;
  constexpr int kChunks = S::kChunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gi = lane >> 2, qi = lane & 3;
  const int Hkv = p.num_kv_heads, G = p.num_q_heads / Hkv, R = p.q_len * G;
  // the first tile's loads start before the rows are rounded
  const int32_t* bt = p.block_table + (size_t)b * p.max_blocks_per_seq;
  struct Tile {
    uint4 a0[2 * kChunks], a1[2 * kChunks];  // blocks gi and gi + 8: upper, then lower codes, pieces qi, qi + 4, ...
    float s0, s1;
    bool ok0, ok1;
  };
  auto id_at = [&](int col) { return col < ncols ? bt[col] : -1; };
  auto load = [&](Tile& t, int id0, int id1) {
    t.ok0 = id0 >= 0 && id0 < p.num_blocks;
    t.ok1 = id1 >= 0 && id1 < p.num_blocks;
    const size_t page0 = (size_t)(t.ok0 ? id0 : 0) * Hkv + g, page1 = (size_t)(t.ok1 ? id1 : 0) * Hkv + g;
    const uint4* r0 = reinterpret_cast<const uint4*>(p.bounds + page0 * (2 * D)) + qi;
    const uint4* r1 = reinterpret_cast<const uint4*>(p.bounds + page1 * (2 * D)) + qi;
#pragma unroll
    for (int k = 0; k < 2 * kChunks; ++k) {
      t.a0[k] = t.ok0 ? r0[4 * k] : make_uint4(0u, 0u, 0u, 0u);
      t.a1[k] = t.ok1 ? r1[4 * k] : make_uint4(0u, 0u, 0u, 0u);
    }
    t.s0 = p.bound_scale[page0];
    t.s1 = p.bound_scale[page1];
  };
  Tile cur;
  load(cur, id_at(first * 16 + gi), id_at(first * 16 + gi + 8));
  int id0 = id_at((first + stride) * 16 + gi), id1 = id_at((first + stride) * 16 + gi + 8);

  // the codes of row gi of each n-tile, pieces qi and qi + 4 of its d dims, positive and negative parts
  for (int nt = WARP ? 0 : warp; nt < NT; nt += WARP ? 1 : kScoreWarps) {
    const int c = 8 * nt + gi;
    const bool real = c < R;
    const __nv_bfloat16* row =
        p.q + (((size_t)b * p.q_len + (real ? c / G : 0)) * p.num_q_heads + g * G + (real ? c % G : 0)) * D;
    uint32_t x[kChunks][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const uint4* src = reinterpret_cast<const uint4*>(row + (qi + 4 * k) * 16);
      const uint4 a = real ? src[0] : make_uint4(0u, 0u, 0u, 0u), d = real ? src[1] : make_uint4(0u, 0u, 0u, 0u);
      x[k][0] = a.x; x[k][1] = a.y; x[k][2] = a.z; x[k][3] = a.w;
      x[k][4] = d.x; x[k][5] = d.y; x[k][6] = d.z; x[k][7] = d.w;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = bf16x2_to_f2(x[k][j]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int f = code_exp(amax);
    const float down = exp2_int(-f);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      uint32_t pos[8], neg[8];
      if constexpr (S::kInt8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          pos[w] = neg[w] = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = bf16x2_to_f2(x[k][2 * w + e / 2]);
            const int code = max(-127, min(127, __float2int_rn((e & 1 ? v.y : v.x) * down)));
            pos[w] |= (uint32_t)(max(code, 0) & 0xff) << (8 * e);
            neg[w] |= (uint32_t)(min(code, 0) & 0xff) << (8 * e);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 v = bf16x2_to_f2(x[k][w]);
          const float a = fminf(fmaxf(rintf(v.x * down), -127.f), 127.f), d = fminf(fmaxf(rintf(v.y * down), -127.f), 127.f);
          pos[w] = pack_f16(fmaxf(a, 0.f), fmaxf(d, 0.f));
          neg[w] = pack_f16(fminf(a, 0.f), fminf(d, 0.f));
        }
      }
#pragma unroll
      for (int h = 0; h < (S::kInt8 ? 1 : 2); ++h) {
        sh.q_frag[nt][k][h][lane] = make_uint4(pos[4 * h], pos[4 * h + 1], pos[4 * h + 2], pos[4 * h + 3]);
        sh.q_frag[nt][kChunks + k][h][lane] = make_uint4(neg[4 * h], neg[4 * h + 1], neg[4 * h + 2], neg[4 * h + 3]);
      }
    }
    if (qi == 0) sh.q_up[c] = exp2_int(f);
  }
  if constexpr (WARP)
    __syncwarp();
  else
    __syncthreads();
  float up[NT][2];  // of rows 2qi, 2qi + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    up[nt][0] = sh.q_up[8 * nt + 2 * qi];
    up[nt][1] = sh.q_up[8 * nt + 2 * qi + 1];
  }

  for (int t = 0; t < most; ++t) {
    const int col0 = (first + t * stride) * 16;
    if (col0 >= ncols) break;
    Tile next;
    const bool more = t + 1 < most && col0 + stride * 16 < ncols;
    if (more) {
      load(next, id0, id1);
      id0 = id_at(col0 + 2 * stride * 16 + gi);
      id1 = id_at(col0 + 2 * stride * 16 + gi + 8);
    }
    if (((!cur.ok0 && col0 + gi < ncols) || (!cur.ok1 && col0 + gi + 8 < ncols)) && qi == 0)
      record_error(p.err, kErrBlockId);
    // products: [0..1] of block gi, rows 2qi, 2qi + 1; [2..3] of block gi + 8
    float best0 = -INFINITY, best1 = -INFINITY;
    auto rows_of = [&](int nt, float x0, float x1, float x2, float x3) {
      if (8 * nt + 2 * qi < R) {
        best0 = fmaxf(best0, x0 * up[nt][0]);
        best1 = fmaxf(best1, x2 * up[nt][0]);
      }
      if (8 * nt + 2 * qi + 1 < R) {
        best0 = fmaxf(best0, x1 * up[nt][1]);
        best1 = fmaxf(best1, x3 * up[nt][1]);
      }
    };
    if constexpr (S::kInt8) {
      int acc[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 2 * kChunks; ++k) {
        const uint4 q = sh.q_frag[0][k][0][lane];
        mma_s8(acc, cur.a0[k].x, cur.a1[k].x, cur.a0[k].y, cur.a1[k].y, q.x, q.y);
        mma_s8(acc, cur.a0[k].z, cur.a1[k].z, cur.a0[k].w, cur.a1[k].w, q.z, q.w);
      }
      rows_of(0, (float)acc[0], (float)acc[1], (float)acc[2], (float)acc[3]);
    } else {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * kChunks; ++k) {
        const uint32_t w0[4] = {cur.a0[k].x, cur.a0[k].y, cur.a0[k].z, cur.a0[k].w};
        const uint32_t w1[4] = {cur.a1[k].x, cur.a1[k].y, cur.a1[k].z, cur.a1[k].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s8x4_to_f16(w0[2 * h + e], a[e][0], a[e][2]);
            s8x4_to_f16(w1[2 * h + e], a[e][1], a[e][3]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 q = sh.q_frag[nt][k][S::kInt8 ? 0 : h][lane];
            mma_16816<false>(acc[nt], a[0][0], a[0][1], a[0][2], a[0][3], q.x, q.y);
            mma_16816<false>(acc[nt], a[1][0], a[1][1], a[1][2], a[1][3], q.z, q.w);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) rows_of(nt, acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, o));
      best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, o));
    }
    if (qi == 0) {  // (a block that is not there comes last)
      if (col0 + gi < ncols) sink(col0 + gi, cur.ok0 ? best0 * cur.s0 : -INFINITY);
      if (col0 + gi + 8 < ncols) sink(col0 + gi + 8, cur.ok1 ? best1 * cur.s1 : -INFINITY);
    }
    if (more) cur = next;
  }
}

// The sequence's blocks, its length cut to the bound (and flagged by one thread).
__device__ __forceinline__ int select_cols(const SelectParams& p, int b, bool flag) {
  const int L = p.context_lens[b];
  if (flag && L > p.max_context_len) record_error(p.err, kErrShortContext);
  return (max(0, min(L, p.max_context_len)) + 15) / 16;
}

constexpr int kClusterCtas = 8;     // at most
constexpr int kClusterCols = 4096;  // keys in the first CTA's shared memory
constexpr int kClusterColsMany = 1024;  // where there are more pairs than SMs

// Whether a call takes the one kernel.
bool in_clusters(int num_seqs, int num_kv_heads, int max_context_len, int num_sms) {
  const bool few = (int64_t)num_seqs * num_kv_heads <= num_sms;
  return max_context_len <= (few ? kClusterCols : kClusterColsMany) * 16;
}

template <int D, int NT>
__global__ void __launch_bounds__(kScoreWarps * 32) block_select_kernel(const SelectParams p) {
  extern __shared__ uint32_t smem_keys[];  // of the first CTA: one for each block
  __shared__ ScoreShared<D, NT> sh;
  __shared__ TopkShared top;
  const int rank = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int ncols = select_cols(p, b, rank == 0 && g == 0 && threadIdx.x == 0);
  int32_t* out = p.blocks + ((size_t)b * p.num_kv_heads + g) * p.count;
  if (ncols <= p.count) {  // (the whole cluster) every block
    if (rank == 0)
      for (int i = threadIdx.x; i < p.count; i += blockDim.x) {
        out[i] = i < ncols ? i : -1;
        if (g == 0 && i < ncols) {  // (nothing is scored here: the ids are looked at for the flag alone)
          const int id = p.block_table[(size_t)b * p.max_blocks_per_seq + i];
          if (id < 0 || id >= p.num_blocks) record_error(p.err, kErrBlockId);
        }
      }
    return;
  }
  cluster_arrive();
  uint32_t keys0;  // the first CTA's keys
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(keys0) : "r"(smem_addr(smem_keys)), "r"(0));
  cluster_wait();  // every CTA runs: its shared memory may be written
  const int first = rank * kScoreWarps + (threadIdx.x >> 5);
  score_tiles<D, NT, false>(p, b, g, ncols, first, gridDim.x * kScoreWarps, kClusterCols, sh, [&](int col, float score) {
    const uint32_t key = col < p.sinks || col >= ncols - p.recent ? kKeyAlways : order_key(score);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys0 + col * 4), "r"(key) : "memory");
  });
  cluster_arrive();
  cluster_wait();
  if (rank == 0) topk_in_order(smem_keys, ncols, p.count, top, [&](int at, int i) { out[at] = i; });
}

// HEADS: the warps take neighbouring kv heads of the same blocks, whose bounds are neighbours in memory (kScoreWarps
// or more heads); else the tiles of one head in turn.
template <int D, int NT, bool HEADS>
__global__ void __launch_bounds__(kScoreWarps * 32) block_score_kernel(const SelectParams p, int tiles_per_warp) {
  __shared__ ScoreShared<D, NT> sh[HEADS ? kScoreWarps : 1];
  const int warp = threadIdx.x >> 5, b = blockIdx.z;
  const int g = HEADS ? blockIdx.y * kScoreWarps + warp : blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ncols = select_cols(p, b, blockIdx.x == 0 && g == 0 && threadIdx.x == 0);
  const int first = blockIdx.x * (HEADS ? 1 : kScoreWarps) * tiles_per_warp;
  if (first * 16 >= ncols || g >= p.num_kv_heads) return;  // (the whole CTA, or a warp that works alone)
  float* out = p.scores + ((size_t)b * p.num_kv_heads + g) * p.max_cols;
  auto sink = [&](int col, float score) { out[col] = score; };
  if constexpr (HEADS)
    score_tiles<D, NT, true>(p, b, g, ncols, first, 1, tiles_per_warp, sh[warp], sink);
  else
    score_tiles<D, NT, false>(p, b, g, ncols, first + warp, kScoreWarps, tiles_per_warp, sh[0], sink);
}

// One CTA per (kv head, sequence).  IN_SMEM: the keys are kept in shared memory, else turned in place in the scores.
template <bool IN_SMEM>
__global__ void __launch_bounds__(1024) block_pick_kernel(const SelectParams p) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ TopkShared sh;
  const int g = blockIdx.x, b = blockIdx.y;
  const int n = select_cols(p, b, false);
  int32_t* out = p.blocks + ((size_t)b * p.num_kv_heads + g) * p.count;
  const int k = min(n, p.count);
  for (int i = k + threadIdx.x; i < p.count; i += blockDim.x) out[i] = -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n <= p.count) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = i;
    return;
  }
  float* scores = p.scores + ((size_t)b * p.num_kv_heads + g) * p.max_cols;
  uint32_t* keys = IN_SMEM ? smem_keys : reinterpret_cast<uint32_t*>(scores);
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    keys[i] = i < p.sinks || i >= n - p.recent ? kKeyAlways : order_key(scores[i]);
  __syncthreads();
  topk_in_order(keys, n, k, sh, [&](int at, int i) { out[at] = i; });
}

constexpr int kPickSmemCols = 50000;  // keys that fit in shared memory

template <int D, int NT>
cudaError_t score(const SelectParams& p, int num_sms, cudaStream_t st) {
  if (in_clusters(p.num_seqs, p.num_kv_heads, p.max_context_len, num_sms)) {  // scored and selected
    // CTAs of a cluster: no more than there are tiles for, nor than one wave of four CTAs an SM holds
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads, tiles = (p.max_cols + 15) / 16;
    int ctas = kClusterCtas;
    while (ctas > 1 && (units * ctas > 4 * (int64_t)num_sms || (ctas / 2) * kScoreWarps >= tiles)) ctas /= 2;
    const void* fn = reinterpret_cast<const void*>(block_select_kernel<D, NT>);
    SelectParams pp = p;
    void* args[] = {&pp};
    return launch_clusters(fn, dim3(ctas, p.num_kv_heads, p.num_seqs), dim3(kScoreWarps * 32), p.max_cols * 4, ctas, st, args);
  }
  // a tile a warp until there are several waves of warps; then up to sixteen, so that a warp's loads run ahead (64 contexts
  // of 8000 to 32768 tokens, 8 heads, with selection and attention: 2 tiles 147 us, 4 143, 8 141, 16 139, 32 155)
  const int64_t tiles = p.max_cols > 0 ? (p.max_cols + 15) / 16 : 1, units = (int64_t)p.num_seqs * p.num_kv_heads;
  int64_t per = tiles * units / ((int64_t)num_sms * 32);
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  constexpr bool kHeads = NT <= 2;  // (the rows of four heads fit in shared memory)
  const bool heads = kHeads && p.num_kv_heads >= kScoreWarps;
  const int64_t cover = per * (heads ? 1 : kScoreWarps);
  const dim3 grid((unsigned)((tiles + cover - 1) / cover),
                  heads ? (p.num_kv_heads + kScoreWarps - 1) / kScoreWarps : p.num_kv_heads, p.num_seqs);
  if (heads)
    block_score_kernel<D, NT, kHeads><<<grid, kScoreWarps * 32, 0, st>>>(p, (int)per);
  else
    block_score_kernel<D, NT, false><<<grid, kScoreWarps * 32, 0, st>>>(p, (int)per);
  return cudaGetLastError();
}

template <int D>
cudaError_t score_rows(const SelectParams& p, int num_sms, cudaStream_t st) {
  switch ((p.q_len * (p.num_q_heads / p.num_kv_heads) + 7) / 8) {
    case 1: return score<D, 1>(p, num_sms, st);
    case 2: return score<D, 2>(p, num_sms, st);
    case 3: return score<D, 3>(p, num_sms, st);
    case 4: return score<D, 4>(p, num_sms, st);
    default: return cudaErrorInvalidConfiguration;
  }
}

}  // namespace

size_t select_scratch_bytes(int num_seqs, int num_kv_heads, int max_context_len, int num_sms) {
  const size_t cols = ((size_t)max_context_len + 15) / 16;
  return in_clusters(num_seqs, num_kv_heads, max_context_len, num_sms) ? 0
                                                                       : (size_t)num_seqs * num_kv_heads * cols * sizeof(float);
}

cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, int num_sms, cudaStream_t st) {
  const cudaError_t e = head_dim == 128 ? score_rows<128>(p, num_sms, st)
                        : head_dim == 64 ? score_rows<64>(p, num_sms, st)
                                         : cudaErrorInvalidConfiguration;
  if (e != cudaSuccess || in_clusters(p.num_seqs, p.num_kv_heads, p.max_context_len, num_sms)) return e;
  const bool in_smem = p.max_cols <= kPickSmemCols;
  const void* fn = in_smem ? reinterpret_cast<const void*>(block_pick_kernel<true>)
                           : reinterpret_cast<const void*>(block_pick_kernel<false>);
  const int smem = in_smem ? p.max_cols * 4 : 0;
  if (in_smem) {
    const cudaError_t e2 = set_smem_once(fn, kPickSmemCols * 4);
    if (e2 != cudaSuccess) return e2;
  }
  SelectParams pp = p;
  void* args[] = {&pp};
  const int threads = p.max_cols <= 4096 ? 256 : 1024;  // (512 lists of up to 2048: 512 threads cost 4 us more)
  return launch_dependent(fn, dim3(p.num_kv_heads, p.num_seqs), dim3(threads), smem, st, args);
}

}  // namespace pa
