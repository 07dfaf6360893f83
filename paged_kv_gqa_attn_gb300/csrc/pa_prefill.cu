// Prefill and split verify: the planner's work list, the dense (no window) bf16 and E4M3 forms of the
// tile kernel, and the choice between the forms.
#include "pa_prefill.cuh"

namespace pa {
namespace {

// Work order: the (sequence, tile) pairs sorted by their number of 64-token steps, largest first
// (longest-processing-time order: the block scheduler hands out CTAs in blockIdx order, so the
// heaviest tiles start first and the light ones fill the tail).  One CTA: per-sequence checks,
// a histogram of step counts, its exclusive scan from the top, a scatter.  tiles[0] = number of
// pairs, tiles[1 + k] = work_item(b, tile).
// Up to 32 threads share a sequence's tiles where there are few sequences (4 chunks of 2048: 6.3 -> 4.5 us;
// one thread walked 64 tiles), and the window's step count is a variant of its own (as a branch it cost the
// dense call 2 us of 6.7).
constexpr int kCostBuckets = 8192;

template <bool WIN>
__global__ void __launch_bounds__(1024) prefill_plan_kernel(const AttnParams p, int tiles_per_row, int32_t* tiles) {
  __shared__ int hist[kCostBuckets];
  __shared__ int warp_tot[32];
  __shared__ int total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kCostBuckets; i += 1024) hist[i] = 0;
  if (tid == 0) total = 0;
  __syncthreads();
  const int Tt = tiles_per_row;
  int share = 1;  // threads that share a sequence's tiles
  while (share < 32 && p.num_seqs <= 512 / share) share *= 2;
  auto seq_info = [&](int b, int& QL, int& first_new) {
    const int qs = p.query_start_loc[b], qe = p.query_start_loc[b + 1];
    if (qs < 0 || qe < qs || qe > p.total_q || qe - qs > p.q_len) {  // (in this order no difference wraps)
      record_error(p.err, kErrBadInput);  // rows outside the packed q: the sequence is skipped
      QL = 0;
    } else {
      QL = qe - qs;
    }
    int L = p.context_lens[b];
    if (L > p.max_context_len) {
      record_error(p.err, kErrShortContext);
      L = p.max_context_len;
    }
    first_new = max(L, 0) - QL;
  };
  auto cost = [&](int QL, int first_new, int t) {
    const int n_max = first_new + min((t + 1) * Tt, QL);
    int steps = n_max > 0 ? (n_max + 63) / 64 : 0;
    if (WIN && n_max > 0)
      steps = (page_span((n_max + 15) / 16, max(0, first_new + t * Tt + 1 - p.window), p.sinks, 4).count + 3) / 4;
    return kCostBuckets - 1 - min(steps, kCostBuckets - 1);  // order index: costliest first
  };
  for (int b = tid / share; b < p.num_seqs; b += 1024 / share) {
    int QL, first_new;
    seq_info(b, QL, first_new);
    const int nt = (QL + Tt - 1) / Tt;
    for (int t = tid % share; t < nt; t += share) atomicAdd(&hist[cost(QL, first_new, t)], 1);
  }
  __syncthreads();
  // exclusive scan of the histogram (8 buckets per thread)
  int loc[kCostBuckets / 1024];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kCostBuckets / 1024; ++i) {
    loc[i] = hist[tid * (kCostBuckets / 1024) + i];
    sum += loc[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += v;
    }
    warp_tot[lane] = w;  // inclusive over warps
  }
  __syncthreads();
  int run = inc - sum + (warp > 0 ? warp_tot[warp - 1] : 0);
#pragma unroll
  for (int i = 0; i < kCostBuckets / 1024; ++i) {
    hist[tid * (kCostBuckets / 1024) + i] = run;
    run += loc[i];
  }
  if (tid == 1023) total = run;
  __syncthreads();
  for (int b = tid / share; b < p.num_seqs; b += 1024 / share) {
    int QL, first_new;
    seq_info(b, QL, first_new);
    const int nt = (QL + Tt - 1) / Tt;
    for (int t = tid % share; t < nt; t += share) {
      const int pos = atomicAdd(&hist[cost(QL, first_new, t)], 1);
      tiles[1 + pos] = work_item(b, t);
    }
  }
  if (tid == 0) tiles[0] = total;
  // the attention kernel (a programmatic dependent) waits for this grid before reading the list
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace

cudaError_t launch_prefill_plan(const AttnParams& p, int tiles_per_row, int32_t* tiles, cudaStream_t st) {
  if (p.window > 0)
    prefill_plan_kernel<true><<<1, 1024, 0, st>>>(p, tiles_per_row, tiles);
  else
    prefill_plan_kernel<false><<<1, 1024, 0, st>>>(p, tiles_per_row, tiles);
  return cudaGetLastError();
}

namespace {

cudaError_t dense_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles, const CUtensorMap& tk,
                       const CUtensorMap& tv) {
  if (l.head_dim == 128)
    return l.kv == kKvE4m3 ? prefill_form<128, kKvE4m3, kFormAll>(p, l, max_q_len, tiles, tk, tv)
                           : prefill_form<128, kKvBf16, kFormAll>(p, l, max_q_len, tiles, tk, tv);
  if (l.head_dim == 64)
    return l.kv == kKvE4m3 ? prefill_form<64, kKvE4m3, kFormAll>(p, l, max_q_len, tiles, tk, tv)
                           : prefill_form<64, kKvBf16, kFormAll>(p, l, max_q_len, tiles, tk, tv);
  return cudaErrorInvalidConfiguration;
}

cudaError_t any_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles, const CUtensorMap& tk,
                     const CUtensorMap& tv) {
  if (l.form == kFormOwn) return tiles_own_form(p, l, tk, tv);
  if (l.kv == kKvFp4) return prefill_fp4_form(p, l, max_q_len, tiles);
  if (p.window > 0) return prefill_window_form(p, l, max_q_len, tiles, tk, tv);
  return dense_form(p, l, max_q_len, tiles, tk, tv);
}

}  // namespace

size_t prefill_scratch_bytes(int num_seqs, int max_q_len, int group) {
  const int tt = PfTraits<128>::kRows / group;
  return (1 + (size_t)num_seqs * ((max_q_len + tt - 1) / tt)) * sizeof(int32_t);
}

cudaError_t launch_verify_split(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  if (l.group * p.q_len > PfTraits<128>::kRows || p.pages_per_partition % PfTraits<128>::kTP != 0)
    return cudaErrorInvalidConfiguration;
  return any_form(p, l, 0, nullptr, tk, tv);
}

cudaError_t launch_prefill_tc(const AttnParams& p, const Launch& l, int max_q_len, void* scratch, const CUtensorMap& tk,
                              const CUtensorMap& tv) {
  if (l.group < 1 || PfTraits<128>::kRows % l.group != 0) return cudaErrorInvalidConfiguration;
  return any_form(p, l, max_q_len, static_cast<int32_t*>(scratch), tk, tv);
}

#ifdef PA_TIMELINE
}  // namespace pa
// Instrumented build only: copy the per-CTA slots ([CTA][12] u64) to host, then zero them, so
// that CTAs of the next launch that return before their first stamp read as all-zero.
extern "C" int paged_attn_timeline_read_prefill(unsigned long long* host, int max_ctas) {
  const int n = max_ctas < pa::kPfTlCtas ? max_ctas : pa::kPfTlCtas;
  const size_t bytes = (size_t)n * pa::kPfTlSlots * sizeof(unsigned long long);
  if (cudaMemcpyFromSymbol(host, pa::g_prefill_timeline, bytes) != cudaSuccess) return 3;
  void* dev = nullptr;
  if (cudaGetSymbolAddress(&dev, pa::g_prefill_timeline) != cudaSuccess) return 3;
  if (cudaMemset(dev, 0, sizeof(unsigned long long) * pa::kPfTlCtas * pa::kPfTlSlots) != cudaSuccess) return 3;
  return cudaDeviceSynchronize() == cudaSuccess ? 0 : 3;
}
namespace pa {
#endif

}  // namespace pa
