// sort.hip -- one stable counting-sort pass: the dispatch plan (one pass
// over the experts) and the radix passes that sort an embedding gradient's
// tokens.
//
// The items are cut into `blocks` runs.  With one run a single workgroup
// counts and places them; otherwise sort_hist_kernel counts every run's bins
// and sort_place_kernel places: item i goes to
//     (items of lower bins) + (items of its bin in earlier runs)
//       + (items of its bin before it in its run).
// Every workgroup works the first two out for itself from the counts of all
// runs (they stay in L2), which costs less than a launch of its own.  In a
// run each wave owns a contiguous part and its own 16-bit counters, and a
// lane's rank among equal bins of its wave comes from ballots over the bin's
// bits, so that the order needs no atomics and is the same every time.
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// key of item position i
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
  if (a.key_in) return a.key_in[i];
  const int64_t id = load_id(a.ids, a.id_bytes, i);
  // the difference wraps for far ids; as unsigned it is then no key either
  const uint64_t k = (uint64_t)id - (uint64_t)a.first;
  return k < a.vocab && id != a.pad ? (uint32_t)k : (uint32_t)a.vocab;
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(const SortArgs a) {
  __shared__ uint32_t count[kSortMaxBins];
  for (uint32_t b = threadIdx.x; b < a.bins; b += kSortThreads) count[b] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * a.chunk;
  const uint32_t hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  for (uint32_t i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&count[(sort_key(a, i) >> a.shift) & a.mask], 1u);
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < a.bins; b += kSortThreads) a.hist[(uint64_t)blockIdx.x * a.bins + b] = count[b];
}

// Lanes of the wave with the same bin (those with `on` only).
__device__ __forceinline__ uint64_t same_bin(uint32_t bin, bool on, uint32_t bits) {
  uint64_t m = __ballot(on);
  for (uint32_t b = 0; b < bits; ++b) {
    const bool set = (bin >> b) & 1u;
    const uint64_t v = __ballot(set);
    m &= set ? v : ~v;
  }
  return m;
}

template <bool PLAN>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const SortArgs a) {
  __shared__ uint16_t wave_count[kSortWaves][kSortMaxBins + 1];
  __shared__ uint32_t base[kSortMaxBins];
  __shared__ uint32_t scan[kSortWaves + 1];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = wave_id();
  const uint32_t bits = 32u - (uint32_t)__clz((int)(a.bins - 1) | 1);
  for (uint32_t i = tid; i < kSortWaves * (kSortMaxBins + 1); i += kSortThreads) (&wave_count[0][0])[i] = 0;
  __syncthreads();
  // this wave's part of the run
  const uint32_t lo = blockIdx.x * a.chunk;
  const uint32_t hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  const uint32_t per = ((hi - lo + kSortThreads - 1) / kSortThreads) * 64u;
  const uint32_t wlo = lo + wave * per < hi ? lo + wave * per : hi;
  const uint32_t whi = hi - wlo < per ? hi : wlo + per;
  uint16_t* mine = wave_count[wave];
  for (uint32_t i0 = wlo; i0 < whi; i0 += 64) {
    const bool on = i0 + lane < whi;
    const uint32_t bin = on ? (sort_key(a, i0 + lane) >> a.shift) & a.mask : 0;
    const uint64_t same = same_bin(bin, on, bits);
    if (on && (same >> lane) == 1) mine[bin] = (uint16_t)(mine[bin] + __popcll(same));
  }
  __syncthreads();
  // per bin: counts of the waves before each wave, the run's own total, and
  // the totals over all runs and over the earlier ones.  Thread i takes bins
  // 2 i and 2 i + 1 (kSortMaxBins < 2 kSortThreads).
  uint32_t total[2] = {0, 0}, early[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = 2 * tid + h;
    if (b < a.bins) {
      uint32_t run = 0;
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = wave_count[w][b];
        wave_count[w][b] = (uint16_t)run;
        run += c;
      }
      if (a.blocks == 1) {
        total[h] = run;
      } else {
        for (uint32_t k = 0; k < a.blocks; ++k) {
          const uint32_t c = a.hist[(uint64_t)k * a.bins + b];
          total[h] += c;
          early[h] += k < blockIdx.x ? c : 0;
        }
      }
    }
  }
  // exclusive sum of the totals over the bins
  uint32_t sum = total[0] + total[1];
  const uint32_t own = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(sum, d);
    if (lane >= (uint32_t)d) sum += o;
  }
  if (lane == 63) scan[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    uint32_t run = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = scan[w];
      scan[w] = run;
      run += c;
    }
  }
  __syncthreads();
  const uint32_t before = scan[wave] + sum - own;
  if (2 * tid < a.bins) base[2 * tid] = before + early[0];
  if (2 * tid + 1 < a.bins) base[2 * tid + 1] = before + total[0] + early[1];
  if (PLAN && blockIdx.x == 0) {
    if (2 * tid < a.vocab) a.counts[2 * tid] = (int32_t)total[0];
    if (2 * tid + 1 < a.vocab) a.counts[2 * tid + 1] = (int32_t)total[1];
  }
  __syncthreads();
  for (uint32_t i0 = wlo; i0 < whi; i0 += 64) {
    const uint32_t i = i0 + lane;
    const bool on = i < whi;
    const uint32_t key = on ? sort_key(a, i) : 0;
    const uint32_t bin = (key >> a.shift) & a.mask;
    const uint64_t same = same_bin(on ? bin : 0, on, bits);
    if (on) {
      const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
      const uint32_t seen = mine[bin];
      const uint32_t at = base[bin] + seen + rank;
      if ((same >> lane) == 1) mine[bin] = (uint16_t)(seen + rank + 1);
      if constexpr (PLAN) {
        const bool kept = bin < a.vocab;
        a.row_of_slot[i] = kept ? (int32_t)at : -1;
        a.slot_of_row[at] = kept ? (int32_t)i : -1;
      } else {
        a.key_out[at] = key;
        a.item_out[at] = a.item_in ? a.item_in[i] : (int32_t)i;
      }
    }
  }
}

}  // namespace

// One run up to 8192 items (one launch); else runs of at least 4096 items,
// at most 256 of them while a run's items fit the 16-bit counters.
void sort_shape(uint32_t n, uint32_t* blocks, uint32_t* chunk) {
  if (n <= 8192) {
    *blocks = 1;
    *chunk = n ? n : 1;
    return;
  }
  uint32_t c = 4096;
  while (c < 32768 && (n + c - 1) / c > 256) c *= 2;
  *chunk = c;
  *blocks = (n + c - 1) / c;
}

hipError_t launch_sort_pass(const SortArgs& a, bool plan, hipStream_t stream) {
  if (a.blocks > 1) {
    hipLaunchKernelGGL(sort_hist_kernel, dim3(a.blocks), dim3(kSortThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (plan) hipLaunchKernelGGL((sort_place_kernel<true>), dim3(a.blocks), dim3(kSortThreads), 0, stream, a);
  else hipLaunchKernelGGL((sort_place_kernel<false>), dim3(a.blocks), dim3(kSortThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace snac
