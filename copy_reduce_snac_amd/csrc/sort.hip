// sort.hip -- one stable counting-sort pass: the dispatch plan (one pass
// over the experts) and the radix passes that sort an embedding gradient's
// tokens.
//
// The items are cut into `blocks` runs.  With one run a single workgroup
// counts and places them (all passes of a radix sort in one launch); otherwise
// sort_hist_kernel counts every run's bins and sort_place_kernel places: item i
// goes to
//     (items of lower bins) + (items of its bin in earlier runs)
//       + (items of its bin before it in its run).
// Every workgroup works the first two out for itself from the counts of all
// runs (they stay in L2), which costs less than a launch of its own.  In a
// run each wave owns a contiguous part and its own 16-bit counters, and a
// lane's rank among equal bins of its wave comes from ballots over the bin's
// bits, so that the order needs no atomics and is the same every time.
// (Counting a radix pass's bins with integer atomics while the pass before it
// places took 19 us more than a launch of sort_hist_kernel, 4.8 us: frequent
// tokens make them meet.)
//
// The passes are bound by latency, launches and first loads: 131072 slots of
// 256 experts take 4.8 us (counting) and 8.3 us (placing) in 64 runs of 2048;
// placing took 21 us in 32 runs of 4096 by 1024 threads with the bins'
// ballots made twice.  The code is kept short (no source of keys but the
// pass's own is built in), since each launch fetches it anew.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kRunThreads = 512;    // several runs
constexpr int kAloneThreads = 1024;  // one run: the whole sort is one workgroup's

// Where a pass finds its keys: in an earlier pass's output (in memory, or of
// one run in LDS), or from ids of 4 or 8 bytes.
enum : int { kFromKeys = 0, kFromLds = 1, kFromIds4 = 4, kFromIds8 = 8 };

// key of item position i
template <int FROM>
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
  if constexpr (FROM == kFromKeys) {
    return a.key_in[i];
  } else {
    const int64_t id = load_id(a.ids, FROM, i);
    // the difference wraps for far ids; as unsigned it is then no key either
    const uint64_t k = (uint64_t)id - (uint64_t)a.first;
    return k < a.vocab && id != a.pad ? (uint32_t)k : (uint32_t)a.vocab;
  }
}

__device__ __forceinline__ uint32_t sort_bin(const SortArgs& a, uint32_t key) { return (key >> a.shift) & a.mask; }

template <int FROM>
__global__ __launch_bounds__(kRunThreads) void sort_hist_kernel(const SortArgs a) {
  __shared__ uint32_t count[kSortMaxBins];
  if (blockIdx.x >= a.blocks) {
    write_zeros(a.zero_hist, blockIdx.x - a.blocks);
    return;
  }
  for (uint32_t b = threadIdx.x; b < a.bins; b += kRunThreads) count[b] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * a.chunk;
  const uint32_t hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
#pragma unroll 4
  for (uint32_t i = lo + threadIdx.x; i < hi; i += kRunThreads) atomicAdd(&count[sort_bin(a, sort_key<FROM>(a, i))], 1u);
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < a.bins; b += kRunThreads) a.hist[b * a.hist_ld + blockIdx.x] = count[b];
}

// Lanes of the wave with the same bin (those with `on` only).
__device__ __forceinline__ uint64_t same_bin(uint32_t bin, bool on, uint32_t bits) {
  const uint64_t all = __ballot(on);
  uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
  for (uint32_t b = 0; b < bits; ++b) {
    const uint32_t set = (uint32_t)((int32_t)(bin << (31 - b)) >> 31);  // the bit in all places
    const uint64_t v = __ballot(set != 0);
    lo &= ~((uint32_t)v ^ set);
    hi &= ~((uint32_t)(v >> 32) ^ set);
  }
  return (uint64_t)hi << 32 | lo;
}

// Two of the 16-bit counters at a time.
typedef uint32_t __attribute__((may_alias)) two_counts;

// Place of this lane's item among the wave's items of its bin, counting it for
// the lanes of the next call.
__device__ __forceinline__ uint32_t place_in_wave(uint16_t* count, uint32_t bin, bool on, uint32_t bits, uint32_t lane) {
  const uint64_t same = same_bin(bin, on, bits);
  uint32_t place = 0;
  if (on) {
    place = count[bin] + (uint32_t)__popcll(same & ((1ull << lane) - 1));
    if ((same >> lane) == 1) count[bin] = (uint16_t)(place + 1);  // the last of them
  }
  wave_lds_order();
  return place;
}

constexpr uint32_t kSortBins = kSortMaxBins + 1;  // an even number
template <int TH>
struct SortLds {
  __align__(4) uint16_t wave_count[TH / 64][kSortBins];
  uint32_t base[kSortBins], early[kSortBins];
  uint32_t scan[TH / 64];
};
// and the keys and items between the passes over one run
struct AloneLds : SortLds<kAloneThreads> {
  uint32_t key[kSortAlone];
  uint16_t item[kSortAlone];
};

// One pass over this workgroup's run.  `stay`: its output is the next pass's
// in LDS, which takes the place of its input: every key and item has been
// read by then, since a run of kSortAlone has no more than R steps a wave.
template <bool PLAN, int TH, int FROM, typename Lds>
__device__ __forceinline__ void place_run(const SortArgs& a, Lds& lds, bool stay = false) {
  constexpr uint32_t W = TH / 64;
  constexpr uint32_t BINS = kSortBins;
  auto& wave_count = lds.wave_count;
  auto& base = lds.base;
  auto& early = lds.early;
  auto& scan = lds.scan;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = wave_id();
  const uint32_t bits = 32u - (uint32_t)__clz((int)(a.bins - 1) | 1);
  // this wave's part of the run
  const uint32_t lo = blockIdx.x * a.chunk;
  const uint32_t hi = a.n - lo < a.chunk ? a.n : lo + a.chunk;
  const uint32_t per = ((hi - lo + TH - 1) / TH) * 64u;
  const uint32_t wlo = lo + wave * per < hi ? lo + wave * per : hi;
  const uint32_t whi = hi - wlo < per ? hi : wlo + per;
  uint16_t* mine = wave_count[wave];
  for (uint32_t b = lane; b < BINS / 2; b += 64) reinterpret_cast<two_counts*>(mine)[b] = 0;
  wave_lds_order();
  // R keys a lane at a time; a wave's part is seldom more, and then they stay
  constexpr uint32_t R = TH == kAloneThreads ? 8 : 4;
  uint32_t key[R], place[R], item[R];
  auto load = [&](uint32_t i0) {
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
      const uint32_t i = i0 + r * 64 + lane;
      item[r] = i;
      if constexpr (FROM == kFromLds) {
        key[r] = i < whi ? lds.key[i] : 0;
        item[r] = i < whi ? lds.item[i] : 0;
      } else {
        key[r] = i < whi ? sort_key<FROM>(a, i) : 0;
      }
    }
  };
  for (uint32_t i0 = wlo; i0 < whi; i0 += 64 * R) {
    load(i0);
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
      if (i0 + r * 64 >= whi) break;
      const bool on = i0 + r * 64 + lane < whi;
      place[r] = place_in_wave(mine, on ? sort_bin(a, key[r]) : 0, on, bits, lane);
    }
  }
  // per bin: the totals over all runs and over the earlier ones
  if (a.blocks > 1) {
    for (uint32_t b = tid; b < a.bins; b += TH) {
      const u32x4* h = reinterpret_cast<const u32x4*>(a.hist + (uint64_t)b * a.hist_ld);
      uint32_t all = 0, bef = 0;
#pragma unroll 4
      for (uint32_t k = 0; k < a.blocks; k += 4) {
        const u32x4 c = h[k / 4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t v = k + i < a.blocks ? c[i] : 0;
          all += v;
          bef += k + i < blockIdx.x ? v : 0;
        }
      }
      base[b] = all;
      early[b] = bef;
    }
  }
  __syncthreads();
  // and the counts of the waves before each wave
  for (uint32_t b = tid; b < a.bins; b += TH) {
    uint32_t run = 0;
#pragma unroll
    for (uint32_t w = 0; w < W; ++w) {
      const uint32_t c = wave_count[w][b];
      wave_count[w][b] = (uint16_t)run;
      run += c;
    }
    if (a.blocks == 1) base[b] = run, early[b] = 0;
  }
  __syncthreads();
  // exclusive sum of the totals over the bins, `span` neighbours a thread
  const uint32_t span = (a.bins + TH - 1) / TH;
  uint32_t own = 0;
  for (uint32_t b = tid * span; b < (tid + 1) * span && b < a.bins; ++b) own += base[b];
  uint32_t sum = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(sum, d);
    if (lane >= (uint32_t)d) sum += o;
  }
  if (lane == 63) scan[wave] = sum;
  __syncthreads();
  uint32_t before = sum - own;
#pragma unroll
  for (uint32_t w = 0; w < W; ++w) before += w < wave ? scan[w] : 0;
  for (uint32_t b = tid * span; b < (tid + 1) * span && b < a.bins; ++b) {
    const uint32_t all = base[b];
    if (PLAN && blockIdx.x == 0 && b < a.vocab) a.counts[b] = (int32_t)all;
    base[b] = before + early[b];
    before += all;
  }
  __syncthreads();
  // the place in the wave is known from counting; with more than R steps it is
  // counted again, on from the waves before
  const bool once = whi - wlo <= 64 * R;
  for (uint32_t i0 = wlo; i0 < whi; i0 += 64 * R) {
    if (!once) load(i0);
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
      if (i0 + r * 64 >= whi) break;
      const uint32_t i = i0 + r * 64 + lane;
      const bool on = i < whi;
      const uint32_t bin = on ? sort_bin(a, key[r]) : 0;
      const uint32_t in = once ? mine[bin] + place[r] : place_in_wave(mine, bin, on, bits, lane);
      if (on) {
        const uint32_t at = base[bin] + in;
        if constexpr (PLAN) {
          const bool kept = bin < a.vocab;
          a.row_of_slot[i] = kept ? (int32_t)at : -1;
          a.slot_of_row[at] = kept ? (int32_t)i : -1;
        } else {
          if constexpr (std::is_same_v<Lds, AloneLds>) {
            if (stay) {
              lds.key[at] = key[r];
              lds.item[at] = (uint16_t)item[r];
              continue;
            }
          }
          a.key_out[at] = key[r];
          a.item_out[at] = FROM == kFromKeys ? a.item_in[i] : (int32_t)item[r];
        }
      }
    }
  }
}

template <bool PLAN, int TH, int FROM>
__global__ __launch_bounds__(TH) void sort_place_kernel(const SortArgs a) {
  __shared__ SortLds<TH> lds;
  if (!PLAN && blockIdx.x >= a.blocks) {
    write_zeros(a.zero_place, blockIdx.x - a.blocks);
    return;
  }
  place_run<PLAN, TH, FROM>(a, lds);
}

// All passes of a radix sort of one run, by one workgroup: `digit` bits a
// pass, keys and items in LDS in between (by way of memory the gradient of 4096
// tokens, 32768 x 4096 bf16, took 65 us instead of 59; 2929 tokens, 4117 x 2048
// 18.5 instead of 17.8).
template <int FROM>
__global__ __launch_bounds__(kAloneThreads) void sort_alone_kernel(const SortArgs a, uint32_t passes, uint32_t digit) {
  __shared__ AloneLds lds;
  if (blockIdx.x >= 1) {
    write_zeros(a.zero_place, blockIdx.x - 1);
    return;
  }
  SortArgs b = a;
  place_run<false, kAloneThreads, FROM>(b, lds, passes > 1);
  for (uint32_t i = 1; i < passes; ++i) {
    __syncthreads();  // what was placed is seen by all, and the counters are free
    b.shift = i * digit;
    place_run<false, kAloneThreads, kFromLds>(b, lds, i + 1 < passes);
  }
}

}  // namespace

// One run up to kSortAlone items (one launch); else runs of 2048 items or,
// past 256 of them, of as many more as keep to that, while a run's items fit
// the 16-bit counters.
void sort_shape(uint32_t n, uint32_t* blocks, uint32_t* chunk) {
  if (n <= kSortAlone) {
    *blocks = 1;
    *chunk = n ? n : 1;
    return;
  }
  uint32_t c = 2048;
  while (c < 32768 && (n + c - 1) / c > 256) c *= 2;
  *chunk = c;
  *blocks = (n + c - 1) / c;
}

uint64_t sort_hist_words(uint32_t blocks, uint32_t bins) {
  return blocks > 1 ? (uint64_t)bins * sort_hist_ld(blocks) : 0;
}

namespace {

uint32_t zero_groups(const ZeroRows& z) { return z.rows ? (z.rows + z.per - 1) / z.per : 0; }

template <bool PLAN, int FROM>
hipError_t sort_pass(const SortArgs& a, hipStream_t stream) {
  if constexpr (PLAN) {
    if (a.blocks == 1) {
      hipLaunchKernelGGL((sort_place_kernel<true, kAloneThreads, FROM>), dim3(1), dim3(kAloneThreads), 0, stream, a);
      return hipGetLastError();
    }
  }
  const dim3 place(a.blocks + zero_groups(a.zero_place));
  hipLaunchKernelGGL((sort_hist_kernel<FROM>), dim3(a.blocks + zero_groups(a.zero_hist)), dim3(kRunThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sort_place_kernel<PLAN, kRunThreads, FROM>), place, dim3(kRunThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_plan(const SortArgs& a, hipStream_t stream) {
  return a.id_bytes == 8 ? sort_pass<true, kFromIds8>(a, stream) : sort_pass<true, kFromIds4>(a, stream);
}

hipError_t launch_radix_pass(const SortArgs& a, hipStream_t stream) {
  if (a.key_in) return sort_pass<false, kFromKeys>(a, stream);
  return a.id_bytes == 8 ? sort_pass<false, kFromIds8>(a, stream) : sort_pass<false, kFromIds4>(a, stream);
}

hipError_t launch_radix_alone(const SortArgs& a, uint32_t passes, uint32_t digit, hipStream_t stream) {
  const dim3 grid(1 + zero_groups(a.zero_place)), block(kAloneThreads);
  if (a.id_bytes == 8) hipLaunchKernelGGL((sort_alone_kernel<kFromIds8>), grid, block, 0, stream, a, passes, digit);
  else hipLaunchKernelGGL((sort_alone_kernel<kFromIds4>), grid, block, 0, stream, a, passes, digit);
  return hipGetLastError();
}

}  // namespace snac
