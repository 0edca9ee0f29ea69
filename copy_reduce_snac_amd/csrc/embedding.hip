// embedding.hip -- rows of a vocabulary shard and the shard's gradient
// (snac_embedding, snac_embedding_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kEmbWaves = kEmbThreads / 64;
template <typename T, int U>
constexpr uint32_t kEmbElems = 64u * U * kUnit<T>;

// One wave a piece (U units a lane) of one token's row.  32768 rows of 4 KiB:
// 31 us (38 with stores that stay in the caches).
template <typename T, int U>
__global__ __launch_bounds__(kEmbThreads) void embedding_kernel(const EmbeddingArgs a, uint32_t pieces, uint64_t items) {
  constexpr uint32_t N = kUnit<T>;
  for (uint64_t it = (uint64_t)blockIdx.x * kEmbWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kEmbWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kEmbElems<T, U>;
    const uint64_t off = (uint64_t)first * T::kSize;
    // the difference wraps for far ids; as unsigned it is then no row either
    const uint64_t row = uniform64((uint64_t)load_id(a.ids, a.id_bytes, t) - (uint64_t)a.first);
    u32x4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = u32x4{0, 0, 0, 0};
    if (row < a.vocab) {
      ld_piece<T, U, false>(a.table + row * a.ld_table + off, a.width - first, v);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[N];
        unpack<T>(v[j], f);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) f[c] = f[c] * a.scale;
        v[j] = pack<T>(f);
      }
    }
    st_piece<T, U, true>(a.out + t * a.ld_out + off, a.width - first, v);
  }
}

// ------------------------------------------------------------- gradient
//
// The sorted positions are cut into chunks of C (embed_chunk).  One wave takes
// a chunk's slab of columns (a unit a lane), adds the rows of equal tokens in
// order and writes a run that lies inside the chunk; the sums of the runs
// that cross its ends go to partial[chunk][0] (begun before it) and [1]
// (begun in it), and embedding_join_kernel adds those up in order.  So a
// token that makes up half the text is spread over as many waves as a
// hundred rare ones, no atomics are needed, and the order of every sum is
// fixed by the ids alone.  However long a run, its sum is off by one rounding
// of each chunk's sum and one of the whole.  The work is bound by HBM (dout once, dtable once),
// and the sort before it and the joining after it by latency, so the zeros of
// the rows without a token are written beside all of them: workgroups past a
// launch's own write zeros to a part of the table, before the keys are sorted
// to all of its rows, after that to those that no key names.
//
// 32768 tokens (10500 different ones) of 2048 bf16 into 65536 x 2048 f32, 671
// MB, take 134 us (5.0 TB/s).  A chunk's rows are all in flight before the
// first sum is written, since a load issued after a store waits for it: 32
// rows at a time 164 us, 16: 173, 8: 178, 4: 182 (before the zeros moved
// beside the other launches).  Zeros stream (150 us for 159); the sums do not,
// whose lanes write 16 of every 32 bytes at a time (177 us for 150).

// A lane's sums within a chunk.  Rows of binary32 are added in binary64: 32 of
// them in binary32 are off by up to 31 half steps.  Rows of bf16 in binary32,
// which holds a sum of 32 of them exactly unless some are 2^11 times smaller
// than others; twice the registers would take a wave of three off each SIMD.
template <typename T>
using Sum = std::conditional_t<T::kSize == 4, double, float>;

// A sum scaled, and (ACC) added to `old`, with one rounding to binary32.
template <bool ACC>
__device__ __forceinline__ float scaled(float sum, float scale, float old) {
  return ACC ? __builtin_fmaf(sum, scale, old) : sum * scale;
}
template <bool ACC>
__device__ __forceinline__ float scaled(double sum, float scale, float old) {
  return (float)(ACC ? __builtin_fma(sum, (double)scale, (double)old) : sum * (double)scale);
}

// kUnit<T> sums of one lane -> columns first .. first + n of row `key`.
template <typename T, typename TG, bool ACC>
__device__ __forceinline__ void put_unit(const EmbedGradArgs& a, uint32_t key, uint32_t first, uint32_t n,
                                         const Sum<T> (&acc)[kUnit<T>]) {
  constexpr uint32_t N = kUnit<T>, NG = kUnit<TG>;
  char* p = a.dtable + (uint64_t)key * a.ld_dtable + (uint64_t)first * TG::kSize;
  // pieces of whole units of the gradient's type, or of half a unit (f32
  // rows of dout, bf16 gradient)
#pragma unroll
  for (uint32_t c0 = 0; c0 < N; c0 += N < NG ? N : NG) {
    constexpr uint32_t M = N < NG ? N : NG;
    if (c0 >= n) return;
    char* q = p + c0 * TG::kSize;
    const uint32_t m = n - c0 < M ? n - c0 : M;
    if (M == NG && m == M) {
      float f[NG], old[NG] = {};
      if constexpr (ACC) unpack<TG>(ld_unit<false>(q), old);
#pragma unroll
      for (uint32_t c = 0; c < NG; ++c) f[c] = c < M ? scaled<ACC>(acc[c0 + (c < M ? c : 0)], a.scale, old[c]) : 0.0f;
      st_unit<false>(q, pack<TG>(f));
    } else {
#pragma unroll
      for (uint32_t c = 0; c < M; ++c) {
        if (c < m) {
          char* to = q + c * TG::kSize;
          store_elem<TG>(to, scaled<ACC>(acc[c0 + c], a.scale, ACC ? load_elem<TG>(to) : 0.0f));
        }
      }
    }
  }
}

// Zeros for the rows that no token names, kZeroBytes of them a workgroup where
// they are that long: `per` rows, or `cols` columns of one.  It finds its
// rows' part of the sorted keys and marks those that it meets.  Small groups
// keep what is written at a time close together; the search, of kProbes keys
// a step, must not read more lines than they write.  us, 16384 tokens into
// 131072 x 4096 f32: with 32 keys a step, groups of 12 / 16 / 32 KiB 628 / 369 /
// 426, of 16 rows 418; with groups of 16 KiB, 8 / 16 / 32 / 48 / 256 keys a step
// 418 / 392 / 369 / 367 / 447.
constexpr uint32_t kZeroRows = 16;  // at most
constexpr uint32_t kZeroBytes = 16384;
constexpr uint32_t kProbes = 48;
constexpr uint64_t kJoinZeroBytes = 32ull << 20;  // of zeros beside the joining
struct ZeroShape {
  uint32_t per, cols, slabs;  // slabs: of cols columns in a row
  __host__ __device__ uint64_t groups(uint64_t rows) const { return (rows + per - 1) / per * slabs; }
};

template <typename TG>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, uint32_t wg, uint32_t from, uint32_t to, const ZeroShape z,
                                          uint32_t* met, uint32_t* start) {
  uint32_t set = wg, col = 0;
  if (z.slabs > 1) set = wg / z.slabs, col = (wg - set * z.slabs) * z.cols;
  const uint32_t lo = from + set * z.per, rows = to - lo < z.per ? to - lo : z.per;
  const uint32_t cols = a.width - col < z.cols ? a.width - col : z.cols;
  if (threadIdx.x < kZeroRows) met[threadIdx.x] = 0;
  if (wave_id() == 0) {
    // the first position whose key is not below lo, kProbes at a time
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t b = 0, e = a.n;
    while (b < e) {
      const uint32_t step = (e - b + kProbes - 1) / kProbes;
      const uint32_t at = b + lane * step;  // a probe past the end answers no
      const bool probe = lane < kProbes && at < e;
      const uint32_t below = (uint32_t)__popcll(__ballot(probe && a.keys[probe ? at : b] < lo));
      // probes 0 .. below - 1 are below: the answer lies after the last of them
      if (below == 0) {
        e = b;
      } else {
        e = below < kProbes && b + below * step < e ? b + below * step : e;
        b += (below - 1) * step + 1;
      }
    }
    if (lane == 0) *start = b;
  }
  __syncthreads();
  for (uint32_t i = *start + threadIdx.x; i < a.n; i += kEmbThreads) {
    const uint32_t r = a.keys[i] - lo;
    if (r >= rows) break;
    met[r] = 1;
  }
  __syncthreads();
  put_zeros<TG>(a.dtable + (uint64_t)lo * a.ld_dtable + (uint64_t)col * TG::kSize, a.ld_dtable, cols, rows,
                [&](uint32_t r) { return met[r] != 0; });
}

// One chunk's slab of 64 units of columns from `col0` on, by one wave.  WHOLE:
// all of them exist; the form without their checks is a third of the code,
// which the unrolled loop repeats for each row.
template <typename T, typename TG, bool ACC, bool WHOLE, uint32_t C>
__device__ __forceinline__ void add_chunk(const EmbedGradArgs& a, uint32_t chunk, uint32_t col0) {
  constexpr uint32_t N = kUnit<T>;
  static_assert(C + 2 <= 64, "a lane for each key of a chunk and its neighbours");
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wide = (a.width + 7u) & ~7u;
  const uint32_t first = col0 + lane * N;
  const uint32_t left = first < a.width ? a.width - first : 0;
  const uint32_t n = WHOLE ? N : left < N ? left : N;
  constexpr int kLoads = WHOLE || C < 8 ? C : 8;  // rows of dout in flight
  const uint32_t lo = chunk * C, hi = a.n - lo < C ? a.n : lo + C;
  // lane i: the key and token of position lo + i; lane 62: the key before the
  // chunk, lane 63: the key after it (`vocab`, no gradient, where there is none)
  uint32_t my_key = a.vocab, my_token = 0;
  if (lane < hi - lo) my_key = a.keys[lo + lane], my_token = (uint32_t)a.tokens[lo + lane];
  if (lane == 62 && lo > 0) my_key = a.keys[lo - 1];
  if (lane == 63 && hi < a.n) my_key = a.keys[hi];
  // the positions that have a gradient come first
  const uint32_t count = (uint32_t)__popcll(__ballot(lane < hi - lo && my_key < a.vocab));
  if (count == 0) return;
  auto key_of = [&](uint32_t i) { return (uint32_t)__builtin_amdgcn_readlane((int)my_key, (int)i); };
  uint32_t cur = key_of(0);
  bool head = key_of(62) == cur && lo > 0;
  Sum<T> acc[N];
#pragma unroll
  for (uint32_t c = 0; c < N; ++c) acc[c] = 0;
  auto flush = [&](bool tail) {
    if (head || tail) {
      float* p = a.partial + ((uint64_t)chunk * 2 + (head ? 0 : 1)) * wide + first;
      // rows of `wide` floats: a lane's columns up to the next multiple of 8
      if (n) {
#pragma unroll
        for (uint32_t c = 0; c < N; c += 4)
          st_unit<false>(reinterpret_cast<char*>(p + c),
                         u32x4{__float_as_uint((float)acc[c]), __float_as_uint((float)acc[c + 1]),
                               __float_as_uint((float)acc[c + 2]), __float_as_uint((float)acc[c + 3])});
      }
    } else {
      put_unit<T, TG, ACC>(a, cur, first, n, acc);
    }
  };
  const char* col = a.dout + (uint64_t)first * T::kSize;
  for (uint32_t i0 = 0; i0 < count; i0 += kLoads) {
    u32x4 v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t i = i0 + j < count ? i0 + j : count - 1;  // past the end: the last row again, not used
      const char* p = col + (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)my_token, (int)i) * a.ld_dout;
      if constexpr (WHOLE) {
        v[j] = ld_unit<true>(p);
      } else {
        v[j] = u32x4{0, 0, 0, 0};
        if (n == N) v[j] = ld_unit<true>(p);
        else if (n) v[j] = ld_part<T>(p, n);
      }
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if (i0 + j < count) {
        const uint32_t key = key_of(i0 + j);
        if (key != cur) {
          flush(false);
          head = false;
          cur = key;
#pragma unroll
          for (uint32_t c = 0; c < N; ++c) acc[c] = 0;
        }
        float f[N];
        unpack<T>(v[j], f);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) acc[c] += f[c];
      }
    }
  }
  flush(key_of(63) == cur);
}

// The first `adds` workgroups add, the rest write zeros as those finish.  Three
// waves a SIMD, but where the registers for that do not suffice.
template <typename T, typename TG, bool ACC>
constexpr int kGradWaves = ACC && T::kSize > TG::kSize ? 2 : 3;

template <typename T, typename TG, bool ACC, uint32_t C>
__global__ __launch_bounds__(kEmbThreads, (kGradWaves<T, TG, ACC>)) void embedding_grad_kernel(
    const EmbedGradArgs a, uint32_t slabs, uint64_t items, uint32_t adds, uint32_t zero_to, const ZeroShape z) {
  __shared__ uint32_t met[kZeroRows];
  __shared__ uint32_t start;
  if (!ACC && blockIdx.x >= adds) {
    zero_rows<TG>(a, blockIdx.x - adds, a.zero_from, zero_to, z, met, &start);
    return;
  }
  const uint64_t it = (uint64_t)blockIdx.x * kEmbWaves + wave_id();
  if (it >= items) return;
  const uint32_t chunk = (uint32_t)(it / slabs), slab = (uint32_t)(it % slabs);
  constexpr uint32_t S = 64u * kUnit<T>;
  uint32_t col0 = slab * S;
  // a row's last slab reaches back to be whole: the wave before it writes the
  // same sums to the columns they share (which must not be when they are
  // added to what is there)
  if (!ACC && a.width >= S && col0 + S > a.width) col0 = a.width - S;
  if (col0 + S <= a.width) add_chunk<T, TG, ACC, true, C>(a, chunk, col0);
  else add_chunk<T, TG, ACC, false, C>(a, chunk, col0);
}

// The runs that cross chunks: the chunk that a run begins in adds up its
// partial sums, a lane for each 4 columns, kJoinLoads rows of them in flight.
// They are binary32 (as binary64 they would need twice the scratch), off by
// half a step of each, but added in binary64: a run may have 2^19 of them, whose
// sum in binary32 lost 1e-3 of itself.  65536 tokens into 1000 x 1024: 69 us
// in all, 67 with a binary32 sum.
constexpr int kJoinLoads = 16;

template <typename TG, bool ACC, uint32_t C>
__global__ __launch_bounds__(kEmbThreads) void embedding_join_kernel(const EmbedGradArgs a, uint32_t slabs, uint32_t joins,
                                                                     uint32_t zero_from, const ZeroShape z) {
  __shared__ uint32_t met[kZeroRows];
  __shared__ uint32_t start;
  if (!ACC && blockIdx.x >= joins) {
    zero_rows<TG>(a, blockIdx.x - joins, zero_from, a.vocab, z, met, &start);
    return;
  }
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wide = (a.width + 7u) & ~7u;
  const uint32_t chunk = blockIdx.x / slabs;
  const uint32_t lo = chunk * C, hi = lo + C;  // hi < a.n: not the last chunk
  const uint32_t key = a.keys[hi - 1], next = a.keys[hi], begin = a.keys[lo], prev = a.keys[lo ? lo - 1 : 0];
  // only where a run begins in this chunk and goes on after it
  if (key >= a.vocab || next != key || (begin == key && lo > 0 && prev == key)) return;
  // how many chunks after this one it reaches into
  uint32_t more = 0;
  while (true) {
    const uint64_t end = ((uint64_t)chunk + 2 + more + lane) * C;  // past the more + lane + 1st
    const uint64_t on = __ballot(end < a.n && a.keys[end < a.n ? end : 0] == key);
    more += on == ~0ull ? 64 : (uint32_t)__ffsll((unsigned long long)~on) - 1;
    if (on != ~0ull) break;
  }
  ++more;
  const uint32_t col = ((blockIdx.x % slabs) * kEmbThreads + threadIdx.x) * 4;
  if (col >= a.width) return;
  const float* p = a.partial + (uint64_t)chunk * 2 * wide + col;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  const f32x4 own = *reinterpret_cast<const f32x4*>(p + wide);
  double sum[4] = {own[0], own[1], own[2], own[3]};
  for (uint32_t m = 1; m <= more; m += kJoinLoads) {
    f32x4 v[kJoinLoads];
#pragma unroll
    for (int j = 0; j < kJoinLoads; ++j)
      v[j] = *reinterpret_cast<const f32x4*>(p + (uint64_t)(m + j <= more ? m + j : more) * 2 * wide);
#pragma unroll
    for (int j = 0; j < kJoinLoads; ++j)
      if (m + j <= more) {
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] += v[j][c];
      }
  }
  put_unit<F32, TG, ACC>(a, key, col, a.width - col < 4 ? a.width - col : 4, sum);
}

uint32_t emb_grid(uint64_t items) {
  const uint64_t want = (items + kEmbWaves - 1) / kEmbWaves;
  return (uint32_t)(want < (1u << 22) ? want : 1u << 22);
}

template <typename T, int U>
hipError_t embedding_in(const EmbeddingArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kEmbElems<T, U> - 1) / kEmbElems<T, U>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((embedding_kernel<T, U>), dim3(emb_grid(items)), dim3(kEmbThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

// Pieces of one unit where those of four would leave SIMDs without a wave.
template <typename T>
hipError_t embedding_any(const EmbeddingArgs& a, hipStream_t stream) {
  const int cus = device_cu_count();
  const uint64_t simds = (uint64_t)(cus > 0 ? cus : 1) * 4;
  const uint32_t pieces = (a.width + kEmbElems<T, 4> - 1) / kEmbElems<T, 4>;
  return a.tokens < simds && a.tokens * pieces < simds ? embedding_in<T, 1>(a, stream) : embedding_in<T, 4>(a, stream);
}

template <typename T, typename TG, bool ACC, uint32_t C>
hipError_t embedding_grad_in(const EmbedGradArgs& a, hipStream_t stream) {
  const uint32_t chunks = (a.n + C - 1) / C;
  uint32_t slabs = (a.width + 64u * kUnit<T> - 1) / (64u * kUnit<T>);
  const uint64_t items = (uint64_t)chunks * slabs;
  const uint64_t adds = (items + kEmbWaves - 1) / kEmbWaves;
  // zeros: what is left of them, kJoinZeroBytes beside the joining and the
  // rest here
  const uint32_t left = ACC ? 0 : a.vocab - a.zero_from;
  const uint64_t row_bytes = (uint64_t)a.width * TG::kSize, late = kJoinZeroBytes / row_bytes;
  const uint32_t join_zeros = chunks < 2 ? 0 : late < left ? (uint32_t)late : left;
  const uint32_t zero_to = a.vocab - join_zeros;
  constexpr uint32_t kCols = kZeroBytes / TG::kSize;
  const uint32_t fit = a.width > kCols / kZeroRows ? kCols / a.width : kZeroRows;
  const ZeroShape z{fit ? fit : 1, kCols, (a.width + kCols - 1) / kCols};
  uint32_t rows = left - join_zeros;
  // a launch has fewer than 2^32 threads; more rows than that take further ones
  constexpr uint64_t kMostGroups = (1ull << 32) / kEmbThreads - 1;
  if (adds > kMostGroups) return hipErrorInvalidValue;  // dout would be larger than the memory
  EmbedGradArgs c = a;
  for (uint64_t add = adds; add || rows; add = 0) {
    const uint64_t most = (kMostGroups - add) / z.slabs * z.per;  // rows
    const uint32_t now = rows < most ? rows : (uint32_t)most;
    hipLaunchKernelGGL((embedding_grad_kernel<T, TG, ACC, C>), dim3((uint32_t)(add + z.groups(now))), dim3(kEmbThreads), 0,
                       stream, c, slabs, items, (uint32_t)add, zero_to, z);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    c.zero_from += now;
    rows -= now;
  }
  if (chunks < 2) return hipSuccess;
  slabs = (a.width + 4 * kEmbThreads - 1) / (4 * kEmbThreads);
  const uint32_t joins = (chunks - 1) * slabs;
  hipLaunchKernelGGL((embedding_join_kernel<TG, ACC, C>), dim3(joins + (uint32_t)z.groups(join_zeros)),
                     dim3(kEmbThreads), 0, stream, a, slabs, joins, zero_to, z);
  return hipGetLastError();
}

// Chunks of 32 positions write the fewest partial sums; with few tokens their
// waves are few and long.  us, chunks of 8 / 32: 1000 tokens, 2000 x 777: 19 /
// 23; 32768 x 2048 with 2048 tokens 53 / 57, 4096: 57 / 59, 8192: 76 / 70.
template <typename T, typename TG, bool ACC>
hipError_t embedding_grad_any(const EmbedGradArgs& a, hipStream_t stream) {
  return embed_chunk(a.n) == 8 ? embedding_grad_in<T, TG, ACC, 8>(a, stream) : embedding_grad_in<T, TG, ACC, 32>(a, stream);
}

}  // namespace

hipError_t launch_embedding(const EmbeddingArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? embedding_any<BF16>(a, stream) : embedding_any<F32>(a, stream);
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, bool bf16, bool grad_bf16, hipStream_t stream) {
  auto go = [&](auto t, auto tg) {
    using T = decltype(t);
    using TG = decltype(tg);
    return a.accumulate ? embedding_grad_any<T, TG, true>(a, stream) : embedding_grad_any<T, TG, false>(a, stream);
  };
  if (bf16) return grad_bf16 ? go(BF16{}, BF16{}) : go(BF16{}, F32{});
  return grad_bf16 ? go(F32{}, BF16{}) : go(F32{}, F32{});
}

}  // namespace snac
