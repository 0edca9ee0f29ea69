// embedding.hip -- rows of a vocabulary shard and the shard's gradient
// (snac_embedding, snac_embedding_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kEmbWaves = kEmbThreads / 64;
constexpr int kEmbUnits = 4;

template <typename T>
constexpr uint32_t kEmbElems = 64u * kEmbUnits * kUnit<T>;

// One wave a piece of one token's row.
template <typename T>
__global__ __launch_bounds__(kEmbThreads) void embedding_kernel(const EmbeddingArgs a, uint32_t pieces, uint64_t items) {
  constexpr uint32_t N = kUnit<T>;
  for (uint64_t it = (uint64_t)blockIdx.x * kEmbWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kEmbWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kEmbElems<T>;
    const uint64_t off = (uint64_t)first * T::kSize;
    // the difference wraps for far ids; as unsigned it is then no row either
    const uint64_t row = uniform64((uint64_t)load_id(a.ids, a.id_bytes, t) - (uint64_t)a.first);
    u32x4 v[kEmbUnits];
#pragma unroll
    for (int j = 0; j < kEmbUnits; ++j) v[j] = u32x4{0, 0, 0, 0};
    if (row < a.vocab) {
      ld_piece<T, kEmbUnits, false>(a.table + row * a.ld_table + off, a.width - first, v);
#pragma unroll
      for (int j = 0; j < kEmbUnits; ++j) {
        float f[N];
        unpack<T>(v[j], f);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) f[c] = f[c] * a.scale;
        v[j] = pack<T>(f);
      }
    }
    st_piece<T, kEmbUnits, false>(a.out + t * a.ld_out + off, a.width - first, v);
  }
}

// The gradient runs over the sorted positions in chunks of kEmbedChunk.  One
// wave takes a chunk's 64 units of columns, adds the rows of equal tokens in
// order and writes a run that lies inside the chunk; the sums of the runs
// that cross its ends go to partial[chunk][0] (begun before it) and [1]
// (begun in it), and embedding_join_kernel adds those up in order.
template <typename TG>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, uint32_t key, uint32_t first, uint32_t n,
                                        const float* acc) {
  // n elements (at most the lane's) at column `first` of row `key`
  char* p = a.dtable + (uint64_t)key * a.ld_dtable + (uint64_t)first * TG::kSize;
  for (uint32_t c = 0; c < n; ++c) {
    float v = acc[c] * a.scale;
    if (a.accumulate) v = load_elem<TG>(p + c * TG::kSize) + v;
    store_elem<TG>(p + c * TG::kSize, v);
  }
}

template <typename T, typename TG>
__global__ __launch_bounds__(kEmbThreads) void embedding_grad_kernel(const EmbedGradArgs a, uint32_t pieces,
                                                                     uint64_t items) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wide = (a.width + 7u) & ~7u;
  for (uint64_t it = (uint64_t)blockIdx.x * kEmbWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kEmbWaves) {
    const uint32_t chunk = (uint32_t)(it / pieces);
    const uint32_t first = ((uint32_t)(it - (uint64_t)chunk * pieces) * 64u + lane) * N;
    const uint32_t left = first < a.width ? a.width - first : 0;
    const uint32_t n = left < N ? left : N;
    const uint32_t lo = chunk * kEmbedChunk, hi = a.n - lo < kEmbedChunk ? a.n : lo + kEmbedChunk;
    uint32_t cur = a.keys[lo];
    bool head = lo > 0 && a.keys[lo - 1] == cur;
    float acc[N];
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) acc[c] = 0.0f;
    auto flush = [&](bool tail) {
      if (cur >= a.vocab || n == 0) return;
      if (head || tail) {
        float* p = a.partial + ((uint64_t)chunk * 2 + (head ? 0 : 1)) * wide + first;
        for (uint32_t c = 0; c < n; ++c) p[c] = acc[c];
      } else {
        put_row<TG>(a, cur, first, n, acc);
      }
    };
    for (uint32_t i = lo; i < hi; ++i) {
      const uint32_t key = a.keys[i];
      if (key != cur) {
        flush(false);
        head = false;
        cur = key;
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) acc[c] = 0.0f;
      }
      if (key >= a.vocab) break;  // the rest have no gradient
      const char* p = a.dout + (uint64_t)(uint32_t)a.tokens[i] * a.ld_dout + (uint64_t)first * T::kSize;
      u32x4 v = {0, 0, 0, 0};
      if (n == N) v = ld_unit<true>(p);
      else if (n) v = ld_part<T>(p, n);
      float f[N];
      unpack<T>(v, f);
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) acc[c] += f[c];
    }
    flush(hi < a.n && a.keys[hi] == cur);
  }
}

template <typename TG>
__global__ __launch_bounds__(kEmbThreads) void embedding_join_kernel(const EmbedGradArgs a, uint32_t pieces,
                                                                     uint64_t items) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t wide = (a.width + 7u) & ~7u;
  const uint64_t it = (uint64_t)blockIdx.x * kEmbWaves + wave_id();
  if (it >= items) return;
  uint32_t chunk = (uint32_t)(it / pieces);
  const uint32_t col = (uint32_t)(it - (uint64_t)chunk * pieces) * 64u + lane;
  const uint32_t lo = chunk * kEmbedChunk, hi = lo + kEmbedChunk;
  if (hi >= a.n) return;
  const uint32_t key = a.keys[hi - 1];
  // only where a run begins in this chunk and goes on after it
  if (key >= a.vocab || a.keys[hi] != key || (a.keys[lo] == key && lo > 0 && a.keys[lo - 1] == key)) return;
  if (col >= a.width) return;
  float acc = a.partial[((uint64_t)chunk * 2 + 1) * wide + col];
  while (true) {
    ++chunk;
    acc += a.partial[(uint64_t)chunk * 2 * wide + col];
    const uint64_t end = ((uint64_t)chunk + 1) * kEmbedChunk;
    if (end >= a.n || a.keys[end] != key) break;
  }
  put_row<TG>(a, key, col, 1, &acc);
}

// Zeros for the rows that no token names: a workgroup takes kZeroRows rows,
// finds their part of the sorted keys by bisection and marks those that it
// meets.
constexpr uint32_t kZeroRows = 64;

template <typename TG>
__global__ __launch_bounds__(kEmbThreads) void embedding_zero_kernel(const EmbedGradArgs a) {
  __shared__ uint32_t met[kZeroRows];
  __shared__ uint32_t ends[2];
  const uint32_t lo = blockIdx.x * kZeroRows;
  const uint32_t rows = a.vocab - lo < kZeroRows ? a.vocab - lo : kZeroRows;
  if (threadIdx.x < kZeroRows) met[threadIdx.x] = 0;
  if (threadIdx.x < 2) {
    const uint32_t key = lo + (threadIdx.x ? rows : 0);
    uint32_t b = 0, e = a.n;  // the first position whose key is not below `key`
    while (b < e) {
      const uint32_t m = b + (e - b) / 2;
      if (a.keys[m] < key) b = m + 1;
      else e = m;
    }
    ends[threadIdx.x] = b;
  }
  __syncthreads();
  for (uint32_t i = ends[0] + threadIdx.x; i < ends[1]; i += kEmbThreads) met[a.keys[i] - lo] = 1;
  __syncthreads();
  const u32x4 zero[1] = {u32x4{0, 0, 0, 0}};
  constexpr uint32_t step = 64u * kUnit<TG>;
  for (uint32_t r = wave_id(); r < rows; r += kEmbWaves) {
    if (met[r]) continue;
    char* row = a.dtable + (uint64_t)(lo + r) * a.ld_dtable;
    for (uint32_t e = 0; e < a.width; e += step) st_piece<TG, 1, true>(row + (uint64_t)e * TG::kSize, a.width - e, zero);
  }
}

uint32_t emb_grid(uint64_t items) {
  const int cus = device_cu_count();
  const uint64_t most = (uint64_t)(cus > 0 ? cus : 1) * 16;
  const uint64_t want = (items + kEmbWaves - 1) / kEmbWaves;
  return (uint32_t)(want < most ? want : most);
}

template <typename T>
hipError_t embedding_any(const EmbeddingArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kEmbElems<T> - 1) / kEmbElems<T>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((embedding_kernel<T>), dim3(emb_grid(items)), dim3(kEmbThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

template <typename T, typename TG>
hipError_t embedding_grad_any(const EmbedGradArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (!a.accumulate) {
    hipLaunchKernelGGL((embedding_zero_kernel<TG>), dim3((a.vocab + kZeroRows - 1) / kZeroRows), dim3(kEmbThreads), 0,
                       stream, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.n == 0) return e;
  const uint32_t chunks = (a.n + kEmbedChunk - 1) / kEmbedChunk;
  uint32_t pieces = (a.width + 64u * kUnit<T> - 1) / (64u * kUnit<T>);
  uint64_t items = (uint64_t)chunks * pieces;
  hipLaunchKernelGGL((embedding_grad_kernel<T, TG>), dim3(emb_grid(items)), dim3(kEmbThreads), 0, stream, a, pieces,
                     items);
  e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  pieces = (a.width + 63u) / 64u;
  items = (uint64_t)(chunks - 1) * pieces;
  hipLaunchKernelGGL((embedding_join_kernel<TG>), dim3((uint32_t)((items + kEmbWaves - 1) / kEmbWaves)),
                     dim3(kEmbThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding(const EmbeddingArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? embedding_any<BF16>(a, stream) : embedding_any<F32>(a, stream);
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, bool bf16, bool grad_bf16, hipStream_t stream) {
  if (bf16) return grad_bf16 ? embedding_grad_any<BF16, BF16>(a, stream) : embedding_grad_any<BF16, F32>(a, stream);
  return grad_bf16 ? embedding_grad_any<F32, BF16>(a, stream) : embedding_grad_any<F32, F32>(a, stream);
}

}  // namespace snac
