// grads.hip -- the global norm over a list of tensors and clipping by it
// (snac_grad_norm, snac_clip_grads in include/snac_ops.h).
//
// Both stream the list's tiles (at most kGradTileBytes of one tensor each)
// and are bound by HBM.  A tensor's tiles begin on 256-byte boundaries of its
// output but for the first, so that only a tensor's ends share lines (tiles
// on 16-byte boundaries took 669 us where these take 570: workgroups on two
// XCDs wrote halves of one line).
//
// Shapes, measured on 0.27 G bf16 and 0.27 G f32 elements in 300 tensors
// (1.61 GB):
//   norm  512 threads, one workgroup a CU, two tiles in flight: 242 us, 6.6
//         TB/s.  256 threads at 2, 3, 4 and 8 a CU, one tile: 295, 262, 297
//         and 336 us; 512 threads at 2 a CU, one tile: 250 us.  Squares in
//         binary32 a unit at a time would not be faster (266 against 267).
//   clip  512 threads, two workgroups a CU, after 8 grid-stride rounds tiles
//         in order from 4 counters: 506 us, 6.4 TB/s of reads and writes; all
//         grid-stride 590 us, 8 counters 527, one 1200.  Taking the tiles from
//         the last one back, to find some in the Infinity Cache, gained 1 us.
#include <hip/hip_runtime.h>

#include "internal.hpp"
#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kGradThreads = 512;
constexpr int kGradUnits = (int)(kGradTileBytes / 16 / kGradThreads);  // of a lane, in a full tile

// single elements of global memory (see ld_unit)
template <typename T>
__device__ __forceinline__ float ld_one(const char* p) {
  if constexpr (T::kSize == 4) return *(global_ptr<const float>)p;
  else return bf16_lo(*(global_ptr<const uint16_t>)p);
}
template <typename T>
__device__ __forceinline__ void st_one(char* p, float v) {
  if constexpr (T::kSize == 4) *(global_ptr<float>)p = v;
  else *(global_ptr<uint16_t>)p = to_bf16(v);
}

template <typename T>
__device__ __forceinline__ double unit_squares(const u32x4& w, double acc) {
  float f[kUnit<T>];
  unpack<T>(w, f);
#pragma unroll
  for (uint32_t c = 0; c < kUnit<T>; ++c) acc = __builtin_fma((double)f[c], (double)f[c], acc);
  return acc;
}

__device__ __forceinline__ bool full_tile(const GradTile& g) { return g.n == kGradTileBytes >> (2 - g.bf16); }

__device__ __forceinline__ void load_tile(const GradTile& g, u32x4 (&v)[kGradUnits]) {
#pragma unroll
  for (int j = 0; j < kGradUnits; ++j) v[j] = ld_unit<true>(g.src + threadIdx.x * 16u + j * kGradThreads * 16);
}

// Squares of a full tile, its units loaded before.
template <typename T>
__device__ __forceinline__ double full_squares(const u32x4 (&v)[kGradUnits], double acc) {
  double more = 0.0;
#pragma unroll
  for (int j = 0; j < kGradUnits; j += 2) {
    acc = unit_squares<T>(v[j], acc);
    more = unit_squares<T>(v[j + 1], more);
  }
  return acc + more;
}

// Squares of a shorter tile: units one by one, its last part of a unit by
// elements.
template <typename T>
__device__ __forceinline__ double part_squares(const GradTile& g, double acc) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t units = g.n / N;
  for (uint32_t u = threadIdx.x; u < units; u += kGradThreads) acc = unit_squares<T>(ld_unit<true>(g.src + u * 16u), acc);
  const uint32_t e = units * N + threadIdx.x;
  if (e < g.n) {
    const double x = ld_one<T>(g.src + e * T::kSize);
    acc = __builtin_fma(x, x, acc);
  }
  return acc;
}

// Sum over the workgroup in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double x, double* lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63u) == 0) lds[wave_id()] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kGradThreads / 64; ++w) s += lds[w];
  __syncthreads();
  return s;
}

// The norm of n partial sums, added up in a fixed order by the workgroup; in
// every thread.
template <typename Load>
__device__ __forceinline__ float norm_of(uint32_t n, double* lds, Load load) {
  double sum = 0.0;
  for (uint32_t b = threadIdx.x; b < n; b += kGradThreads) sum += load(b);
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) lds[0] = sum;
  __syncthreads();
  return (float)sqrt(lds[0]);
}

// Every workgroup leaves its sum in partial[].  JOIN: the last one to do so
// makes the norm of them and leaves the ticket at 0 for the next call; else
// clip_kernel does.
template <bool JOIN>
__global__ __launch_bounds__(kGradThreads) void norm_kernel(const GradTile* __restrict__ tiles, uint32_t ntiles, double* partial,
                                                            uint32_t* ticket, float* norm) {
  __shared__ double lds[kGradThreads / 64];
  __shared__ uint32_t last;
  double acc = 0.0;
  // two neighbouring tiles at a time
  const uint32_t pairs = (ntiles + 1) / 2;
  auto tile = [&](uint32_t t) { return t < ntiles ? tiles[t] : GradTile{nullptr, nullptr, 0, 0}; };
  GradTile next0 = tile(2 * blockIdx.x), next1 = tile(2 * blockIdx.x + 1);
  for (uint32_t p = blockIdx.x; p < pairs; p += gridDim.x) {
    const GradTile g0 = next0, g1 = next1;
    if (pairs - p > gridDim.x) next0 = tile(2 * (p + gridDim.x)), next1 = tile(2 * (p + gridDim.x) + 1);
    u32x4 v0[kGradUnits], v1[kGradUnits];
    const bool full0 = full_tile(g0), full1 = full_tile(g1);
    if (full0) load_tile(g0, v0);
    if (full1) load_tile(g1, v1);
    if (full0) acc = g0.bf16 ? full_squares<BF16>(v0, acc) : full_squares<F32>(v0, acc);
    else acc = g0.bf16 ? part_squares<BF16>(g0, acc) : part_squares<F32>(g0, acc);
    if (full1) acc = g1.bf16 ? full_squares<BF16>(v1, acc) : full_squares<F32>(v1, acc);
    else acc = g1.bf16 ? part_squares<BF16>(g1, acc) : part_squares<F32>(g1, acc);
  }
  const double s = block_sum(acc, lds);
  if constexpr (!JOIN) {
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
    return;
  }
  if (threadIdx.x == 0) {
    __hip_atomic_store(&partial[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  const float total = norm_of(gridDim.x, lds, [&](uint32_t b) {
    return __hip_atomic_load(&partial[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  });
  if (threadIdx.x == 0) {
    *norm = total;
    __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

__global__ void zero_norm_kernel(float* norm) { *norm = 0.0f; }

template <typename T>
__device__ __forceinline__ u32x4 unit_scale(const u32x4& w, float factor) {
  float f[kUnit<T>];
  unpack<T>(w, f);
#pragma unroll
  for (uint32_t c = 0; c < kUnit<T>; ++c) f[c] = f[c] * factor;
  return pack<T>(f);
}

template <typename T>
__device__ __forceinline__ void tile_scale(const GradTile& g, float factor) {
  constexpr uint32_t N = kUnit<T>;
  if (full_tile(g)) {
    u32x4 v[kGradUnits];
    load_tile(g, v);
#pragma unroll
    for (int j = 0; j < kGradUnits; ++j) st_unit<true>(g.dst + threadIdx.x * 16u + j * kGradThreads * 16, unit_scale<T>(v[j], factor));
    return;
  }
  const uint32_t units = g.n / N;
  for (uint32_t u = threadIdx.x; u < units; u += kGradThreads)
    st_unit<true>(g.dst + u * 16u, unit_scale<T>(ld_unit<true>(g.src + u * 16u), factor));
  const uint32_t e = units * N + threadIdx.x;
  if (e < g.n) st_one<T>(g.dst + e * T::kSize, ld_one<T>(g.src + e * T::kSize) * factor);
}

// JOIN: the norm is that of `parts` partial sums, which every workgroup adds up
// for itself and the first one writes to `norm`.
template <bool JOIN>
__global__ __launch_bounds__(kGradThreads) void clip_kernel(const GradTile* __restrict__ tiles, uint32_t ntiles,
                                                            const double* __restrict__ partial, uint32_t parts, float* norm,
                                                            const PoolArg pa, float max_norm) {
  float total;
  if constexpr (JOIN) {
    __shared__ double lds[kGradThreads / 64];
    total = norm_of(parts, lds, [&](uint32_t b) { return partial[b]; });
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  } else {
    total = *norm;
  }
  float factor = max_norm / (total + 1e-6f);
  if (factor > 1.0f) factor = 1.0f;  // a NaN stays
  __shared__ unsigned long long xchg[2];
  const TilePool pool{(global_u64*)pa.next, (global_u64*)(pa.next + (uint64_t)pa.counters * kFlagStride), xchg,
                      pa.rounds, pa.counters};
  for_each_tile(blockIdx.x, gridDim.x, ntiles, pool, [&](uint32_t t) {
    const GradTile g = tiles[t];
    if (factor == 1.0f && g.src == g.dst) return;
    if (g.bf16) tile_scale<BF16>(g, factor);
    else tile_scale<F32>(g, factor);
  });
}

uint32_t grad_grid(uint32_t ntiles, uint32_t per_cu) {
  const int cus = device_cu_count();
  uint32_t most = (uint32_t)(cus > 0 ? cus : 1) * per_cu;
  if (most > kGradMaxBlocks) most = kGradMaxBlocks;
  return ntiles < most ? ntiles : most;
}

uint32_t norm_grid(uint32_t ntiles) { return grad_grid((ntiles + 1) / 2, 1); }

// counters where there are rounds left for them after the grid-stride ones
PoolArg clip_pool(uint32_t ntiles, uint32_t grid, unsigned long long* pool) {
  return ntiles / grid >= 16 ? PoolArg{pool, 8, kGradCounters} : PoolArg{nullptr, 0, 1};
}

}  // namespace

hipError_t launch_grad_norm(const GradTile* tiles, uint32_t ntiles, double* partial, uint32_t* ticket, float* norm,
                            hipStream_t stream) {
  if (ntiles == 0)
    hipLaunchKernelGGL(zero_norm_kernel, dim3(1), dim3(1), 0, stream, norm);
  else
    hipLaunchKernelGGL((norm_kernel<true>), dim3(norm_grid(ntiles)), dim3(kGradThreads), 0, stream, tiles, ntiles,
                       partial, ticket, norm);
  return hipGetLastError();
}

hipError_t launch_clip(const GradTile* tiles, uint32_t ntiles, const float* norm, float max_norm,
                       unsigned long long* pool, hipStream_t stream) {
  if (ntiles == 0) return hipSuccess;
  const uint32_t grid = grad_grid(ntiles, 2);
  hipLaunchKernelGGL((clip_kernel<false>), dim3(grid), dim3(kGradThreads), 0, stream, tiles, ntiles, nullptr, 0,
                     const_cast<float*>(norm), clip_pool(ntiles, grid, pool), max_norm);
  return hipGetLastError();
}

hipError_t launch_norm_and_clip(const GradTile* tiles, uint32_t ntiles, double* partial, float* norm, float max_norm,
                                unsigned long long* pool, hipStream_t stream) {
  if (ntiles == 0) return launch_grad_norm(tiles, 0, partial, nullptr, norm, stream);
  const uint32_t parts = norm_grid(ntiles), grid = grad_grid(ntiles, 2);
  hipLaunchKernelGGL((norm_kernel<false>), dim3(parts), dim3(kGradThreads), 0, stream, tiles, ntiles, partial, nullptr,
                     nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((clip_kernel<true>), dim3(grid), dim3(kGradThreads), 0, stream, tiles, ntiles, partial, parts, norm,
                     clip_pool(ntiles, grid, pool), max_norm);
  return hipGetLastError();
}

}  // namespace snac
