// grads.hip -- the global norm over a list of tensors and clipping by it
// (snac_grad_norm, snac_clip_grads in include/snac_ops.h).
//
// Both stream the list's tiles (at most kGradTileBytes of one tensor each)
// and are bound by HBM.  Tiles begin on 16-byte boundaries of their tensor
// except where the tensor does not.
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kGradThreads = 256;

// f(first element, units or elements) over a tile: whole units by all
// lanes, then the last part of a unit by single elements.
template <typename T>
__device__ __forceinline__ double tile_squares(const GradTile& g, double acc) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t units = g.n / N;
  for (uint32_t u = threadIdx.x; u < units; u += kGradThreads) {
    float f[N];
    unpack<T>(ld_unit<true>(g.src + (uint64_t)u * 16u), f);
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) acc = __builtin_fma((double)f[c], (double)f[c], acc);
  }
  const uint32_t e = units * N + threadIdx.x;
  if (e < g.n) {
    const double x = load_elem<T>(g.src + (uint64_t)e * T::kSize);
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

// Every workgroup leaves its sum in partial[]; the last one to do so adds
// them up in their order and leaves the ticket at 0 for the next call.
__global__ __launch_bounds__(kGradThreads) void norm_kernel(const GradTile* tiles, uint32_t ntiles, double* partial,
                                                            uint32_t* ticket, float* norm) {
  __shared__ double lds[kGradThreads / 64];
  __shared__ uint32_t last;
  double acc = 0.0;
  for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const GradTile g = tiles[t];
    acc = g.bf16 ? tile_squares<BF16>(g, acc) : tile_squares<F32>(g, acc);
  }
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    __hip_atomic_store(&partial[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double sum = 0.0;
  for (uint32_t b = threadIdx.x; b < gridDim.x; b += kGradThreads)
    sum += __hip_atomic_load(&partial[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) {
    *norm = (float)sqrt(sum);
    __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

__global__ void zero_norm_kernel(float* norm) { *norm = 0.0f; }

template <typename T>
__device__ __forceinline__ void tile_scale(const GradTile& g, float factor) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t units = g.n / N;
  for (uint32_t u = threadIdx.x; u < units; u += kGradThreads) {
    float f[N];
    unpack<T>(ld_unit<true>(g.src + (uint64_t)u * 16u), f);
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) f[c] = f[c] * factor;
    st_unit<true>(g.dst + (uint64_t)u * 16u, pack<T>(f));
  }
  const uint32_t e = units * N + threadIdx.x;
  if (e < g.n) store_elem<T>(g.dst + (uint64_t)e * T::kSize, load_elem<T>(g.src + (uint64_t)e * T::kSize) * factor);
}

__global__ __launch_bounds__(kGradThreads) void clip_kernel(const GradTile* tiles, uint32_t ntiles, const float* norm,
                                                            float max_norm) {
  float factor = max_norm / (*norm + 1e-6f);
  if (factor > 1.0f) factor = 1.0f;  // a NaN stays
  for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const GradTile g = tiles[t];
    if (factor == 1.0f && g.src == g.dst) continue;
    if (g.bf16) tile_scale<BF16>(g, factor);
    else tile_scale<F32>(g, factor);
  }
}

uint32_t grad_grid(uint32_t ntiles) {
  const int cus = device_cu_count();
  uint32_t most = (uint32_t)(cus > 0 ? cus : 1) * 8;
  if (most > kGradMaxBlocks) most = kGradMaxBlocks;
  return ntiles < most ? ntiles : most;
}

}  // namespace

hipError_t launch_grad_norm(const GradTile* tiles, uint32_t ntiles, double* partial, uint32_t* ticket, float* norm,
                            hipStream_t stream) {
  if (ntiles == 0)
    hipLaunchKernelGGL(zero_norm_kernel, dim3(1), dim3(1), 0, stream, norm);
  else
    hipLaunchKernelGGL(norm_kernel, dim3(grad_grid(ntiles)), dim3(kGradThreads), 0, stream, tiles, ntiles, partial,
                       ticket, norm);
  return hipGetLastError();
}

hipError_t launch_clip(const GradTile* tiles, uint32_t ntiles, const float* norm, float max_norm, hipStream_t stream) {
  if (ntiles == 0) return hipSuccess;
  hipLaunchKernelGGL(clip_kernel, dim3(grad_grid(ntiles)), dim3(kGradThreads), 0, stream, tiles, ntiles, norm, max_norm);
  return hipGetLastError();
}

}  // namespace snac
