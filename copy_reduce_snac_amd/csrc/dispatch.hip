// dispatch.hip -- rows of tokens packed by expert, and the weighted sum of
// the rows that come back, with its gradient (snac_dispatch, snac_combine,
// snac_combine_backward in include/snac_ops.h).
//
// All three move rows and are bound by HBM.  A wave takes one piece of one
// token's row (kPieceUnits units of 16 bytes a lane) and walks the token's
// topk slots, so that a token's row is read once (dispatch) or written once
// (combine), and its slots' rows are whole lines each.
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kPieceUnits = 4;

template <typename T>
constexpr uint32_t kPieceElems = 64u * kPieceUnits * kUnit<T>;

template <typename T>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const DispatchArgs a, uint32_t pieces, uint64_t items) {
  for (uint64_t it = (uint64_t)blockIdx.x * kRowWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kRowWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kPieceElems<T>;
    const uint64_t off = (uint64_t)first * T::kSize;
    u32x4 v[kPieceUnits];
    ld_piece<T, kPieceUnits, false>(a.x + t * a.ld_x + off, a.width - first, v);
    for (int32_t k = 0; k < a.topk; ++k) {
      const uint32_t row = uniform((uint32_t)a.row_of_slot[t * a.topk + k]);
      if (row < a.rows) st_piece<T, kPieceUnits, true>(a.out + (uint64_t)row * a.ld_out + off, a.width - first, v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const CombineArgs a, uint32_t pieces, uint64_t items) {
  constexpr uint32_t N = kUnit<T>;
  for (uint64_t it = (uint64_t)blockIdx.x * kRowWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kRowWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kPieceElems<T>;
    const uint64_t off = (uint64_t)first * T::kSize;
    float acc[kPieceUnits][N];
#pragma unroll
    for (int j = 0; j < kPieceUnits; ++j)
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) acc[j][c] = 0.0f;
    for (int32_t k = 0; k < a.topk; ++k) {
      const uint32_t row = uniform((uint32_t)a.row_of_slot[t * a.topk + k]);
      if (row >= a.rows) continue;
      const float w = a.weights ? a.weights[t * a.topk + k] : 1.0f;
      u32x4 v[kPieceUnits];
      ld_piece<T, kPieceUnits, true>(a.y + (uint64_t)row * a.ld_y + off, a.width - first, v);
#pragma unroll
      for (int j = 0; j < kPieceUnits; ++j) {
        float f[N];
        unpack<T>(v[j], f);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) acc[j][c] = __builtin_fmaf(w, f[c], acc[j][c]);
      }
    }
    u32x4 v[kPieceUnits];
#pragma unroll
    for (int j = 0; j < kPieceUnits; ++j) v[j] = pack<T>(acc[j]);
    st_piece<T, kPieceUnits, true>(a.out + t * a.ld_out + off, a.width - first, v);
  }
}

// One wave a slot: its rows of dout (read again by the token's other slots,
// from L2) and of y once through, the dot product in binary32 per lane and
// then over the lanes.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(const CombineBackwardArgs a, uint64_t slots) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t lane = threadIdx.x & 63u;
  for (uint64_t s = (uint64_t)blockIdx.x * kRowWaves + wave_id(); s < slots; s += (uint64_t)gridDim.x * kRowWaves) {
    const uint32_t row = uniform((uint32_t)a.row_of_slot[s]);
    if (row >= a.rows) {
      if (lane == 0) a.dweights[s] = 0.0f;
      continue;
    }
    const uint64_t t = s / (uint32_t)a.topk;
    const float w = a.weights[s];
    const char* g = a.dout + t * a.ld_dout;
    const char* y = a.y + (uint64_t)row * a.ld_y;
    char* dy = a.dy + (uint64_t)row * a.ld_dy;
    float dot = 0.0f;
    for (uint32_t e = 0; e < a.width; e += kPieceElems<T>) {
      const uint64_t off = (uint64_t)e * T::kSize;
      u32x4 vg[kPieceUnits], vy[kPieceUnits];
      ld_piece<T, kPieceUnits, false>(g + off, a.width - e, vg);
      ld_piece<T, kPieceUnits, true>(y + off, a.width - e, vy);
#pragma unroll
      for (int j = 0; j < kPieceUnits; ++j) {
        float fg[N], fy[N];
        unpack<T>(vg[j], fg);
        unpack<T>(vy[j], fy);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) {
          dot = __builtin_fmaf(fg[c], fy[c], dot);
          fg[c] = w * fg[c];
        }
        vg[j] = pack<T>(fg);
      }
      st_piece<T, kPieceUnits, true>(dy + off, a.width - e, vg);
    }
    dot = wave_sum(dot);
    if (lane == 0) a.dweights[s] = dot;
  }
}

// workgroups for `items` waves of work, grid-stride past 16 a CU
uint32_t row_grid(uint64_t items) {
  const int cus = device_cu_count();
  const uint64_t most = (uint64_t)(cus > 0 ? cus : 1) * 16;
  const uint64_t want = (items + kRowWaves - 1) / kRowWaves;
  return (uint32_t)(want < most ? want : most);
}

template <typename T>
hipError_t dispatch_any(const DispatchArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kPieceElems<T> - 1) / kPieceElems<T>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((dispatch_kernel<T>), dim3(row_grid(items)), dim3(kRowThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

template <typename T>
hipError_t combine_any(const CombineArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kPieceElems<T> - 1) / kPieceElems<T>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((combine_kernel<T>), dim3(row_grid(items)), dim3(kRowThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

template <typename T>
hipError_t combine_backward_any(const CombineBackwardArgs& a, hipStream_t stream) {
  const uint64_t slots = a.tokens * (uint64_t)a.topk;
  hipLaunchKernelGGL((combine_backward_kernel<T>), dim3(row_grid(slots)), dim3(kRowThreads), 0, stream, a, slots);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? dispatch_any<BF16>(a, stream) : dispatch_any<F32>(a, stream);
}

hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? combine_any<BF16>(a, stream) : combine_any<F32>(a, stream);
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? combine_backward_any<BF16>(a, stream) : combine_backward_any<F32>(a, stream);
}

}  // namespace snac
