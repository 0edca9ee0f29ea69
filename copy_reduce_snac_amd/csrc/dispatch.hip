// dispatch.hip -- rows of tokens packed by expert, and the weighted sum of
// the rows that come back, with its gradient (snac_dispatch, snac_combine,
// snac_combine_backward in include/snac_ops.h).
//
// All three move rows and are bound by HBM.  A wave takes one piece of one
// token's row (U units of 16 bytes a lane) and walks the token's topk slots,
// so that a token's row is read once (dispatch) or written once (combine), and
// its slots' rows are whole lines each.  Rows that are used once stream
// (stores that stay in the caches: 130 us for 115, 121 for 103).  16384 tokens,
// rows of 4 KiB: dispatch to 8 rows 100 us (5.9 TB/s), combine of 8 rows 101 us
// (6.0 TB/s; two or four rows in flight at a time 102 to 104), combine_backward
// of 4 rows 95 us (6.1 TB/s).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kPieceUnits = 4;  // of combine_backward

template <typename T, int U>
constexpr uint32_t kPieceElems = 64u * U * kUnit<T>;

template <typename T, int U>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const DispatchArgs a, uint32_t pieces, uint64_t items) {
  for (uint64_t it = (uint64_t)blockIdx.x * kRowWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kRowWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kPieceElems<T, U>;
    const uint64_t off = (uint64_t)first * T::kSize;
    u32x4 v[U];
    ld_piece<T, U, false>(a.x + t * a.ld_x + off, a.width - first, v);
    for (int32_t k = 0; k < a.topk; ++k) {
      const uint32_t row = uniform((uint32_t)a.row_of_slot[t * a.topk + k]);
      if (row < a.rows) st_piece<T, U, true>(a.out + (uint64_t)row * a.ld_out + off, a.width - first, v);
    }
  }
}

template <typename T, int U>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const CombineArgs a, uint32_t pieces, uint64_t items) {
  constexpr uint32_t N = kUnit<T>;
  for (uint64_t it = (uint64_t)blockIdx.x * kRowWaves + wave_id(); it < items; it += (uint64_t)gridDim.x * kRowWaves) {
    const uint64_t t = it / pieces;
    const uint32_t first = (uint32_t)(it - t * pieces) * kPieceElems<T, U>;
    const uint64_t off = (uint64_t)first * T::kSize;
    float acc[U][N];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) acc[j][c] = 0.0f;
    for (int32_t k = 0; k < a.topk; ++k) {
      const uint32_t row = uniform((uint32_t)a.row_of_slot[t * a.topk + k]);
      if (row >= a.rows) continue;
      const float w = a.weights ? a.weights[t * a.topk + k] : 1.0f;
      u32x4 v[U];
      ld_piece<T, U, true>(a.y + (uint64_t)row * a.ld_y + off, a.width - first, v);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[N];
        unpack<T>(v[j], f);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) acc[j][c] = __builtin_fmaf(w, f[c], acc[j][c]);
      }
    }
    u32x4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = pack<T>(acc[j]);
    st_piece<T, U, true>(a.out + t * a.ld_out + off, a.width - first, v);
  }
}

// One wave a slot: its rows of dout (read again by the token's other slots,
// from L2) and of y once through.  The dot product is binary32 within a 16-byte
// unit and binary64 from there on, so that its error does not grow with the
// width.
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
    double dot = 0.0;
    for (uint32_t e = 0; e < a.width; e += kPieceElems<T, kPieceUnits>) {
      const uint64_t off = (uint64_t)e * T::kSize;
      u32x4 vg[kPieceUnits], vy[kPieceUnits];
      ld_piece<T, kPieceUnits, false>(g + off, a.width - e, vg);
      ld_piece<T, kPieceUnits, true>(y + off, a.width - e, vy);
#pragma unroll
      for (int j = 0; j < kPieceUnits; ++j) {
        float fg[N], fy[N];
        unpack<T>(vg[j], fg);
        unpack<T>(vy[j], fy);
        float part = 0.0f;
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) {
          part = __builtin_fmaf(fg[c], fy[c], part);
          fg[c] = w * fg[c];
        }
        dot += part;
        vg[j] = pack<T>(fg);
      }
      st_piece<T, kPieceUnits, true>(dy + off, a.width - e, vg);
    }
    dot = wave_sum(dot);
    if (lane == 0) a.dweights[s] = (float)dot;
  }
}

// Workgroups for `items` waves of work: one item a wave (grid-stride only past
// 2^22 workgroups).  combine_backward of 65536 rows of 4 KiB: 95 us, against
// 103, 107 and 102 with 16, 8 and 4 workgroups a CU striding over the items.
uint32_t row_grid(uint64_t items) {
  const uint64_t want = (items + kRowWaves - 1) / kRowWaves;
  return (uint32_t)(want < (1u << 22) ? want : 1u << 22);
}

// Units a lane of the pieces that `tokens` rows of `width` elements are cut
// into.  Four read the most at a time; where they would leave SIMDs without a
// wave (4 a CU) one, and with few waves a SIMD (64 a CU) two, since a wave
// walks its token's slots one after another.  us, pieces of 1 / 2 / 4 units:
//   combine   64 tokens of 8 rows of 16 KiB 8.3 / - / 10; 629 of 6 rows of
//             6.4 KiB 14.5 / 14.1 / 19.9; 2600 of 6 rows of 4 KiB 18.2 / 15.3 /
//             15.6; 9000 48.9 / 45.2 / 44.6; 16384 of 8 133 / 103 / 101
//   dispatch  629 15.4 / 15.7 / 16.1; 9000 50.6 / 52.2 / 54.2 (never four)
template <typename T>
int piece_units(uint64_t tokens, uint32_t width, int most) {
  const int cus = device_cu_count();
  const uint64_t cu = (uint64_t)(cus > 0 ? cus : 1);
  const uint32_t pieces = (width + kPieceElems<T, 4> - 1) / kPieceElems<T, 4>;
  if (tokens >= cu * 64) return most;
  return tokens * pieces < cu * 4 ? 1 : tokens * pieces < cu * 64 ? 2 : most;
}

template <typename T, int U>
hipError_t dispatch_in(const DispatchArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kPieceElems<T, U> - 1) / kPieceElems<T, U>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((dispatch_kernel<T, U>), dim3(row_grid(items)), dim3(kRowThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch_any(const DispatchArgs& a, hipStream_t stream) {
  return piece_units<T>(a.tokens, a.width, 2) == 1 ? dispatch_in<T, 1>(a, stream) : dispatch_in<T, 2>(a, stream);
}

template <typename T, int U>
hipError_t combine_in(const CombineArgs& a, hipStream_t stream) {
  const uint32_t pieces = (a.width + kPieceElems<T, U> - 1) / kPieceElems<T, U>;
  const uint64_t items = a.tokens * pieces;
  hipLaunchKernelGGL((combine_kernel<T, U>), dim3(row_grid(items)), dim3(kRowThreads), 0, stream, a, pieces, items);
  return hipGetLastError();
}

template <typename T>
hipError_t combine_any(const CombineArgs& a, hipStream_t stream) {
  switch (piece_units<T>(a.tokens, a.width, 4)) {
    case 1: return combine_in<T, 1>(a, stream);
    case 2: return combine_in<T, 2>(a, stream);
    default: return combine_in<T, 4>(a, stream);
  }
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
