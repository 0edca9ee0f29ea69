// rows.hpp -- device helpers of the operators' kernels: rows of bf16 or
// binary32 elements in 16-byte units at any element alignment, and
// reductions over a 64-lane wave in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops.hpp"
#include "snac_device.hpp"

namespace snac {

// 16 bytes at any element alignment: one dwordx4 access (global accesses of
// gfx950 need no alignment; aligned ones touch fewer lines)
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

// Elements of a 16-byte unit
template <typename T>
constexpr uint32_t kUnit = 16 / T::kSize;

template <typename T>
__device__ __forceinline__ void unpack(const u32x4& w, float (&f)[kUnit<T>]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if constexpr (T::kSize == 4) {
      f[c] = __uint_as_float(w[c]);
    } else {
      f[2 * c] = bf16_lo(w[c]);
      f[2 * c + 1] = bf16_hi(w[c]);
    }
  }
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&f)[kUnit<T>]) {
  u32x4 w;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if constexpr (T::kSize == 4)
      w[c] = __float_as_uint(f[c]);
    else
      w[c] = pack_bf16(f[2 * c], f[2 * c + 1]);
  }
  return w;
}

// The pointers are to global memory and say so: one that was itself loaded
// from memory would otherwise be accessed as a flat address, whose loads also
// wait for LDS.
template <typename U>
using global_ptr = __attribute__((address_space(1))) U*;

template <bool NT>
__device__ __forceinline__ u32x4 ld_unit(const char* p) {
  const auto g = (global_ptr<const u32x4_a2>)(p);
  if constexpr (NT)
    return __builtin_nontemporal_load(g);
  else
    return *g;
}
template <bool NT>
__device__ __forceinline__ void st_unit(char* p, u32x4 v) {
  const auto g = (global_ptr<u32x4_a2>)(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, g);
  else
    *g = v;
}

// The first `n` (0 < n < a unit) elements of a row's last unit; the others
// read as 0.
template <typename T>
__device__ __forceinline__ u32x4 ld_part(const char* p, uint32_t n) {
  u32x4 v = {0, 0, 0, 0};
  if constexpr (T::kSize == 4) {
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i)
      if (i < n) v[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  } else {
#pragma unroll
    for (uint32_t i = 0; i < 7; ++i)
      if (i < n) v[i / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void st_part(char* p, u32x4 v, uint32_t n) {
  if constexpr (T::kSize == 4) {
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i)
      if (i < n) *reinterpret_cast<uint32_t*>(p + 4 * i) = v[i];
  } else {
#pragma unroll
    for (uint32_t i = 0; i < 7; ++i)
      if (i < n) *reinterpret_cast<uint16_t*>(p + 2 * i) = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}

// A wave's piece of a row: U units per lane, unit j of lane l being the
// row's unit u0 + 64 j + l.  `left`: elements of the row from unit u0 on.  A
// whole piece takes the branch-free form, so that its loads go out together.
template <typename T, int U>
__device__ __forceinline__ bool whole_piece(uint32_t left) {
  return left >= 64u * U * kUnit<T>;
}

template <typename T, int U, bool NT>
__device__ __forceinline__ void ld_piece(const char* row, uint32_t left, u32x4 (&v)[U]) {
  const uint32_t lane = threadIdx.x & 63u;
  if (whole_piece<T, U>(left)) {
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = ld_unit<NT>(row + (j * 64u + lane) * 16u);
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t u = j * 64u + lane, e = u * kUnit<T>;
      v[j] = u32x4{0, 0, 0, 0};
      if (e + kUnit<T> <= left)
        v[j] = ld_unit<NT>(row + u * 16u);
      else if (e < left)
        v[j] = ld_part<T>(row + u * 16u, left - e);
    }
  }
}

template <typename T, int U, bool NT>
__device__ __forceinline__ void st_piece(char* row, uint32_t left, const u32x4 (&v)[U]) {
  const uint32_t lane = threadIdx.x & 63u;
  if (whole_piece<T, U>(left)) {
#pragma unroll
    for (int j = 0; j < U; ++j) st_unit<NT>(row + (j * 64u + lane) * 16u, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t u = j * 64u + lane, e = u * kUnit<T>;
      if (e + kUnit<T> <= left)
        st_unit<NT>(row + u * 16u, v[j]);
      else if (e < left)
        st_part<T>(row + u * 16u, v[j], left - e);
    }
  }
}

// 8, 4 or 2 bytes at any element alignment
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

// ld_part and st_part with `n` the same in all lanes: an access for each of its
// bits instead of one for each element.
template <typename T>
__device__ __forceinline__ u32x4 ld_rest(const char* p, uint32_t n) {
  auto two = [&](uint32_t at) { return *(global_ptr<const u32x2_a2>)(p + at); };
  auto one = [&](uint32_t at) { return (uint32_t) * (global_ptr<const u32_a2>)(p + at); };
  auto half = [&](uint32_t at) { return (uint32_t) * (global_ptr<const uint16_t>)(p + at); };
  u32x4 v = {0, 0, 0, 0};
  const uint32_t words = T::kSize == 4 ? n : n / 2;
  if (words & 2) {
    const auto w = two(0);
    v[0] = w[0], v[1] = w[1];
    if (words & 1) v[2] = one(8);
  } else if (words & 1) {
    v[0] = one(0);
  }
  if (T::kSize == 2 && (n & 1)) {
    const uint32_t h = half(words * 4);
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      if (words == c) v[c] = h;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void st_rest(char* p, u32x4 v, uint32_t n) {
  const uint32_t words = T::kSize == 4 ? n : n / 2;
  if (words & 2) {
    *(global_ptr<u32x2_a2>)(p) = u32x2_a2{v[0], v[1]};
    if (words & 1) *(global_ptr<u32_a2>)(p + 8) = v[2];
  } else if (words & 1) {
    *(global_ptr<u32_a2>)(p) = v[0];
  }
  if (T::kSize == 2 && (n & 1)) {
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      if (words == c) *(global_ptr<uint16_t>)(p + words * 4) = (uint16_t)v[c];
  }
}

// Whether every row begins on a line (`ld` in bytes).  Such rows may be read past
// the caches; of others two share a line, and each would fetch it.
__device__ __forceinline__ bool whole_lines(const char* p, uint64_t ld) { return (((uint64_t)(uintptr_t)p | ld) & 127) == 0; }

// Pieces of rows of `width` elements, of which the last may end in a part of a unit;
// `left` is the same in all lanes.  The part is loaded with the others, as the 16
// bytes that end where the row does, and settle_held brings its elements to their
// places when they are unpacked: what waits for them before, waits for every load in
// flight.
template <typename T, int U, bool NT>
__device__ __forceinline__ void ld_held(const char* piece, uint32_t left, uint32_t width, u32x4 (&v)[U]) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t lane = threadIdx.x & 63u;
  if (whole_piece<T, U>(left)) {
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = ld_unit<NT>(piece + (j * 64u + lane) * 16u);
    return;
  }
  const uint32_t units = left / N, rest = left % N;
  if (rest == 0 || width < N) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      v[j] = u32x4{0, 0, 0, 0};
      if (j * 64u + lane < units) v[j] = ld_unit<NT>(piece + (j * 64u + lane) * 16u);
    }
    if (rest != 0 && lane == 0) v[0] = ld_rest<T>(piece, rest);
  } else {
    const char* end = piece + (uint64_t)left * T::kSize - 16;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t u = j * 64u + lane;
      v[j] = u32x4{0, 0, 0, 0};
      if (u <= units) v[j] = ld_unit<NT>(u < units ? piece + u * 16u : end);
    }
  }
}

// Elements first, first + 1 .. of a unit as its elements 0, 1 .., zeros after them,
// where `mine`; `first` (1 .. its number of elements - 1) is the same in all lanes.
template <uint32_t N>
__device__ __forceinline__ void later_elems(float (&f)[N], uint32_t first, bool mine) {
#pragma unroll
  for (uint32_t k = 1; k < N; ++k) {
    if (first != k) continue;
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) f[c] = mine ? (c + k < N ? f[(c + k) % N] : 0.0f) : f[c];
  }
}

template <typename T, int U>
__device__ __forceinline__ void settle_held(uint32_t left, uint32_t width, float (&f)[U][kUnit<T>]) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t units = left / N, rest = left % N;
  if (rest == 0 || units >= 64u * U || width < N) return;
#pragma unroll
  for (uint32_t j = 0; j < U; ++j)
    if (units / 64 == j) later_elems<N>(f[j], N - rest, (threadIdx.x & 63u) == units % 64);
}

template <typename T, int U, bool NT>
__device__ __forceinline__ void st_held(char* row, uint32_t left, const u32x4 (&v)[U]) {
  const uint32_t lane = threadIdx.x & 63u;
  if (whole_piece<T, U>(left)) {
#pragma unroll
    for (int j = 0; j < U; ++j) st_unit<NT>(row + (j * 64u + lane) * 16u, v[j]);
    return;
  }
  const uint32_t units = left / kUnit<T>, rest = left % kUnit<T>;
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (j * 64u + lane < units) st_unit<NT>(row + (j * 64u + lane) * 16u, v[j]);
  if (rest != 0) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j * 64u + lane == units) st_rest<T>(row + units * 16u, v[j], rest);
  }
}

// What this wave's lanes wrote to LDS before is what its lanes read after: LDS
// keeps a wave's order by itself, this keeps the compiler to it (which may
// otherwise take a lane's own store for what it reads back).  No instructions.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

__device__ __forceinline__ uint32_t wave_id() { return uniform(threadIdx.x >> 6); }

// ---- reductions over L = 16, 32 or 64 neighbouring lanes, every lane with
// the same result: exchanges inside a row of 16 lanes by DPP (lanes 1, 2,
// then mirrored halves, so that both sides of a sum add the same two
// numbers), across rows by gfx950's lane swaps.  All 64 lanes must be active.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// x = f(x, the x of the lane's partner) at distance D (1, 2, 4, 8, 16, 32)
template <int D, typename F>
__device__ __forceinline__ uint32_t exchange(uint32_t x, F f) {
  if constexpr (D == 1) return f(x, dpp<kDppXor1>(x));
  else if constexpr (D == 2) return f(x, dpp<kDppXor2>(x));
  else if constexpr (D == 4) return f(x, dpp<kDppHalfMirror>(x));
  else if constexpr (D == 8) return f(x, dpp<kDppMirror>(x));
  else if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return f(r[0], r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return f(r[0], r[1]);
  }
}

template <int L, typename F>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t x, F f) {
  x = exchange<1>(x, f);
  x = exchange<2>(x, f);
  x = exchange<4>(x, f);
  x = exchange<8>(x, f);
  if constexpr (L >= 32) x = exchange<16>(x, f);
  if constexpr (L >= 64) x = exchange<32>(x, f);
  return x;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
  return __uint_as_float(lanes_reduce<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
// x + the x of the lane's partner at distance D (both types here: an overload in an
// inner namespace would hide the other and take its arguments)
template <int D>
__device__ __forceinline__ float exchange_sum(float x) {
  return __uint_as_float(exchange<D>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int D>
__device__ __forceinline__ double exchange_sum(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32), lo2 = lo, hi2 = hi;
  if constexpr (D <= 8) {
    constexpr int C = D == 1 ? kDppXor1 : D == 2 ? kDppXor2 : D == 4 ? kDppHalfMirror : kDppMirror;
    lo2 = dpp<C>(lo), hi2 = dpp<C>(hi);
  } else if constexpr (D == 16) {
    const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    lo = l[0], lo2 = l[1], hi = h[0], hi2 = h[1];
  } else {
    const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    lo = l[0], lo2 = l[1], hi = h[0], hi2 = h[1];
  }
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo)) + __longlong_as_double((long long)((uint64_t)hi2 << 32 | lo2));
}
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
  x = exchange_sum<1>(x);
  x = exchange_sum<2>(x);
  x = exchange_sum<4>(x);
  x = exchange_sum<8>(x);
  if constexpr (L >= 32) x = exchange_sum<16>(x);
  if constexpr (L >= 64) x = exchange_sum<32>(x);
  return x;
}
// the largest of the values that are not NaN
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
  return __uint_as_float(lanes_reduce<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  return lanes_reduce<L>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

__device__ __forceinline__ float wave_sum(float x) { return lanes_sum<64>(x); }
__device__ __forceinline__ float wave_max(float x) { return lanes_max<64>(x); }
__device__ __forceinline__ double wave_sum(double x) { return lanes_sum<64>(x); }

// Zeros to `rows` rows of `width` elements from `p` on, but those that `skip`
// names, by the whole workgroup: a wave a piece, in the order of the addresses.
template <typename T, typename Skip>
__device__ __forceinline__ void put_zeros(char* p, uint64_t ld, uint32_t width, uint32_t rows, Skip skip) {
  const u32x4 zero[4] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  constexpr uint32_t step = 64u * 4 * kUnit<T>;
  const uint32_t pieces = (width + step - 1) / step;
  for (uint32_t i = wave_id(); i < rows * pieces; i += blockDim.x >> 6) {
    const uint32_t r = i / pieces, e = (i - r * pieces) * step;
    if (!skip(r)) st_piece<T, 4, true>(p + r * ld + (uint64_t)e * T::kSize, width - e, zero);
  }
}

// A workgroup's share of ZeroRows, `wg` counted from the first that has one.
__device__ __forceinline__ void write_zeros(const ZeroRows& z, uint32_t wg) {
  const uint32_t lo = wg * z.per, rows = z.rows - lo < z.per ? z.rows - lo : z.per;
  put_zeros<BF16>(z.p + lo * z.ld, z.ld, z.width, rows, [](uint32_t) { return false; });
}

// id of item i of an id array of 4- or 8-byte elements
__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, uint64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

}  // namespace snac
