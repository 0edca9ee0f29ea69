// layernorm.hip -- layer norm and its gradients (snac_layer_norm,
// snac_layer_norm_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

// The widest rows that a workgroup holds in registers: 16 waves of 64 lanes of 4
// units, or 2 where wider parameters (with 4 they spill) or the gradient's sums over
// tokens are held too.
template <typename T, typename P>
constexpr uint64_t kHeldKib = P::kSize > T::kSize ? 32 : 64;
constexpr uint64_t kHeldBackwardKib = 32;
constexpr uint32_t kSumTokens = 32;  // binary32 sums over tokens go no further

// 16 bytes' worth of T elements' parameters of type P, raw.
template <typename T, typename P>
struct Params {
  static constexpr int kWords = kUnit<T> * P::kSize / 4;
  uint32_t w[kWords];
};

// Parameters of the kUnit<T> elements from `e` on.
template <typename T, typename P>
__device__ __forceinline__ void ld_params(const char* p, uint32_t e, Params<T, P>& r) {
  constexpr int K = Params<T, P>::kWords;
  const char* at = p + (uint64_t)e * P::kSize;
  if constexpr (K == 2) {
    const u32x2_a2 v = *(global_ptr<const u32x2_a2>)(at);
    r.w[0] = v[0], r.w[1] = v[1];
  } else {
#pragma unroll
    for (int u = 0; u < K / 4; ++u) {
      const u32x4 v = ld_unit<false>(at + 16 * u);
#pragma unroll
      for (int c = 0; c < 4; ++c) r.w[4 * u + c] = v[c];
    }
  }
}
// The same at the end of a row; those past `width` are 0.
template <typename T, typename P>
__device__ __forceinline__ void ld_params(const char* p, uint32_t e, uint32_t width, Params<T, P>& r) {
  constexpr uint32_t N = kUnit<T>;
  if (e + N <= width) return ld_params<T, P>(p, e, r);
#pragma unroll
  for (int c = 0; c < Params<T, P>::kWords; ++c) r.w[c] = 0;
#pragma unroll
  for (uint32_t i = 0; i < N; ++i) {
    if (e + i >= width) continue;
    const char* at = p + (uint64_t)(e + i) * P::kSize;
    if constexpr (P::kSize == 4) r.w[i] = *(global_ptr<const uint32_t>)(at);
    else r.w[i / 2] |= (uint32_t)*(global_ptr<const uint16_t>)(at) << (16 * (i & 1));
  }
}
// All of them 1 (absent weights) or -0 (absent biases: x + -0 is x, also for -0).
template <typename T, typename P>
__device__ __forceinline__ void fill_params(float v, Params<T, P>& r) {
  const uint32_t w = __float_as_uint(v);
#pragma unroll
  for (int c = 0; c < Params<T, P>::kWords; ++c) r.w[c] = P::kSize == 4 ? w : w | w >> 16;
}
template <typename T, typename P>
__device__ __forceinline__ float param(const Params<T, P>& r, uint32_t i) {
  if constexpr (P::kSize == 4) return __uint_as_float(r.w[i]);
  else return i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
}

// Sum over W neighbouring lanes, W a power of two up to 16, in each of them, in F.
template <int W, typename F>
__device__ __forceinline__ F few_lanes_sum(F x) {
  if constexpr (W > 1) x = exchange_sum<1>(x);
  if constexpr (W > 2) x = exchange_sum<2>(x);
  if constexpr (W > 4) x = exchange_sum<4>(x);
  if constexpr (W > 8) x = exchange_sum<8>(x);
  return x;
}

// Sums of a and b over the L lanes or the W waves of a row (`lds`: room for two numbers of each
// of the workgroup's waves, not used by the call before), in every lane.
template <int L, int W>
__device__ __forceinline__ void row_sum(double& a, double& b, double (*lds)[2]) {
  a = lanes_sum<L>(a);
  b = lanes_sum<L>(b);
  if constexpr (W > 1) {
    const uint32_t lane = threadIdx.x & 63u, w = wave_id(), w0 = w / W * W;
    if (lane == 0) lds[w][0] = a, lds[w][1] = b;
    __syncthreads();
    // A lane reads some of them, which takes fewer instructions than an exchange of
    // binary64: two, of 8 waves four (gradients of 8192 rows of 5003 bf16 60 us instead
    // of 62; of 4 and 16 waves the registers of wider parameters do not allow it).
    constexpr uint32_t P = W == 8 ? 4 : 2, S = W / P;
    a = lds[w0 + lane % S][0], b = lds[w0 + lane % S][1];
#pragma unroll
    for (uint32_t k = 1; k < P; ++k) a += lds[w0 + k * S + lane % S][0], b += lds[w0 + k * S + lane % S][1];
    a = few_lanes_sum<S>(a);
    b = few_lanes_sum<S>(b);
  }
}
template <int L, int W>
__device__ __forceinline__ float row_sum(float a, float* lds) {
  a = lanes_sum<L>(a);
  if constexpr (W > 1) {
    const uint32_t lane = threadIdx.x & 63u, w = wave_id(), w0 = w / W * W;
    if (lane == 0) lds[w] = a;
    __syncthreads();
    a = few_lanes_sum<W>(lds[w0 + lane % W]);
  }
  return a;
}

// 1 / sqrt(v) rounded to binary32: the hardware's estimate (2^-23 or better) and one
// step of Newton's iteration, which leaves 1.5 times its square, 2^-45.
__device__ __forceinline__ float inverse_root(double v) {
  const double r = __builtin_amdgcn_rsq(v);
  return (float)(v > 0.0 && v < HUGE_VAL ? r * __builtin_fma(-0.5 * v * r, r, 1.5) : r);
}

// Sum over a unit of f(element), in binary32.
template <uint32_t N, typename F>
__device__ __forceinline__ float unit_sum(F f) {
  float s = f(0);
#pragma unroll
  for (uint32_t c = 1; c < N; ++c) s += f(c);
  return s;
}

// Sum over a unit of the products, fused in binary32.
template <uint32_t N>
__device__ __forceinline__ float unit_dot(const float (&x)[N], const float (&y)[N]) {
  float s = x[0] * y[0];
#pragma unroll
  for (uint32_t c = 1; c < N; ++c) s = __builtin_fmaf(x[c], y[c], s);
  return s;
}

// A 16-bit element's place in its word.
__device__ __forceinline__ uint32_t with_half(uint32_t w, uint32_t c, uint16_t half) {
  return (c & 1) ? (w & 0xffffu) | (uint32_t)half << 16 : (w & 0xffff0000u) | half;
}

// A wave's piece of a row that stays in registers: U units of each of a row's L
// lanes, unit j of lane l being the piece's unit j L + l; `left` elements of the row
// from the piece on.  REST: a row may end in a part of a unit.  Its lane takes the
// unit that ends where the row does instead, whose first `skip` elements are another
// lane's too: both make the same results of them, and sums leave them out.  A row of
// less than a unit (16 lanes only) is the last elements of one.  (Parts loaded and
// stored in pieces of their own, and moved to their places: 8192 rows of 5003 bf16
// 42 us, this way 33.)
template <typename T, int L, int U, bool REST>
struct Piece {
  static constexpr uint32_t N = kUnit<T>;
  const uint32_t left;
  const bool whole;
  __device__ __forceinline__ Piece(uint32_t left) : left(left), whole(left >= L * U * N) {}
  __device__ __forceinline__ static uint32_t own(int j) { return (j * L + threadIdx.x % L) * N; }
  __device__ __forceinline__ bool has(int j) const { return REST ? own(j) < left : own(j) + N <= left; }
  // the unit's first element, counted from the piece
  __device__ __forceinline__ int32_t at(int j) const {
    const int32_t e = (int32_t)own(j), last = (int32_t)(left - N);
    return REST && e > last ? last : e;
  }
  __device__ __forceinline__ uint32_t skip(int j) const { return own(j) - (uint32_t)at(j); }
  __device__ __forceinline__ bool small() const { return REST && L == 16 && left < N && has(0); }
  template <typename P>
  __device__ __forceinline__ void params(const char* p, uint32_t first, int j, Params<T, P>& r) const {
    if (!p || !has(j)) return;
    const char* from = p + (int64_t)(int32_t)(first + (uint32_t)at(j)) * P::kSize;
    if (small()) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        if (c < skip(j)) continue;
        if constexpr (P::kSize == 4) r.w[c] = *(global_ptr<const uint32_t>)(from + 4 * c);
        else r.w[c / 2] = with_half(r.w[c / 2], c, *(global_ptr<const uint16_t>)(from + 2 * c));
      }
    } else {
      ld_params<T, P>(from, 0, r);
    }
  }
  template <bool NT>
  __device__ __forceinline__ void load(const char* piece, u32x4 (&v)[U]) const {
    const uint32_t l = threadIdx.x % L;
    if (small()) {
      v[0] = u32x4{0, 0, 0, 0};
      const char* from = piece + (int64_t)at(0) * T::kSize;
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        if (c < skip(0)) continue;
        if constexpr (T::kSize == 4) v[0][c] = *(global_ptr<const uint32_t>)(from + 4 * c);
        else v[0][c / 2] = with_half(v[0][c / 2], c, *(global_ptr<const uint16_t>)(from + 2 * c));
      }
    } else if (whole) {
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = ld_unit<NT>(piece + (j * L + l) * 16u);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        v[j] = u32x4{0, 0, 0, 0};
        if (has(j)) v[j] = ld_unit<NT>(piece + (int64_t)at(j) * T::kSize);
      }
    }
  }
  __device__ __forceinline__ void store(char* piece, const u32x4 (&v)[U]) const {
    const uint32_t l = threadIdx.x % L;
    if (small()) {
      char* from = piece + (int64_t)at(0) * T::kSize;
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        if (c < skip(0)) continue;
        if constexpr (T::kSize == 4) *(global_ptr<uint32_t>)(from + 4 * c) = v[0][c];
        else *(global_ptr<uint16_t>)(from + 2 * c) = (uint16_t)(v[0][c / 2] >> (16 * (c & 1)));
      }
    } else if (whole) {
#pragma unroll
      for (int j = 0; j < U; ++j) st_unit<true>(piece + (j * L + l) * 16u, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (has(j)) st_unit<true>(piece + (int64_t)at(j) * T::kSize, v[j]);
    }
  }
  // an element as sums take it
  __device__ __forceinline__ float counted(int j, uint32_t c, float f) const { return !REST || c >= skip(j) ? f : 0.0f; }
};

// ------------------------------------------------------------------ forward

// What a row's sums give.  The mean `near` of the first pass is binary32
// throughout and off by its sum's roundings, which matter where the row is far
// from 0 and hardly varies: so the second pass sums the distances d from it as
// well as their squares, and takes their mean off, in a fused product with rstd.
// Where that is more than a deviation, its roundings would show: then its binary32
// `rest` goes off first, exactly so from such d.
struct Moments {
  float mean, rstd, rest, shift;  // h = (d - rest) * rstd + shift
  // the sums of the d's and of their squares; `inv`: 1 / width
  __device__ __forceinline__ Moments(float near, double sum_d, double sum_dd, double width, double inv, float eps) {
    // The quotient is rounded once, by its remainder, and the squares lose it in one
    // rounding: of equal d's it is d, and their variance is 0.
    const double q = sum_d * inv, mean_d = __builtin_fma(__builtin_fma(-q, width, sum_d), inv, q);
    const double var = __builtin_fma(-sum_d, mean_d, sum_dd) * inv;
    mean = (float)((double)near + mean_d);
    rstd = inverse_root((var < 0.0 ? 0.0 : var) + (double)eps);
    rest = __builtin_fabs(mean_d) * (double)rstd > 1.0 ? (float)mean_d : 0.0f;
    shift = (float)(((double)rest - mean_d) * (double)rstd);
  }
  // whether a row of this wave has one: taken off in a branch, since it costs 8192
  // rows of 5003 bf16 2 us of 33
  __device__ __forceinline__ bool any_rest() const { return __any(rest != 0.0f); }
};

constexpr int kNormWaves = 4;  // of a workgroup whose rows take up to 4 waves

// out = (x - mean) rstd weight + bias, mean and variance those of the row, rstd =
// (variance + eps)^-1/2.  L lanes of one wave a row (L < 64: W and U are 1), or W
// waves of U units a lane: the row stays in registers, so that it is read once
// although its mean is needed before its variance and that before the result.  Sums
// go over a unit in binary32 and on in binary64.
//
// Bound by HBM: each element is read and written once.  A workgroup takes `per` rows
// one after another, so that its parameters are loaded once for them.  Calls in a row
// (one kernel alone has its ramp and drain, 88 us of the first), TB/s read and
// written: 32768 x 4096 bf16 83 us, 6.4; 16384 x 4096 f32 84 us, 6.4; 65536 x 1024
// bf16 43 us, 6.2; 262144 x 128 bf16 (16 lanes a row; with 64, 3 of 4 of them idle)
// 23 us, 5.9; 8192 x 16384 f32 194 us, 5.5: one workgroup a CU there, whose waves load
// and store at the same times.  Rows that fill a part of a shape hold its waves and
// registers all the same, with lanes idle: 20000 x 5999 bf16 (12 of 16 KiB) 98 to 101,
// 4.8.  One row of 8192 takes 3.2 us, two joins of four
// waves' sums through LDS after its load.
template <typename T, typename P, int L, int W, int U, bool REST>
__global__ __launch_bounds__(64 * (W > kNormWaves ? W : kNormWaves)) void layer_norm_kernel(const LayerNormArgs a,
                                                                                                     const uint32_t per) {
  constexpr int NW = W > kNormWaves ? W : kNormWaves, G = NW / W * (64 / L);
  constexpr uint32_t N = kUnit<T>;
  __shared__ float first_sums[NW];
  __shared__ double lds[NW][2];
  const uint32_t l = threadIdx.x % L, w = wave_id();
  const uint32_t g = L < 64 ? threadIdx.x / L : w / W;  // the row of those side by side
  const uint32_t first = (w % W) * 64u * U * N * (L == 64);  // the wave's piece of it
  const uint32_t left = first < a.width ? a.width - first : 0;
  const Piece<T, L, U, REST> piece(left);
  // the next row is loaded while this one is worked on (4096 rows of 32768 bf16 111 us
  // without, 100 with it), and the parameters are kept where registers allow it
  constexpr bool kKeep = W * U < 64;
  Params<T, P> weight[U], bias[U];
  auto params = [&](int j, const Piece<T, L, U, REST>& piece) {
    const char *pw = a.weight, *pb = a.bias;
    // opaque here, so that they are not loaded before the loop after all
    if constexpr (!kKeep) asm volatile("" : "+s"(pw), "+s"(pb));
    fill_params<T, P>(1.0f, weight[j]);
    fill_params<T, P>(-0.0f, bias[j]);
    piece.params(pw, first, j, weight[j]);
    piece.params(pb, first, j, bias[j]);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int j = 0; j < U; ++j) params(j, piece);
  }
  const double width = (double)a.width, inv = 1.0 / width;
  const float inv_f = (float)inv;
  const uint64_t t0 = (uint64_t)blockIdx.x * per, end = a.tokens - t0 < per ? a.tokens : t0 + per;
  u32x4 next[U] = {};
  const bool lines = whole_lines(a.x, a.ld_x);
  auto load = [&](uint64_t row, const Piece<T, L, U, REST>& piece) {
    if (row >= end) return;
    const char* x = a.x + row * a.ld_x + (uint64_t)first * T::kSize;
    if (L == 64 && lines) piece.template load<true>(x, next);
    else piece.template load<false>(x, next);
  };
  load(t0 + g, piece);
  // every wave of the workgroup goes round as often as its first
  for (uint64_t s = t0; s < end; s += G) {
    const uint64_t t = s + g;
    // places and masks worked out again for every row: kept, they spill
    uint32_t left_here = left;
    if constexpr (REST && !kKeep) {
      left_here = __builtin_amdgcn_readfirstlane(left);
      asm volatile("" : "+s"(left_here));
    }
    const Piece<T, L, U, REST> piece(left_here);
    u32x4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = next[j];
    load(t + G, piece);
    float f[U][N], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) unpack<T>(v[j], f[j]);
#pragma unroll
    for (int j = 0; j < U; ++j) sum += unit_sum<N>([&](uint32_t c) { return piece.counted(j, c, f[j][c]); });
    const float near = row_sum<L, W>(sum, first_sums) * inv_f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) f[j][c] = f[j][c] - near;
    double sd = 0.0, sq = 0.0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!piece.whole && !piece.has(j)) continue;
      float d[N];
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) d[c] = piece.counted(j, c, f[j][c]);
      sd += unit_sum<N>([&](uint32_t c) { return d[c]; });
      sq += unit_dot<N>(d, d);
    }
    row_sum<L, W>(sd, sq, lds);
    const Moments m(near, sd, sq, width, inv, a.eps);
    if (m.any_rest()) {
      asm volatile("");  // a branch, and not always
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) f[j][c] = f[j][c] - m.rest;
    }
    if (t < end) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if constexpr (!kKeep) {
          __builtin_amdgcn_sched_barrier(0);  // not all of them at once
          params(j, piece);
        }
#pragma unroll
        for (uint32_t c = 0; c < N; ++c)
          f[j][c] = __builtin_fmaf(__builtin_fmaf(f[j][c], m.rstd, m.shift), param<T, P>(weight[j], c), param<T, P>(bias[j], c));
        v[j] = pack<T>(f[j]);
      }
      piece.store(a.out + t * a.ld_out + (uint64_t)first * T::kSize, v);
      if (a.stats && w % W == 0 && l == 0) {
        a.stats[2 * t] = m.mean;
        a.stats[2 * t + 1] = m.rstd;
      }
    }
  }
}

// Rows of any width by one workgroup of 16 waves, which reads them three times, the
// later times from the caches where they hold it: 4096 x 32768 f32 305 us, 3.5 TB/s
// of what it cannot do without.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(const LayerNormArgs a) {
  constexpr int NW = 16;
  constexpr uint32_t N = kUnit<T>, kStep = 64u * NW * N;
  __shared__ float first_sums[NW];
  __shared__ double lds[NW][2];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  const double width = (double)a.width, inv = 1.0 / width;
  for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const char* x = a.x + t * a.ld_x;
    char* out = a.out + t * a.ld_out;
    // f(element offset, elements left from the wave's first on, the unit)
    auto row = [&](auto f) {
      for (uint64_t e0 = (uint64_t)w * 64 * N; e0 < a.width; e0 += kStep) {
        u32x4 v[1];
        ld_piece<T, 1, false>(x + e0 * T::kSize, a.width - (uint32_t)e0, v);
        float u[N];
        unpack<T>(v[0], u);
        f((uint32_t)e0, a.width - (uint32_t)e0, u);
      }
    };
    double sum = 0.0, sd = 0.0, sq = 0.0;
    row([&](uint32_t, uint32_t, float (&u)[N]) { sum += unit_sum<N>([&](uint32_t c) { return u[c]; }); });
    const float near = row_sum<64, NW>((float)sum, first_sums) * (float)inv;
    row([&](uint32_t, uint32_t left, float (&u)[N]) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) u[c] = lane * N + c < left ? u[c] - near : 0.0f;
      sd += unit_sum<N>([&](uint32_t c) { return u[c]; });
      sq += unit_dot<N>(u, u);
    });
    row_sum<64, NW>(sd, sq, lds);
    const Moments m(near, sd, sq, width, inv, a.eps);
    row([&](uint32_t e0, uint32_t left, float (&u)[N]) {
      Params<T, P> weight, bias;
      const uint32_t e = e0 + lane * N;
      if (a.weight && e < a.width) ld_params<T, P>(a.weight, e, a.width, weight);
      else fill_params<T, P>(1.0f, weight);
      if (a.bias && e < a.width) ld_params<T, P>(a.bias, e, a.width, bias);
      else fill_params<T, P>(-0.0f, bias);
#pragma unroll
      for (uint32_t c = 0; c < N; ++c)
        u[c] = __builtin_fmaf(__builtin_fmaf((u[c] - near) - m.rest, m.rstd, m.shift), param<T, P>(weight, c), param<T, P>(bias, c));
      const u32x4 v[1] = {pack<T>(u)};
      st_piece<T, 1, true>(out + (uint64_t)e0 * T::kSize, left, v);
    });
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * t] = m.mean;
      a.stats[2 * t + 1] = m.rstd;
    }
    __syncthreads();  // lds is free
  }
}

// ----------------------------------------------------------------- backward

constexpr int kGradWaves = 16;  // of a workgroup
constexpr uint32_t kGradBlocks = 256;
constexpr uint64_t kGradPartial = 32ull << 20;  // bytes of partial sums
constexpr uint64_t kGradAgain = 256;            // times kGradBlocks in a launch at most
constexpr uint32_t kAloneTurns = 2;

// N binary32 values to `p`, but the first `skip`.
template <uint32_t N>
__device__ __forceinline__ void st_sums(float* p, uint32_t skip, const float (&f)[N]) {
  if (skip == 0) {
#pragma unroll
    for (uint32_t c = 0; c < N; c += 4)
      st_unit<false>(reinterpret_cast<char*>(p + c), u32x4{__float_as_uint(f[c]), __float_as_uint(f[c + 1]),
                                                           __float_as_uint(f[c + 2]), __float_as_uint(f[c + 3])});
  } else {
#pragma unroll
    for (uint32_t c = 0; c < N; ++c)
      if (c >= skip) *(global_ptr<float>)(reinterpret_cast<char*>(p + c)) = f[c];
  }
}

// A sum over the tokens into a gradient.
__device__ __forceinline__ void put_grad(void* grad, bool bf16, bool accumulate, uint64_t i, double sum) {
  char* p = static_cast<char*>(grad);
  if (bf16) {
    if (accumulate) sum += load_elem<BF16>(p + i * 2);
    store_elem<BF16>(p + i * 2, (float)sum);
  } else {
    if (accumulate) sum += load_elem<F32>(p + i * 4);
    store_elem<F32>(p + i * 4, (float)sum);
  }
}

// With h = (x - mean) rstd and g = dout weight: dx = rstd (g - mean(g) - h mean(g h)),
// dweight = sum over the tokens of dout h, dbias of dout.  L lanes of one wave a row
// (L < 64: W and U are 1), or W waves of U units a lane; x and dout are read once, for
// dx and for the sums over tokens, which stay in registers in binary32 for up to
// kSumTokens rows; those of the rows that went side by side are added up in binary64
// and leave as one partial sum a workgroup, rounded to binary32.  More tokens than
// kGradPartial bytes of partial sums serve take several launches, each with a join
// into the call's sums.
//
// Bound by HBM: two streams read, one written, 16384 x 4096 bf16 65 us, 6.4 TB/s
// (8192 x 8192 66), the join 4.  One workgroup of 16 waves a CU leaves the fewest
// partial sums (8.4 MB there), and its waves' registers are what one CU has: the row
// after this one is on its way while this one is worked on, but not before this one's
// mean and rstd, loaded at the head of its turn, are there.  That wait in each turn,
// and that turns are dealt out evenly (171 of 256 CUs have the 3 of 2049 rows), is
// what few or short rows spend besides launch and ramp: 2049 x 1030 f32 11 us for 27
// MB and the join 3.9; 131072 x 128 bf16 21 us, 4.7 TB/s.
template <typename T, typename P, int L, int W, int U, bool REST>
__global__ __launch_bounds__(64 * kGradWaves) void layer_norm_backward_kernel(
    const LayerNormBackwardArgs a, const uint32_t per) {
  constexpr int NW = kGradWaves, Q = NW / W, G = Q * (64 / L);
  constexpr uint32_t N = kUnit<T>, kPiece = 64u * U * N;
  __shared__ double lds[2][NW][2];
  // of the rows side by side: of a wave, and of all waves of a row; columns of a thread
  // at a time, and whether weight's and bias's sums are joined at once
  constexpr uint32_t kRow = L * U * N, kCols = W * kRow;
  constexpr bool kBoth = 2 * kCols <= 64 * NW;
  constexpr uint32_t V = kBoth ? 1 : 4;
  __shared__ __align__(16) float join[kBoth ? 2 : 1][Q > 1 ? NW : 1][Q > 1 ? kPiece : 4];
  const uint32_t lane = threadIdx.x & 63u, l = lane % L, w = wave_id(), q = w / W;
  const uint32_t g = L < 64 ? threadIdx.x / L : q;  // the row of those side by side
  const uint32_t first = (w % W) * kPiece * (L == 64);
  const uint32_t left = first < a.width ? a.width - first : 0;
  const Piece<T, L, U, REST> piece(left);
  const uint64_t off = (uint64_t)first * T::kSize;
  Params<T, P> weight[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    fill_params<T, P>(1.0f, weight[j]);
    piece.params(a.weight, first, j, weight[j]);
  }
  float dw[U][N], db[U][N];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) dw[j][c] = db[j][c] = 0.0f;
  const double inv = 1.0 / (double)a.width;
  const bool lines = whole_lines(a.x, a.ld_x) && whole_lines(a.dout, a.ld_dout);
  // kGradBlocks workgroups go at once, the rows of their same turn side by side; as many
  // again take the rows after theirs
  const uint32_t before = blockIdx.x / kGradBlocks * kGradBlocks;
  const uint32_t at_once = gridDim.x - before < kGradBlocks ? gridDim.x - before : kGradBlocks;
  const uint64_t step = (uint64_t)at_once * G, first_row = (uint64_t)before * per;
  const uint64_t start = first_row + (blockIdx.x - before) * G;
  const uint64_t end = a.tokens - first_row < (uint64_t)at_once * per ? a.tokens : first_row + (uint64_t)at_once * per;
  u32x4 next_x[U] = {}, next_g[U] = {};
  auto load = [&](uint64_t t, const Piece<T, L, U, REST>& piece) {
    if (t >= end) return;
    if (L == 64 && lines) {
      piece.template load<true>(a.x + t * a.ld_x + off, next_x);
      piece.template load<true>(a.dout + t * a.ld_dout + off, next_g);
    } else {
      piece.template load<false>(a.x + t * a.ld_x + off, next_x);
      piece.template load<false>(a.dout + t * a.ld_dout + off, next_g);
    }
  };
  load(start + g, piece);
  uint32_t turn = 0;
  for (uint64_t s = start; s < end; s += step, turn ^= 1) {
    const uint64_t t = s + g;
    const bool live = t < end;
    // its places and masks are worked out again for every row: kept, they spill
    uint32_t left_here = left;
    if constexpr (REST) {
      left_here = __builtin_amdgcn_readfirstlane(left);
      asm volatile("" : "+s"(left_here));
    }
    const Piece<T, L, U, REST> piece(left_here);
    float h[U][N], up[U][N];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      unpack<T>(next_x[j], h[j]);
      unpack<T>(next_g[j], up[j]);
    }
    const float mean = live ? a.stats[2 * t] : 0.0f, rstd = live ? a.stats[2 * t + 1] : 0.0f;
    load(t + step, piece);
    double c1 = 0.0, c2 = 0.0;
    if (live) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) h[j][c] = (h[j][c] - mean) * rstd;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        // what is not of the row has no part: its h is -mean rstd, which may be infinite
        if (!piece.whole && !piece.has(j)) continue;
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) {
          if (c % (N / Params<T, P>::kWords ? N / Params<T, P>::kWords : 1) == 0)  // kept as it is stored
            asm volatile("" : "+v"(weight[j].w[c * Params<T, P>::kWords / N]));
          dw[j][c] = __builtin_fmaf(up[j][c], h[j][c], dw[j][c]);
          db[j][c] += up[j][c];
          up[j][c] = up[j][c] * param<T, P>(weight[j], c);
        }
        float d[N];
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) d[c] = piece.counted(j, c, up[j][c]);
        c1 += unit_sum<N>([&](uint32_t c) { return d[c]; });
        if constexpr (L == 16) {  // nor have the elements before a row of less than a unit
          float dh[N];
#pragma unroll
          for (uint32_t c = 0; c < N; ++c) dh[c] = piece.counted(j, c, h[j][c]);
          c2 += unit_dot<N>(d, dh);
        } else {
          c2 += unit_dot<N>(d, h[j]);
        }
      }
    }
    row_sum<L, W>(c1, c2, lds[turn]);
    const float m1 = (float)(c1 * inv), m2 = (float)(c2 * inv);
    u32x4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) h[j][c] = rstd * __builtin_fmaf(-h[j][c], m2, up[j][c] - m1);
      v[j] = pack<T>(h[j]);
    }
    if (live) piece.store(a.dx + t * a.ld_dx + off, v);
  }
  if (!a.dweight && !a.dbias) return;
  float* part = a.partial + (uint64_t)blockIdx.x * 2 * a.width;
  const bool alone = gridDim.x == 1 && !a.whole;  // nothing to join
  if constexpr (Q > 1) {
    // The sums of the rows that went side by side, in the order of a row's elements:
    // a thread adds up a column's in binary64.
    auto put = [&](const float (&f)[U][N], float (&to)[kPiece]) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (uint32_t c = 0; c < N; c += 4)
          *reinterpret_cast<u32x4*>(&to[(j * 64 + lane) * N + c]) =
              u32x4{__float_as_uint(f[j][c]), __float_as_uint(f[j][c + 1]), __float_as_uint(f[j][c + 2]), __float_as_uint(f[j][c + 3])};
    };
    auto columns = [&](const float (&from)[NW][kPiece], uint32_t col, void* grad, float* part) {
      const uint32_t own = col / N * N;
      if (own >= a.width) return;
      double sum[V];
#pragma unroll
      for (uint32_t c = 0; c < V; ++c) sum[c] = 0.0;
#pragma unroll
      for (uint32_t k = 0; k < Q; ++k)
#pragma unroll
        for (uint32_t sub = 0; sub < 64 / L; ++sub) {
          const float* f = &from[k * W + col / kRow][sub * kRow + col % kRow];
          if constexpr (V == 4) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(f);
#pragma unroll
            for (uint32_t c = 0; c < V; ++c) sum[c] += __uint_as_float(v[c]);
          } else {
            sum[0] += *f;
          }
        }
      // of the unit that ends where the row does another has the first elements
      const int32_t e = (int32_t)(REST && own + N > a.width ? col + a.width - N - own : col);
      if (V == 4 && !alone && e >= (int32_t)own) {
        u32x4 v;
#pragma unroll
        for (uint32_t c = 0; c < V; ++c) v[c] = __float_as_uint((float)sum[c]);
        return st_unit<false>(reinterpret_cast<char*>(part + e), v);
      }
#pragma unroll
      for (uint32_t c = 0; c < V; ++c) {
        const int32_t at = e + (int32_t)c;
        if (at < (int32_t)own) continue;
        if (!alone) part[at] = (float)sum[c];
        else if (grad) put_grad(grad, a.grad_bf16, a.accumulate, at, sum[c]);
      }
    };
    if constexpr (kBoth) {
      put(dw, join[0][w]);
      put(db, join[1][w]);
      __syncthreads();
      const uint32_t i = threadIdx.x;
      if (i < kCols) columns(join[0], i, a.dweight, part);
      else if (i < 2 * kCols) columns(join[1], i - kCols, a.dbias, part + a.width);
    } else {
      // one after the other, four columns at a time (both at once and by single columns
      // took 128 KiB of LDS and 8192 rows of 5003 bf16 4 us more of 60)
      put(dw, join[0][w]);
      __syncthreads();
#pragma unroll
      for (uint32_t i = V * threadIdx.x; i < kCols; i += V * 64 * NW) columns(join[0], i, a.dweight, part);
      __syncthreads();
      put(db, join[0][w]);
      __syncthreads();
#pragma unroll
      for (uint32_t i = V * threadIdx.x; i < kCols; i += V * 64 * NW) columns(join[0], i, a.dbias, part + a.width);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (!piece.has(j)) continue;
    const int64_t e = (int32_t)(first + (uint32_t)piece.at(j));
    if (alone) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        if (c < piece.skip(j)) continue;
        if (a.dweight) put_grad(a.dweight, a.grad_bf16, a.accumulate, e + c, dw[j][c]);
        if (a.dbias) put_grad(a.dbias, a.grad_bf16, a.accumulate, e + c, db[j][c]);
      }
    } else {
      st_sums<N>(part + e, piece.skip(j), dw[j]);
      st_sums<N>(part + a.width + e, piece.skip(j), db[j]);
    }
  }
}

// Rows wider than the above holds: the two sums of each first, sum g / width and sum
// g h / width, a row a workgroup, and then dx and the sums over tokens by columns,
// which reads both streams again: 2048 x 16384 f32 115 us, half of what reading them
// once would allow.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void layer_norm_row_sums_kernel(const LayerNormBackwardArgs a) {
  constexpr int NW = 16;
  constexpr uint32_t N = kUnit<T>, kStep = 64u * NW * N;
  __shared__ double lds[NW][2];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const float mean = a.stats[2 * t], rstd = a.stats[2 * t + 1];
    double c1 = 0.0, c2 = 0.0;
    for (uint64_t e0 = (uint64_t)w * 64 * N; e0 < a.width; e0 += kStep) {
      const uint32_t left = a.width - (uint32_t)e0, e = (uint32_t)e0 + lane * N;
      u32x4 vx[1], vg[1];
      ld_piece<T, 1, false>(a.x + t * a.ld_x + e0 * T::kSize, left, vx);
      ld_piece<T, 1, false>(a.dout + t * a.ld_dout + e0 * T::kSize, left, vg);
      float h[N], up[N];
      unpack<T>(vx[0], h);
      unpack<T>(vg[0], up);
      Params<T, P> weight;
      if (a.weight && e < a.width) ld_params<T, P>(a.weight, e, a.width, weight);
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        h[c] = lane * N + c < left ? (h[c] - mean) * rstd : 0.0f;
        if (a.weight && e < a.width) up[c] = up[c] * param<T, P>(weight, c);
      }
      c1 += unit_sum<N>([&](uint32_t c) { return up[c]; });
      c2 += unit_sum<N>([&](uint32_t c) { return up[c] * h[c]; });
    }
    row_sum<64, NW>(c1, c2, lds);
    if (threadIdx.x == 0) {
      a.row_sums[2 * t] = (float)(c1 / (double)a.width);
      a.row_sums[2 * t + 1] = (float)(c2 / (double)a.width);
    }
    __syncthreads();  // lds is free
  }
}

// Wide rows by columns: a wave takes 64 units of `per` rows.
template <typename T, typename P>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(const LayerNormBackwardArgs a, const uint32_t per) {
  constexpr uint32_t N = kUnit<T>;
  const uint32_t lane = threadIdx.x & 63u;
  const uint64_t e0 = ((uint64_t)blockIdx.x * 4 + wave_id()) * 64 * N;
  if (e0 >= a.width) return;
  const uint32_t left = a.width - (uint32_t)e0, e = (uint32_t)e0 + lane * N;
  Params<T, P> weight;
  if (a.weight && e < a.width) ld_params<T, P>(a.weight, e, a.width, weight);
  const uint64_t t0 = (uint64_t)blockIdx.y * per, end = a.tokens - t0 < per ? a.tokens : t0 + per;
  double sum_w[N], sum_b[N];
#pragma unroll
  for (uint32_t c = 0; c < N; ++c) sum_w[c] = sum_b[c] = 0.0;
  for (uint64_t r0 = t0; r0 < end; r0 += kSumTokens) {
    const uint64_t r1 = end - r0 < kSumTokens ? end : r0 + kSumTokens;
    float dw[N], db[N];
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) dw[c] = db[c] = 0.0f;
    for (uint64_t t = r0; t < r1; ++t) {
      u32x4 vx[1], vg[1];
      ld_piece<T, 1, true>(a.x + t * a.ld_x + e0 * T::kSize, left, vx);
      ld_piece<T, 1, true>(a.dout + t * a.ld_dout + e0 * T::kSize, left, vg);
      const float mean = a.stats[2 * t], rstd = a.stats[2 * t + 1];
      const float m1 = a.row_sums[2 * t], m2 = a.row_sums[2 * t + 1];
      float h[N], up[N];
      unpack<T>(vx[0], h);
      unpack<T>(vg[0], up);
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        h[c] = (h[c] - mean) * rstd;
        dw[c] = __builtin_fmaf(up[c], h[c], dw[c]);
        db[c] += up[c];
        if (a.weight) up[c] = up[c] * param<T, P>(weight, c);
        h[c] = rstd * __builtin_fmaf(-h[c], m2, up[c] - m1);
      }
      vx[0] = pack<T>(h);
      st_piece<T, 1, true>(a.dx + t * a.ld_dx + e0 * T::kSize, left, vx);
    }
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) sum_w[c] += dw[c], sum_b[c] += db[c];
  }
  if (!a.partial) return;
  float* part = a.partial + (uint64_t)blockIdx.y * 2 * a.width;
#pragma unroll
  for (uint32_t c = 0; c < N; ++c) {
    if (e + c >= a.width) continue;
    part[e + c] = (float)sum_w[c];
    part[(uint64_t)a.width + e + c] = (float)sum_b[c];
  }
}

// dweight and dbias from the partial sums: 64 columns a workgroup, its waves
// taking every 16th partial sum.  256 of 4096 columns each (8.4 MB) 4.2 us.  Those of
// a call's several launches go through its sums in binary64.
constexpr int kJoinWaves = 16;
constexpr uint64_t kJoinGrid = 1u << 20;
__global__ __launch_bounds__(64 * kJoinWaves) void layer_norm_join_kernel(const LayerNormBackwardArgs a, const uint32_t blocks,
                                                                          const bool later, const bool last) {
  __shared__ double lds[kJoinWaves][64];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  const bool second = blockIdx.y != 0;
  void* out = second ? a.dbias : a.dweight;
  if (!out) return;
  for (uint64_t c0 = (uint64_t)blockIdx.x * 64; c0 < a.width; c0 += (uint64_t)gridDim.x * 64) {
    const uint64_t col = c0 + lane, at = (second ? a.width : 0) + col;
    double sum = 0.0;
    if (col < a.width) {
      const float* p = a.partial + at;
#pragma unroll 8
      for (uint32_t b = w; b < blocks; b += kJoinWaves) sum += p[(uint64_t)b * 2 * a.width];
    }
    lds[w][lane] = sum;
    __syncthreads();
    if (w == 0 && col < a.width) {
#pragma unroll
      for (int i = 1; i < kJoinWaves; ++i) sum += lds[i][lane];
      if (later) sum += a.whole[at];
      if (last) put_grad(out, a.grad_bf16, a.accumulate, col, sum);
      else a.whole[at] = sum;
    }
    __syncthreads();  // lds is free
  }
}

uint32_t cus() {
  const int n = device_cu_count();
  return n > 0 ? (uint32_t)n : 1;
}

// The rows of a workgroup, one after another: its parameters are loaded once for
// them.
template <typename T, typename P, int L, int W, int U>
void layer_norm_in(const LayerNormArgs& a, hipStream_t stream) {
  constexpr int NW = W > kNormWaves ? W : kNormWaves, G = NW / W * (64 / L);
  const uint32_t kib = (a.width * T::kSize * G + 1023) / 1024;  // of the rows side by side
  uint32_t per = G * (kib > 16 ? 4 : (32 + kib - 1) / kib);
  const uint64_t fill = (uint64_t)cus() * 4;
  while (per > G && (a.tokens + per - 1) / per < fill) per /= 2;
  const uint64_t most = (uint64_t)per << 22;  // rows of a launch
  LayerNormArgs c = a;
  for (uint64_t t = 0; t < a.tokens; t += most) {
    c.tokens = a.tokens - t < most ? a.tokens - t : most;
    c.x = a.x + t * a.ld_x;
    c.out = a.out + t * a.ld_out;
    c.stats = a.stats ? a.stats + 2 * t : nullptr;
    const dim3 grid((uint32_t)((c.tokens + per - 1) / per)), block(64 * NW);
    if (a.width % kUnit<T> == 0) hipLaunchKernelGGL((layer_norm_kernel<T, P, L, W, U, false>), grid, block, 0, stream, c, per);
    else hipLaunchKernelGGL((layer_norm_kernel<T, P, L, W, U, true>), grid, block, 0, stream, c, per);
  }
}

// The narrowest shape that holds a row, in units of 1 KiB (64 lanes), and of those of
// one size the one with the fewest waves whose registers leave 3 of them a SIMD: 32768
// x 4096 bf16 by 2 waves of 4 units 84 us, 4 of 2 90, 8 of 1 98, 1 of 8 94; 16384 x
// 8192 by 4 of 4 84, 2 of 8 97, 8 of 2 94.
template <typename T, typename P>
void layer_norm_any(const LayerNormArgs& a, hipStream_t stream) {
  const uint64_t bytes = (uint64_t)a.width * T::kSize, kib = (bytes + 1023) / 1024;
  if (bytes <= 256) layer_norm_in<T, P, 16, 1, 1>(a, stream);
  else if (bytes <= 512) layer_norm_in<T, P, 32, 1, 1>(a, stream);
  else if (kib <= 1) layer_norm_in<T, P, 64, 1, 1>(a, stream);
  else if (kib <= 2) layer_norm_in<T, P, 64, 1, 2>(a, stream);
  else if (kib <= 4) layer_norm_in<T, P, 64, 1, 4>(a, stream);
  else if (kib <= 8) layer_norm_in<T, P, 64, 2, 4>(a, stream);
  else if (kib <= 16) layer_norm_in<T, P, 64, 4, 4>(a, stream);
  else if (kib <= 32) layer_norm_in<T, P, 64, 8, 4>(a, stream);
  else if (kib <= kHeldKib<T, P>) {
    if constexpr (kHeldKib<T, P> > 32) layer_norm_in<T, P, 64, 16, 4>(a, stream);
  } else {
    const uint64_t most = (uint64_t)cus() * 2;
    hipLaunchKernelGGL((layer_norm_wide_kernel<T, P>), dim3((uint32_t)(a.tokens < most ? a.tokens : most)), dim3(1024),
                       0, stream, a);
  }
}

void layer_norm_join(const LayerNormBackwardArgs& a, uint64_t blocks, bool later, bool last, hipStream_t stream) {
  const uint64_t cols = ((uint64_t)a.width + 63) / 64;
  hipLaunchKernelGGL(layer_norm_join_kernel, dim3((uint32_t)(cols < kJoinGrid ? cols : kJoinGrid), 2), dim3(64 * kJoinWaves),
                     0, stream, a, (uint32_t)blocks, later, last);
}

template <typename T, typename P, int L, int W, int U>
void layer_norm_backward_in(const LayerNormBackwardArgs& a, const LayerNormShape& s, hipStream_t stream) {
  const uint64_t most = s.blocks * s.per;  // tokens of a launch
  LayerNormBackwardArgs c = a;
  for (uint64_t t = 0; t < a.tokens; t += most) {
    c.tokens = a.tokens - t < most ? a.tokens - t : most;
    c.dout = a.dout + t * a.ld_dout;
    c.x = a.x + t * a.ld_x;
    c.stats = a.stats + 2 * t;
    c.dx = a.dx + t * a.ld_dx;
    const uint64_t blocks = (c.tokens + s.per - 1) / s.per;
    const dim3 grid((uint32_t)blocks), block(64 * kGradWaves);
    if (a.width % kUnit<T> == 0) hipLaunchKernelGGL((layer_norm_backward_kernel<T, P, L, W, U, false>), grid, block, 0, stream, c, s.per);
    else hipLaunchKernelGGL((layer_norm_backward_kernel<T, P, L, W, U, true>), grid, block, 0, stream, c, s.per);
    if ((a.dweight || a.dbias) && (blocks != 1 || a.whole))
      layer_norm_join(c, blocks, t != 0, a.tokens - t <= most, stream);
  }
}

template <typename T, typename P>
void layer_norm_backward_any(const LayerNormBackwardArgs& a, const LayerNormShape& s, hipStream_t stream) {
  const uint64_t bytes = (uint64_t)a.width * T::kSize, kib = (bytes + 1023) / 1024;
  if (s.row_sums) {
    const uint64_t most = (uint64_t)cus() * 2;
    hipLaunchKernelGGL((layer_norm_row_sums_kernel<T, P>), dim3((uint32_t)(a.tokens < most ? a.tokens : most)),
                       dim3(1024), 0, stream, a);
    hipLaunchKernelGGL((layer_norm_columns_kernel<T, P>), dim3((uint32_t)((kib + 3) / 4), (uint32_t)s.blocks), dim3(256), 0,
                       stream, a, s.per);
    if (a.dweight || a.dbias) layer_norm_join(a, s.blocks, false, true, stream);
  } else if (bytes <= 256) layer_norm_backward_in<T, P, 16, 1, 1>(a, s, stream);
  else if (bytes <= 512) layer_norm_backward_in<T, P, 32, 1, 1>(a, s, stream);
  else if (kib <= 1) layer_norm_backward_in<T, P, 64, 1, 1>(a, s, stream);
  else if (kib <= 2) layer_norm_backward_in<T, P, 64, 1, 2>(a, s, stream);
  else if (kib <= 4) layer_norm_backward_in<T, P, 64, 2, 2>(a, s, stream);
  else if (kib <= 8) layer_norm_backward_in<T, P, 64, 4, 2>(a, s, stream);
  else if (kib <= 16) layer_norm_backward_in<T, P, 64, 8, 2>(a, s, stream);
  else layer_norm_backward_in<T, P, 64, 16, 2>(a, s, stream);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, bool bf16, bool param_bf16, hipStream_t stream) {
  if (bf16) param_bf16 ? layer_norm_any<BF16, BF16>(a, stream) : layer_norm_any<BF16, F32>(a, stream);
  else param_bf16 ? layer_norm_any<F32, BF16>(a, stream) : layer_norm_any<F32, F32>(a, stream);
  return hipGetLastError();
}

LayerNormShape layer_norm_shape(uint64_t tokens, uint64_t width, uint64_t esize) {
  const uint64_t bytes = width * esize;
  LayerNormShape s{0, kSumTokens, bytes > kHeldBackwardKib * 1024, false};
  if (tokens == 0) return s;
  // rows side by side in a workgroup of layer_norm_backward_kernel, and how many
  // workgroups they are dealt out to
  const uint64_t kib = (bytes + 1023) / 1024;
  uint64_t rows = 1, most = kGradBlocks;
  if (s.row_sums) most = kGradBlocks * 16 / kib + 1;
  else rows = bytes <= 256 ? 64 : bytes <= 512 ? 32 : kib <= 2 ? 16 : kib <= 4 ? 8 : kib <= 8 ? 4 : kib <= 16 ? 2 : 1;
  uint64_t turns = (tokens + rows * most - 1) / (rows * most);
  // one workgroup has no other's sums to wait for: the join's launch is saved
  if (tokens <= rows * kAloneTurns) turns = (tokens + rows - 1) / rows;
  // more tokens than those have turns for: as many workgroups again, and as even
  // (20000 rows of 6000 bf16 in turns of 32, 313 workgroups of one a CU, 180 us;
  // evenly 137), while their partial sums are few; then several launches, so that the
  // scratch does not grow with the tokens (131072 rows of 8192 bf16 in one 1150 us and
  // 134 MB of partial sums, in four 1075; 20000 of 5999 in two 155, in one 147).  A
  // workgroup of layer_norm_columns_kernel takes any number of tokens.
  uint64_t launches = 1;
  if (turns > kSumTokens && !s.row_sums) {
    const uint64_t groups = (turns + kSumTokens - 1) / kSumTokens;
    uint64_t again = kGradPartial / (most * 2 * width * 4);
    again = again < 1 ? 1 : again > kGradAgain ? kGradAgain : again;
    again = again < groups ? again : groups;
    launches = (groups + again - 1) / again;
    most *= again;
    turns = (tokens + rows * most * launches - 1) / (rows * most * launches);
  }
  s.runs = launches > 1;
  s.per = (uint32_t)(rows * turns);
  s.blocks = s.runs ? most : (tokens + s.per - 1) / s.per;
  return s;
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, const LayerNormShape& s, bool bf16,
                                      bool param_bf16, hipStream_t stream) {
  if (a.tokens == 0) layer_norm_join(a, 0, false, true, stream);  // zeros
  else if (bf16) param_bf16 ? layer_norm_backward_any<BF16, BF16>(a, s, stream) : layer_norm_backward_any<BF16, F32>(a, s, stream);
  else param_bf16 ? layer_norm_backward_any<F32, BF16>(a, s, stream) : layer_norm_backward_any<F32, F32>(a, s, stream);
  return hipGetLastError();
}

}  // namespace snac
