// layernorm.hip -- layer norm and its gradients (snac_layer_norm,
// snac_layer_norm_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

// The widest rows that a workgroup holds in registers: 16 waves of 64 lanes of 4
// units, or 2 where the gradient's sums over tokens are held too.
constexpr uint64_t kHeldKib = 64, kHeldBackwardKib = 32;
constexpr uint32_t kSumTokens = 32;  // binary32 sums over tokens go no further

// 16 bytes' worth of T elements' parameters of type P, raw.
template <typename T, typename P>
struct Params {
  static constexpr int kWords = kUnit<T> * P::kSize / 4;
  uint32_t w[kWords];
};
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

// Parameters of the kUnit<T> elements from `e` on; those past `width` read as 0.
template <typename T, typename P>
__device__ __forceinline__ void ld_params(const char* p, uint32_t e, uint32_t width, Params<T, P>& r) {
  constexpr uint32_t N = kUnit<T>;
  const char* at = p + (uint64_t)e * P::kSize;
#pragma unroll
  for (int c = 0; c < Params<T, P>::kWords; ++c) r.w[c] = 0;
  if (e + N <= width) {
    if constexpr (Params<T, P>::kWords == 2) {
      const u32x2_a2 v = *(global_ptr<const u32x2_a2>)(at);
      r.w[0] = v[0], r.w[1] = v[1];
    } else {
#pragma unroll
      for (int u = 0; u < Params<T, P>::kWords / 4; ++u) {
        const u32x4 v = ld_unit<false>(at + 16 * u);
#pragma unroll
        for (int c = 0; c < 4; ++c) r.w[4 * u + c] = v[c];
      }
    }
  } else {
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
      if (e + i >= width) continue;
      if constexpr (P::kSize == 4) r.w[i] = *(global_ptr<const uint32_t>)(at + 4 * i);
      else r.w[i / 2] |= (uint32_t)*(global_ptr<const uint16_t>)(at + 2 * i) << (16 * (i & 1));
    }
  }
}
template <typename T, typename P>
__device__ __forceinline__ float param(const Params<T, P>& r, uint32_t i) {
  if constexpr (P::kSize == 4) return __uint_as_float(r.w[i]);
  else return i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
}

// Sums of a and b over the W waves of a row (`lds`: room for two numbers of each
// of the workgroup's waves, not used by the call before), in every lane.
template <int W, int NW>
__device__ __forceinline__ void row_sum(double& a, double& b, double (*lds)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    const uint32_t lane = threadIdx.x & 63u, w = wave_id(), w0 = w / W * W;
    if (lane == 0) lds[w][0] = a, lds[w][1] = b;
    __syncthreads();
    if constexpr (W == 16) {
      a = lanes_sum<16>(lds[lane & 15][0]);
      b = lanes_sum<16>(lds[lane & 15][1]);
    } else {
      a = lds[w0][0], b = lds[w0][1];
#pragma unroll
      for (int i = 1; i < W; ++i) a += lds[w0 + i][0], b += lds[w0 + i][1];
    }
  }
}
template <int W, int NW>
__device__ __forceinline__ double row_sum(double a, double (*lds)[2]) {
  a = wave_sum(a);
  if constexpr (W > 1) {
    const uint32_t lane = threadIdx.x & 63u, w = wave_id(), w0 = w / W * W;
    if (lane == 0) lds[w][0] = a;
    __syncthreads();
    if constexpr (W == 16) {
      a = lanes_sum<16>(lds[lane & 15][0]);
    } else {
      a = lds[w0][0];
#pragma unroll
      for (int i = 1; i < W; ++i) a += lds[w0 + i][0];
    }
  }
  return a;
}

// 1 / sqrt(v), off by a few of binary64's last bits: the hardware's estimate
// (2^-23 or better) and one step of Newton's iteration.
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

// ------------------------------------------------------------------ forward

// What a row's sums give.  The first sum over x is off by its own size's
// roundings, which matter where the row is far from 0 and hardly varies: so the
// second pass sums the distances d from that mean `near` too, and d - rest is
// as good as x - mean with the exact mean.
struct Moments {
  float mean, rest, rstd;
  __device__ __forceinline__ Moments(float near, double mean_d, double mean_dd, float eps) {
    const double var = mean_dd - mean_d * mean_d;
    rest = (float)mean_d;
    mean = (float)((double)near + mean_d);
    rstd = inverse_root((var < 0.0 ? 0.0 : var) + (double)eps);
  }
};

constexpr int kNormWaves = 4;  // of a workgroup whose rows take up to 4 waves

// W waves a row, U units a lane: the row stays in registers, so that it is read
// once although its mean is needed before its variance and that before the
// result.
template <typename T, typename P, int W, int U>
__global__ __launch_bounds__(64 * (W > kNormWaves ? W : kNormWaves)) void layer_norm_kernel(const LayerNormArgs a) {
  constexpr int NW = W > kNormWaves ? W : kNormWaves, G = NW / W;
  constexpr uint32_t N = kUnit<T>;
  __shared__ double lds[2][NW][2];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id(), g = w / W;
  const uint32_t first = (w % W) * 64u * U * N;  // the wave's piece of a row
  const uint32_t left = first < a.width ? a.width - first : 0;
  // the parameters are kept, and the next row is loaded while this one is worked
  // on, where registers allow it
  constexpr bool kAhead = W * U < 64;
  Params<T, P> weight[U], bias[U];
  auto params = [&](int j) {
    const uint32_t e = first + (j * 64u + lane) * N;
    if (a.weight) ld_params<T, P>(a.weight, e, a.width, weight[j]);
    if (a.bias) ld_params<T, P>(a.bias, e, a.width, bias[j]);
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < U; ++j) params(j);
  }
  const double inv = 1.0 / (double)a.width;
  const uint64_t step = (uint64_t)gridDim.x * G;
  uint64_t t = (uint64_t)blockIdx.x * G + g;
  u32x4 next[U] = {};
  auto load = [&](uint64_t row) {
    if (row < a.tokens) ld_piece<T, U, true>(a.x + row * a.ld_x + (uint64_t)first * T::kSize, left, next);
  };
  if constexpr (kAhead) load(t);
  // every wave of the workgroup goes round as often as its first
  for (uint64_t t0 = (uint64_t)blockIdx.x * G; t0 < a.tokens; t0 += step, t += step) {
    if constexpr (!kAhead) load(t);
    u32x4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = next[j];
    if constexpr (kAhead) load(t + step);
    float f[U][N];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      unpack<T>(v[j], f[j]);
      sum += unit_sum<N>([&](uint32_t c) { return f[j][c]; });
    }
    const float near = (float)(row_sum<W, NW>(sum, lds[0]) * inv);
    double sd = 0.0, sq = 0.0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t e = (j * 64u + lane) * N;  // within the wave's piece
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) f[j][c] = e + c < left ? f[j][c] - near : 0.0f;
      sd += unit_sum<N>([&](uint32_t c) { return f[j][c]; });
      sq += unit_sum<N>([&](uint32_t c) { return f[j][c] * f[j][c]; });
    }
    row_sum<W, NW>(sd, sq, lds[1]);
    const Moments m(near, sd * inv, sq * inv, a.eps);
    if (t < a.tokens) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if constexpr (!kAhead) params(j);
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) {
          f[j][c] = (f[j][c] - m.rest) * m.rstd;
          if (a.weight) f[j][c] = f[j][c] * param<T, P>(weight[j], c);
          if (a.bias) f[j][c] = f[j][c] + param<T, P>(bias[j], c);
        }
        v[j] = pack<T>(f[j]);
      }
      st_piece<T, U, true>(a.out + t * a.ld_out + (uint64_t)first * T::kSize, left, v);
      if (a.stats && w % W == 0 && lane == 0) {
        a.stats[2 * t] = m.mean;
        a.stats[2 * t + 1] = m.rstd;
      }
    }
  }
}

// Rows of any width by one workgroup of 16 waves, which reads them three times.
template <typename T, typename P>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(const LayerNormArgs a) {
  constexpr int NW = 16;
  constexpr uint32_t N = kUnit<T>, kStep = 64u * NW * N;
  __shared__ double lds[2][NW][2];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  const double inv = 1.0 / (double)a.width;
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
    const float near = (float)(row_sum<NW, NW>(sum, lds[0]) * inv);
    row([&](uint32_t, uint32_t left, float (&u)[N]) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) u[c] = lane * N + c < left ? u[c] - near : 0.0f;
      sd += unit_sum<N>([&](uint32_t c) { return u[c]; });
      sq += unit_sum<N>([&](uint32_t c) { return u[c] * u[c]; });
    });
    row_sum<NW, NW>(sd, sq, lds[1]);
    const Moments m(near, sd * inv, sq * inv, a.eps);
    row([&](uint32_t e0, uint32_t left, float (&u)[N]) {
      Params<T, P> weight, bias;
      const uint32_t e = e0 + lane * N;
      if (a.weight && e < a.width) ld_params<T, P>(a.weight, e, a.width, weight);
      if (a.bias && e < a.width) ld_params<T, P>(a.bias, e, a.width, bias);
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) {
        u[c] = ((u[c] - near) - m.rest) * m.rstd;
        if (a.weight) u[c] = u[c] * param<T, P>(weight, c);
        if (a.bias) u[c] = u[c] + param<T, P>(bias, c);
      }
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

constexpr int kGradWaves = 8;  // of a workgroup whose rows take up to 8 waves
constexpr uint32_t kGradBlocks = 512;

// N binary32 values to `p`, the first `left` of them.
template <uint32_t N>
__device__ __forceinline__ void st_sums(float* p, uint32_t left, const float (&f)[N]) {
  char* at = reinterpret_cast<char*>(p);
#pragma unroll
  for (uint32_t c = 0; c < N; c += 4) {
    const u32x4 v = {__float_as_uint(f[c]), __float_as_uint(f[c + 1]), __float_as_uint(f[c + 2]), __float_as_uint(f[c + 3])};
    if (c + 4 <= left) st_unit<false>(at + 4 * c, v);
    else if (c < left) st_part<F32>(at + 4 * c, v, left - c);
  }
}

// W waves a row, U units a lane, G rows at a time; the sums over tokens stay in
// registers and leave as one partial sum a workgroup.
template <typename T, typename P, int W, int U>
__global__ __launch_bounds__(64 * (W > kGradWaves ? W : kGradWaves)) void layer_norm_backward_kernel(
    const LayerNormBackwardArgs a, const uint32_t per) {
  constexpr int NW = W > kGradWaves ? W : kGradWaves, G = NW / W;
  constexpr uint32_t N = kUnit<T>, kPiece = 64u * U * N;
  __shared__ double lds[2][NW][2];
  __shared__ __align__(16) float join[G > 1 ? G / 2 * W : 1][2][G > 1 ? kPiece : 1];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id(), g = w / W;
  const uint32_t first = (w % W) * kPiece;
  const uint32_t left = first < a.width ? a.width - first : 0;
  const uint64_t off = (uint64_t)first * T::kSize;
  Params<T, P> weight[U];
  if (a.weight) {
#pragma unroll
    for (int j = 0; j < U; ++j) ld_params<T, P>(a.weight, first + (j * 64u + lane) * N, a.width, weight[j]);
  }
  float dw[U][N], db[U][N];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) dw[j][c] = db[j][c] = 0.0f;
  const float inv = (float)(1.0 / (double)a.width);
  const uint64_t t0 = (uint64_t)blockIdx.x * per;
  const uint64_t end = a.tokens - t0 < per ? a.tokens : t0 + per;
  u32x4 next_x[U] = {}, next_g[U] = {};
  auto load = [&](uint64_t t) {
    ld_piece<T, U, true>(a.x + t * a.ld_x + off, left, next_x);
    ld_piece<T, U, true>(a.dout + t * a.ld_dout + off, left, next_g);
  };
  if (t0 + g < end) load(t0 + g);
  uint32_t turn = 0;
  for (uint64_t s = t0; s < end; s += G, turn ^= 1) {
    const uint64_t t = s + g;
    const bool live = t < end;
    u32x4 vx[U], vg[U];
#pragma unroll
    for (int j = 0; j < U; ++j) vx[j] = next_x[j], vg[j] = next_g[j];
    const float mean = live ? a.stats[2 * t] : 0.0f, rstd = live ? a.stats[2 * t + 1] : 0.0f;
    if (t + G < end) load(t + G);
    double c1 = 0.0, c2 = 0.0;
    float h[U][N], up[U][N];
    if (live) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        unpack<T>(vx[j], h[j]);
        unpack<T>(vg[j], up[j]);
        const uint32_t e = (j * 64u + lane) * N;
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) {
          h[j][c] = e + c < left ? (h[j][c] - mean) * rstd : 0.0f;
          dw[j][c] = __builtin_fmaf(up[j][c], h[j][c], dw[j][c]);
          db[j][c] += up[j][c];
          if (a.weight) up[j][c] = up[j][c] * param<T, P>(weight[j], c);
        }
        c1 += unit_sum<N>([&](uint32_t c) { return up[j][c]; });
        c2 += unit_sum<N>([&](uint32_t c) { return up[j][c] * h[j][c]; });
      }
    }
    row_sum<W, NW>(c1, c2, lds[turn]);
    if (!live) continue;
    const float m1 = (float)c1 * inv, m2 = (float)c2 * inv;
#pragma unroll
    for (int j = 0; j < U; ++j) {
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) h[j][c] = rstd * __builtin_fmaf(-h[j][c], m2, up[j][c] - m1);
      vx[j] = pack<T>(h[j]);
    }
    st_piece<T, U, true>(a.dx + t * a.ld_dx + off, left, vx);
  }
  if (!a.partial) return;
  // the rows that went beside each other: the upper half of them to the lower
  if constexpr (G > 1) {
#pragma unroll
    for (uint32_t half = G / 2; half > 0; half /= 2) {
      __syncthreads();
      if (g >= half && g < 2 * half) {
        float(&to)[2][kPiece] = join[w - half * W];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (uint32_t c = 0; c < N; c += 4) {
            *reinterpret_cast<u32x4*>(&to[0][(j * N + c) * 64 + lane * 4]) =
                u32x4{__float_as_uint(dw[j][c]), __float_as_uint(dw[j][c + 1]), __float_as_uint(dw[j][c + 2]),
                      __float_as_uint(dw[j][c + 3])};
            *reinterpret_cast<u32x4*>(&to[1][(j * N + c) * 64 + lane * 4]) =
                u32x4{__float_as_uint(db[j][c]), __float_as_uint(db[j][c + 1]), __float_as_uint(db[j][c + 2]),
                      __float_as_uint(db[j][c + 3])};
          }
      }
      __syncthreads();
      if (g < half) {
        const float(&from)[2][kPiece] = join[w];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (uint32_t c = 0; c < N; c += 4) {
            const u32x4 p = *reinterpret_cast<const u32x4*>(&from[0][(j * N + c) * 64 + lane * 4]);
            const u32x4 q = *reinterpret_cast<const u32x4*>(&from[1][(j * N + c) * 64 + lane * 4]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dw[j][c + i] += __uint_as_float(p[i]);
              db[j][c + i] += __uint_as_float(q[i]);
            }
          }
      }
    }
  }
  if (g != 0) return;
  float* part = a.partial + (uint64_t)blockIdx.x * 2 * a.width;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t e = first + (j * 64u + lane) * N;
    if (e >= a.width) continue;
    st_sums<N>(part + e, a.width - e, dw[j]);
    st_sums<N>(part + a.width + e, a.width - e, db[j]);
  }
}

// Sums of one row of any width, by one workgroup: sum g / width and
// sum g h / width.
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
    row_sum<NW, NW>(c1, c2, lds);
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
  const uint64_t blocks = (a.tokens + per - 1) / per;
  for (uint64_t b = blockIdx.y; b < blocks; b += gridDim.y) {
    const uint64_t t0 = b * per, end = a.tokens - t0 < per ? a.tokens : t0 + per;
    float dw[N], db[N];
#pragma unroll
    for (uint32_t c = 0; c < N; ++c) dw[c] = db[c] = 0.0f;
    for (uint64_t t = t0; t < end; ++t) {
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
    if (!a.partial) continue;
    float* part = a.partial + b * 2 * a.width;
    if (e >= a.width) continue;
    st_sums<N>(part + e, a.width - e, dw);
    st_sums<N>(part + a.width + e, a.width - e, db);
  }
}

// dweight and dbias from the partial sums: 64 columns a workgroup, its waves
// taking every 16th partial sum.
constexpr int kJoinWaves = 16;
template <typename GT>
__global__ __launch_bounds__(64 * kJoinWaves) void layer_norm_join_kernel(const LayerNormBackwardArgs a, const uint32_t blocks) {
  __shared__ double lds[kJoinWaves][64];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  const uint64_t col = (uint64_t)blockIdx.x * 64 + lane;
  const bool second = blockIdx.y != 0;
  char* out = static_cast<char*>(second ? a.dbias : a.dweight);
  if (!out) return;
  double sum = 0.0;
  if (col < a.width) {
    const float* p = a.partial + (second ? a.width : 0) + col;
#pragma unroll 8
    for (uint32_t b = w; b < blocks; b += kJoinWaves) sum += p[(uint64_t)b * 2 * a.width];
  }
  lds[w][lane] = sum;
  __syncthreads();
  if (w != 0 || col >= a.width) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) sum += lds[i][lane];
  char* at = out + col * GT::kSize;
  if (a.accumulate) sum += load_elem<GT>(at);
  store_elem<GT>(at, (float)sum);
}

uint32_t cus() {
  const int n = device_cu_count();
  return n > 0 ? (uint32_t)n : 1;
}

template <typename T, typename P, int W, int U>
void layer_norm_in(const LayerNormArgs& a, hipStream_t stream) {
  constexpr int NW = W > kNormWaves ? W : kNormWaves, G = NW / W;
  const uint64_t want = (a.tokens + G - 1) / G, most = (uint64_t)cus() * 32 / NW;
  hipLaunchKernelGGL((layer_norm_kernel<T, P, W, U>), dim3((uint32_t)(want < most ? want : most)), dim3(64 * NW), 0,
                     stream, a);
}

// The narrowest shape that holds a row, in units of 1 KiB (64 lanes).
template <typename T, typename P>
void layer_norm_any(const LayerNormArgs& a, hipStream_t stream) {
  const uint64_t kib = ((uint64_t)a.width * T::kSize + 1023) / 1024;
  if (kib <= 1) layer_norm_in<T, P, 1, 1>(a, stream);
  else if (kib <= 2) layer_norm_in<T, P, 1, 2>(a, stream);
  else if (kib <= 4) layer_norm_in<T, P, 1, 4>(a, stream);
  else if (kib <= 8) layer_norm_in<T, P, 4, 2>(a, stream);
  else if (kib <= 16) layer_norm_in<T, P, 4, 4>(a, stream);
  else if (kib <= 32) layer_norm_in<T, P, 16, 2>(a, stream);
  else if (kib <= kHeldKib) layer_norm_in<T, P, 16, 4>(a, stream);
  else {
    const uint64_t most = (uint64_t)cus() * 2;
    hipLaunchKernelGGL((layer_norm_wide_kernel<T, P>), dim3((uint32_t)(a.tokens < most ? a.tokens : most)), dim3(1024),
                       0, stream, a);
  }
}

template <typename T, typename P, int W, int U>
void layer_norm_backward_in(const LayerNormBackwardArgs& a, const LayerNormShape& s, hipStream_t stream) {
  constexpr int NW = W > kGradWaves ? W : kGradWaves;
  hipLaunchKernelGGL((layer_norm_backward_kernel<T, P, W, U>), dim3(s.blocks), dim3(64 * NW), 0, stream, a, s.per);
}

template <typename T, typename P>
void layer_norm_backward_any(const LayerNormBackwardArgs& a, const LayerNormShape& s, hipStream_t stream) {
  const uint64_t kib = ((uint64_t)a.width * T::kSize + 1023) / 1024;
  if (s.row_sums) {
    const uint64_t most = (uint64_t)cus() * 2;
    hipLaunchKernelGGL((layer_norm_row_sums_kernel<T, P>), dim3((uint32_t)(a.tokens < most ? a.tokens : most)),
                       dim3(1024), 0, stream, a);
    const uint32_t y = s.blocks < 32768 ? s.blocks : 32768;
    hipLaunchKernelGGL((layer_norm_columns_kernel<T, P>), dim3((uint32_t)((kib + 3) / 4), y), dim3(256), 0, stream, a,
                       s.per);
  } else if (kib <= 1) layer_norm_backward_in<T, P, 1, 1>(a, s, stream);
  else if (kib <= 2) layer_norm_backward_in<T, P, 1, 2>(a, s, stream);
  else if (kib <= 4) layer_norm_backward_in<T, P, 1, 4>(a, s, stream);
  else if (kib <= 8) layer_norm_backward_in<T, P, 4, 2>(a, s, stream);
  else if (kib <= 16) layer_norm_backward_in<T, P, 4, 4>(a, s, stream);
  else layer_norm_backward_in<T, P, 16, 2>(a, s, stream);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, bool bf16, bool param_bf16, hipStream_t stream) {
  if (bf16) param_bf16 ? layer_norm_any<BF16, BF16>(a, stream) : layer_norm_any<BF16, F32>(a, stream);
  else param_bf16 ? layer_norm_any<F32, BF16>(a, stream) : layer_norm_any<F32, F32>(a, stream);
  return hipGetLastError();
}

LayerNormShape layer_norm_shape(uint64_t tokens, uint64_t width, uint64_t esize) {
  const uint64_t bytes = width * esize;
  LayerNormShape s{0, kSumTokens, bytes > kHeldBackwardKib * 1024};
  if (tokens == 0) return s;
  // rows beside each other in a workgroup of layer_norm_backward_kernel
  const uint64_t rows = s.row_sums || bytes > 16384 ? 1 : bytes > 4096 ? kGradWaves / 4 : kGradWaves;
  uint64_t turns = (tokens + rows * kGradBlocks - 1) / (rows * kGradBlocks);
  if (turns > kSumTokens) turns = kSumTokens;
  s.per = (uint32_t)(rows * turns);
  s.blocks = (uint32_t)((tokens + s.per - 1) / s.per);
  return s;
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, const LayerNormShape& s, bool bf16,
                                      bool param_bf16, bool grad_bf16, hipStream_t stream) {
  if (a.tokens) {
    if (bf16) param_bf16 ? layer_norm_backward_any<BF16, BF16>(a, s, stream) : layer_norm_backward_any<BF16, F32>(a, s, stream);
    else param_bf16 ? layer_norm_backward_any<F32, BF16>(a, s, stream) : layer_norm_backward_any<F32, F32>(a, s, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dweight || a.dbias) {
    const dim3 grid((uint32_t)(((uint64_t)a.width + 63) / 64), 2), block(64 * kJoinWaves);
    if (grad_bf16) hipLaunchKernelGGL((layer_norm_join_kernel<BF16>), grid, block, 0, stream, a, s.blocks);
    else hipLaunchKernelGGL((layer_norm_join_kernel<F32>), grid, block, 0, stream, a, s.blocks);
  }
  return hipGetLastError();
}

}  // namespace snac
