// route.hip -- routing of tokens to experts and its gradient
// (snac_route, snac_route_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// A binary64 as an unsigned number of the same order; 0 for -infinity
// (masked), NaN above everything, -0 as +0.
__device__ __forceinline__ uint64_t order64(double x) {
  if (x != x) return ~0ull;
  if (x == -HUGE_VAL) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) {
    const uint64_t y = __shfl_xor((unsigned long long)x, m);
    x = y > x ? y : x;
  }
  return x;
}

template <typename T>
__device__ __forceinline__ float load_logit(const char* row, uint32_t e) {
  return load_elem<T>(row + (uint64_t)e * T::kSize);
}

// One wave a token, lane l holding experts l V .. l V + V - 1, so that the
// lowest lane of several with equal keys holds the lowest expert.
template <typename T, int V>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t E = (uint32_t)a.r.experts, G = (uint32_t)a.r.groups, K = (uint32_t)a.r.topk;
  const uint32_t gs = E / G;
  const bool softmax = a.r.score == SNAC_SCORE_SOFTMAX;
  const float inf = __builtin_inff();
  for (uint64_t t = (uint64_t)blockIdx.x * kRouteWaves + wave_id(); t < a.tokens;
       t += (uint64_t)gridDim.x * kRouteWaves) {
    const char* row = static_cast<const char*>(a.logits) + t * a.ld * T::kSize;
    float x[V];
    bool bad = false;
    float top = -inf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = lane * V + j;
      x[j] = e < E ? load_logit<T>(row, e) : -inf;
      bad |= x[j] != x[j];
      top = fmaxf(top, x[j]);
    }
    top = snac::wave_max(top);
    // softmax of a row with a NaN or +infinity is NaN throughout
    const bool poison = softmax && (__any(bad) || top == inf);
    double s[V];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (softmax) {
        s[j] = x[j] == -inf ? 0.0 : exp((double)x[j] - (double)top);
        sum += s[j];
      } else {
        s[j] = 1.0 / (1.0 + exp(-(double)x[j]));
      }
    }
    if (softmax) sum = wave_sum(sum);
    uint64_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = lane * V + j;
      if (softmax) s[j] = poison ? __builtin_nan("") : s[j] / sum;
      const double k = x[j] == -inf ? -HUGE_VAL : (a.bias && e < E ? s[j] + (double)a.bias[e] : s[j]);
      key[j] = order64(k);
      s[j] = k;  // from here on the key itself
    }
    if (G > 1) {
      // lane g: the worth of group g
      uint64_t worth = 0;
      for (uint32_t g = 0; g < G; ++g) {
        uint64_t best[2] = {0, 0};
        double val[2] = {-HUGE_VAL, -HUGE_VAL};
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const uint32_t e = lane * V + j;
          if (e < E && e / gs == g) {
            if (key[j] > best[0]) {
              best[1] = best[0], val[1] = val[0];
              best[0] = key[j], val[0] = s[j];
            } else if (key[j] > best[1]) {
              best[1] = key[j], val[1] = s[j];
            }
          }
        }
        const uint64_t m0 = wave_max(best[0]);
        const uint64_t at0 = __ballot(best[0] == m0);
        const uint32_t l0 = (uint32_t)__ffsll((unsigned long long)at0) - 1;
        double w = __shfl(val[0], (int)l0);
        if (a.r.group_top == 2 && gs > 1) {
          if (lane == l0) best[0] = best[1], val[0] = val[1];
          const uint64_t m1 = wave_max(best[0]);
          const uint32_t l1 = (uint32_t)__ffsll((unsigned long long)__ballot(best[0] == m1)) - 1;
          w = w + __shfl(val[0], (int)l1);
        }
        if (lane == g) worth = order64(w);
      }
      uint32_t before = 0;
      for (uint32_t g = 0; g < G; ++g) {
        const uint64_t o = __shfl((unsigned long long)worth, (int)g);
        before += o > worth || (o == worth && g < lane);
      }
      const uint64_t kept = __ballot(lane < G && worth != 0 && before < (uint32_t)a.r.topk_groups);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = lane * V + j;
        if (e >= E || !((kept >> (e / gs)) & 1)) key[j] = 0;
      }
    }
    // lane k: the k-th choice
    int32_t my_id = -1;
    float my_x = -inf;
    for (uint32_t k = 0; k < K; ++k) {
      uint64_t best = key[0];
      int at = 0;
      float bx = x[0];
#pragma unroll
      for (int j = 1; j < V; ++j)
        if (key[j] > best) best = key[j], at = j, bx = x[j];
      const uint64_t m = wave_max(best);
      if (m == 0) break;
      const int l = __ffsll((unsigned long long)__ballot(best == m)) - 1;
      const int id = __shfl((int)(lane * V) + at, l);
      const float vx = __shfl(bx, l);
      if (lane == k) my_id = id, my_x = vx;
      if ((int)lane == l) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j == at) key[j] = 0;
      }
    }
    const bool have = my_id >= 0;
    float w;
    if (softmax) {
      const float m = a.r.renorm ? snac::wave_max(my_x) : top;
      const float p = have ? expf(my_x - m) : 0.0f;
      float total;
      if (a.r.renorm) {
        total = wave_sum(p);
      } else {
        total = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) total += x[j] == -inf ? 0.0f : expf(x[j] - m);
        total = wave_sum(total);
      }
      w = poison ? __builtin_nanf("") : p / total;
    } else if (a.r.renorm) {
      // s_i / sum s_j with both sides times exp(-m), m the largest chosen
      // logit where that is negative: nothing underflows
      const float m = fminf(snac::wave_max(my_x), 0.0f);
      const float p = !have ? 0.0f : m < 0.0f ? expf(my_x - m) / (1.0f + expf(my_x)) : 1.0f / (1.0f + expf(-my_x));
      w = p / wave_sum(p);
    } else {
      w = 1.0f / (1.0f + expf(-my_x));
    }
    if (lane < K) {
      a.weights[t * K + lane] = have ? w * a.r.scale : 0.0f;
      a.ids[t * K + lane] = my_id;
    }
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(const RouteBackwardArgs a) {
  __shared__ float lds[kRouteWaves][64 * V];
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t E = (uint32_t)a.r.experts, K = (uint32_t)a.r.topk;
  const bool softmax = a.r.score == SNAC_SCORE_SOFTMAX;
  const float inf = __builtin_inff();
  float* up = lds[wave_id()];
  for (uint64_t t = (uint64_t)blockIdx.x * kRouteWaves + wave_id(); t < a.tokens;
       t += (uint64_t)gridDim.x * kRouteWaves) {
    const char* row = static_cast<const char*>(a.logits) + t * a.ld * T::kSize;
    char* drow = static_cast<char*>(a.dlogits) + t * a.ld_d * T::kSize;
    const int32_t id = lane < K ? a.ids[t * K + lane] : -1;
    const bool have = id >= 0 && (uint32_t)id < E;
    const float dw = have ? a.dweights[t * K + lane] * a.r.scale : 0.0f;
    const float cx = have ? load_logit<T>(row, (uint32_t)id) : -inf;
#pragma unroll
    for (int j = 0; j < V; ++j) up[j * 64 + lane] = 0.0f;
    if (softmax && !a.r.renorm) {
      float x[V];
      float top = -inf;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 64u + lane;
        x[j] = e < E ? load_logit<T>(row, e) : -inf;
        top = fmaxf(top, x[j]);
      }
      top = snac::wave_max(top);
      float total = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] = x[j] == -inf ? 0.0f : expf(x[j] - top);
        total += x[j];
      }
      total = wave_sum(total);
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // 0: every logit masked
      const float r = !have || cx == -inf ? 0.0f : expf(cx - top) * inv;
      const float dot = wave_sum(have ? r * dw : 0.0f);
      if (have) atomicAdd(&up[id], dw);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 64u + lane;
        if (e < E) store_elem<T>(drow + (uint64_t)e * T::kSize, x[j] * inv * (up[e] - dot));
      }
    } else {
      float g;
      if (softmax) {
        const float m = snac::wave_max(cx);
        const float p = !have || cx == -inf ? 0.0f : expf(cx - m);
        const float total = wave_sum(p);
        const float r = total == 0.0f ? 0.0f : p / total;
        g = r * (dw - wave_sum(have ? r * dw : 0.0f));
      } else {
        const float far = 1.0f / (1.0f + expf(cx));
        if (a.r.renorm) {
          const float m = fminf(snac::wave_max(cx), 0.0f);
          const float p = !have || cx == -inf ? 0.0f : m < 0.0f ? expf(cx - m) * far : 1.0f / (1.0f + expf(-cx));
          const float total = wave_sum(p);
          const float r = total == 0.0f ? 0.0f : p / total;
          g = r * far * (dw - wave_sum(have ? r * dw : 0.0f));
        } else {
          g = dw * far / (1.0f + expf(-cx));
        }
      }
      if (have) atomicAdd(&up[id], g);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 64u + lane;
        if (e < E) store_elem<T>(drow + (uint64_t)e * T::kSize, up[e]);
      }
    }
  }
}

uint32_t route_grid(uint64_t tokens) {
  const int cus = device_cu_count();
  const uint64_t most = (uint64_t)(cus > 0 ? cus : 1) * 16;
  const uint64_t want = (tokens + kRouteWaves - 1) / kRouteWaves;
  return (uint32_t)(want < most ? want : most);
}

template <typename T>
void route_any(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid(route_grid(a.tokens)), block(kRouteThreads);
  const int e = a.r.experts;
  if (e <= 64) hipLaunchKernelGGL((route_kernel<T, 1>), grid, block, 0, stream, a);
  else if (e <= 128) hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, 0, stream, a);
  else if (e <= 256) hipLaunchKernelGGL((route_kernel<T, 4>), grid, block, 0, stream, a);
  else if (e <= 512) hipLaunchKernelGGL((route_kernel<T, 8>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, 0, stream, a);
}

template <typename T>
void route_backward_any(const RouteBackwardArgs& a, hipStream_t stream) {
  const dim3 grid(route_grid(a.tokens)), block(kRouteThreads);
  const int e = a.r.experts;
  if (e <= 64) hipLaunchKernelGGL((route_backward_kernel<T, 1>), grid, block, 0, stream, a);
  else if (e <= 128) hipLaunchKernelGGL((route_backward_kernel<T, 2>), grid, block, 0, stream, a);
  else if (e <= 256) hipLaunchKernelGGL((route_backward_kernel<T, 4>), grid, block, 0, stream, a);
  else if (e <= 512) hipLaunchKernelGGL((route_backward_kernel<T, 8>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_backward_kernel<T, 16>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) route_any<BF16>(a, stream);
  else route_any<F32>(a, stream);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) route_backward_any<BF16>(a, stream);
  else route_backward_any<F32>(a, stream);
  return hipGetLastError();
}

}  // namespace snac
