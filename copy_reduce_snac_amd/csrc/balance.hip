// balance.hip -- how evenly a router's choices load the experts, as a loss, and
// its gradient (snac_balance_load, snac_balance_loss, snac_balance_backward in
// include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504f;

// 1 / x for a normal binary64 x, off by a few of its last bits: the hardware's
// estimate (2^-24 or better) and one step of Newton's iteration.
__device__ __forceinline__ double reciprocal(double x) {
  const double r = __builtin_amdgcn_rcp(x);
  return r * __builtin_fma(-x, r, 2.0);
}

// The tokens of a wave: L lanes a token, V logits a lane.  UNITS: in 16-byte
// units, unit u of lane l being the row's unit u L + l, for rows of whole units;
// else by elements, j L + l.
template <typename T, int L, int V, bool UNITS>
struct Row {
  static constexpr int N = kUnit<T>;
  uint32_t l, E;
  __device__ __forceinline__ Row(uint32_t experts) : l(threadIdx.x % L), E(experts) {}
  // the row's element that is this lane's j-th
  __device__ __forceinline__ uint32_t at(int j) const { return UNITS ? ((j / N) * L + l) * N + j % N : j * L + l; }

  // a lane without an element reads the row's first; `rest` is put in its place
  __device__ __forceinline__ void load(const char* row, float rest, float (&x)[V]) const {
    if constexpr (UNITS) {
      u32x4 w[V / N];
#pragma unroll
      for (int u = 0; u < V / N; ++u) w[u] = ld_unit<false>(row + (at(u * N) < E ? at(u * N) : 0) * T::kSize);
#pragma unroll
      for (int u = 0; u < V / N; ++u) {
        float f[N];
        unpack<T>(w[u], f);
#pragma unroll
        for (int c = 0; c < N; ++c) x[u * N + c] = at(u * N) < E ? f[c] : rest;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = load_elem<T>(row + (at(j) < E ? at(j) : 0) * T::kSize);
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = at(j) < E ? x[j] : rest;
    }
  }
  __device__ __forceinline__ void store(char* row, const float (&x)[V]) const {
    if constexpr (UNITS) {
#pragma unroll
      for (int u = 0; u < V / N; ++u) {
        float f[N];
#pragma unroll
        for (int c = 0; c < N; ++c) f[c] = x[u * N + c];
        if (at(u * N) < E) st_unit<true>(row + at(u * N) * T::kSize, pack<T>(f));
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at(j) < E) store_elem<T>(row + at(j) * T::kSize, x[j]);
    }
  }
};

// A row's scores x -> e and 1 over their sum: e * inv are the shares.
// Exponentials are binary32, their sum binary64.  Sigmoids where all are small
// are taken times exp(-m), m the largest logit, so that they do not underflow.
// far: 1 - sigmoid of each logit.
template <int L, int V, bool FAR>
__device__ __forceinline__ double shares(bool softmax, float (&x)[V], float (&far)[FAR ? V : 1]) {
  const float inf = __builtin_inff();
  float top = -inf;
#pragma unroll
  for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
  top = lanes_max<L>(top);
  if (top == -inf) top = 0.0f;  // every logit masked (or NaN)
  double total = 0.0;
  if (softmax) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = __builtin_amdgcn_exp2f((x[j] - top) * kLog2e);
      total += x[j];
    }
  } else {
    const float m = fminf(top, 0.0f);
    const bool low = __any(m < 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a = __builtin_amdgcn_exp2f(-fabsf(x[j]) * kLog2e);
      const float r = __builtin_amdgcn_rcpf(1.0f + a);
      float up = x[j] < 0.0f ? a : 1.0f;
      if (low && m < 0.0f) up = __builtin_amdgcn_exp2f((x[j] - m) * kLog2e);
      if constexpr (FAR) far[j] = (x[j] < 0.0f ? 1.0f : a) * r;
      x[j] = up * r;
      total += x[j];
    }
  }
  total = lanes_sum<L>(total);
  return total == 0.0 ? 0.0 : reciprocal(total);
}

// Whether the token of this lane's L lanes has an id in range; with COUNT, its
// ids are counted.
template <int L, bool COUNT>
__device__ __forceinline__ bool counts(const BalanceArgs& a, uint64_t t, bool live, uint32_t l, uint32_t* hist) {
  bool any = false;
  for (uint32_t k = l; k < (uint32_t)a.topk; k += L) {
    const int32_t id = live ? a.ids[t * (uint32_t)a.topk + k] : -1;
    if ((uint32_t)id < (uint32_t)a.experts) {
      any = true;
      if constexpr (COUNT) atomicAdd(&hist[id], 1u);
    }
  }
  const uint64_t mask = __ballot(any), lanes = L == 64 ? ~0ull : ((1ull << (L & 63)) - 1) << ((threadIdx.x & 63u) / L * L);
  return (mask & lanes) != 0;
}

// Sums of the shares and counts of the ids of this workgroup's tokens.
template <typename T, int L, int V, bool UNITS>
__global__ __launch_bounds__(kThreads) void balance_load_kernel(const BalanceArgs a) {
  constexpr uint32_t TPW = 64 / L, kRows = kWaves * TPW;
  __shared__ uint32_t hist[L * V];
  __shared__ double sums[kRows][L * V <= 256 ? L * V : 256];
  const Row<T, L, V, UNITS> r((uint32_t)a.experts);
  const uint32_t sub = (threadIdx.x & 63u) / L;
  const bool softmax = a.score == SNAC_SCORE_SOFTMAX;
  for (uint32_t e = threadIdx.x; e < L * V; e += kThreads) hist[e] = 0;
  __syncthreads();
  double acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0;
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows + wave_id() * TPW; t0 < a.tokens; t0 += step) {
    const bool live = t0 + sub < a.tokens;
    const uint64_t t = live ? t0 + sub : t0;
    float x[V], none[1];
    r.load(static_cast<const char*>(a.logits) + t * a.ld * T::kSize, -__builtin_inff(), x);
    const bool in = counts<L, true>(a, t, live, r.l, hist);
    const double inv = shares<L, V, false>(softmax, x, none);
    if (in) {
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = __builtin_fma((double)x[j], inv, acc[j]);
    }
  }
  // the workgroup's rows are added up in order, up to 256 experts at a time
  constexpr int kPer = L * V <= 256 ? V : 256 / L;
  double* out = a.sums + (uint64_t)blockIdx.x * r.E;
#pragma unroll
  for (int j0 = 0; j0 < V; j0 += kPer) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) sums[wave_id() * TPW + sub][j * L + r.l] = acc[j0 + j];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < (uint32_t)(kPer * L); i += kThreads) {
      double s = 0.0;
#pragma unroll
      for (uint32_t k = 0; k < kRows; ++k) s += sums[k][i];
      Row<T, L, V, UNITS> other(r.E);
      other.l = i % L;
      const uint32_t e = other.at((int)(j0 + i / L));
      if (e < r.E) out[e] = s;
    }
  }
  for (uint32_t e = threadIdx.x; e < r.E; e += kThreads) a.counts[(uint64_t)blockIdx.x * r.E + e] = hist[e];
}

// load from the workgroups' sums and counts: 64 experts a workgroup, its waves
// taking every 16th.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void balance_join_kernel(const BalanceArgs a) {
  __shared__ double sums[kJoinWaves][64];
  __shared__ uint32_t counts[kJoinWaves][64];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id(), E = (uint32_t)a.experts, e = blockIdx.x * 64 + lane;
  double s = 0.0;
  uint32_t c = 0;
  if (e < E) {
#pragma unroll 4
    for (uint32_t b = w; b < a.blocks; b += kJoinWaves) {
      s += a.sums[(uint64_t)b * E + e];
      c += a.counts[(uint64_t)b * E + e];
    }
  }
  sums[w][lane] = s;
  counts[w][lane] = c;
  __syncthreads();
  if (w != 0 || e >= E) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) s += sums[i][lane], c += counts[i][lane];
  a.load[e] = (float)c;
  a.load[E + e] = (float)s;
}

__global__ __launch_bounds__(64) void balance_loss_kernel(const float* load, uint32_t experts, float coefficient, float* loss) {
  double c = 0.0, s = 0.0, dot = 0.0;
  for (uint32_t e = threadIdx.x; e < experts; e += 64) {
    const double ce = load[e], se = load[experts + e];
    c += ce;
    s += se;
    dot = __builtin_fma(ce, se, dot);
  }
  c = wave_sum(c);
  s = wave_sum(s);
  dot = wave_sum(dot);
  if (threadIdx.x == 0) loss[0] = c == 0.0 || s == 0.0 ? 0.0f : (float)((double)coefficient * experts * dot / (c * s));
}

// The gradient.  A token's shares sum to 1, so a constant may be taken off every
// expert's slope: counts are taken less their mean, which leaves small numbers
// where the loads are nearly even.  Sums over a row are binary64.
template <typename T, int L, int V, bool UNITS>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(const BalanceArgs a) {
  constexpr uint32_t TPW = 64 / L, kRows = kWaves * TPW;
  const Row<T, L, V, UNITS> r((uint32_t)a.experts);
  const uint32_t sub = (threadIdx.x & 63u) / L;
  const bool softmax = a.score == SNAC_SCORE_SOFTMAX;
  float slope[V];
  double c = 0.0, s = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool in = r.at(j) < r.E;
    slope[j] = in ? a.load[r.at(j)] : 0.0f;
    c += slope[j];
    s += in ? a.load[r.E + r.at(j)] : 0.0f;
  }
  c = lanes_sum<L>(c);
  s = lanes_sum<L>(s);
  const double mean = c / (double)r.E;
  const double scale = c == 0.0 || s == 0.0 ? 0.0
                                            : (a.dloss ? (double)a.dloss[0] : 1.0) * (double)a.coefficient * (double)r.E / (c * s);
#pragma unroll
  for (int j = 0; j < V; ++j) slope[j] = (float)(((double)slope[j] - mean) * scale);
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows + wave_id() * TPW; t0 < a.tokens; t0 += step) {
    const bool live = t0 + sub < a.tokens;
    const uint64_t t = live ? t0 + sub : t0;
    float x[V], far[V], old[V];
    r.load(static_cast<const char*>(a.logits) + t * a.ld * T::kSize, -__builtin_inff(), x);
    char* out = static_cast<char*>(a.dlogits) + t * a.ld_d * T::kSize;
    if (a.accumulate) r.load(out, 0.0f, old);
    uint32_t* nothing = nullptr;
    const bool in = counts<L, false>(a, t, live, r.l, nothing);
    const double inv = shares<L, V, true>(softmax, x, far);
    double dot = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) dot = __builtin_fma((double)x[j], (double)slope[j], dot);
    dot = lanes_sum<L>(dot) * inv;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d = (float)((double)x[j] * inv * ((double)slope[j] - dot));
      if (!softmax) d = d * far[j];
      x[j] = in ? d : 0.0f;
      if (a.accumulate) x[j] = in ? old[j] + d : old[j];
    }
    if (live) r.store(out, x);
  }
}

template <typename T, int L, int V, typename F>
void with_units(int experts, F launch) {
  if constexpr (V >= (int)kUnit<T>) {
    if (experts % kUnit<T> == 0) return launch.template operator()<T, L, V, true>();
  }
  launch.template operator()<T, L, V, false>();
}

// The narrowest shape that holds the experts.
template <typename T, typename F>
void by_experts(int e, F launch) {
  if (e <= 16) with_units<T, 16, 1>(e, launch);
  else if (e <= 64) with_units<T, 16, 4>(e, launch);
  else if (e <= 128) with_units<T, 16, 8>(e, launch);
  else if (e <= 256) with_units<T, 16, 16>(e, launch);
  else if (e <= 512) with_units<T, 32, 16>(e, launch);
  else with_units<T, 64, 16>(e, launch);
}

struct LoadLauncher {
  const BalanceArgs& a;
  hipStream_t stream;
  template <typename T, int L, int V, bool UNITS>
  void operator()() const {
    hipLaunchKernelGGL((balance_load_kernel<T, L, V, UNITS>), dim3(a.blocks), dim3(kThreads), 0, stream, a);
  }
};
struct BackwardLauncher {
  const BalanceArgs& a;
  hipStream_t stream;
  template <typename T, int L, int V, bool UNITS>
  void operator()() const {
    constexpr uint64_t rows = kWaves * (64 / L);
    const int n = device_cu_count();
    const uint64_t want = (a.tokens + rows - 1) / rows, most = (uint64_t)(n > 0 ? n : 1) * 8;
    hipLaunchKernelGGL((balance_backward_kernel<T, L, V, UNITS>), dim3((uint32_t)(want < most ? want : most)),
                       dim3(kThreads), 0, stream, a);
  }
};

}  // namespace

uint32_t balance_blocks(uint64_t tokens, int experts) {
  const uint64_t rows = kWaves * (experts <= 256 ? 4 : experts <= 512 ? 2 : 1);
  const uint64_t want = (tokens + rows - 1) / rows;
  return (uint32_t)(want < kBalanceMaxBlocks ? want : kBalanceMaxBlocks);
}

hipError_t launch_balance_load(const BalanceArgs& a, bool bf16, hipStream_t stream) {
  if (a.blocks) {
    if (bf16) by_experts<BF16>(a.experts, LoadLauncher{a, stream});
    else by_experts<F32>(a.experts, LoadLauncher{a, stream});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(balance_join_kernel, dim3((a.experts + 63) / 64), dim3(64 * kJoinWaves), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_balance_loss(const float* load, int experts, float coefficient, float* loss, hipStream_t stream) {
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(64), 0, stream, load, (uint32_t)experts, coefficient, loss);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) by_experts<BF16>(a.experts, BackwardLauncher{a, stream});
  else by_experts<F32>(a.experts, BackwardLauncher{a, stream});
  return hipGetLastError();
}

}  // namespace snac
