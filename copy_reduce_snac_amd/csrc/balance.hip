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

// 1 / x for a normal binary64 x: the hardware's estimate (2^-24 or better) and one step
// of Newton's iteration, which leaves its square, 2^-48.
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

  // a lane without an element reads the row's first
  struct Raw {
    u32x4 unit[UNITS ? V / N : 1];
    float one[UNITS ? 1 : V];
  };
  __device__ __forceinline__ void fetch(const char* row, Raw& raw) const {
    if constexpr (UNITS) {
#pragma unroll
      for (int u = 0; u < V / N; ++u) raw.unit[u] = ld_unit<false>(row + (at(u * N) < E ? at(u * N) : 0) * T::kSize);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) raw.one[j] = load_elem<T>(row + (at(j) < E ? at(j) : 0) * T::kSize);
    }
  }
  // what was fetched; `rest` is put in the place of what a lane has not
  __device__ __forceinline__ void take(const Raw& raw, float rest, float (&x)[V]) const {
    if constexpr (UNITS) {
#pragma unroll
      for (int u = 0; u < V / N; ++u) {
        float f[N];
        unpack<T>(raw.unit[u], f);
#pragma unroll
        for (int c = 0; c < N; ++c) x[u * N + c] = at(u * N) < E ? f[c] : rest;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = at(j) < E ? raw.one[j] : rest;
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

// The largest of a row's logits; 0 where all are masked.
template <int L, int V>
__device__ __forceinline__ float row_top(const float (&x)[V]) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < V; ++j) top = fmaxf(top, x[j]);
  top = lanes_max<L>(top);
  return top == -__builtin_inff() || top != top ? 0.0f : top;
}

// A row's scores x -> e and 1 over their sum: e * inv are the shares.
// Exponentials are binary32, their sum binary64.  Sigmoids where all are small
// are taken times exp(-m), m the largest logit, so that they do not underflow.
// far: 1 - sigmoid of each logit.
template <int L, int V, bool FAR>
__device__ __forceinline__ double shares(bool softmax, float top, float (&x)[V], float (&far)[FAR ? V : 1]) {
  double total = 0.0;
  if (softmax) {
    asm volatile("");  // a branch, and not both sides and a choice
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = __builtin_amdgcn_exp2f((x[j] - top) * kLog2e);
      total += x[j];
    }
  } else {
    asm volatile("");
    const float m = fminf(top, 0.0f);
    const bool low = __any(m < 0.0f);
    constexpr int P = V < 8 ? V : 8;  // at a time: more would cost registers
#pragma unroll
    for (int j0 = 0; j0 < V; j0 += P) {
      float up[P], r[P];
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float a = __builtin_amdgcn_exp2f(-fabsf(x[j0 + j]) * kLog2e);
        r[j] = __builtin_amdgcn_rcpf(1.0f + a);
        if constexpr (FAR) far[j0 + j] = (x[j0 + j] < 0.0f ? 1.0f : a) * r[j];
        up[j] = x[j0 + j] < 0.0f ? a : 1.0f;
      }
      if (low) {
        asm volatile("");
#pragma unroll
        for (int j = 0; j < P; ++j) up[j] = m < 0.0f ? __builtin_amdgcn_exp2f((x[j0 + j] - m) * kLog2e) : up[j];
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        x[j0 + j] = up[j] * r[j];
        total += x[j0 + j];
      }
    }
  }
  total = lanes_sum<L>(total);
  return total == 0.0 ? 0.0 : reciprocal(total);
}

// The ids of a token's choices, choice c L + l in slot c of lane l.
template <int L>
struct Ids {
  static constexpr int C = (SNAC_MAX_TOPK + L - 1) / L;
  int32_t id[C];
  __device__ __forceinline__ void fetch(const BalanceArgs& a, uint64_t t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t k = c * L + threadIdx.x % L;
      id[c] = k < (uint32_t)a.topk ? a.ids[t * (uint32_t)a.topk + k] : -1;
    }
  }
  // whether the token of this lane's L lanes has an id in range
  __device__ __forceinline__ bool any(uint32_t experts) const {
    bool mine = false;
#pragma unroll
    for (int c = 0; c < C; ++c) mine |= (uint32_t)id[c] < experts;
    const uint64_t lanes = L == 64 ? ~0ull : ((1ull << (L & 63)) - 1) << ((threadIdx.x & 63u) / L * L);
    return (__ballot(mine) & lanes) != 0;
  }
};

constexpr int kLoadThreads = 1024;
constexpr int kLoadWaves = kLoadThreads / 64;

// load[e] = how many of the ids are e, load[E + e] = sum over the tokens of expert
// e's share of the scores: sums of the shares (binary64, a lane's columns in its
// registers) and counts of the ids (integer atomics in LDS) of this workgroup's
// tokens.
//
// 32768 x 256 f32 sigmoid 11.2 us of kernel for 35 MB, of which the launch and the
// first row's load take 5 and two turns of 4 tokens a wave the rest; longer ones are
// bound by instructions, of which a sigmoid's logit takes two transcendental ones and
// four of binary64: two conversions, an addition to the row's sum and a fused product
// to the expert's (131072 x 256: 29 us, 4.6 TB/s; 16384 x 1000 softmax, one
// transcendental and those four, 18 us, 3.7).  256 workgroups of 16 waves, so that the
// join has no more than 256 sums an expert; a turn's logits are fetched during the
// turn before.
template <typename T, int L, int V, bool UNITS>
__global__ __launch_bounds__(kLoadThreads) void balance_load_kernel(const BalanceArgs a) {
  constexpr uint32_t TPW = 64 / L, kRows = kLoadWaves * TPW;
  constexpr int kPer = L * V <= 512 ? V : 512 / L;  // elements of a lane that are added up at a time
  __shared__ uint32_t hist[L * V];
  __shared__ double sums[kLoadWaves][kPer * L];
  using R = Row<T, L, V, UNITS>;
  const R r((uint32_t)a.experts);
  const uint32_t lane = threadIdx.x & 63u, sub = lane / L;
  const bool softmax = a.score == SNAC_SCORE_SOFTMAX;
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  uint64_t t = (uint64_t)blockIdx.x * kRows + wave_id() * TPW + sub;
  typename R::Raw next;
  Ids<L> ids;
  auto fetch = [&](uint64_t token) {  // (one past the last reads the last, and counts for nothing)
    const uint64_t at = token < a.tokens ? token : a.tokens - 1;
    r.fetch(static_cast<const char*>(a.logits) + at * a.ld * T::kSize, next);
    ids.fetch(a, at);
  };
  constexpr bool kAhead = UNITS;  // else it costs too many registers
  if (kAhead) fetch(t);
  for (uint32_t e = threadIdx.x; e < L * V; e += kLoadThreads) hist[e] = 0;
  __syncthreads();
  double acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0;
  for (uint64_t t0 = t - sub; t0 < a.tokens; t0 += step, t += step) {
    float x[V], none[1];
    if (!kAhead) fetch(t);
    r.take(next, -__builtin_inff(), x);
    const bool in = ids.any(r.E) && t < a.tokens;
    if (t < a.tokens) {
#pragma unroll
      for (int c = 0; c < ids.C; ++c)
        if ((uint32_t)ids.id[c] < r.E) atomicAdd(&hist[ids.id[c]], 1u);
    }
    if (kAhead && t0 + step < a.tokens) fetch(t + step);
    const double inv = shares<L, V, false>(softmax, row_top<L>(x), x, none);
    if (in) {
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = __builtin_fma((double)x[j], inv, acc[j]);
    }
  }
  // the tokens side by side in a wave, then the waves, in order
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (L <= 16) acc[j] = exchange_sum<16>(acc[j]);
    if constexpr (L <= 32) acc[j] = exchange_sum<32>(acc[j]);
  }
  double* out = a.sums + (uint64_t)blockIdx.x * r.E;
#pragma unroll
  for (int j0 = 0; j0 < V; j0 += kPer) {
    __syncthreads();
    if (sub == 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) sums[wave_id()][j * L + r.l] = acc[j0 + j];
    }
    __syncthreads();
    const uint32_t i = threadIdx.x;
    if (i < (uint32_t)(kPer * L)) {
      double s = 0.0;
#pragma unroll
      for (uint32_t k = 0; k < kLoadWaves; ++k) s += sums[k][i];
      R other(r.E);
      other.l = i % L;
      const uint32_t e = other.at((int)(j0 + i / L));
      if (e >= r.E) continue;
      if (gridDim.x == 1) a.load[r.E + e] = (float)s;  // nothing to join
      else out[e] = s;
    }
  }
  for (uint32_t e = threadIdx.x; e < r.E; e += kLoadThreads) {
    if (gridDim.x == 1) a.load[e] = (float)hist[e];
    else a.counts[(uint64_t)blockIdx.x * r.E + e] = hist[e];
  }
}

// load from the workgroups' sums and counts: 16 experts a workgroup, a lane
// taking every 64th of an expert's numbers.  Latency: 256 x 256 of them 4 us, and
// always in the same order.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void balance_join_kernel(const BalanceArgs a) {
  __shared__ double sums[kJoinWaves][16];
  __shared__ uint32_t counts[kJoinWaves][16];
  const uint32_t lane = threadIdx.x & 63u, w = wave_id(), E = (uint32_t)a.experts, e = blockIdx.x * 16 + lane % 16;
  double s = 0.0;
  uint32_t c = 0;
  if (e < E) {
#pragma unroll 4
    for (uint32_t b = threadIdx.x / 16; b < a.blocks; b += 4 * kJoinWaves) {
      s += a.sums[(uint64_t)b * E + e];
      c += a.counts[(uint64_t)b * E + e];
    }
  }
  auto add = [](uint32_t x, uint32_t y) { return x + y; };
  s = exchange_sum<32>(exchange_sum<16>(s));
  c = exchange<32>(exchange<16>(c, add), add);
  if (lane < 16) sums[w][lane] = s, counts[w][lane] = c;
  __syncthreads();
  if (threadIdx.x >= 16 || e >= E) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) s += sums[i][lane], c += counts[i][lane];
  a.load[e] = (float)c;
  a.load[E + e] = (float)s;
}

// coefficient E sum c s / (sum c sum s): one wave, 1.3 us of launch.
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

// The gradient: scale p[e] (c[e] - sum over j of p[j] c[j]) for softmax, and times
// 1 - sigmoid(x[e]) for sigmoids, p the token's shares and c the counts.  The shares
// sum to 1, so a constant may be taken off every count: that of the token's best
// expert is.  These differences of whole numbers are exact, and the best expert's own
// term, which is what the others leave, is not a small difference of large ones.
//
// Launch and ramp, then HBM: 32768 x 128 f32 softmax 7.9 us of kernel for 35 MB, 4.2
// TB/s; 131072 x 256 f32 sigmoid 51 us, 5.3.  Three workgroups a CU, each of which
// loads the counts once; a token's logits are fetched during the one before.
template <typename T, int L, int V, bool UNITS>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(const BalanceArgs a) {
  constexpr uint32_t TPW = 64 / L, kRows = kWaves * TPW;
  using R = Row<T, L, V, UNITS>;
  const R r((uint32_t)a.experts);
  const float inf = __builtin_inff();
  const uint32_t sub = (threadIdx.x & 63u) / L;
  const bool softmax = a.score == SNAC_SCORE_SOFTMAX;
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  uint64_t t = (uint64_t)blockIdx.x * kRows + wave_id() * TPW + sub;
  typename R::Raw next;
  Ids<L> ids;
  auto fetch = [&](uint64_t token) {  // (one past the last reads the last)
    const uint64_t at = token < a.tokens ? token : a.tokens - 1;
    r.fetch(static_cast<const char*>(a.logits) + at * a.ld * T::kSize, next);
    ids.fetch(a, at);
  };
  fetch(t);
  // 16 bytes at a time (by single numbers, which lie 32 bytes apart from lane to
  // lane, 32768 x 256 bf16 took 19.9 us instead of 10.9)
  float count[V];
  if constexpr (UNITS) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const uint32_t e = r.at(j);
      const u32x4 v = ld_unit<false>(reinterpret_cast<const char*>(a.load + (e < r.E ? e : 0)));
#pragma unroll
      for (int i = 0; i < 4; ++i) count[j + i] = e < r.E ? __uint_as_float(v[i]) : 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) count[j] = r.at(j) < r.E ? a.load[r.at(j)] : 0.0f;
  }
  double c = 0.0, s = 0.0;
  for (uint32_t e = threadIdx.x & 63u; e < r.E; e += 64) c += a.load[e], s += a.load[r.E + e];
  c = wave_sum(c);
  s = wave_sum(s);
  const double scale = c == 0.0 || s == 0.0 ? 0.0
                                            : (a.dloss ? (double)a.dloss[0] : 1.0) * (double)a.coefficient * (double)r.E / (c * s);
  // A scale that binary32 holds not at all, or with few bits, is taken by a power of two
  // that the products get back; 2^60 of it stays, for the smallest shares to be normal
  // numbers with it.
  const int power = scale != 0.0 && isfinite(scale) && !(fabs(scale) > 0x1p-60 && fabs(scale) < 0x1p60) ? ilogb(scale) - 60 : 0;
  const double scale_f = ldexp(scale, -power);
  for (uint64_t t0 = t - sub; t0 < a.tokens; t0 += step, t += step) {
    float x[V], far[V];
    r.take(next, -inf, x);
    const bool in = ids.any(r.E);
    if (t0 + step < a.tokens) fetch(t + step);
    const float top = row_top<L>(x);
    float best = -inf;
#pragma unroll
    for (int j = 0; j < V; ++j) best = x[j] == top ? fmaxf(best, count[j]) : best;
    best = lanes_max<L>(best);
    if (best == -inf) best = 0.0f;
    const double inv = shares<L, V, true>(softmax, top, x, far);
    float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) dot[j % 4] = __builtin_fmaf(x[j], count[j] - best, dot[j % 4]);
    const float mean = (float)((double)lanes_sum<L>((dot[0] + dot[1]) + (dot[2] + dot[3])) * inv);
    const float f = (float)(inv * scale_f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = x[j] * f * ((count[j] - best) - mean);
      if (!softmax) x[j] = x[j] * far[j];
    }
    if (power != 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = ldexpf(x[j], power);
    }
    char* out = static_cast<char*>(a.dlogits) + (t < a.tokens ? t : a.tokens - 1) * a.ld_d * T::kSize;
    if (a.accumulate) {
      typename R::Raw raw;
      float old[V];
      r.fetch(out, raw);
      r.take(raw, 0.0f, old);
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = old[j] + x[j];
      if (t < a.tokens && in) r.store(out, x);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = in ? x[j] : 0.0f;
      if (t < a.tokens) r.store(out, x);
    }
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
    hipLaunchKernelGGL((balance_load_kernel<T, L, V, UNITS>), dim3(a.blocks), dim3(kLoadThreads), 0, stream, a);
  }
};
struct BackwardLauncher {
  const BalanceArgs& a;
  hipStream_t stream;
  template <typename T, int L, int V, bool UNITS>
  void operator()() const {
    constexpr uint64_t rows = kWaves * (64 / L);
    const int n = device_cu_count();
    const uint64_t want = (a.tokens + rows - 1) / rows, most = (uint64_t)(n > 0 ? n : 1) * 3;
    hipLaunchKernelGGL((balance_backward_kernel<T, L, V, UNITS>), dim3((uint32_t)(want < most ? want : most)),
                       dim3(kThreads), 0, stream, a);
  }
};

}  // namespace

uint32_t balance_blocks(uint64_t tokens, int experts) {
  const uint64_t rows = kLoadWaves * (experts <= 256 ? 4 : experts <= 512 ? 2 : 1);
  // one workgroup has no other's sums to wait for: the join's launch is saved.  Load
  // and loss of 200 x 60 bf16 11.3 us a call among others and 6.6 in a graph, with the
  // join 14.4 and 7.2; 509 x 60, which takes 8 turns, 11.2 and 10.3 or 14.4 and 7.1;
  // 250 x 256 f32, 4 turns of 16 logits a lane, 14.8 and 14.7 or 14.3 and 10.8.
  const uint64_t alone = experts <= 64 ? 4 : 2;  // turns
  if (tokens != 0 && tokens <= alone * rows) return 1;
  const uint64_t want = (tokens + rows - 1) / rows;
  return (uint32_t)(want < kBalanceMaxBlocks ? want : kBalanceMaxBlocks);
}

hipError_t launch_balance_load(const BalanceArgs& a, bool bf16, hipStream_t stream) {
  if (a.blocks) {
    if (bf16) by_experts<BF16>(a.experts, LoadLauncher{a, stream});
    else by_experts<F32>(a.experts, LoadLauncher{a, stream});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.blocks == 1) return e;
  }
  hipLaunchKernelGGL(balance_join_kernel, dim3((a.experts + 15) / 16), dim3(64 * kJoinWaves), 0, stream, a);
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
