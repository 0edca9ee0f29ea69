// route.hip -- routing of tokens to experts and its gradient
// (snac_route, snac_route_backward in include/snac_ops.h).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr float kLog2e = 1.44269504f;
// Above this, several tokens a wave (fewer instructions a token), else a wave a
// token (shorter chains).  us, several / one: 256 experts 6.3 / 5.5 at 2048
// tokens, 6.6 / 7.9 at 4096, 11.0 / 18.8 at 16384; 64 experts 4.3 / 4.3 at
// 1024, 4.2 / 4.8 at 2048, 7.0 / 15.7 at 16384.
constexpr uint64_t kRouteManyTokens = 2048;
constexpr int kMoreRounds = 3;  // choices looked at past the next one, where two are too near

// A binary64 as an unsigned number of the same order; 0 for -infinity
// (masked), NaN above everything, -0 as +0.
__device__ __forceinline__ uint64_t order64(double x) {
  if (x != x) return ~0ull;
  if (x == -HUGE_VAL) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t x) {
  const uint32_t hi = lanes_max<64>((uint32_t)(x >> 32));
  const uint32_t lo = lanes_max<64>((uint32_t)(x >> 32) == hi ? (uint32_t)x : 0);
  return (uint64_t)hi << 32 | lo;
}

// The value that lane `l` (the same in all lanes) holds.
__device__ __forceinline__ uint32_t from_lane(uint32_t x, uint32_t l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, (int)l);
}
__device__ __forceinline__ uint64_t from_lane(uint64_t x, uint32_t l) {
  return (uint64_t)from_lane((uint32_t)(x >> 32), l) << 32 | from_lane((uint32_t)x, l);
}
__device__ __forceinline__ double from_lane(double x, uint32_t l) {
  return __longlong_as_double((long long)from_lane((uint64_t)__double_as_longlong(x), l));
}

// 1 / x for a normal binary64 x, off by a few of its last bits: the
// hardware's estimate (2^-24 or better) and one step of Newton's iteration.
__device__ __forceinline__ double reciprocal(double x) {
  const double r = __builtin_amdgcn_rcp(x);
  return r * __builtin_fma(-x, r, 2.0);
}

// A chosen expert's share of `total`, scaled.  Scores are binary32, sums and
// quotients of them binary64, so that a weight is off by its own exponential
// and one rounding.  32768 x 256: 15.5 us (15.4 with binary32 throughout, whose
// weights are off by half as much again), softmax 20.5 (19.8).
__device__ __forceinline__ float share(float score, double total, float scale) {
  return (float)((double)score * (double)scale * reciprocal(total));
}

// scale * sigmoid(x)
__device__ __forceinline__ float scaled_sigmoid(float x, float scale) {
  const float a = expf(-fabsf(x));
  return share(x < 0.0f ? a : 1.0f, 1.0 + (double)a, scale);
}

template <typename T>
__device__ __forceinline__ float load_logit(const char* row, uint32_t e) {
  return load_elem<T>(row + (uint64_t)e * T::kSize);
}

// One token by a whole wave with its keys in binary64, lane l holding experts
// l V .. l V + V - 1, so that the lowest lane of several with equal keys holds
// the lowest expert.  Right for every input; route_kernel calls it for the
// tokens whose order it cannot be sure of.
template <typename T, int V>
__device__ void route_exact(const RouteArgs& a, uint64_t t) {
  uint32_t lane = threadIdx.x & 63u, E = (uint32_t)a.r.experts;
  // opaque here, so that nothing of this rare path is worked out before the
  // branch to it (it took 290 of 1000 instructions of route_kernel)
  asm volatile("" : "+v"(lane), "+s"(E));
  const uint32_t G = (uint32_t)a.r.groups, K = (uint32_t)a.r.topk;
  const uint32_t gs = E / G;
  const bool softmax = a.r.score == SNAC_SCORE_SOFTMAX;
  const float inf = __builtin_inff();
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
  top = wave_max(top);
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
      const uint64_t m0 = wave_max64(best[0]);
      const uint64_t at0 = __ballot(best[0] == m0);
      const uint32_t l0 = (uint32_t)__ffsll((unsigned long long)at0) - 1;
      double w = from_lane(val[0], l0);
      if (a.r.group_top == 2 && gs > 1) {
        if (lane == l0) best[0] = best[1], val[0] = val[1];
        const uint64_t m1 = wave_max64(best[0]);
        const uint32_t l1 = (uint32_t)__ffsll((unsigned long long)__ballot(best[0] == m1)) - 1;
        w = w + from_lane(val[0], l1);
      }
      if (lane == g) worth = order64(w);
    }
    uint32_t before = 0;
    for (uint32_t g = 0; g < G; ++g) {
      const uint64_t o = from_lane(worth, g);
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
    const uint64_t m = wave_max64(best);
    if (m == 0) break;
    const int l = __ffsll((unsigned long long)__ballot(best == m)) - 1;
    const int id = (int)from_lane(lane * V + (uint32_t)at, (uint32_t)l);
    const float vx = __uint_as_float(from_lane(__float_as_uint(bx), (uint32_t)l));
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
    const float m = a.r.renorm ? wave_max(my_x) : top;
    const float p = have ? expf(my_x - m) : 0.0f;
    w = poison ? __builtin_nanf("") : share(p, a.r.renorm ? wave_sum((double)p) : sum, a.r.scale);
  } else if (a.r.renorm) {
    // s_i / sum s_j with both sides times exp(-m), m the largest chosen
    // logit where that is negative: nothing underflows
    const float m = fminf(wave_max(my_x), 0.0f);
    const float p = !have ? 0.0f : m < 0.0f ? expf(my_x - m) / (1.0f + expf(my_x)) : 1.0f / (1.0f + expf(-my_x));
    w = share(p, wave_sum((double)p), a.r.scale);
  } else {
    w = scaled_sigmoid(my_x, a.r.scale);
  }
  if (lane < K) {
    a.weights[t * K + lane] = have ? w : 0.0f;
    a.ids[t * K + lane] = my_id;
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kRouteThreads) void route_exact_kernel(const RouteArgs a) {
  for (uint64_t t = (uint64_t)blockIdx.x * kRouteWaves + wave_id(); t < a.tokens;
       t += (uint64_t)gridDim.x * kRouteWaves)
    route_exact<T, V>(a, t);
}

// Batcher's odd-even merge sort of N (a power of two) registers, largest
// first.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + q];
            k[i + j] = x > y ? x : y;
            k[i + j + q] = x > y ? y : x;
          }
}

// V neighbouring elements of a row from element e0 on, the first `n` of them
// (those past it as `rest`).  whole: n is 0 or V in every lane, full: V.  No
// branch per lane: a lane without an element reads the row's first.
template <typename T, int V>
__device__ __forceinline__ void load_elems(const char* row, uint32_t e0, uint32_t n, bool whole, bool full, float rest,
                                           float (&x)[V]) {
  constexpr int N = kUnit<T>;
  if constexpr (V >= N) {
    if (whole) {
      const char* p = row + (uint64_t)(n ? e0 : 0) * T::kSize;
      u32x4 w[V / N];
#pragma unroll
      for (int u = 0; u < V / N; ++u) w[u] = ld_unit<false>(p + u * 16);
#pragma unroll
      for (int u = 0; u < V / N; ++u) {
        float f[N];
        unpack<T>(w[u], f);
#pragma unroll
        for (int c = 0; c < N; ++c) x[u * N + c] = f[c];
      }
      if (!full) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = n ? x[j] + 0.0f : rest;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = load_elem<T>(row + (uint64_t)((uint32_t)j < n ? e0 + j : 0) * T::kSize);
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = (uint32_t)j < n ? x[j] + 0.0f : rest;
}

// What a key is: kByLogit where there is no bias and no sum of scores (keys
// order as the logits), else the score (with its bias).
enum : int { kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2 };

// L lanes a token, V experts a lane (in neighbouring slots; a group of
// experts begins at a lane of its own and has 1 << ps lanes).
//
// Choosing is bound by instructions, not by memory: 32768 tokens of 256 f32
// logits, 8 of them from 4 of 8 groups, take 15.4 us, 863 vector instructions
// (32 of them transcendental) a wave of 4 tokens, 12.7 us of issue; the same
// logits are read in 5.4 us.  (All keys in binary64, by a wave a token: 147.)
// So a key is one 32-bit number: the score's distance from the row's best, QB
// bits of it, above the complement of the slot's number.  All keys of a token
// differ, they order as the scores do down to their last bits, and the maximum
// over lanes is 4 to 6 instructions.  A lane sorts its V keys once; a round
// takes the largest head over the lanes and shifts that lane's keys down.
//
// What QB bits and binary32 scores cannot tell apart is seen by comparing every
// choice with the next one (one round more than topk), and the last group that
// stays with the first that does not.  Where two come as near as `tol` steps
// without being equal in logit and bias, the choices and kMoreRounds after them
// (or the groups, by their two largest keys) are ordered by their binary64
// scores; a token that this does not settle, or that is not finite, is done
// again by route_exact.
//   no bias (keys order as the logits): the distance as a floating number of
//     QB bits.  Distance and cut keep the order, so only equal codes of
//     different logits are in doubt.
//   else: the distance in fixed point over S = 2 max(|best|, largest score).
//     A binary32 score with its bias is off by less than 3.5 S 2^-24 (sigmoid)
//     or 16 S 2^-24 (softmax: its exponent is a rounded product), the subtraction and the
//     scaling by at most S 2^-24 each, cutting by one step: two keys by 12 or
//     37 steps at QB = 24.
template <typename T, int L, int V, int KB, int KEY>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a, const uint32_t ps, const uint32_t gs) {
  constexpr uint32_t TPW = 64 / L;
  constexpr uint32_t IB = __builtin_ctz(L * V), QB = IB < 8 ? 24 : 32 - IB, QMAX = (1u << QB) - 1;
  constexpr int VX = L * V <= 64 ? 1 : L * V / 64;
  const uint32_t lane = threadIdx.x & 63u, l = lane % L, sub = lane / L;
  const uint32_t G = (uint32_t)a.r.groups, K = (uint32_t)a.r.topk;
  const bool softmax = KEY == kBySoftmax || (KEY == kByLogit && a.r.score == SNAC_SCORE_SOFTMAX);
  constexpr bool by_logit = KEY == kByLogit;
  const float inf = __builtin_inff();
  // the lane's experts
  const uint32_t g = l >> ps, in = (l & ((1u << ps) - 1)) * V;
  const uint32_t e0 = g * gs + in, n = g >= G || in >= gs ? 0 : gs - in < V ? gs - in : V;
  const bool whole = gs % V == 0, full = G << ps == L && gs == (uint32_t)V << ps;
  float b[V];
#pragma unroll
  for (int j = 0; j < V; ++j) b[j] = 0.0f;
  if (!by_logit && a.bias) load_elems<F32, V>(reinterpret_cast<const char*>(a.bias), e0, n, whole, full, 0.0f, b);

  // a packed key's expert (0: none), its logit and bias
  struct Choice {
    int32_t id;
    float x, b;
  };
  auto chosen = [&](const char* row, uint32_t won) {
    const uint32_t slot = L * V - 1 - (won & ((1u << IB) - 1)), wl = slot / V;
    const uint32_t id = (wl >> ps) * gs + (wl & ((1u << ps) - 1)) * V + slot % V;
    return Choice{won ? (int32_t)id : -1, won ? load_logit<T>(row, id) : -inf, won && a.bias ? a.bias[id] : 0.0f};
  };

  const uint64_t t0 = ((uint64_t)blockIdx.x * kRouteWaves + wave_id()) * TPW;
  if (t0 >= a.tokens) return;
  const uint64_t t = t0 + sub;
  const bool live = t < a.tokens;
  const char* row = static_cast<const char*>(a.logits) + (live ? t : t0) * a.ld * T::kSize;
  float x[V];
  load_elems<T, V>(row, e0, n, whole, full, -inf, x);
  bool doubt = false;
  float top = -inf;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    doubt |= x[j] != x[j];
    top = fmaxf(top, x[j]);
  }
  top = lanes_max<L>(top);
  doubt |= top == inf;
  // in binary64: softmax's sum over the row (read again: doubts are rare), and
  // a score with its bias
  double sum64 = 1.0;
  auto make_sum64 = [&]() {
    if constexpr (KEY == kBySoftmax) {
      float y[V];
      load_elems<T, V>(row, e0, n, whole, full, -inf, y);
      sum64 = 0.0;
#pragma unroll 1
      for (int j = 0; j < V; ++j) {
        float v = y[0];
#pragma unroll
        for (int i = 1; i < V; ++i) v = i == j ? y[i] + 0.0f : v;
        sum64 += v == -inf ? 0.0 : exp((double)v - (double)top);
      }
#pragma unroll
      for (int m = 1; m < L; m *= 2) sum64 += __shfl_xor(sum64, m, L);
    }
  };
  auto score64 = [&](float x, float b) {
    const double s = softmax ? exp((double)x - (double)top) / sum64 : 1.0 / (1.0 + exp(-(double)x));
    return by_logit ? s : s + (double)b;
  };
  double total = 0.0;  // softmax: sum of exp(x - top)
  if (softmax && !(by_logit && a.r.renorm)) {
#pragma unroll
    for (int j = 0; j < V; ++j) total += x[j] == -inf ? 0.0f : __builtin_amdgcn_exp2f((x[j] - top) * kLog2e);
    total = lanes_sum<L>(total);
  }
  uint32_t key[V];
  uint32_t tol = 0;
  if constexpr (by_logit) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t q = (0x7fffffffu - __float_as_uint(top - x[j])) >> (31 - QB);
      key[j] = x[j] == -inf ? 0 : q << IB | (L * V - 1 - (l * V + j));
    }
  } else {
    float v[V];
    float best = -inf;
    const float inv = 1.0f / (float)total;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float s = softmax ? __builtin_amdgcn_exp2f((x[j] - top) * kLog2e) * inv
                              : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x[j]));
      v[j] = x[j] == -inf ? -inf : s + b[j];
      doubt |= v[j] != v[j];
      best = fmaxf(best, v[j]);
    }
    best = lanes_max<L>(best);
    doubt |= best == inf;
    const float most = softmax ? inv : 1.0f;  // the largest score
    const float scale = (float)(1u << (QB - 1)) / fmaxf(fabsf(best), most);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t d = (uint32_t)fminf((best - v[j]) * scale, (float)(QMAX - 1));
      key[j] = v[j] == -inf ? 0 : (QMAX - d) << IB | (L * V - 1 - (l * V + j));
    }
    tol = ((softmax ? 37u : 12u) >> (24 - QB)) + (QB < 24);
  }
  sort_down<V>(key);
  if (G > 1) {
    // the group's two largest keys, over its lanes
    uint32_t m0 = key[0], m1 = V > 1 ? key[V > 1 ? 1 : 0] : 0;
    auto merge = [&](auto d) {
      constexpr int D = decltype(d)::value;
      uint32_t o0, o1;
      if constexpr (D <= 8) {
        constexpr int C = D == 1 ? kDppXor1 : D == 2 ? kDppXor2 : D == 4 ? kDppHalfMirror : kDppMirror;
        o0 = dpp<C>(m0), o1 = dpp<C>(m1);
      } else if constexpr (D == 16) {
        const auto r0 = __builtin_amdgcn_permlane16_swap(m0, m0, false, false);
        const auto r1 = __builtin_amdgcn_permlane16_swap(m1, m1, false, false);
        m0 = r0[0], o0 = r0[1], m1 = r1[0], o1 = r1[1];
      } else {
        const auto r0 = __builtin_amdgcn_permlane32_swap(m0, m0, false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(m1, m1, false, false);
        m0 = r0[0], o0 = r0[1], m1 = r1[0], o1 = r1[1];
      }
      const uint32_t lo = m0 < o0 ? m0 : o0, hi = m1 > o1 ? m1 : o1;
      m0 = m0 > o0 ? m0 : o0;
      m1 = lo > hi ? lo : hi;
    };
    if (ps > 0) merge(std::integral_constant<int, 1>{});
    if (ps > 1) merge(std::integral_constant<int, 2>{});
    if (ps > 2) merge(std::integral_constant<int, 4>{});
    if (ps > 3) merge(std::integral_constant<int, 8>{});
    if (L > 16 && ps > 4) merge(std::integral_constant<int, 16>{});
    const bool two = a.r.group_top == 2 && gs > 1;
    uint32_t worth = m0 >> IB;
    if (two) worth = m1 ? worth + (m1 >> IB) : 0;
    const bool cut = !by_logit && ((m0 >> IB) == 1 || (two && (m1 >> IB) == 1));
    const uint32_t mine = worth && g < G ? worth << 6 | (63 - g) : 0;
    // the topk_groups-th largest, and the next
    uint32_t left = mine, last = 0, next = 0;
    for (uint32_t k = 0; k < (uint32_t)a.r.topk_groups; ++k) {
      last = lanes_max<L>(left);
      left = left == last ? 0 : left;
    }
    next = lanes_max<L>(left);
    bool kept = mine && mine >= last;
    bool near = last && next && (last >> 6) - (next >> 6) <= 2 * tol;
    // logits this near the best have equal scores in binary64 at times
    if (by_logit) near |= last && next >> 6 >= (0x7fffffffu - __float_as_uint(1e-10f)) >> (31 - QB);
    if (__any(near && live)) {
      make_sum64();
      // by the worths in binary64, every lane its own group's; the keys
      // that they sum have to be clear of the next one
      uint32_t third = 0;
#pragma unroll
      for (int j = V > 2 ? 2 : V - 1; j >= 0; --j) third = key[j] != m0 && (!two || key[j] != m1) ? key[j] + 0 : third;
      for (uint32_t d = 1; d < 1u << ps; d *= 2) {
        const uint32_t o = __shfl_xor(third, (int)d, L);
        third = o > third ? o : third;
      }
      const int away = (int)(mine >> 6) - (int)(last >> 6);
      doubt |= near && mine && third && (uint32_t)abs(away) <= 4 * tol &&
               ((two ? m1 : m0) >> IB) - (third >> IB) <= tol;
      uint64_t w64 = 0;
      if (mine) {
        const Choice c0 = chosen(row, m0), c1 = chosen(row, two ? m1 : m0);
        const double s0 = score64(c0.x, c0.b), s1 = score64(c1.x, c1.b);
        w64 = order64(two ? s0 + s1 : s0);
      }
      uint32_t before = 0;
      for (uint32_t o = 0; o < G; ++o) {
        const uint64_t v = __shfl((unsigned long long)w64, (int)(o << ps), L);
        before += v > w64 || (v == w64 && o < g);
      }
      kept = near ? mine && before < (uint32_t)a.r.topk_groups : kept;
    }
    doubt |= kept && cut;
    if (!kept) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = 0;
    }
  }
  // lane k: the k-th choice (0: none); lane topk: the next one
  uint32_t won = 0;
  auto round = [&](uint32_t k, int keep) {
    const uint32_t m = lanes_max<L>(key[0]);
    won = l == k ? m : won;
    const bool pop = key[0] == m;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < keep) {
        const uint32_t stay = key[j], next = j + 1 < V ? key[j + 1 < V ? j + 1 : j] + 0 : 0;
        key[j] = pop ? next : stay;
      }
  };
#pragma unroll
  for (int k = 0; k <= KB; ++k)
    if ((uint32_t)k <= K) round((uint32_t)k, KB + kMoreRounds - k);
  Choice c = chosen(row, won);
  const uint32_t q = won >> IB, next = from_next_lane(won, 0);
  const float nx = __uint_as_float(from_next_lane(__float_as_uint(c.x), 0));
  const float nb = __uint_as_float(from_next_lane(__float_as_uint(c.b), 0));
  bool near = false;
  if (l < K && won) {
    const float cx = c.x, cb = c.b;
    // binary64 scores of different logits may be equal where they saturate
    // (sigmoids of logits above 20 nearly so), underflow or lie too near
    doubt |= by_logit ? (softmax ? top - cx > 700.0f : cx > 20.0f || cx < -700.0f) : q == 1;
    doubt |= by_logit && next && cx != nx && cx - nx < 1e-13f;
    if (next && q - (next >> IB) <= tol) {
      const bool equal = cx == nx && cb == nb;
      // past an equal pair at the end there may be more, not looked at: two
      // bf16 logits of one code are equal unless far below the best
      const bool sure = l + 1 < K || (T::kSize == 2 && by_logit && (float)(1u << (QB - 17)) * fabsf(cx) >= top - cx);
      near = !(equal && sure);
    }
  }
  if (__any(near && live)) {
    make_sum64();
    // by the binary64 scores of the choices and of kMoreRounds after
    // them, the last of which has to be clear of the topk-th
#pragma unroll
    for (int r = 1; r <= kMoreRounds; ++r) round(K + r, kMoreRounds - r);
    const uint32_t end = __shfl(won, (int)(K + kMoreRounds), L);
    doubt |= l + 1 == K && end && q - (end >> IB) <= tol;
    c = chosen(row, won);
    const uint64_t k64 = won ? order64(score64(c.x, c.b)) : 0;
    uint32_t rank = 0;
    for (uint32_t o = 0; o <= K + kMoreRounds; ++o) {
      const uint64_t v = __shfl((unsigned long long)k64, (int)o, L);
      const int32_t v_id = __shfl(c.id, (int)o, L);
      rank += v > k64 || (v == k64 && v_id < c.id);
    }
    // to the lane of its rank (the lanes that nothing is sent to get 0)
    const uint32_t to = won ? rank : L - 1;
    won = (uint32_t)__builtin_amdgcn_ds_permute((int)((sub * L + to) * 4), (int)won);
    c = chosen(row, won);
  }
  const uint64_t again = __ballot(doubt && live);
  const float cx = c.x;
  // the weights of the chosen, lane k the k-th
  const bool have = l < K && won;
  const float sx = have ? cx : -inf;
  float w;
  if (softmax) {
    const float m = a.r.renorm ? lanes_max<L>(sx) : top;
    const float p = have ? expf(cx - m) : 0.0f;
    w = share(p, a.r.renorm ? lanes_sum<L>((double)p) : total, a.r.scale);
  } else if (a.r.renorm) {
    const float m = fminf(lanes_max<L>(sx), 0.0f);
    const float p = !have ? 0.0f : m < 0.0f ? expf(cx - m) / (1.0f + expf(cx)) : 1.0f / (1.0f + expf(-cx));
    w = share(p, lanes_sum<L>((double)p), a.r.scale);
  } else {
    w = scaled_sigmoid(cx, a.r.scale);
  }
  const uint64_t sub_lanes = (L == 64 ? ~0ull : (1ull << (L & 63)) - 1) << (sub * L % 64);
  if (l < K && live && !(again & sub_lanes)) {
    a.weights[t * K + l] = have ? w : 0.0f;
    a.ids[t * K + l] = have ? c.id : -1;
  }
  for (uint32_t s = 0; s < TPW; ++s)
    if (again >> (s * L % 64) & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1)) route_exact<T, VX>(a, t0 + s);
}

// The gradient, L lanes a token, V logits a lane.  UNITS: in 16-byte units,
// unit u of lane l being the row's unit u L + l, for rows of whole units; else
// by elements, j L + l.  Either way neighbouring lanes touch neighbouring
// memory (32768 x 128 f32: 7.7 us a call among others, the kernel 7.8 to 8.6;
// when that was 8.5, a lane's 8 logits side by side, in two units of every other
// 16 bytes, took 10.1, and 32 lanes of 4 logits 9.3).  The chosen
// experts' terms come to their lanes by way of LDS: lane k < topk works choice
// k out and adds it to the row's slot.  Sums over the row and quotients are
// binary64, the exponentials binary32.  Bound by HBM: the row is read once (not
// at all where only the chosen logits matter) and written once.
template <typename T, int L, int V, bool UNITS>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(const RouteBackwardArgs a) {
  constexpr uint32_t TPW = 64 / L;
  constexpr int N = kUnit<T>;
  __shared__ __align__(16) float lds[kRouteWaves][TPW][L * V];
  const uint32_t lane = threadIdx.x & 63u, l = lane % L, sub = lane / L;
  const uint32_t E = (uint32_t)a.r.experts, K = (uint32_t)a.r.topk;
  const bool softmax = a.r.score == SNAC_SCORE_SOFTMAX, renorm = a.r.renorm != 0;
  const float inf = __builtin_inff();
  float* row_up = lds[wave_id()][sub];
  // the row's element that is this lane's j-th
  auto at = [&](int j) { return UNITS ? ((j / N) * L + l) * N + j % N : j * L + l; };
  const uint64_t t0 = ((uint64_t)blockIdx.x * kRouteWaves + wave_id()) * TPW;
  if (t0 >= a.tokens) return;
  const bool live = t0 + sub < a.tokens;
  const uint64_t t = live ? t0 + sub : t0;
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * T::kSize;
  float x[V];
  if (softmax && !renorm) {
    // a lane without an element reads the row's first
    if constexpr (UNITS) {
      u32x4 w[V / N];
#pragma unroll
      for (int u = 0; u < V / N; ++u) w[u] = ld_unit<false>(row + (at(u * N) < E ? at(u * N) : 0) * T::kSize);
#pragma unroll
      for (int u = 0; u < V / N; ++u) {
        float f[N];
        unpack<T>(w[u], f);
#pragma unroll
        for (int c = 0; c < N; ++c) x[u * N + c] = at(u * N) < E ? f[c] + 0.0f : -inf;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = load_elem<T>(row + (at(j) < E ? at(j) : 0) * T::kSize);
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = at(j) < E ? x[j] + 0.0f : -inf;
    }
  }
  // the choices of this lane: one, or two where topk is above L
  constexpr int C = L < SNAC_MAX_TOPK ? 2 : 1;
  int32_t id[C];
  bool have[C];
  float dw[C], cx[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t k = l + c * L;
    id[c] = k < K ? a.ids[t * K + k] : -1;
    have[c] = id[c] >= 0 && (uint32_t)id[c] < E;
    dw[c] = have[c] ? a.dweights[t * K + k] * a.r.scale : 0.0f;
    cx[c] = have[c] ? load_logit<T>(row, (uint32_t)id[c]) : -inf;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) row_up[at(j)] = 0.0f;
  float g[C];  // what goes to the chosen slots
  double inv = 0.0, dot = 0.0;
  float top = -inf;
  if (softmax && !renorm) {
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
    top = lanes_max<L>(top);
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = x[j] == -inf ? 0.0f : __builtin_amdgcn_exp2f((x[j] - top) * kLog2e);
      total += x[j];
    }
    total = lanes_sum<L>(total);
    inv = total == 0.0 ? 0.0 : reciprocal(total);  // 0: every logit masked
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const double r = !have[c] || cx[c] == -inf ? 0.0 : expf(cx[c] - top) * inv;
      dot += have[c] ? r * dw[c] : 0.0;
    }
    dot = lanes_sum<L>(dot);
    // dw - dot is made in binary64: for a score near 1 hardly anything is left
    // of dw.  f32: with the product, below.  bf16: here, where a lane has one or
    // two of them (512 experts 14.3 us; below 15.4, all in binary32 13.4); a slot
    // of 0 is then one that was not chosen, so what is chosen is not 0.
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float up = (float)(dw[c] - dot);
      g[c] = T::kSize == 4 ? dw[c] : fabsf(up) < 0x1p-126f ? 0x1p-126f : up;
    }
  } else {
    float m = cx[0], r[C];
    double total = 0.0, part[C];
    if constexpr (C == 2) m = fmaxf(m, cx[1]);
    if (renorm) m = lanes_max<L>(m);
    if (!softmax) m = fminf(m, 0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      r[c] = 0.0f;
      if (have[c] && cx[c] != -inf)
        r[c] = softmax || (renorm && m < 0.0f) ? expf(cx[c] - m) : 1.0f / (1.0f + expf(-cx[c]));
      // the sigmoid's slope is its score times that of -x
      g[c] = softmax ? 1.0f : 1.0f / (1.0f + expf(cx[c]));
      if (!softmax && renorm && m < 0.0f) r[c] *= g[c];
      total += r[c];
    }
    if (renorm) total = lanes_sum<L>(total);
    inv = !renorm ? 1.0 : total == 0.0 ? 0.0 : reciprocal(total);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      part[c] = r[c] * inv;
      dot += have[c] ? part[c] * dw[c] : 0.0;
    }
    dot = renorm ? lanes_sum<L>(dot) : 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) g[c] = (float)(part[c] * g[c] * (dw[c] - dot));
  }
  // zeros, then the other lanes' terms, then this lane's slots
  wave_lds_order();
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (have[c]) atomicAdd(&row_up[id[c]], g[c]);
  wave_lds_order();
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = row_up[at(j)];
  if (softmax && !renorm) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (T::kSize == 4) d[j] = (float)(x[j] * __builtin_fma((double)d[j], inv, -inv * dot));
      else d[j] = x[j] * (float)inv * (d[j] == 0.0f ? (float)-dot : d[j]);
    }
  }
  if (!live) return;
  char* p = static_cast<char*>(a.dlogits) + t * a.ld_d * T::kSize;
  if constexpr (UNITS) {
#pragma unroll
    for (int u = 0; u < V / N; ++u) {
      float f[N];
#pragma unroll
      for (int c = 0; c < N; ++c) f[c] = d[u * N + c];
      if (at(u * N) < E) st_unit<true>(p + at(u * N) * T::kSize, pack<T>(f));
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (at(j) < E) store_elem<T>(p + at(j) * T::kSize, d[j]);
  }
}

uint32_t route_grid(uint64_t tokens) {
  const int cus = device_cu_count();
  const uint64_t most = (uint64_t)(cus > 0 ? cus : 1) * 16;
  const uint64_t want = (tokens + kRouteWaves - 1) / kRouteWaves;
  return (uint32_t)(want < most ? want : most);
}

// Lanes of a group when a lane holds V experts: 1 << ps.
uint32_t group_shift(const snac_router& r, uint32_t V) {
  const uint32_t gs = (uint32_t)(r.experts / r.groups);
  uint32_t ps = 0;
  while ((V << ps) < gs) ++ps;
  return ps;
}

template <typename T, int L, int V, int KB, int KEY>
bool route_fits(const RouteArgs& a, hipStream_t stream) {
  uint32_t ps = group_shift(a.r, V);
  if (a.r.topk > KB || a.r.topk + kMoreRounds + 1 > L || (uint64_t)a.r.groups << ps > L) return false;
  if (a.r.groups == 1) ps = __builtin_ctz(L);
  // a wave a set of tokens; in launches of fewer than 2^32 threads
  const uint64_t per = kRouteWaves * (64 / L), most = per << 23;
  RouteArgs c = a;
  for (uint64_t t = 0; t < a.tokens; t += most) {
    c.tokens = a.tokens - t < most ? a.tokens - t : most;
    c.logits = static_cast<const char*>(a.logits) + t * a.ld * T::kSize;
    c.weights = a.weights + t * (uint64_t)a.r.topk;
    c.ids = a.ids + t * (uint64_t)a.r.topk;
    hipLaunchKernelGGL((route_kernel<T, L, V, KB, KEY>), dim3((uint32_t)((c.tokens + per - 1) / per)),
                       dim3(kRouteThreads), 0, stream, c, ps, (uint32_t)(a.r.experts / a.r.groups));
  }
  return true;
}

// The narrowest shape that holds the experts; few tokens take a wave each.
template <typename T, int KEY>
void route_any(const RouteArgs& a, hipStream_t stream) {
  if (a.tokens > kRouteManyTokens &&
      (route_fits<T, 16, 1, 8, KEY>(a, stream) || route_fits<T, 16, 4, 8, KEY>(a, stream) || route_fits<T, 16, 8, 8, KEY>(a, stream) ||
       route_fits<T, 16, 16, 8, KEY>(a, stream) || route_fits<T, 32, 16, 8, KEY>(a, stream) ||
       route_fits<T, 16, 4, 12, KEY>(a, stream) || route_fits<T, 16, 16, 12, KEY>(a, stream) ||
       route_fits<T, 32, 16, 12, KEY>(a, stream)))
    return;
  if (route_fits<T, 64, 1, 8, KEY>(a, stream) || route_fits<T, 64, 4, 8, KEY>(a, stream) || route_fits<T, 64, 16, 8, KEY>(a, stream))
    return;
  if (route_fits<T, 64, 1, 32, KEY>(a, stream) || route_fits<T, 64, 4, 32, KEY>(a, stream) || route_fits<T, 64, 16, 32, KEY>(a, stream))
    return;
  // more than 560 experts in groups that take more than 64 lanes between them,
  // each a power of two of them (3 groups of 340: 32 lanes each): 32768 tokens of
  // 1020 f32 in 3 groups 283 us, where 1024 in 4 groups take 69
  hipLaunchKernelGGL((route_exact_kernel<T, 16>), dim3(route_grid(a.tokens)), dim3(kRouteThreads), 0, stream, a);
}

template <typename T>
void route_by_key(const RouteArgs& a, hipStream_t stream) {
  const snac_router& r = a.r;
  if (!a.bias && (r.groups == 1 || r.group_top == 1 || r.groups == r.experts)) route_any<T, kByLogit>(a, stream);
  else if (r.score == SNAC_SCORE_SIGMOID) route_any<T, kBySigmoid>(a, stream);
  else route_any<T, kBySoftmax>(a, stream);
}

template <typename T, int L, int V>
void route_backward_in(const RouteBackwardArgs& a, hipStream_t stream) {
  const uint64_t per = kRouteWaves * (64 / L), most = per << 23;
  RouteBackwardArgs c = a;
  for (uint64_t t = 0; t < a.tokens; t += most) {
    c.tokens = a.tokens - t < most ? a.tokens - t : most;
    c.logits = static_cast<const char*>(a.logits) + t * a.ld * T::kSize;
    c.ids = a.ids + t * (uint64_t)a.r.topk;
    c.dweights = a.dweights + t * (uint64_t)a.r.topk;
    c.dlogits = static_cast<char*>(a.dlogits) + t * a.ld_d * T::kSize;
    const dim3 grid((uint32_t)((c.tokens + per - 1) / per)), block(kRouteThreads);
    bool units = false;
    if constexpr (V >= (int)kUnit<T>) {
      units = a.r.experts % kUnit<T> == 0;
      if (units) hipLaunchKernelGGL((route_backward_kernel<T, L, V, true>), grid, block, 0, stream, c);
    }
    if (!units) hipLaunchKernelGGL((route_backward_kernel<T, L, V, false>), grid, block, 0, stream, c);
  }
}

template <typename T>
void route_backward_any(const RouteBackwardArgs& a, hipStream_t stream) {
  const int e = a.r.experts;
  if (e <= 16) route_backward_in<T, 16, 1>(a, stream);
  else if (e <= 64) route_backward_in<T, 16, 4>(a, stream);
  else if (e <= 128) route_backward_in<T, 16, 8>(a, stream);
  else if (e <= 256) route_backward_in<T, 16, 16>(a, stream);
  else if (e <= 512) route_backward_in<T, 32, 16>(a, stream);
  else route_backward_in<T, 64, 16>(a, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) route_by_key<BF16>(a, stream);
  else route_by_key<F32>(a, stream);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) route_backward_any<BF16>(a, stream);
  else route_backward_any<F32>(a, stream);
  return hipGetLastError();
}

}  // namespace snac
