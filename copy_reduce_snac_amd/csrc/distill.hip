// distill.hip -- the divergence from a teacher's top logits, over the whole
// vocabulary or a shard of it, and its gradient (snac_distill and its kin in
// include/snac_ops.h).
#include <hip/hip_runtime.h>

#include "ops.hpp"
#include "rows.hpp"

namespace snac {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxSlots = SNAC_MAX_TEACHER / 64;  // of a lane, see Choices
constexpr double kLog2e = 1.4426950408889634;

// A token's choices, up to 64 C of them, choice c * 64 + lane in slot c of a lane:
// their columns (-1: not valid), the teacher's logits, and after weigh() their q.
template <int C>
struct Choices {
  int64_t id[C];
  float t[C], q[C];
  float top;     // the largest valid logit
  double total;  // sum of exp((t - top) / temperature)
  bool any;      // a valid choice: the token has a part

  __device__ __forceinline__ void load(const snac_teacher& a, uint64_t token) {
    const uint32_t lane = threadIdx.x & 63u;
    const float inf = __builtin_inff();
    const uint64_t at = token * (uint32_t)a.topk;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t k = c * 64 + lane;
      id[c] = -1;
      t[c] = -inf;
      if (c * 64 >= a.topk) continue;
      if (k < (uint32_t)a.topk) {
        id[c] = load_id(a.ids, a.id_bytes, at + k);
        t[c] = a.dtype == SNAC_BF16 ? bf16_lo(static_cast<const uint16_t*>(a.logits)[at + k])
                                    : static_cast<const float*>(a.logits)[at + k];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if ((uint64_t)id[c] >= (uint64_t)a.vocab || t[c] == -inf) id[c] = -1, t[c] = -inf;
  }
  // scale: log2(e) / temperature
  __device__ __forceinline__ void weigh(float scale) {
    const float inf = __builtin_inff();
    top = -inf;
    bool mine = false;
#pragma unroll
    for (int c = 0; c < C; ++c) top = fmaxf(top, t[c]), mine |= id[c] >= 0;
    any = __any(mine);
    top = wave_max(top);
    if (top == -inf) top = 0.0f;
    total = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      q[c] = __builtin_amdgcn_exp2f((t[c] - top) * scale);
      total += q[c];
    }
    total = wave_sum(total);
    const double inv = total == 0.0 ? 0.0 : 1.0 / total;
#pragma unroll
    for (int c = 0; c < C; ++c) q[c] = (float)(q[c] * inv);
  }
  // sum of q log q
  __device__ __forceinline__ double entropy(double inv_tau) const {
    const double log_total = total == 0.0 ? 0.0 : log(total);
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (q[c] != 0.0f) s += (double)q[c] * (((double)t[c] - (double)top) * inv_tau - log_total);
    return wave_sum(s);
  }
};

__device__ __forceinline__ float choice_scale(const snac_teacher& a) { return (float)(kLog2e / (double)a.temperature); }

// Largest logit and sum of exponentials of what a lane has seen of a row.  The
// sum is taken relative to the largest so far: one pass.
struct Running {
  float m;
  double s;
  __device__ __forceinline__ void start() { m = -__builtin_inff(), s = 0.0; }
  // brought to another maximum
  __device__ __forceinline__ double at(float top, float scale) const {
    return m == -__builtin_inff() ? s : s * (double)__builtin_amdgcn_exp2f((m - top) * scale);
  }
  template <int U, uint32_t N>
  __device__ __forceinline__ void add(const float (&f)[U][N], float scale) {
    float top = m;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) top = fmaxf(top, f[j][c]);
    if (__any(top > m)) {
      s = at(top, scale);
      m = top;
    }
    const float ref = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float part = 0.0f;
#pragma unroll
      for (uint32_t c = 0; c < N; ++c) part += __builtin_amdgcn_exp2f((f[j][c] - ref) * scale);
      s += part;
    }
  }
  __device__ __forceinline__ void over_wave(float scale) {
    const float top = wave_max(m);
    s = wave_sum(at(top, scale));
    m = top;
  }
};

constexpr int kUnits = 4;  // of a lane at a time

// loss = sum over the choices of q (log q - log p), q the softmax of their logits, p
// that of the row, both at the teacher's temperature: sum q log q - sum q (x - max) /
// temperature + log(sum exp((x - max) / temperature)).  A shard's part is the maximum,
// the sum and its choices' sums of q (x - max) / temperature and of q.
//
// A row by W waves (kWaves rows a workgroup where W is 1), once through.  The last
// wave, which has the fewest pieces, sees to the choices before it begins and
// makes the loss of them in the end.
//
// Bound by HBM: 4096 x 131072 bf16 163 us, 6.6 TB/s read; 2048 x 131072 f32 157, 6.8.
// Units are counted from a row's first element, so rows that begin off the 16 bytes
// straddle with every access, and the lines that two accesses share are not read past
// the caches: 4096 x 50258 bf16 77 us, 5.3, and of 50257, off the 4 bytes, 89.  A unit's
// exponentials are summed in binary32 and units in binary64; the maximum so far moves
// for a whole wave at a time, which it seldom does.  7 x 32768 f32 takes 6.5 us, one
// workgroup of 16 waves a row.
template <typename T, int W, int C>
__global__ __launch_bounds__(W == 1 ? kThreads : 64 * W) void distill_kernel(const DistillArgs a) {
  constexpr uint32_t N = kUnit<T>, kPiece = 64u * kUnits * N;
  constexpr uint32_t kRows = W == 1 ? kWaves : 1;
  __shared__ float tops[W];
  __shared__ double totals[W];
  const uint32_t lane = threadIdx.x & 63u, w = W == 1 ? 0 : wave_id();
  const float inf = __builtin_inff(), scale = choice_scale(a.teacher);
  const double inv_tau = 1.0 / (double)a.teacher.temperature;
  const uint32_t pieces = (uint32_t)(((uint64_t)a.width + kPiece - 1) / kPiece);
  const bool lines = whole_lines(a.logits, a.ld);
  for (uint64_t t = (uint64_t)blockIdx.x * kRows + (W == 1 ? wave_id() : 0); t < a.tokens; t += (uint64_t)gridDim.x * kRows) {
    const char* row = a.logits + t * a.ld;
    u32x4 next[kUnits] = {};
    auto load = [&](uint32_t p) {
      const char* at = row + (uint64_t)p * kPiece * T::kSize;
      if (lines) ld_held<T, kUnits, true>(at, a.width - p * kPiece, a.width, next);
      else ld_held<T, kUnits, false>(at, a.width - p * kPiece, a.width, next);
    };
    if (w < pieces) load(w);
    Choices<C> k;
    float z[C];
    bool here[C];
    auto choices = [&] {
      k.load(a.teacher, t);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t at = k.id[c] - a.first;
        here[c] = k.id[c] >= 0 && (uint64_t)at < a.width;
        z[c] = here[c] ? load_elem<T>(row + at * (int64_t)T::kSize) : 0.0f;
      }
      k.weigh(scale);
    };
    constexpr bool kEarly = C == 1 && W < 16;  // else they cost the loop registers
    if (kEarly && w == W - 1) choices();
    Running r;
    r.start();
    for (uint32_t p = w; p < pieces; p += W) {
      float f[kUnits][N];
      const uint32_t left = a.width - p * kPiece;
#pragma unroll
      for (int j = 0; j < kUnits; ++j) unpack<T>(next[j], f[j]);
      if (pieces - p > W) load(p + W);
      if (left < kPiece) {
        settle_held<T, kUnits>(left, a.width, f);
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
#pragma unroll
          for (uint32_t c = 0; c < N; ++c)
            if ((j * 64u + lane) * N + c >= left) f[j][c] = -inf;
      }
      r.add(f, scale);
    }
    r.over_wave(scale);
    if constexpr (W > 1) {
      if (lane == 0) tops[w] = r.m, totals[w] = r.s;
      __syncthreads();
      if (w == W - 1) {
        r.start();
        if (lane < W) r.m = tops[lane], r.s = totals[lane];
        r.over_wave(scale);
      }
      if (a.tokens - t > gridDim.x) __syncthreads();  // they are read
      if (w != W - 1) continue;
    }
    if (!kEarly) choices();
    double d = 0.0, q = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!here[c] || k.q[c] == 0.0f) continue;
      d += (double)k.q[c] * (z[c] == -inf ? -HUGE_VAL : ((double)z[c] - (double)r.m) * inv_tau);
      q += k.q[c];
    }
    d = wave_sum(d);
    if (a.loss) {
      const double ent = k.entropy(inv_tau);
      if (lane == 0) {
        a.loss[t] = !k.any || r.s == 0.0 ? 0.0f : (float)(ent - d + log(r.s));
        a.stats[2 * t] = r.m;
        a.stats[2 * t + 1] = (float)r.s;
      }
    } else {
      q = wave_sum(q);
      if (lane == 0) {
        float* part = a.part + 4 * t;
        part[0] = r.m;
        part[1] = (float)r.s;
        part[2] = (float)d;
        part[3] = (float)q;
      }
    }
  }
}

// The shards' parts brought to the largest maximum and added up, in binary64.  A token
// a wave, a shard's part a lane: latency, 1021 tokens 3.2 us.
template <int C>
__global__ __launch_bounds__(kThreads) void distill_join_kernel(const DistillArgs a) {
  const uint32_t lane = threadIdx.x & 63u;
  const float inf = __builtin_inff();
  const double inv_tau = 1.0 / (double)a.teacher.temperature;
  for (uint64_t t = (uint64_t)blockIdx.x * kWaves + wave_id(); t < a.tokens; t += (uint64_t)gridDim.x * kWaves) {
    float m = -inf, s = 0.0f, d = 0.0f, q = 0.0f;
    if (lane < (uint32_t)a.shards) {
      const float* part = a.parts + 4 * (lane * a.tokens + t);
      m = part[0], s = part[1], d = part[2], q = part[3];
    }
    Choices<C> k;
    k.load(a.teacher, t);
    k.weigh(choice_scale(a.teacher));
    const float top = wave_max(m);
    const double gap = ((double)m - (double)top) * inv_tau;
    const double total = wave_sum(m == -inf ? (double)s : (double)s * exp(gap));
    const double dot = wave_sum(q == 0.0f ? 0.0 : (double)d + (double)q * gap);
    const double ent = k.entropy(inv_tau);
    if (lane == 0) {
      a.loss[t] = !k.any || total == 0.0 ? 0.0f : (float)(ent - dot + log(total));
      a.stats[2 * t] = top;
      a.stats[2 * t + 1] = (float)total;
    }
  }
}

// dlogits = scale dloss / temperature (p - q), q 0 but at the choices' columns.
// One workgroup a run of a row's pieces, a wave every kBackWaves-th of them.  Its
// first wave makes the choices' q while the others' logits are on their way; a
// piece that holds a choice's column takes its q off before the rounding.
//
// Bound by HBM: 4096 x 131072 bf16, 64 choices, 338 us, 6.4 TB/s read and written (256
// choices 391); 509 x 32003 f32 21.8, 6.0.  Runs of 16 KiB: shorter ones make their
// choices' q too often, longer ones leave the CUs unevenly done.
constexpr int kBackWaves = 4;
constexpr int kBackUnits = 2;  // of a lane at a time
constexpr uint32_t kBackTurns = 2;

template <typename T, int C>
__global__ __launch_bounds__(64 * kBackWaves) void distill_backward_kernel(const DistillArgs a, uint32_t pieces, uint32_t per,
                                                                           uint32_t runs, uint64_t items) {
  constexpr uint32_t N = kUnit<T>, kPiece = 64u * kBackUnits * N;
  __shared__ uint32_t columns[C * 64];  // of the run's choices, counted from its first
  __shared__ float offs[C * 64];
  __shared__ uint32_t some;
  const uint32_t lane = threadIdx.x & 63u, w = wave_id();
  const float scale = choice_scale(a.teacher);
  const bool lines = whole_lines(a.logits, a.ld);
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint64_t t = it / runs;
    const uint32_t p0 = (uint32_t)(it - t * runs) * per, p1 = pieces - p0 < per ? pieces : p0 + per;
    const char* row = a.logits + t * a.ld;
    char* out = a.dlogits + t * a.ld_d;
    u32x4 next[kBackUnits];
    auto load = [&](uint32_t p) {
      const char* at = row + (uint64_t)p * kPiece * T::kSize;
      if (lines) ld_held<T, kBackUnits, true>(at, a.width - p * kPiece, a.width, next);
      else ld_held<T, kBackUnits, false>(at, a.width - p * kPiece, a.width, next);
    };
    if (p0 + w < p1) load(p0 + w);
    const float top = a.stats[2 * t], total = a.stats[2 * t + 1];
    const double whole = (double)a.scale / (double)a.teacher.temperature * (a.dloss ? (double)a.dloss[t] : 1.0);
    // beyond binary32 by a power of two that the differences get back; 2^100 of it stays,
    // for the smallest shares to be normal numbers with it
    const int power = (int)uniform(fabs(whole) >= 0x1p126 && isfinite(whole) ? (uint32_t)(ilogb(whole) - 100) : 0u);
    const float factor = (float)ldexp(whole, -power);
    const float f0 = (float)((double)factor / (double)total);
    if (w == 0) {
      Choices<C> k;
      k.load(a.teacher, t);
      k.weigh(scale);
      const int64_t e0 = a.first + (int64_t)p0 * kPiece;
      const uint64_t many = (uint64_t)(p1 - p0) * kPiece, left = a.width - (uint64_t)p0 * kPiece;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t at = k.id[c] - e0;
        columns[c * 64 + lane] = k.id[c] >= 0 && (uint64_t)at < (left < many ? left : many) ? (uint32_t)at : ~0u;
        offs[c * 64 + lane] = factor * k.q[c];
      }
      if (lane == 0) some = k.any;
    }
    __syncthreads();
    const bool part = some != 0 && total != 0.0f;
    uint32_t column[C];
#pragma unroll
    for (int c = 0; c < C; ++c) column[c] = columns[c * 64 + lane];
    for (uint32_t p = p0 + w; p < p1; p += kBackWaves) {
      const uint32_t left = a.width - p * kPiece;
      float f[kBackUnits][N];
#pragma unroll
      for (int j = 0; j < kBackUnits; ++j) unpack<T>(next[j], f[j]);
      if (left < kPiece) settle_held<T, kBackUnits>(left, a.width, f);
      if (p1 - p > kBackWaves) load(p + kBackWaves);
#pragma unroll
      for (int j = 0; j < kBackUnits; ++j)
#pragma unroll
        for (uint32_t c = 0; c < N; ++c) f[j][c] = f0 * __builtin_amdgcn_exp2f((f[j][c] - top) * scale);
      if (part) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t at = column[c] - (p - p0) * kPiece;
          uint64_t hits = __ballot(column[c] != ~0u && at < kPiece);
          while (hits) {
            const uint32_t l = (uint32_t)__builtin_ctzll(hits);
            hits &= hits - 1;
            const uint32_t col = (uint32_t)__builtin_amdgcn_readlane((int)at, (int)l);
            const uint32_t unit = col / N, el = col % N;
            const float off = (unit & 63u) == lane ? offs[c * 64 + l] : 0.0f;
#pragma unroll
            for (uint32_t j = 0; j < kBackUnits; ++j) {
              if (unit / 64 != j) continue;
#pragma unroll
              for (uint32_t i = 0; i < N; ++i)
                if (el == i) f[j][i] = f[j][i] - off;
            }
          }
        }
      }
      u32x4 v[kBackUnits];
#pragma unroll
      for (int j = 0; j < kBackUnits; ++j) v[j] = part ? pack<T>(f[j]) : u32x4{0, 0, 0, 0};
      if (power != 0) {  // exact, also after the rounding; before it it costs 20 registers
#pragma unroll
        for (int j = 0; j < kBackUnits; ++j) {
          float g[N];
          unpack<T>(v[j], g);
#pragma unroll
          for (uint32_t c = 0; c < N; ++c) g[c] = ldexpf(g[c], power);
          v[j] = pack<T>(g);
        }
      }
      st_held<T, kBackUnits, true>(out + (uint64_t)p * kPiece * T::kSize, left, v);
    }
    if (items - it > gridDim.x) __syncthreads();  // the choices are read
  }
}

uint32_t cus() {
  const int n = device_cu_count();
  return n > 0 ? (uint32_t)n : 1;
}

constexpr uint64_t kMaxGrid = 1u << 22;  // workgroups; grid-stride past them

template <typename T, int C>
void distill_any(const DistillArgs& a, hipStream_t stream) {
  const uint64_t bytes = (uint64_t)a.width * T::kSize;
  auto grid = [&](uint64_t rows) {
    const uint64_t want = (a.tokens + rows - 1) / rows;
    return dim3((uint32_t)(want < kMaxGrid ? want : kMaxGrid));
  };
  // Waves a row: one has its sums without a barrier, more have it sooner.  us, 1 / 4
  // waves: 8192 x 9001 bf16 40 / 58, 2000 x 16384 15.9 / 19.5, 700 x 16384 10.4 /
  // 9.0, 8192 x 32768 96 / 97, f32 92 / 84 at 8192 x 16384; 4 / 16: 500 x 9001 bf16
  // 8.2 / 10.2.
  const uint64_t cu = cus();
  if (bytes <= 16384 || (bytes <= 32768 && a.tokens >= cu * 4))
    hipLaunchKernelGGL((distill_kernel<T, 1, C>), grid(kWaves), dim3(kThreads), 0, stream, a);
  else if (bytes <= 65536 || a.tokens >= cu * 2)
    hipLaunchKernelGGL((distill_kernel<T, 4, C>), grid(1), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((distill_kernel<T, 16, C>), grid(1), dim3(1024), 0, stream, a);
}

template <typename T, int C>
void distill_backward_any(const DistillArgs& a, hipStream_t stream) {
  constexpr uint32_t kPiece = 64u * kBackUnits * kUnit<T>;
  const uint32_t pieces = (uint32_t)(((uint64_t)a.width + kPiece - 1) / kPiece);
  // runs of about kBackWaves * kBackTurns pieces, of equal lengths
  constexpr uint32_t kRun = kBackWaves * kBackTurns;
  const uint32_t about = pieces < kRun ? 1 : (pieces + kRun / 2) / kRun;
  const uint32_t per = (pieces + about - 1) / about, runs = (pieces + per - 1) / per;
  const uint64_t items = a.tokens * runs;
  hipLaunchKernelGGL((distill_backward_kernel<T, C>), dim3((uint32_t)(items < kMaxGrid ? items : kMaxGrid)),
                     dim3(64 * kBackWaves), 0, stream, a, pieces, per, runs, items);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, bool bf16, hipStream_t stream) {
  const bool few = a.teacher.topk <= 64;
  if (bf16) few ? distill_any<BF16, 1>(a, stream) : distill_any<BF16, kMaxSlots>(a, stream);
  else few ? distill_any<F32, 1>(a, stream) : distill_any<F32, kMaxSlots>(a, stream);
  return hipGetLastError();
}

hipError_t launch_distill_join(const DistillArgs& a, hipStream_t stream) {
  const uint64_t want = (a.tokens + kWaves - 1) / kWaves;
  const dim3 grid((uint32_t)(want < kMaxGrid ? want : kMaxGrid));
  if (a.teacher.topk <= 64) hipLaunchKernelGGL((distill_join_kernel<1>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((distill_join_kernel<kMaxSlots>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_distill_backward(const DistillArgs& a, bool bf16, hipStream_t stream) {
  const bool few = a.teacher.topk <= 64;
  if (bf16) few ? distill_backward_any<BF16, 1>(a, stream) : distill_backward_any<BF16, kMaxSlots>(a, stream);
  else few ? distill_backward_any<F32, 1>(a, stream) : distill_backward_any<F32, kMaxSlots>(a, stream);
  return hipGetLastError();
}

}  // namespace snac
