// ops.hip -- the C ABI declared in include/snac_ops.h: argument validation,
// sizes and launches of the operators beside the collectives.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "internal.hpp"
#include "ops.hpp"

using namespace snac;

namespace {
// addresses lo .. hi - 1, those of tensor `i` of a list
struct Extent {
  uintptr_t lo, hi;
  size_t i;
};
}  // namespace

struct snac_grads {
  int device;
  std::vector<Extent> outs, all;  // what the list writes; and reads: neither holds a call's norm
  uint32_t ntiles;
  GradTile* tiles;   // device; then the partial sums, the ticket and the counters
  double* partial;   // kGradMaxBlocks
  uint32_t* ticket;  // 0 between calls
  unsigned long long* pool;  // tile counters of snac_clip_grads, 0 between calls
};

namespace {

constexpr uint64_t kMaxWidth = 1ull << 31;  // elements of a row
constexpr uint64_t kMaxRows = 1ull << 31;

uint64_t esize(snac_dtype t) { return t == SNAC_BF16 ? 2 : 4; }
bool is_float(int t) { return t == SNAC_F32 || t == SNAC_BF16; }

// One argument's memory: `rows` rows of `width` bytes, `ld` bytes apart.
struct Span {
  const char* name;
  const void* p;
  uint64_t rows, width, ld;
  bool out;
};

Span array(const char* name, const void* p, uint64_t bytes, bool out) { return {name, p, 1, bytes, bytes, out}; }

bool empty(const Span& s) { return s.rows == 0 || s.width == 0; }

// bytes from the first to past the last (checked against SNAC_MAX_BYTES)
unsigned __int128 extent(const Span& s) {
  return empty(s) ? 0 : (unsigned __int128)(s.rows - 1) * s.ld + s.width;
}

bool overlap(const Span& a, const Span& b) {
  if (empty(a) || empty(b)) return false;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  if (!(pa < pb + (uint64_t)extent(b) && pb < pa + (uint64_t)extent(a))) return false;
  // columns of one wider matrix: the rows interleave without touching (a single
  // row lies in the other's matrix, whatever its own stride)
  const uint64_t ld = a.rows > 1 ? a.ld : b.ld;
  if (b.rows == 1 || b.ld == ld) {
    const uint64_t d = pa < pb ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;
    if (d >= a.width && d + b.width <= ld) return false;
  }
  return true;
}

// Every span: a pointer where there are bytes, its element alignment (given
// in `align`), its extent; and no output over another span.  `may`: the one
// output that may be `with` itself.
template <size_t N>
snac_status check_spans(const Span (&s)[N], const uint64_t (&align)[N], const void* may = nullptr,
                        const void* with = nullptr) {
  for (size_t i = 0; i < N; ++i) {
    if (empty(s[i])) continue;
    if (!s[i].p) return fail(SNAC_E_ARG, "%s is NULL", s[i].name);
    if ((uintptr_t)s[i].p % align[i])
      return fail(SNAC_E_ARG, "%s not aligned to %llu bytes", s[i].name, (unsigned long long)align[i]);
    if (extent(s[i]) > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%s: extent above SNAC_MAX_BYTES", s[i].name);
  }
  for (size_t i = 0; i < N; ++i) {
    if (!s[i].out) continue;
    for (size_t j = 0; j < N; ++j) {
      if (j == i || (s[j].out && j < i) || !overlap(s[i], s[j])) continue;
      if (may && may == with && s[i].p == may && s[j].p == with && s[i].ld == s[j].ld && s[i].width == s[j].width)
        continue;
      return fail(SNAC_E_ARG, "%s overlaps %s", s[i].name, s[j].name);
    }
  }
  return SNAC_OK;
}

snac_status check_dtype(snac_dtype t, const char* what) {
  if (!is_float(t)) return fail(SNAC_E_ARG, "%s must be SNAC_F32 or SNAC_BF16", what);
  return SNAC_OK;
}

snac_status check_id_bytes(int b) {
  if (b != 4 && b != 8) return fail(SNAC_E_ARG, "id_bytes %d is not 4 or 8", b);
  return SNAC_OK;
}

snac_status check_router(const snac_router* r, bool forward) {
  if (!r) return fail(SNAC_E_ARG, "router is NULL");
  if (r->experts < 1 || r->experts > SNAC_MAX_EXPERTS)
    return fail(SNAC_E_ARG, "experts %d outside 1..%d", r->experts, SNAC_MAX_EXPERTS);
  if (r->topk < 1 || r->topk > SNAC_MAX_TOPK || r->topk > r->experts)
    return fail(SNAC_E_ARG, "topk %d outside 1..%d or above experts %d", r->topk, SNAC_MAX_TOPK, r->experts);
  if (r->score != SNAC_SCORE_SOFTMAX && r->score != SNAC_SCORE_SIGMOID) return fail(SNAC_E_ARG, "unknown score %d", r->score);
  if (r->renorm != 0 && r->renorm != 1) return fail(SNAC_E_ARG, "renorm %d is not 0 or 1", r->renorm);
  if (!forward) return SNAC_OK;
  if (r->groups < 1 || r->groups > 64 || r->experts % r->groups)
    return fail(SNAC_E_ARG, "groups %d outside 1..64 or no divisor of experts %d", r->groups, r->experts);
  if (r->topk_groups < 1 || r->topk_groups > r->groups)
    return fail(SNAC_E_ARG, "topk_groups %d outside 1..%d", r->topk_groups, r->groups);
  if (r->group_top != 1 && r->group_top != 2) return fail(SNAC_E_ARG, "group_top %d is not 1 or 2", r->group_top);
  if (r->topk > r->topk_groups * (r->experts / r->groups))
    return fail(SNAC_E_ARG, "topk %d above the %d experts of the groups that stay", r->topk,
                r->topk_groups * (r->experts / r->groups));
  return SNAC_OK;
}

// Extents in ascending order of which no two overlap (then their ends ascend
// too): the first that ends after `at`.
std::vector<Extent>::const_iterator first_after(const std::vector<Extent>& v, uintptr_t at) {
  return std::upper_bound(v.begin(), v.end(), at, [](uintptr_t x, const Extent& e) { return x < e.hi; });
}

bool holds(const std::vector<Extent>& v, const void* p, uint64_t bytes) {
  const auto e = first_after(v, (uintptr_t)p);
  return e != v.end() && e->lo < (uintptr_t)p + bytes;
}

// An output of a list of tensors may be its own tensor's source and nothing
// else of the list: it would be clipped twice, or while others read it.  Sorts
// `outs` by address.
snac_status check_outs(std::vector<Extent>& outs, const std::vector<Extent>& srcs) {
  std::sort(outs.begin(), outs.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  for (size_t k = 1; k < outs.size(); ++k)
    if (outs[k].lo < outs[k - 1].hi)
      return fail(SNAC_E_ARG, "the output of tensor %zu overlaps that of tensor %zu", outs[k].i, outs[k - 1].i);
  for (const Extent& s : srcs)
    for (auto o = first_after(outs, s.lo); o != outs.end() && o->lo < s.hi; ++o)
      if (o->i != s.i) return fail(SNAC_E_ARG, "the output of tensor %zu overlaps src[%zu]", o->i, s.i);
  return SNAC_OK;
}

// Overlapping and touching extents as one, in ascending order.
void merge(std::vector<Extent>& v) {
  std::sort(v.begin(), v.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  size_t n = 0;
  for (const Extent& e : v) {
    if (n && e.lo <= v[n - 1].hi) v[n - 1].hi = std::max(v[n - 1].hi, e.hi);
    else v[n++] = e;
  }
  v.resize(n);
}

// Row strides and counts of a matrix argument.
snac_status check_rows(const char* name, uint64_t rows, uint64_t width, uint64_t ld) {
  if (rows > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%s: %llu rows above SNAC_MAX_BYTES", name, (unsigned long long)rows);
  if (width >= kMaxWidth) return fail(SNAC_E_ARG, "%s: width %llu not below 2^31", name, (unsigned long long)width);
  if (ld < width) return fail(SNAC_E_ARG, "%s: row stride %llu below the width %llu", name, (unsigned long long)ld, (unsigned long long)width);
  if (ld > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%s: row stride above SNAC_MAX_BYTES", name);
  return SNAC_OK;
}

snac_status check_topk(int topk) {
  if (topk < 1 || topk > SNAC_MAX_TOPK) return fail(SNAC_E_ARG, "topk %d outside 1..%d", topk, SNAC_MAX_TOPK);
  return SNAC_OK;
}

#define TRY(x)                        \
  do {                                \
    const snac_status st_ = (x);      \
    if (st_ != SNAC_OK) return st_;   \
  } while (0)

// radix digits of an embedding gradient's keys 0 .. vocab
constexpr uint32_t kDigitBits = 10;
// Zeros written beside a counting and a placing launch, and by a workgroup.
// They go to every row, also to those that get a sum later, so only where
// there are fewer tokens than rows: how many of these are different is not known
// before the sort.  us, with them / without:
//   32768 x 2048 f32   4096 different tokens 57.4 / 67.9; 16384 88.9 / 96.7;
//                      32440 126.1 / 126.5
//   65536 x 2048 f32   32768 tokens, 10399 different 133 / 145; 64880 different
//                      243 / 248
//   32768 x 4096 bf16  4096 different 59.0 / 70.0; 24576 120 / 123; 32440 142 /
//                      138, the only one of 77 cases that they cost anything
// As many tokens as rows and more: 32768 into 8192 x 2048 f32 75 us with these,
// 73 with a quarter of them.  Groups of 16 / 32 / 64 KiB: 32768 tokens into
// 65536 x 2048 f32 135 / 136 / 136.4, 8192 into 16384 x 2048 45.9 / 46.5 / 47.2.
constexpr uint64_t kHistZeroBytes = 40ull << 20, kPlaceZeroBytes = 80ull << 20, kZeroGroupBytes = 16ull << 10;
uint32_t key_bits(uint64_t vocab) { return 64u - (uint32_t)__builtin_clzll(vocab); }
uint32_t key_passes(uint64_t vocab) { return (key_bits(vocab) + kDigitBits - 1) / kDigitBits; }

uint64_t up256(uint64_t x) { return (x + 255) & ~(uint64_t)255; }

// scratch of the embedding gradient: two key and item arrays, the counts of
// a sort pass, the sums of runs that cross a chunk
struct EmbedScratch {
  uint64_t keys[2], items[2], hist, partial, total;
};
EmbedScratch embed_scratch(uint64_t tokens, uint64_t width) {
  EmbedScratch s;
  uint32_t blocks, chunk;
  sort_shape((uint32_t)tokens, &blocks, &chunk);
  const uint64_t arr = up256(tokens * 4);
  uint64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = at, at += arr;
    s.items[i] = at, at += arr;
  }
  s.hist = at;
  at += up256(sort_hist_words(blocks, 1u << kDigitBits) * 4);
  s.partial = at;
  const uint32_t per = embed_chunk(tokens);
  const uint64_t chunks = (tokens + per - 1) / per;
  at += chunks * 2 * ((width + 7) & ~(uint64_t)7) * 4;
  s.total = at;
  return s;
}

}  // namespace

extern "C" {

snac_status snac_route(const snac_router* router, const void* logits, size_t ld, const float* bias, size_t tokens,
                       snac_dtype dtype, float* weights, int32_t* ids, snac_stream stream) {
  TRY(check_router(router, true));
  TRY(check_dtype(dtype, "dtype"));
  const uint64_t E = (uint64_t)router->experts, K = (uint64_t)router->topk, es = esize(dtype);
  TRY(check_rows("logits", tokens, E, ld));
  const Span s[] = {{"logits", logits, tokens, E * es, ld * es, false},
                    array("bias", bias, bias && tokens ? E * 4 : 0, false),
                    array("weights", weights, tokens * K * 4, true),
                    array("ids", ids, tokens * K * 4, true)};
  const uint64_t al[] = {es, 4, 4, 4};
  TRY(check_spans(s, al));
  if (tokens == 0) return ok();
  const RouteArgs a{*router, logits, ld, bias, tokens, weights, ids};
  const hipError_t e = launch_route(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_route launch");
}

snac_status snac_route_backward(const snac_router* router, const void* logits, size_t ld, const int32_t* ids,
                                const float* dweights, size_t tokens, snac_dtype dtype, void* dlogits, size_t ld_d,
                                snac_stream stream) {
  TRY(check_router(router, false));
  TRY(check_dtype(dtype, "dtype"));
  const uint64_t E = (uint64_t)router->experts, K = (uint64_t)router->topk, es = esize(dtype);
  TRY(check_rows("logits", tokens, E, ld));
  TRY(check_rows("dlogits", tokens, E, ld_d));
  const Span s[] = {{"logits", logits, tokens, E * es, ld * es, false},
                    array("ids", ids, tokens * K * 4, false),
                    array("dweights", dweights, tokens * K * 4, false),
                    {"dlogits", dlogits, tokens, E * es, ld_d * es, true}};
  const uint64_t al[] = {es, 4, 4, es};
  TRY(check_spans(s, al));
  if (tokens == 0) return ok();
  const RouteBackwardArgs a{*router, logits, ld, ids, dweights, tokens, dlogits, ld_d};
  const hipError_t e = launch_route_backward(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_route_backward launch");
}

snac_status snac_dispatch_plan(snac_ctx* ctx, const void* ids, int id_bytes, size_t slots, int experts,
                               int32_t* counts, int32_t* row_of_slot, int32_t* slot_of_row, snac_stream stream) {
  TRY(check_id_bytes(id_bytes));
  if (experts < 1 || experts > SNAC_MAX_EXPERTS)
    return fail(SNAC_E_ARG, "experts %d outside 1..%d", experts, SNAC_MAX_EXPERTS);
  if (slots > SNAC_MAX_IDS) return fail(SNAC_E_ARG, "%zu slots above SNAC_MAX_IDS", slots);
  const Span s[] = {array("ids", ids, slots * (uint64_t)id_bytes, false),
                    array("counts", counts, (uint64_t)experts * 4, true),
                    array("row_of_slot", row_of_slot, slots * 4, true),
                    array("slot_of_row", slot_of_row, slots * 4, true)};
  const uint64_t al[] = {(uint64_t)id_bytes, 4, 4, 4};
  TRY(check_spans(s, al));
  SortArgs a{};
  a.ids = ids;
  a.id_bytes = id_bytes;
  a.pad = -1;
  a.vocab = (uint64_t)experts;
  a.n = (uint32_t)slots;
  a.bins = (uint32_t)experts + 1;
  a.mask = 0xffffffffu;
  sort_shape(a.n, &a.blocks, &a.chunk);
  a.hist_ld = sort_hist_ld(a.blocks);
  char* scratch = nullptr;
  TRY(ctx_scratch(ctx, sort_hist_words(a.blocks, a.bins) * 4, "snac_dispatch_plan", &scratch));
  a.hist = reinterpret_cast<uint32_t*>(scratch);
  a.counts = counts;
  a.row_of_slot = row_of_slot;
  a.slot_of_row = slot_of_row;
  const hipError_t e = launch_plan(a, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_dispatch_plan launch");
}

snac_status snac_dispatch(const void* x, size_t ld_x, const int32_t* row_of_slot, size_t tokens, int topk,
                          size_t width, snac_dtype dtype, void* out, size_t ld_out, size_t rows, snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_topk(topk));
  const uint64_t es = esize(dtype);
  TRY(check_rows("x", tokens, width, ld_x));
  TRY(check_rows("out", rows, width, ld_out));
  if (rows >= kMaxRows) return fail(SNAC_E_ARG, "%zu rows not below 2^31", rows);
  const Span s[] = {{"x", x, tokens, width * es, ld_x * es, false},
                    array("row_of_slot", row_of_slot, width ? tokens * (uint64_t)topk * 4 : 0, false),
                    {"out", out, rows, width * es, ld_out * es, true}};
  const uint64_t al[] = {es, 4, es};
  TRY(check_spans(s, al));
  if (tokens == 0 || width == 0 || rows == 0) return ok();
  const DispatchArgs a{static_cast<const char*>(x), ld_x * es, row_of_slot, tokens, topk, (uint32_t)width,
                       static_cast<char*>(out), ld_out * es, (uint32_t)rows};
  const hipError_t e = launch_dispatch(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_dispatch launch");
}

snac_status snac_combine(const void* y, size_t ld_y, size_t rows, const int32_t* row_of_slot, const float* weights,
                         size_t tokens, int topk, size_t width, snac_dtype dtype, void* out, size_t ld_out,
                         snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_topk(topk));
  const uint64_t es = esize(dtype);
  TRY(check_rows("y", rows, width, ld_y));
  TRY(check_rows("out", tokens, width, ld_out));
  if (rows >= kMaxRows) return fail(SNAC_E_ARG, "%zu rows not below 2^31", rows);
  const uint64_t slots = width ? tokens * (uint64_t)topk : 0;
  const Span s[] = {{"y", y, rows, width * es, ld_y * es, false},
                    array("row_of_slot", row_of_slot, slots * 4, false),
                    array("weights", weights, weights ? slots * 4 : 0, false),
                    {"out", out, tokens, width * es, ld_out * es, true}};
  const uint64_t al[] = {es, 4, 4, es};
  TRY(check_spans(s, al));
  if (tokens == 0 || width == 0) return ok();
  const CombineArgs a{static_cast<const char*>(y), ld_y * es, (uint32_t)rows, row_of_slot, weights, tokens, topk,
                      (uint32_t)width, static_cast<char*>(out), ld_out * es};
  const hipError_t e = launch_combine(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_combine launch");
}

snac_status snac_combine_backward(const void* dout, size_t ld_dout, const void* y, size_t ld_y, size_t rows,
                                  const int32_t* row_of_slot, const float* weights, size_t tokens, int topk,
                                  size_t width, snac_dtype dtype, void* dy, size_t ld_dy, float* dweights,
                                  snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_topk(topk));
  const uint64_t es = esize(dtype);
  TRY(check_rows("dout", tokens, width, ld_dout));
  TRY(check_rows("y", rows, width, ld_y));
  TRY(check_rows("dy", rows, width, ld_dy));
  if (rows >= kMaxRows) return fail(SNAC_E_ARG, "%zu rows not below 2^31", rows);
  const uint64_t slots = tokens * (uint64_t)topk;
  const Span s[] = {{"dout", dout, tokens, width * es, ld_dout * es, false},
                    {"y", y, rows, width * es, ld_y * es, false},
                    array("row_of_slot", row_of_slot, slots * 4, false),
                    array("weights", weights, slots * 4, false),
                    {"dy", dy, rows, width * es, ld_dy * es, true},
                    array("dweights", dweights, slots * 4, true)};
  const uint64_t al[] = {es, es, 4, 4, es, 4};
  TRY(check_spans(s, al, dy, y));
  if (tokens == 0) return ok();
  const CombineBackwardArgs a{static_cast<const char*>(dout), ld_dout * es, static_cast<const char*>(y), ld_y * es,
                              (uint32_t)rows, row_of_slot, weights, tokens, topk, (uint32_t)width,
                              static_cast<char*>(dy), ld_dy * es, dweights};
  const hipError_t e = launch_combine_backward(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_combine_backward launch");
}

snac_status snac_embedding(const void* table, size_t ld_table, size_t vocab, int64_t first, const void* ids,
                           int id_bytes, size_t tokens, size_t width, float scale, snac_dtype dtype, void* out,
                           size_t ld_out, snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_id_bytes(id_bytes));
  const uint64_t es = esize(dtype);
  TRY(check_rows("table", vocab, width, ld_table));
  TRY(check_rows("out", tokens, width, ld_out));
  const Span s[] = {{"table", table, vocab, width * es, ld_table * es, false},
                    array("ids", ids, width ? tokens * (uint64_t)id_bytes : 0, false),
                    {"out", out, tokens, width * es, ld_out * es, true}};
  const uint64_t al[] = {es, (uint64_t)id_bytes, es};
  TRY(check_spans(s, al));
  if (tokens == 0 || width == 0) return ok();
  const EmbeddingArgs a{static_cast<const char*>(table), ld_table * es, vocab, first, ids, id_bytes, tokens,
                        (uint32_t)width, scale, static_cast<char*>(out), ld_out * es};
  const hipError_t e = launch_embedding(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_embedding launch");
}

size_t snac_embedding_scratch(size_t tokens, size_t vocab, size_t width) {
  if (tokens > SNAC_MAX_IDS || vocab >= (1u << 30) || width >= kMaxWidth) return 0;
  if (tokens == 0 || vocab == 0 || width == 0) return 0;
  return embed_scratch(tokens, width).total;
}

snac_status snac_embedding_backward(snac_ctx* ctx, const void* dout, size_t ld_dout, snac_dtype dtype,
                                    const void* ids, int id_bytes, size_t tokens, int64_t first, size_t vocab,
                                    int64_t pad_id, size_t width, float scale, void* dtable, size_t ld_dtable,
                                    snac_dtype grad_dtype, int accumulate, snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_dtype(grad_dtype, "grad_dtype"));
  TRY(check_id_bytes(id_bytes));
  if (accumulate != 0 && accumulate != 1) return fail(SNAC_E_ARG, "accumulate %d is not 0 or 1", accumulate);
  if (tokens > SNAC_MAX_IDS) return fail(SNAC_E_ARG, "%zu tokens above SNAC_MAX_IDS", tokens);
  if (vocab >= (1u << 30)) return fail(SNAC_E_ARG, "vocab %zu not below 2^30", vocab);
  const uint64_t es = esize(dtype), gs = esize(grad_dtype);
  TRY(check_rows("dout", tokens, width, ld_dout));
  TRY(check_rows("dtable", vocab, width, ld_dtable));
  const Span s[] = {{"dout", dout, tokens, width * es, ld_dout * es, false},
                    array("ids", ids, width ? tokens * (uint64_t)id_bytes : 0, false),
                    {"dtable", dtable, vocab, width * gs, ld_dtable * gs, true}};
  const uint64_t al[] = {es, (uint64_t)id_bytes, gs};
  TRY(check_spans(s, al));
  if (vocab == 0 || width == 0) return ok();
  const EmbedScratch at = embed_scratch(tokens, width);
  char* scratch = nullptr;
  TRY(ctx_scratch(ctx, tokens ? at.total : 0, "snac_embedding_backward", &scratch));
  EmbedGradArgs g{};
  g.dout = static_cast<const char*>(dout);
  g.ld_dout = ld_dout * es;
  g.n = (uint32_t)tokens;
  g.vocab = (uint32_t)vocab;
  g.width = (uint32_t)width;
  g.scale = scale;
  g.dtable = static_cast<char*>(dtable);
  g.ld_dtable = ld_dtable * gs;
  g.accumulate = accumulate;
  g.partial = reinterpret_cast<float*>(scratch + at.partial);
  if (tokens) {
    SortArgs a{};
    a.ids = ids;
    a.id_bytes = id_bytes;
    a.first = first;
    a.pad = pad_id;
    a.vocab = vocab;
    a.n = (uint32_t)tokens;
    sort_shape(a.n, &a.blocks, &a.chunk);
    a.hist_ld = sort_hist_ld(a.blocks);
    const uint32_t bits = key_bits(vocab), passes = key_passes(vocab);
    const uint32_t digit = (bits + passes - 1) / passes;  // equal digits
    auto zeros = [&](uint64_t bytes) {
      ZeroRows z{};
      if (accumulate || tokens >= vocab) return z;
      const uint64_t row = width * gs, rows = bytes / row, left = vocab - g.zero_from;
      z.p = g.dtable + (uint64_t)g.zero_from * g.ld_dtable;
      z.ld = g.ld_dtable;
      z.width = (uint32_t)(row / 2);
      z.rows = (uint32_t)(rows < left ? rows : left);
      z.per = row < kZeroGroupBytes ? (uint32_t)(kZeroGroupBytes / row) : 1;
      g.zero_from += z.rows;
      return z;
    };
    uint32_t* const keys[2] = {reinterpret_cast<uint32_t*>(scratch + at.keys[0]), reinterpret_cast<uint32_t*>(scratch + at.keys[1])};
    int32_t* const items[2] = {reinterpret_cast<int32_t*>(scratch + at.items[0]), reinterpret_cast<int32_t*>(scratch + at.items[1])};
    a.mask = (1u << digit) - 1;
    a.bins = 1u << digit;
    a.hist = reinterpret_cast<uint32_t*>(scratch + at.hist);
    if (a.blocks == 1) {
      a.zero_place = zeros(kPlaceZeroBytes);
      a.key_out = keys[0];
      a.item_out = items[0];
      const hipError_t e = launch_radix_alone(a, passes, digit, (hipStream_t)stream);
      if (e != hipSuccess) return hip_fail(e, "snac_embedding_backward sort launch");
    } else {
      for (uint32_t p = 0; p < passes; ++p) {
        a.shift = p * digit;
        a.zero_hist = zeros(kHistZeroBytes);
        a.zero_place = zeros(kPlaceZeroBytes);
        a.key_out = keys[p & 1];
        a.item_out = items[p & 1];
        const hipError_t e = launch_radix_pass(a, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "snac_embedding_backward sort launch");
        a.key_in = a.key_out;
        a.item_in = a.item_out;
      }
    }
    g.keys = a.key_out;
    g.tokens = a.item_out;
  }
  const hipError_t e = launch_embedding_grad(g, dtype == SNAC_BF16, grad_dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_embedding_backward launch");
}

snac_status snac_grads_init(const void* const* src, void* const* dst, const size_t* counts, const int32_t* dtypes,
                            size_t n, snac_stream stream, snac_grads** out) {
  if (!out) return fail(SNAC_E_ARG, "out is NULL");
  *out = nullptr;
  if (n && (!src || !counts || !dtypes)) return fail(SNAC_E_ARG, "src, counts and dtypes must not be NULL");
  if (n > SNAC_MAX_IDS) return fail(SNAC_E_ARG, "%zu tensors above SNAC_MAX_IDS", n);
  uint64_t ntiles = 0, total = 0;
  for (size_t i = 0; i < n; ++i) {
    if (!is_float(dtypes[i])) return fail(SNAC_E_ARG, "dtypes[%zu] must be SNAC_F32 or SNAC_BF16", i);
    const uint64_t es = esize((snac_dtype)dtypes[i]);
    if (counts[i] > SNAC_MAX_BYTES || (total += counts[i] * es) > SNAC_MAX_BYTES)
      return fail(SNAC_E_ARG, "counts[%zu]: more than SNAC_MAX_BYTES", i);
    if (counts[i] == 0) continue;
    const void* d = dst ? dst[i] : src[i];
    if (!src[i] || !d) return fail(SNAC_E_ARG, "tensor %zu is NULL", i);
    if ((uintptr_t)src[i] % es || (uintptr_t)d % es) return fail(SNAC_E_ARG, "tensor %zu not aligned to %d bytes", i, (int)es);
    if (d != src[i]) {
      const Span a = array("dst", d, counts[i] * es, true), b = array("src", src[i], counts[i] * es, false);
      if (overlap(a, b)) return fail(SNAC_E_ARG, "dst[%zu] overlaps src[%zu] (not in place)", i, i);
    }
    ntiles += (((uintptr_t)d & (kGradAlign - 1)) + counts[i] * es + kGradTileBytes - 1) / kGradTileBytes;
  }
  if (ntiles > 0x7fffffffull) return fail(SNAC_E_ARG, "too many elements in one list");
  snac_grads* g = nullptr;
  char* mem = nullptr;
  try {
    std::vector<Extent> outs, all;
    for (size_t i = 0; i < n; ++i) {
      if (counts[i] == 0) continue;
      const uintptr_t s = (uintptr_t)src[i], d = dst ? (uintptr_t)dst[i] : s;
      const uint64_t bytes = counts[i] * esize((snac_dtype)dtypes[i]);
      all.push_back({s, s + bytes, i});
      outs.push_back({d, d + bytes, i});
    }
    TRY(check_outs(outs, all));
    all.insert(all.end(), outs.begin(), outs.end());
    merge(all);
    merge(outs);
    std::vector<GradTile> tiles;
    tiles.reserve(ntiles);
    for (size_t i = 0; i < n; ++i) {
      const uint64_t es = esize((snac_dtype)dtypes[i]);
      const char* s = static_cast<const char*>(src[i]);
      char* d = dst ? static_cast<char*>(dst[i]) : static_cast<char*>(const_cast<void*>(src[i]));
      uint64_t left = counts[i] * es;
      // the first tile ends where whole lines begin, the others keep to them
      uint64_t room = kGradTileBytes - ((uintptr_t)d & (kGradAlign - 1));
      while (left) {
        const uint64_t take = left < room ? left : room;
        tiles.push_back({s, d, (uint32_t)(take / es), dtypes[i] == SNAC_BF16 ? 1u : 0u});
        s += take;
        d += take;
        left -= take;
        room = kGradTileBytes;
      }
    }
    g = new snac_grads();
    g->outs.swap(outs);
    g->all.swap(all);
    hipError_t e = hipGetDevice(&g->device);
    if (e != hipSuccess) {
      delete g;
      return hip_fail(e, "hipGetDevice");
    }
    const uint64_t table = up256(tiles.size() * sizeof(GradTile));
    const uint64_t words = (kGradCounters + 2) * (uint64_t)kFlagStride;  // the ticket's line, the counters', the done count's
    const uint64_t bytes = table + kGradMaxBlocks * sizeof(double) + words * 8;
    e = hipMalloc(reinterpret_cast<void**>(&mem), bytes);
    if (e != hipSuccess) {
      delete g;
      return fail(SNAC_E_NOMEM, "hipMalloc(%llu) failed: %s", (unsigned long long)bytes, hipGetErrorString(e));
    }
    g->ntiles = (uint32_t)tiles.size();
    g->tiles = reinterpret_cast<GradTile*>(mem);
    g->partial = reinterpret_cast<double*>(mem + table);
    g->ticket = reinterpret_cast<uint32_t*>(mem + table + kGradMaxBlocks * sizeof(double));
    if (g->ntiles)
      e = hipMemcpyAsync(mem, tiles.data(), tiles.size() * sizeof(GradTile), hipMemcpyHostToDevice, (hipStream_t)stream);
    g->pool = reinterpret_cast<unsigned long long*>(g->ticket) + kFlagStride;
    if (e == hipSuccess) e = fill_u64(reinterpret_cast<uint64_t*>(g->ticket), words, 0, (hipStream_t)stream);
    if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
    if (e != hipSuccess) {
      (void)hipFree(mem);
      delete g;
      return hip_fail(e, "uploading the tensor list");
    }
  } catch (const std::bad_alloc&) {
    return fail(SNAC_E_NOMEM, "host allocation failed");
  }
  *out = g;
  return ok();
}

snac_status snac_grads_finalize(snac_grads* grads, snac_stream stream) {
  if (!grads) return ok();
  hipError_t e = hipStreamSynchronize((hipStream_t)stream);
  const hipError_t f = hipFree(grads->tiles);
  if (e == hipSuccess) e = f;
  delete grads;
  return e == hipSuccess ? ok() : hip_fail(e, "snac_grads_finalize");
}

// `written`: the call writes the norm.
static snac_status check_grads(const snac_grads* g, const float* norm, bool written) {
  if (!g) return fail(SNAC_E_ARG, "grads is NULL");
  if (!norm) return fail(SNAC_E_ARG, "norm is NULL");
  if ((uintptr_t)norm % 4) return fail(SNAC_E_ARG, "norm not aligned to 4 bytes");
  if (holds(written ? g->all : g->outs, norm, 4)) return fail(SNAC_E_ARG, "norm overlaps a tensor of the list");
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return fail(SNAC_E_HIP, "hipGetDevice failed");
  if (dev != g->device) return fail(SNAC_E_STATE, "list belongs to device %d, current device is %d", g->device, dev);
  return SNAC_OK;
}

static snac_status check_max_norm(float max_norm) {
  if (!(max_norm >= 0.0f)) return fail(SNAC_E_ARG, "max_norm %g is not >= 0", (double)max_norm);
  return SNAC_OK;
}

snac_status snac_grad_norm(snac_grads* grads, float* norm, snac_stream stream) {
  TRY(check_grads(grads, norm, true));
  const hipError_t e = launch_grad_norm(grads->tiles, grads->ntiles, grads->partial, grads->ticket, norm, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_grad_norm launch");
}

snac_status snac_clip_grads(snac_grads* grads, const float* norm, float max_norm, snac_stream stream) {
  TRY(check_max_norm(max_norm));
  TRY(check_grads(grads, norm, false));
  const hipError_t e = launch_clip(grads->tiles, grads->ntiles, norm, max_norm, grads->pool, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_clip_grads launch");
}

snac_status snac_clip_grad_norm(snac_grads* grads, float max_norm, float* norm, snac_stream stream) {
  TRY(check_max_norm(max_norm));
  TRY(check_grads(grads, norm, true));
  const hipError_t e = launch_norm_and_clip(grads->tiles, grads->ntiles, grads->partial, norm, max_norm, grads->pool,
                                            (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_clip_grad_norm launch");
}

}  // extern "C"
