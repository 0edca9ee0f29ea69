// ops_checks.hpp -- checks of arguments that the operators' entry points share
// (ops.hip, ops_step.hip).
#pragma once

#include "ops.hpp"

namespace snac {

constexpr uint64_t kMaxWidth = 1ull << 31;  // elements of a row
constexpr uint64_t kMaxRows = 1ull << 31;

inline uint64_t esize(snac_dtype t) { return t == SNAC_BF16 ? 2 : 4; }
inline bool is_float(int t) { return t == SNAC_F32 || t == SNAC_BF16; }

// One argument's memory: `rows` rows of `width` bytes, `ld` bytes apart.
struct Span {
  const char* name;
  const void* p;
  uint64_t rows, width, ld;
  bool out;
};

inline Span array(const char* name, const void* p, uint64_t bytes, bool out) { return {name, p, 1, bytes, bytes, out}; }

inline bool empty(const Span& s) { return s.rows == 0 || s.width == 0; }

// bytes from the first to past the last (checked against SNAC_MAX_BYTES)
inline unsigned __int128 extent(const Span& s) {
  return empty(s) ? 0 : (unsigned __int128)(s.rows - 1) * s.ld + s.width;
}

inline bool overlap(const Span& a, const Span& b) {
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

inline snac_status check_dtype(snac_dtype t, const char* what) {
  if (!is_float(t)) return fail(SNAC_E_ARG, "%s must be SNAC_F32 or SNAC_BF16", what);
  return SNAC_OK;
}

inline snac_status check_id_bytes(int b) {
  if (b != 4 && b != 8) return fail(SNAC_E_ARG, "id_bytes %d is not 4 or 8", b);
  return SNAC_OK;
}

inline snac_status check_router(const snac_router* r, bool forward) {
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

// Row strides and counts of a matrix argument.
inline snac_status check_rows(const char* name, uint64_t rows, uint64_t width, uint64_t ld) {
  if (rows > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%s: %llu rows above SNAC_MAX_BYTES", name, (unsigned long long)rows);
  if (width >= kMaxWidth) return fail(SNAC_E_ARG, "%s: width %llu not below 2^31", name, (unsigned long long)width);
  if (ld < width) return fail(SNAC_E_ARG, "%s: row stride %llu below the width %llu", name, (unsigned long long)ld, (unsigned long long)width);
  if (ld > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%s: row stride above SNAC_MAX_BYTES", name);
  return SNAC_OK;
}

inline snac_status check_topk(int topk) {
  if (topk < 1 || topk > SNAC_MAX_TOPK) return fail(SNAC_E_ARG, "topk %d outside 1..%d", topk, SNAC_MAX_TOPK);
  return SNAC_OK;
}

#define TRY(x)                        \
  do {                                \
    const snac_status st_ = (x);      \
    if (st_ != SNAC_OK) return st_;   \
  } while (0)

inline uint64_t up256(uint64_t x) { return (x + 255) & ~(uint64_t)255; }

}  // namespace snac
