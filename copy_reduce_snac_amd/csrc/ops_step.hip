// ops_step.hip -- the C ABI of layer norm, the balance loss and distillation
// (include/snac_ops.h): argument validation, sizes and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "ops.hpp"
#include "ops_checks.hpp"

using namespace snac;

namespace {

constexpr float kMaxTemperature = 0x1p64f;

snac_status check_accumulate(int accumulate) {
  if (accumulate != 0 && accumulate != 1) return fail(SNAC_E_ARG, "accumulate %d is not 0 or 1", accumulate);
  return SNAC_OK;
}

snac_status check_teacher(const snac_teacher* t) {
  if (!t) return fail(SNAC_E_ARG, "teacher is NULL");
  TRY(check_id_bytes(t->id_bytes));
  if (!is_float(t->dtype)) return fail(SNAC_E_ARG, "the teacher's dtype must be SNAC_F32 or SNAC_BF16");
  if (t->topk < 1 || t->topk > SNAC_MAX_TEACHER) return fail(SNAC_E_ARG, "topk %d outside 1..%d", t->topk, SNAC_MAX_TEACHER);
  if (!(t->temperature >= 1.0f / kMaxTemperature && t->temperature <= kMaxTemperature))
    return fail(SNAC_E_ARG, "temperature %g outside 2^-64..2^64", (double)t->temperature);
  if (t->vocab < 1 || (uint64_t)t->vocab > SNAC_MAX_BYTES)
    return fail(SNAC_E_ARG, "vocab %lld outside 1..SNAC_MAX_BYTES", (long long)t->vocab);
  return SNAC_OK;
}

snac_status check_shard(const snac_teacher* t, int64_t first, uint64_t width) {
  if (first < 0 || first > t->vocab || width > (uint64_t)(t->vocab - first))
    return fail(SNAC_E_ARG, "columns %lld.. of %llu are not in the vocabulary of %lld", (long long)first,
                (unsigned long long)width, (long long)t->vocab);
  return SNAC_OK;
}

snac_status check_tokens(uint64_t tokens) {
  if (tokens > SNAC_MAX_BYTES) return fail(SNAC_E_ARG, "%llu tokens above SNAC_MAX_BYTES", (unsigned long long)tokens);
  return SNAC_OK;
}

Span teacher_ids(const snac_teacher* t, uint64_t tokens) {
  return array("the teacher's ids", t->ids, tokens * (uint64_t)t->topk * (uint64_t)t->id_bytes, false);
}
Span teacher_logits(const snac_teacher* t, uint64_t tokens) {
  return array("the teacher's logits", t->logits, tokens * (uint64_t)t->topk * esize((snac_dtype)t->dtype), false);
}

// snac_distill and snac_distill_shard: loss and stats, or part.
snac_status distill(const snac_teacher* t, const void* logits, size_t ld, int64_t first, size_t width, size_t tokens,
                    snac_dtype dtype, float* loss, float* stats, float* part, bool shard, const char* what,
                    snac_stream stream) {
  const uint64_t es = esize(dtype);
  TRY(check_rows("logits", tokens, width, ld));
  const Span s[] = {teacher_ids(t, tokens),
                    teacher_logits(t, tokens),
                    {"logits", logits, tokens, width * es, ld * es, false},
                    array("loss", loss, shard ? 0 : tokens * 4, true),
                    array("stats", stats, shard ? 0 : tokens * 8, true),
                    array("part", part, shard ? tokens * 16 : 0, true)};
  const uint64_t al[] = {(uint64_t)t->id_bytes, esize((snac_dtype)t->dtype), es, 4, 4, 4};
  TRY(check_spans(s, al));
  if (tokens == 0) return ok();
  DistillArgs a{};
  a.teacher = *t;
  a.logits = static_cast<const char*>(logits);
  a.ld = ld * es;
  a.first = first;
  a.width = (uint32_t)width;
  a.tokens = tokens;
  a.loss = shard ? nullptr : loss;
  a.stats = stats;
  a.part = part;
  const hipError_t e = launch_distill(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

}  // namespace

extern "C" {

snac_status snac_layer_norm(const void* x, size_t ld_x, const void* weight, const void* bias, snac_dtype param_dtype,
                            size_t tokens, size_t width, float eps, snac_dtype dtype, void* out, size_t ld_out,
                            float* stats, snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_dtype(param_dtype, "param_dtype"));
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SNAC_E_ARG, "eps %g is not finite and >= 0", (double)eps);
  const uint64_t es = esize(dtype), ps = esize(param_dtype);
  TRY(check_rows("x", tokens, width, ld_x));
  TRY(check_rows("out", tokens, width, ld_out));
  const bool some = tokens && width;
  const Span s[] = {{"x", x, tokens, width * es, ld_x * es, false},
                    array("weight", weight, weight && some ? width * ps : 0, false),
                    array("bias", bias, bias && some ? width * ps : 0, false),
                    {"out", out, tokens, width * es, ld_out * es, true},
                    array("stats", stats, stats && some ? tokens * 8 : 0, true)};
  const uint64_t al[] = {es, ps, ps, es, 4};
  TRY(check_spans(s, al, out, x));
  if (!some) return ok();
  const LayerNormArgs a{static_cast<const char*>(x), ld_x * es, static_cast<const char*>(weight),
                        static_cast<const char*>(bias), tokens, (uint32_t)width, eps, static_cast<char*>(out),
                        ld_out * es, stats};
  const hipError_t e = launch_layer_norm(a, dtype == SNAC_BF16, param_dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_layer_norm launch");
}

size_t snac_layer_norm_scratch(size_t tokens, size_t width, snac_dtype dtype) {
  if (!is_float(dtype) || tokens > SNAC_MAX_BYTES || width >= kMaxWidth || tokens == 0 || width == 0) return 0;
  if (tokens >= kLayerNormMaxTokens) return 0;
  const LayerNormShape s = layer_norm_shape(tokens, width, esize(dtype));
  return up256(s.blocks * 2 * width * 4) + (s.runs ? up256(2 * width * 8) : 0) + (s.row_sums ? tokens * 8 : 0);
}

snac_status snac_layer_norm_backward(snac_ctx* ctx, const void* dout, size_t ld_dout, const void* x, size_t ld_x,
                                     const void* weight, snac_dtype param_dtype, const float* stats, size_t tokens,
                                     size_t width, snac_dtype dtype, void* dx, size_t ld_dx, void* dweight, void* dbias,
                                     snac_dtype grad_dtype, int accumulate, snac_stream stream) {
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_dtype(param_dtype, "param_dtype"));
  TRY(check_dtype(grad_dtype, "grad_dtype"));
  TRY(check_accumulate(accumulate));
  const uint64_t es = esize(dtype), ps = esize(param_dtype), gs = esize(grad_dtype);
  TRY(check_rows("dout", tokens, width, ld_dout));
  TRY(check_rows("x", tokens, width, ld_x));
  TRY(check_rows("dx", tokens, width, ld_dx));
  const bool some = tokens && width;
  const Span s[] = {{"dout", dout, tokens, width * es, ld_dout * es, false},
                    {"x", x, tokens, width * es, ld_x * es, false},
                    array("weight", weight, weight && some ? width * ps : 0, false),
                    array("stats", stats, some ? tokens * 8 : 0, false),
                    {"dx", dx, tokens, width * es, ld_dx * es, true},
                    array("dweight", dweight, dweight ? width * gs : 0, true),
                    array("dbias", dbias, dbias ? width * gs : 0, true)};
  const uint64_t al[] = {es, es, ps, 4, es, gs, gs};
  TRY(check_spans(s, al, dx, dout));
  if (width == 0) return ok();
  if (tokens >= kLayerNormMaxTokens) return fail(SNAC_E_ARG, "%zu tokens: more than one call takes", tokens);
  const LayerNormShape shape = layer_norm_shape(tokens, width, es);
  const uint64_t partial = dweight || dbias ? up256(shape.blocks * 2 * width * 4) : 0;
  const uint64_t whole = partial && shape.runs ? up256(2 * width * 8) : 0;
  const uint64_t bytes = partial + whole + (shape.row_sums ? tokens * 8 : 0);
  char* scratch = nullptr;
  if (bytes) TRY(ctx_scratch(ctx, bytes, "snac_layer_norm_backward", &scratch));
  if (tokens == 0 && (accumulate || !(dweight || dbias))) return ok();
  LayerNormBackwardArgs a{};
  a.dout = static_cast<const char*>(dout);
  a.ld_dout = ld_dout * es;
  a.x = static_cast<const char*>(x);
  a.ld_x = ld_x * es;
  a.weight = static_cast<const char*>(weight);
  a.stats = stats;
  a.tokens = tokens;
  a.width = (uint32_t)width;
  a.dx = static_cast<char*>(dx);
  a.ld_dx = ld_dx * es;
  a.dweight = dweight;
  a.dbias = dbias;
  a.grad_bf16 = grad_dtype == SNAC_BF16;
  a.accumulate = accumulate != 0;
  a.partial = partial ? reinterpret_cast<float*>(scratch) : nullptr;
  a.whole = whole ? reinterpret_cast<double*>(scratch + partial) : nullptr;
  a.row_sums = shape.row_sums ? reinterpret_cast<float*>(scratch + partial + whole) : nullptr;
  const hipError_t e =
      launch_layer_norm_backward(a, shape, dtype == SNAC_BF16, param_dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_layer_norm_backward launch");
}

snac_status snac_balance_load(snac_ctx* ctx, const snac_router* router, const void* logits, size_t ld,
                              const int32_t* ids, size_t tokens, snac_dtype dtype, float* load, snac_stream stream) {
  TRY(check_router(router, false));
  TRY(check_dtype(dtype, "dtype"));
  const uint64_t E = (uint64_t)router->experts, K = (uint64_t)router->topk, es = esize(dtype);
  TRY(check_rows("logits", tokens, E, ld));
  if (tokens * K > SNAC_MAX_IDS) return fail(SNAC_E_ARG, "%llu slots above SNAC_MAX_IDS", (unsigned long long)(tokens * K));
  const Span s[] = {{"logits", logits, tokens, E * es, ld * es, false},
                    array("ids", ids, tokens * K * 4, false),
                    array("load", load, E * 8, true)};
  const uint64_t al[] = {es, 4, 4};
  TRY(check_spans(s, al));
  BalanceArgs a{};
  a.experts = router->experts;
  a.topk = router->topk;
  a.score = router->score;
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.tokens = tokens;
  a.blocks = balance_blocks(tokens, router->experts);
  a.load = load;
  const uint64_t sums = up256(a.blocks * E * 8);
  char* scratch = nullptr;
  TRY(ctx_scratch(ctx, sums + a.blocks * E * 4, "snac_balance_load", &scratch));
  a.sums = reinterpret_cast<double*>(scratch);
  a.counts = reinterpret_cast<uint32_t*>(scratch + sums);
  const hipError_t e = launch_balance_load(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_balance_load launch");
}

static snac_status check_experts(int experts) {
  if (experts < 1 || experts > SNAC_MAX_EXPERTS)
    return fail(SNAC_E_ARG, "experts %d outside 1..%d", experts, SNAC_MAX_EXPERTS);
  return SNAC_OK;
}

snac_status snac_balance_loss(const float* load, int experts, float coefficient, float* loss, snac_stream stream) {
  TRY(check_experts(experts));
  const Span s[] = {array("load", load, (uint64_t)experts * 8, false), array("loss", loss, 4, true)};
  const uint64_t al[] = {4, 4};
  TRY(check_spans(s, al));
  const hipError_t e = launch_balance_loss(load, experts, coefficient, loss, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_balance_loss launch");
}

snac_status snac_balance_backward(const snac_router* router, const void* logits, size_t ld, const int32_t* ids,
                                  const float* load, float coefficient, const float* dloss, size_t tokens,
                                  snac_dtype dtype, void* dlogits, size_t ld_d, int accumulate, snac_stream stream) {
  TRY(check_router(router, false));
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_accumulate(accumulate));
  const uint64_t E = (uint64_t)router->experts, K = (uint64_t)router->topk, es = esize(dtype);
  TRY(check_rows("logits", tokens, E, ld));
  TRY(check_rows("dlogits", tokens, E, ld_d));
  const Span s[] = {{"logits", logits, tokens, E * es, ld * es, false},
                    array("ids", ids, tokens * K * 4, false),
                    array("load", load, tokens ? E * 8 : 0, false),
                    array("dloss", dloss, dloss && tokens ? 4 : 0, false),
                    {"dlogits", dlogits, tokens, E * es, ld_d * es, true}};
  const uint64_t al[] = {es, 4, 4, 4, es};
  TRY(check_spans(s, al));
  if (tokens == 0) return ok();
  BalanceArgs a{};
  a.experts = router->experts;
  a.topk = router->topk;
  a.score = router->score;
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.tokens = tokens;
  a.load = const_cast<float*>(load);
  a.coefficient = coefficient;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.ld_d = ld_d;
  a.accumulate = accumulate;
  const hipError_t e = launch_balance_backward(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_balance_backward launch");
}

snac_status snac_distill(const snac_teacher* teacher, const void* logits, size_t ld, size_t tokens, snac_dtype dtype,
                         float* loss, float* stats, snac_stream stream) {
  TRY(check_teacher(teacher));
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_tokens(tokens));
  return distill(teacher, logits, ld, 0, (size_t)teacher->vocab, tokens, dtype, loss, stats, nullptr, false,
                 "snac_distill launch", stream);
}

snac_status snac_distill_shard(const snac_teacher* teacher, const void* logits, size_t ld, int64_t first, size_t width,
                               size_t tokens, snac_dtype dtype, float* part, snac_stream stream) {
  TRY(check_teacher(teacher));
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_tokens(tokens));
  TRY(check_shard(teacher, first, width));
  return distill(teacher, logits, ld, first, width, tokens, dtype, nullptr, nullptr, part, true,
                 "snac_distill_shard launch", stream);
}

snac_status snac_distill_join(const snac_teacher* teacher, const float* parts, int shards, size_t tokens, float* loss,
                              float* stats, snac_stream stream) {
  TRY(check_teacher(teacher));
  TRY(check_tokens(tokens));
  if (shards < 1 || shards > SNAC_MAX_RANKS) return fail(SNAC_E_ARG, "shards %d outside 1..%d", shards, SNAC_MAX_RANKS);
  const Span s[] = {teacher_ids(teacher, tokens), teacher_logits(teacher, tokens),
                    array("parts", parts, tokens * (uint64_t)shards * 16, false), array("loss", loss, tokens * 4, true),
                    array("stats", stats, tokens * 8, true)};
  const uint64_t al[] = {(uint64_t)teacher->id_bytes, esize((snac_dtype)teacher->dtype), 4, 4, 4};
  TRY(check_spans(s, al));
  if (tokens == 0) return ok();
  DistillArgs a{};
  a.teacher = *teacher;
  a.parts = parts;
  a.shards = shards;
  a.tokens = tokens;
  a.loss = loss;
  a.stats = stats;
  const hipError_t e = launch_distill_join(a, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_distill_join launch");
}

snac_status snac_distill_backward(const snac_teacher* teacher, const void* logits, size_t ld, int64_t first,
                                  size_t width, const float* stats, const float* dloss, float scale, size_t tokens,
                                  snac_dtype dtype, void* dlogits, size_t ld_d, snac_stream stream) {
  TRY(check_teacher(teacher));
  TRY(check_dtype(dtype, "dtype"));
  TRY(check_tokens(tokens));
  TRY(check_shard(teacher, first, width));
  const uint64_t es = esize(dtype);
  TRY(check_rows("logits", tokens, width, ld));
  TRY(check_rows("dlogits", tokens, width, ld_d));
  const bool some = tokens && width;
  const Span s[] = {teacher_ids(teacher, some ? tokens : 0),
                    teacher_logits(teacher, some ? tokens : 0),
                    {"logits", logits, tokens, width * es, ld * es, false},
                    array("stats", stats, some ? tokens * 8 : 0, false),
                    array("dloss", dloss, dloss && some ? tokens * 4 : 0, false),
                    {"dlogits", dlogits, tokens, width * es, ld_d * es, true}};
  const uint64_t al[] = {(uint64_t)teacher->id_bytes, esize((snac_dtype)teacher->dtype), es, 4, 4, es};
  TRY(check_spans(s, al, dlogits, logits));
  if (!some) return ok();
  DistillArgs a{};
  a.teacher = *teacher;
  a.logits = static_cast<const char*>(logits);
  a.ld = ld * es;
  a.first = first;
  a.width = (uint32_t)width;
  a.tokens = tokens;
  a.stats = const_cast<float*>(stats);
  a.dloss = dloss;
  a.scale = scale;
  a.dlogits = static_cast<char*>(dlogits);
  a.ld_d = ld_d * es;
  const hipError_t e = launch_distill_backward(a, dtype == SNAC_BF16, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "snac_distill_backward launch");
}

}  // extern "C"
