// ops.hpp -- host-side interface between the operators' C ABI
// (include/snac_ops.h, ops.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "snac.h"
#include "snac_ops.h"

namespace snac {

// The calling thread's last error (api.hip): fail() records it and returns
// its status, ok() clears it.
snac_status fail(snac_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
snac_status ok();
snac_status hip_fail(hipError_t e, const char* what);

// The context's staging rings as `bytes` bytes of scratch (api.hip);
// SNAC_E_ARG when they hold fewer, SNAC_E_STATE on another device.
snac_status ctx_scratch(snac_ctx* ctx, uint64_t bytes, const char* what, char** out);

int device_cu_count();

// ------------------------------------------------------------- routing
struct RouteArgs {
  snac_router r;
  const void* logits;
  uint64_t ld;
  const float* bias;
  uint64_t tokens;
  float* weights;
  int32_t* ids;
};
hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream);

struct RouteBackwardArgs {
  snac_router r;
  const void* logits;
  uint64_t ld;
  const int32_t* ids;
  const float* dweights;
  uint64_t tokens;
  void* dlogits;
  uint64_t ld_d;
};
hipError_t launch_route_backward(const RouteBackwardArgs& a, bool bf16, hipStream_t stream);

// ---------------------------------------------------------------- zeros
// Rows that workgroups past a launch's own write zeros to: `rows` rows of
// `width` 2-byte words, `per` of them a workgroup.
struct ZeroRows {
  char* p;
  uint64_t ld;  // bytes
  uint32_t width, rows, per;
};

// ---------------------------------------------------------------- sort
// One stable counting-sort pass over n items: positions by bin, ascending
// item order within a bin.
constexpr uint32_t kSortMaxBins = SNAC_MAX_EXPERTS + 1;
struct SortArgs {
  // the items' keys: from ids (key = id - first where that is in 0 .. vocab
  // - 1 and id is not pad, else vocab), or from an earlier pass
  const void* ids;
  int32_t id_bytes;
  int64_t first, pad;
  uint64_t vocab;
  const uint32_t* key_in;  // nullptr: from ids, item i being i
  const int32_t* item_in;
  uint32_t n;
  uint32_t shift, bins;  // bin = (key >> shift) % (mask + 1)
  uint32_t mask;
  uint32_t* hist;    // [bins][hist_ld] when blocks > 1: every run's counts
  uint32_t hist_ld;  // sort_hist_ld(blocks)
  uint32_t blocks, chunk;
  // outputs of a radix pass
  uint32_t* key_out;
  int32_t* item_out;
  // outputs of a dispatch plan (bin = expert, vocab = experts: dropped)
  int32_t* counts;
  int32_t* row_of_slot;
  int32_t* slot_of_row;
  // written beside the counting and the placing: both leave most of the GPU
  // idle for their latency
  ZeroRows zero_hist, zero_place;
};
// Most items that one workgroup sorts alone; a radix sort of so many is one
// launch.
constexpr uint32_t kSortAlone = 8192;
// blocks and chunk of a pass over n items
void sort_shape(uint32_t n, uint32_t* blocks, uint32_t* chunk);
constexpr uint32_t sort_hist_ld(uint32_t blocks) { return (blocks + 3) & ~3u; }
uint64_t sort_hist_words(uint32_t blocks, uint32_t bins);  // of one pass
hipError_t launch_plan(const SortArgs& a, hipStream_t stream);
hipError_t launch_radix_pass(const SortArgs& a, hipStream_t stream);  // several runs
// one run: all passes of `digit` bits each
hipError_t launch_radix_alone(const SortArgs& a, uint32_t passes, uint32_t digit, hipStream_t stream);

// ------------------------------------------------- dispatch and combine
struct DispatchArgs {
  const char* x;
  uint64_t ld_x;  // bytes
  const int32_t* row_of_slot;
  uint64_t tokens;
  int32_t topk;
  uint32_t width;  // elements
  char* out;
  uint64_t ld_out;  // bytes
  uint32_t rows;
};
hipError_t launch_dispatch(const DispatchArgs& a, bool bf16, hipStream_t stream);

struct CombineArgs {
  const char* y;
  uint64_t ld_y;  // bytes
  uint32_t rows;
  const int32_t* row_of_slot;
  const float* weights;
  uint64_t tokens;
  int32_t topk;
  uint32_t width;
  char* out;
  uint64_t ld_out;  // bytes
};
hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream);

struct CombineBackwardArgs {
  const char* dout;
  uint64_t ld_dout;  // bytes
  const char* y;
  uint64_t ld_y;  // bytes
  uint32_t rows;
  const int32_t* row_of_slot;
  const float* weights;
  uint64_t tokens;
  int32_t topk;
  uint32_t width;
  char* dy;
  uint64_t ld_dy;  // bytes
  float* dweights;
};
hipError_t launch_combine_backward(const CombineBackwardArgs& a, bool bf16, hipStream_t stream);

// ----------------------------------------------------------- embedding
struct EmbeddingArgs {
  const char* table;
  uint64_t ld_table;  // bytes
  uint64_t vocab;
  int64_t first;
  const void* ids;
  int32_t id_bytes;
  uint64_t tokens;
  uint32_t width;
  float scale;
  char* out;
  uint64_t ld_out;  // bytes
};
hipError_t launch_embedding(const EmbeddingArgs& a, bool bf16, hipStream_t stream);

// Sorted positions that a wave of the gradient adds up (embedding.hip).
constexpr uint32_t kFewTokens = 4096;
constexpr uint32_t embed_chunk(uint64_t tokens) { return tokens > 32 && tokens <= kFewTokens ? 8 : 32; }
struct EmbedGradArgs {
  const char* dout;
  uint64_t ld_dout;  // bytes
  const uint32_t* keys;   // sorted, vocab: no gradient
  const int32_t* tokens;  // of each sorted position
  uint32_t n;
  uint32_t vocab;
  uint32_t width;
  float scale;
  char* dtable;
  uint64_t ld_dtable;  // bytes
  int32_t accumulate;
  float* partial;  // [chunks][2][width rounded up to 8]
  // rows from here on without a token are still to be zeroed (vocab: none)
  uint32_t zero_from;
};
hipError_t launch_embedding_grad(const EmbedGradArgs& a, bool bf16, bool grad_bf16, hipStream_t stream);

// --------------------------------------------------- norm and clipping
// One tile of one tensor: `n` elements (n > 0).
struct GradTile {
  const char* src;
  char* dst;
  uint32_t n;
  uint32_t bf16;
};
constexpr uint32_t kGradTileBytes = 16384;
constexpr uint32_t kGradAlign = 256;  // tiles of a tensor begin on such addresses, but the first
constexpr uint32_t kGradMaxBlocks = 2048;
hipError_t launch_grad_norm(const GradTile* tiles, uint32_t ntiles, double* partial, uint32_t* ticket, float* norm,
                            hipStream_t stream);
// `pool`: kGradCounters zeroed counters and a done count, kFlagStride words
// apart; a launch leaves them zeroed.
constexpr uint32_t kGradCounters = 4;
hipError_t launch_clip(const GradTile* tiles, uint32_t ntiles, const float* norm, float max_norm,
                       unsigned long long* pool, hipStream_t stream);
// both, the norm made of the partial sums by the second launch
hipError_t launch_norm_and_clip(const GradTile* tiles, uint32_t ntiles, double* partial, float* norm, float max_norm,
                                unsigned long long* pool, hipStream_t stream);

}  // namespace snac
