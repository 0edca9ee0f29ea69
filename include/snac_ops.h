/*
 * snac_ops.h -- C ABI of the operators that stand on either side of a
 * collective in one step of a sharded language model, for AMD Instinct
 * MI355X (gfx950).  They fill the buffers that the collectives of snac.h
 * exchange, and use what comes back:
 *
 *   snac_route, snac_route_backward
 *       routing of tokens to experts: scores, groups, top-k, weights
 *   snac_dispatch_plan, snac_dispatch
 *       rows of tokens packed by expert: AllToAllV's send buffer and counts
 *   snac_combine, snac_combine_backward
 *       the weighted sum of the rows that came back, and its gradient
 *   snac_embedding, snac_embedding_backward
 *       rows of a vocabulary shard (an AllReduce sums the shards), and the
 *       shard's gradient by sorted tokens
 *   snac_grads_init, snac_grad_norm, snac_clip_grads, snac_clip_grad_norm
 *       the global norm over many tensors, and clipping by it
 *
 * The conventions are those of snac.h: device pointers that the caller owns,
 * asynchronous on `stream`, argument errors reported at once with nothing
 * enqueued, no allocation per call (so every call may be captured into a
 * graph), no exception crosses the interface.  Further:
 *   - A matrix of `width` elements a row has its rows `ld` elements apart
 *     (ld >= width); rows may start at any element, so a matrix may be a
 *     column slice of a wider one.  Pointers need the alignment of their
 *     element type only; 16-byte aligned rows are fastest.
 *   - An output may not overlap any other argument, except where a call says
 *     so.  Columns of one wider matrix do not overlap.
 *   - dtype is SNAC_F32 or SNAC_BF16.  Every sum is held in binary32 or
 *     binary64 in a fixed order and rounded once, so results are bitwise
 *     repeatable.
 *   - Indexes read on the device (experts, rows, tokens) are checked there:
 *     one that is out of range counts as absent, it never leaves a buffer.
 */
#ifndef SNAC_OPS_H
#define SNAC_OPS_H

#include "snac.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SNAC_MAX_EXPERTS 1024
#define SNAC_MAX_TOPK 32
/* most ids (tokens, or tokens * topk) that one plan or embedding gradient sorts */
#define SNAC_MAX_IDS (1u << 24)

/* ------------------------------------------------------------- routing */

typedef enum snac_score { SNAC_SCORE_SOFTMAX = 0, SNAC_SCORE_SIGMOID = 1 } snac_score;

/*
 * snac_router -- how a router chooses.  For token t with logits x[0..experts):
 *   score   s = softmax(x) or sigmoid(x)
 *   key     k = s + bias (k orders as s without a bias)
 *   groups  the experts in `groups` runs of experts / groups each; a group's
 *           worth is the sum of its `group_top` largest keys, and the
 *           `topk_groups` worthiest stay
 *   ids     the `topk` largest keys of the groups that stay, largest first
 *   weights scale * s of the chosen, or with `renorm` scale * s / (sum of the
 *           chosen s)
 * Keys and worths are ordered as in binary64, so logits one step apart in
 * their own type fall on their right sides; equal ones by the lower index.
 * A masked expert (logit or key of -infinity) is never chosen, nor is a group
 * whose worth is -infinity (one of fewer than group_top unmasked experts
 * among them); where fewer than topk are left the row ends in id -1 with
 * weight 0.  Renormalised scores do not underflow: very low logits keep their
 * ratios.  NaN orders above everything, and spreads by the formulas (softmax:
 * over the whole row, as +infinity does).
 */
typedef struct snac_router {
  int32_t experts;     /* 1 .. SNAC_MAX_EXPERTS, a multiple of groups */
  int32_t topk;        /* 1 .. min(SNAC_MAX_TOPK, topk_groups * experts / groups) */
  int32_t groups;      /* 1 .. 64 */
  int32_t topk_groups; /* 1 .. groups */
  int32_t group_top;   /* 1 or 2 (a group of one expert has one key to sum) */
  int32_t score;       /* snac_score */
  int32_t renorm;      /* 0 or 1 */
  float scale;
} snac_router;

/*
 * snac_route -- weights[tokens][topk] and ids[tokens][topk] of
 * logits[tokens][experts] (row stride ld, `dtype`).  bias: NULL, or
 * `experts` binary32 values (the balance bias: it moves the choice and not
 * the weights, and has no gradient).
 */
snac_status snac_route(const snac_router* router, const void* logits, size_t ld, const float* bias, size_t tokens,
                       snac_dtype dtype, float* weights, int32_t* ids, snac_stream stream);

/*
 * snac_route_backward -- dlogits[tokens][experts] (row stride ld_d, `dtype`,
 * every element written) from dweights[tokens][topk] for the ids that
 * snac_route chose (a row's ids differ from each other).  Of the router,
 * experts, topk, score, renorm and scale are used.  An id outside
 * 0 .. experts - 1 has no part in it.
 */
snac_status snac_route_backward(const snac_router* router, const void* logits, size_t ld, const int32_t* ids,
                                const float* dweights, size_t tokens, snac_dtype dtype, void* dlogits, size_t ld_d,
                                snac_stream stream);

/* ------------------------------------------------- dispatch and combine */

/*
 * snac_dispatch_plan -- the packed order of `slots` slots (token t's k-th
 * choice is slot t * topk + k) by expert, slots of one expert in ascending
 * order: what AllToAllV sends, experts of one rank being neighbours.
 *   ids          slots ids of id_bytes (4 or 8) bytes each; one outside
 *                0 .. experts - 1 drops its slot
 *   counts       [experts] rows of each expert
 *   row_of_slot  [slots] packed row of each slot, -1 where it is dropped
 *   slot_of_row  [slots] slot of each packed row, -1 past the last one
 * Scratch is the context's staging rings (as in SNAC_REDUCE_ATOMIC), none up
 * to 8192 slots and at most 2 KiB * (experts + 1); SNAC_E_ARG if they are
 * smaller.
 */
snac_status snac_dispatch_plan(snac_ctx* ctx, const void* ids, int id_bytes, size_t slots, int experts,
                               int32_t* counts, int32_t* row_of_slot, int32_t* slot_of_row, snac_stream stream);

/*
 * snac_dispatch -- out[row_of_slot[t * topk + k]] = x[t]: x[tokens][width]
 * (row stride ld_x) into the packed rows out[rows][width] (row stride
 * ld_out).  Rows that no slot names are left as they are.  topk
 * 1 .. SNAC_MAX_TOPK, rows < 2^31.  Its gradient is snac_combine without
 * weights.
 */
snac_status snac_dispatch(const void* x, size_t ld_x, const int32_t* row_of_slot, size_t tokens, int topk,
                          size_t width, snac_dtype dtype, void* out, size_t ld_out, size_t rows, snac_stream stream);

/*
 * snac_combine -- out[t] = sum over k of weights[t][k] * y[row_of_slot[t][k]]
 * in binary32, k ascending, one rounding; weights NULL: all 1.  A dropped
 * slot has no part in it (not even a NaN of its weight); a token without any
 * gets zeros.
 */
snac_status snac_combine(const void* y, size_t ld_y, size_t rows, const int32_t* row_of_slot, const float* weights,
                         size_t tokens, int topk, size_t width, snac_dtype dtype, void* out, size_t ld_out,
                         snac_stream stream);

/*
 * snac_combine_backward -- from dout[tokens][width]:
 *   dy[row_of_slot[t][k]] = weights[t][k] * dout[t]   (other rows are left)
 *   dweights[t][k] = <dout[t], y[row_of_slot[t][k]]>  (0 for a dropped slot)
 * the products dy in binary32; the sums in binary32 within 16 bytes of a row,
 * in binary64 over them, rounded once.  dy may be y itself (same ld).
 */
snac_status snac_combine_backward(const void* dout, size_t ld_dout, const void* y, size_t ld_y, size_t rows,
                                  const int32_t* row_of_slot, const float* weights, size_t tokens, int topk,
                                  size_t width, snac_dtype dtype, void* dy, size_t ld_dy, float* dweights,
                                  snac_stream stream);

/* ------------------------------------------------------------ embedding */

/*
 * snac_embedding -- out[t] = scale * table[ids[t] - first], in binary32 and
 * rounded once; zeros where ids[t] - first is outside 0 .. vocab - 1, so that
 * the sum of the shards' outputs is the whole table's.  ids of id_bytes
 * (4 or 8) bytes.
 */
snac_status snac_embedding(const void* table, size_t ld_table, size_t vocab, int64_t first, const void* ids,
                           int id_bytes, size_t tokens, size_t width, float scale, snac_dtype dtype, void* out,
                           size_t ld_out, snac_stream stream);

/*
 * snac_embedding_backward -- the gradient of the shard:
 *   dtable[v] = scale * sum of dout[t] over the tokens t with id first + v
 * with tokens in ascending order: up to 32 of them make a partial sum (rows
 * of binary32 added in binary64, rows of bf16 in binary32), rounded to binary32;
 * a token's partial sums are added in order in binary64, and the scaled sum is
 * rounded to binary32 and that to dtable's type.
 *   pad_id      ids equal to it have no gradient (any absent id: none)
 *   dtype, grad_dtype   types of dout and of dtable
 *   accumulate  0: dtable is written whole, zeros where no token came;
 *               1: the scaled sums are added to it before that rounding, other
 *               rows stay
 * Scratch is the context's staging rings: snac_embedding_scratch bytes
 * (SNAC_E_ARG if the rings together are smaller).  vocab < 2^30.
 */
snac_status snac_embedding_backward(snac_ctx* ctx, const void* dout, size_t ld_dout, snac_dtype dtype,
                                    const void* ids, int id_bytes, size_t tokens, int64_t first, size_t vocab,
                                    int64_t pad_id, size_t width, float scale, void* dtable, size_t ld_dtable,
                                    snac_dtype grad_dtype, int accumulate, snac_stream stream);

/* Scratch of snac_embedding_backward: staging bytes per rank times ranks
 * must be at least this (0 for arguments that the call refuses). */
size_t snac_embedding_scratch(size_t tokens, size_t vocab, size_t width);

/* ---------------------------------------------------- norm and clipping */

/*
 * snac_grads -- a list of tensors whose places are fixed, such as a
 * program's gradient buckets or the shards that a ReduceScatter leaves.
 */
typedef struct snac_grads snac_grads;

/*
 * snac_grads_init -- describe n tensors on the current device: src[i] with
 * counts[i] elements of dtypes[i] (snac_dtype values), clipped into dst[i].
 * dst NULL: in place; dst[i] may equal src[i], and may not otherwise overlap
 * any tensor of the list (SNAC_E_ARG; nor may a call's norm).  Any number of tensors, any length from 0, any
 * element alignment.  The list's own device memory is allocated here, once;
 * the tensors' addresses are kept and their contents are not.  Making a list
 * uploads its tiles and waits for `stream`: 0.15 ms for 96 tensors of 1 M
 * elements in all, 0.55 ms for 300 of 0.5 G, so a list is for tensors that stay
 * where they are from step to step (gradients that a program keeps and zeroes,
 * or writes in place), not for ones that are allocated anew each time.  Errors:
 * SNAC_E_ARG, SNAC_E_NOMEM, SNAC_E_HIP.  Not to be captured.
 */
snac_status snac_grads_init(const void* const* src, void* const* dst, const size_t* counts, const int32_t* dtypes,
                            size_t n, snac_stream stream, snac_grads** out);

/* Wait for `stream` and free the list (NULL: a no-op). */
snac_status snac_grads_finalize(snac_grads* grads, snac_stream stream);

/*
 * snac_grad_norm -- norm[0] = sqrt(sum of the squares of every element of
 * every src), squares and sums in binary64 (no element's square overflows),
 * rounded to binary32.  NaN and infinity spread by the formula.  An empty
 * list has norm 0.  A list is used on one stream at a time.
 */
snac_status snac_grad_norm(snac_grads* grads, float* norm, snac_stream stream);

/*
 * snac_clip_grads -- dst = src * min(1, max_norm / (norm[0] + 1e-6)) in
 * binary32 with one rounding.  A factor of 1 leaves in-place tensors
 * untouched and copies the others; a NaN factor reaches every element.
 * max_norm >= 0.
 */
snac_status snac_clip_grads(snac_grads* grads, const float* norm, float max_norm, snac_stream stream);

/* snac_clip_grad_norm -- snac_grad_norm, then snac_clip_grads by it. */
snac_status snac_clip_grad_norm(snac_grads* grads, float max_norm, float* norm, snac_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SNAC_OPS_H */
