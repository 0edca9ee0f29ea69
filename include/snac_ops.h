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
 *   snac_layer_norm, snac_layer_norm_backward
 *       rows of mean 0 and variance 1, weighted, and the gradients
 *   snac_balance_load, snac_balance_loss, snac_balance_backward
 *       how evenly a router's choices load the experts, as a loss, and its
 *       gradient (an AllReduce sums the ranks' loads)
 *   snac_distill, snac_distill_shard, snac_distill_join, snac_distill_backward
 *       the divergence from a teacher's top logits, over the whole vocabulary
 *       or in shards of it (an AllGather brings their parts together), and
 *       its gradient
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

/* ----------------------------------------------------------- layer norm */

/*
 * snac_layer_norm -- for each row x of x[tokens][width]:
 *   mean = sum x / width,  var = sum (x - mean)^2 / width,
 *   rstd = 1 / sqrt(var + eps),  out = (x - mean) * rstd * weight + bias
 * weight and bias: `width` values of param_dtype, or NULL (1 and 0; they may be
 * given one without the other).  stats: NULL, or [tokens][2] binary32 that
 * receive mean and rstd for the gradient.  A mean near the row's is made in
 * binary32; the distances from it and their squares are summed in binary32 within
 * 16 bytes of a row and in binary64 over them, which gives the mean and the
 * variance of rows far from 0 too.  (Sums and squares that pass binary32's range
 * are infinite.)  Each output is rounded once.  eps finite and >= 0 (with 0 a
 * constant row gives NaN, by the formula).  out may be x itself (same ld).
 */
snac_status snac_layer_norm(const void* x, size_t ld_x, const void* weight, const void* bias, snac_dtype param_dtype,
                            size_t tokens, size_t width, float eps, snac_dtype dtype, void* out, size_t ld_out,
                            float* stats, snac_stream stream);

/*
 * snac_layer_norm_backward -- from dout[tokens][width], with
 * h = (x - mean) * rstd and g = dout * weight:
 *   dx      = rstd * (g - sum g / width - h * (sum g h) / width)
 *   dweight = sum over the tokens of dout * h   (NULL: not wanted)
 *   dbias   = sum over the tokens of dout       (NULL: not wanted)
 * stats: what snac_layer_norm left for these rows.  A row's sums are binary32
 * within 16 bytes and binary64 over them; the sums over tokens are binary32 over
 * at most 32 tokens and binary64 over those.  On the way a workgroup's sum (of 32
 * tokens, of rows of up to 16 KiB 64 to 2048) is rounded to binary32, the whole to
 * binary32 and that to grad_dtype.
 *   accumulate  0: dweight and dbias are written; 1: the sums are added to them
 *               before the rounding
 * dx may be dout itself (same ld).  Scratch is the context's staging rings:
 * snac_layer_norm_scratch bytes (SNAC_E_ARG if the rings together are smaller);
 * without dweight and dbias rows of up to 32 KiB need none, and ctx may be NULL.
 * Calls of 2^33 tokens and more are refused (SNAC_E_ARG).
 */
snac_status snac_layer_norm_backward(snac_ctx* ctx, const void* dout, size_t ld_dout, const void* x, size_t ld_x,
                                     const void* weight, snac_dtype param_dtype, const float* stats, size_t tokens,
                                     size_t width, snac_dtype dtype, void* dx, size_t ld_dx, void* dweight, void* dbias,
                                     snac_dtype grad_dtype, int accumulate, snac_stream stream);

/* Scratch of snac_layer_norm_backward with dweight or dbias, rows of `dtype`:
 * staging bytes per rank times ranks must be at least this (0 for arguments that
 * the call refuses).  For rows of up to 32 KiB at most 32 MiB, 16 bytes an element
 * of the width and 512, whatever the tokens; for wider ones at most 32 MiB and 8
 * bytes an element of the width, and 8 bytes a token.  (A context of one rank has 64
 * MiB by default.) */
size_t snac_layer_norm_scratch(size_t tokens, size_t width, snac_dtype dtype);

/* --------------------------------------------------------- balance loss */

/*
 * A token with at least one id in 0 .. experts - 1 counts, others (padding) have
 * no part.  For token t with logits x, its shares are
 *   p = softmax(x), or sigmoid(x) / sum of sigmoid(x)     (router->score)
 * (0 for a masked expert; all 0 where every logit is masked), and
 *   c[e] = how many of the counting tokens' slots have id e
 *   s[e] = sum of p[e] over the counting tokens
 *   loss = coefficient * experts * sum over e of (c[e] / C) * (s[e] / S)
 * with C and S the sums of c and s over the experts (0 where C or S is 0).  C is
 * the number of slots in use and S of the counting tokens: even loads give
 * `coefficient`.  The choice has no gradient, the shares have.  Very low logits
 * keep their ratios; NaN spreads by the formulas.
 */

/*
 * snac_balance_load -- load[0][experts] = c and load[1][experts] = s, binary32
 * (c exactly, up to 2^24), from logits[tokens][experts] (row stride ld, `dtype`)
 * and the ids[tokens][topk] that snac_route chose.  Of the router, experts, topk
 * and score are used.  The sums over tokens are binary64.  An AllReduce of
 * `load` gives the ranks' common load.  tokens * topk at most SNAC_MAX_IDS.
 * Scratch is the context's staging rings, 12 bytes * experts * 256 at most;
 * SNAC_E_ARG if they are smaller.
 */
snac_status snac_balance_load(snac_ctx* ctx, const snac_router* router, const void* logits, size_t ld,
                              const int32_t* ids, size_t tokens, snac_dtype dtype, float* load, snac_stream stream);

/* snac_balance_loss -- loss[0] of load[2][experts], sums in binary64. */
snac_status snac_balance_loss(const float* load, int experts, float coefficient, float* loss, snac_stream stream);

/*
 * snac_balance_backward -- dlogits[tokens][experts] (row stride ld_d, `dtype`,
 * every element written) of this rank's tokens, for the `load` that the loss was
 * made of (the ranks' common one, where there are several):
 *   a[e]    = dloss * coefficient * experts * c[e] / (C S)
 *   dlogits = p[e] * (a[e] - sum over j of p[j] a[j])     (softmax)
 *             the same * (1 - sigmoid(x[e]))              (sigmoid)
 * and 0 for a token that does not count.  dloss: one binary32 on the device,
 * NULL: 1.
 *   accumulate  1: added to what dlogits holds (snac_route_backward's), rounded
 *               once; a token that does not count is left as it is
 */
snac_status snac_balance_backward(const snac_router* router, const void* logits, size_t ld, const int32_t* ids,
                                  const float* load, float coefficient, const float* dloss, size_t tokens,
                                  snac_dtype dtype, void* dlogits, size_t ld_d, int accumulate, snac_stream stream);

/* --------------------------------------------------------- distillation */

/* most choices of a teacher that are given for a token */
#define SNAC_MAX_TEACHER 256

/*
 * snac_teacher -- a teacher's top logits.  For a token with teacher's choices
 * id_k, t_k (k = 0 .. topk - 1) and student's logits z over the vocabulary:
 *   q_k  = softmax over its valid choices of t / temperature
 *   p    = softmax over the vocabulary of z / temperature
 *   loss = sum over k with q_k > 0 of q_k * (log q_k - log p[id_k])
 * A choice is valid where 0 <= id_k < vocab and t_k is not -infinity; ids need
 * not be ordered, and one that comes twice counts twice.  A masked z (-infinity)
 * has p = 0; a valid choice of one makes the loss infinite.  A token without a
 * valid choice, or whose logits are all masked, has no part: loss 0, gradient 0.
 * NaN spreads by the formulas, +infinity as in softmax.  No factor of
 * temperature^2 is applied; dloss and scale of the gradient can hold it.
 */
typedef struct snac_teacher {
  const void* ids;     /* [tokens][topk], columns of the whole vocabulary */
  const void* logits;  /* [tokens][topk] */
  int64_t vocab;       /* columns of the whole vocabulary, 1 .. SNAC_MAX_BYTES */
  int32_t id_bytes;    /* 4 or 8 */
  int32_t dtype;       /* SNAC_F32 or SNAC_BF16, of `logits` here */
  int32_t topk;        /* 1 .. SNAC_MAX_TEACHER */
  float temperature;   /* 2^-64 .. 2^64 */
} snac_teacher;

/*
 * snac_distill -- loss[tokens] and stats[tokens][2] of logits[tokens][vocab]
 * (row stride ld, `dtype`).  stats: a row's largest logit m and
 * S = sum of exp((z - m) / temperature), for the gradient.  Exponentials are
 * binary32; they are summed in binary32 within 16 bytes of a row and in binary64
 * over them; the loss is made in binary64 and rounded once.
 */
snac_status snac_distill(const snac_teacher* teacher, const void* logits, size_t ld, size_t tokens, snac_dtype dtype,
                         float* loss, float* stats, snac_stream stream);

/*
 * snac_distill_shard -- the same for a rank that holds columns
 * first .. first + width - 1 of the vocabulary, logits[tokens][width]:
 * part[tokens][4] receives m and S of the shard's columns,
 * D = sum of q_k * (z[id_k] - m) / temperature and Q = sum of q_k over the choices
 * in the shard (q over all valid choices; a term of q_k = 0 is 0).
 */
snac_status snac_distill_shard(const snac_teacher* teacher, const void* logits, size_t ld, int64_t first, size_t width,
                               size_t tokens, snac_dtype dtype, float* part, snac_stream stream);

/*
 * snac_distill_join -- loss and stats of the shards' parts
 * parts[shards][tokens][4] (what an AllGather of `part` leaves), 1 ..
 * SNAC_MAX_RANKS shards whose columns make up the vocabulary, in any order.
 * Every rank that joins them gets the same bits.
 */
snac_status snac_distill_join(const snac_teacher* teacher, const float* parts, int shards, size_t tokens, float* loss,
                              float* stats, snac_stream stream);

/*
 * snac_distill_backward -- the gradient of columns first .. first + width - 1:
 *   dlogits[t][j] = scale * dloss[t] / temperature * (p_j - sum of q_k, id_k = j)
 * with p from `stats` of the whole row.  dloss: [tokens] binary32, NULL: all 1.
 * In binary32, choices in ascending k, rounded once.  dlogits may be logits
 * itself (same ld).
 */
snac_status snac_distill_backward(const snac_teacher* teacher, const void* logits, size_t ld, int64_t first,
                                  size_t width, const float* stats, const float* dloss, float scale, size_t tokens,
                                  snac_dtype dtype, void* dlogits, size_t ld_d, snac_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SNAC_OPS_H */
