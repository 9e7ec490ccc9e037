/*
 * dspark_logits.h -- what a request has said so far, and the target's logits
 * adjusted by it before the accept: penalties for repeated tokens, biases of
 * single tokens, and masks of the tokens that may come next (the same library as
 * dspark_markov.h; its error codes and conventions apply).
 *
 * In a step of a serving loop dspark_logits_adjust comes between the target's
 * logits and dspark_greedy_accept (BF16 out) or dspark_logits_to_probs (FP32
 * out), and dspark_tokens_count adds the accepted tokens.  No entry point
 * synchronises the host or allocates, and all are safe to capture in a CUDA
 * graph.
 */
#ifndef DSPARK_LOGITS_H
#define DSPARK_LOGITS_H

#include "dspark_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSPARK_ADJUST_MAX_DRAFTS 1023

/*
 * The tokens of the requests in `max_slots` slots.
 *   counts: device int32 [max_slots][vocab], row stride counts_stride: how often
 *   a token occurs among a slot's outputs.
 *   marks: device int32 [max_slots][2][(vocab + 31) / 32], slot stride
 *   marks_stride: bit v % 32 of word v / 32 of plane 0 is set where token v occurs
 *   in the slot's prompt, of plane 1 where it occurs among its outputs (counts
 *   above 0).
 * All owned by the caller; a new table is zeros.  vocab 1 to 2^30.
 */
typedef struct dspark_token_table {
  int32_t *counts;
  int64_t counts_stride;
  int32_t *marks;
  int64_t marks_stride;
  int32_t vocab;
  int32_t max_slots;
} dspark_token_table;

/*
 * dspark_tokens_count -- adds tokens[i * stride + t], t < lens[i] (held to
 * [0, width]), to slot slots[i] (i itself when slots is NULL), i < n: to its
 * prompt with `prompt` not 0, else to its outputs.  With `reset` not 0 the slots
 * listed are cleared first.  tokens: device, int64 (wide not 0) or int32, stride
 * >= width; lens: device int32 [n]; ids outside [0, vocab) and slots outside
 * [0, max_slots) are skipped; a slot may be listed more than once.  n, width >= 0.
 * What dspark_greedy_accept writes (accepted, accept_len) may be given as it is.
 * One kernel on `stream`, with `reset` two.
 */
DSPARK_API int dspark_tokens_count(const dspark_token_table *table, int32_t n, const int32_t *slots,
                                   const void *tokens, int32_t wide, int64_t stride, int32_t width,
                                   const int32_t *lens, int32_t prompt, int32_t reset, cudaStream_t stream);

/*
 * dspark_logits_adjust -- the logits l of batch requests with drafts + 1 rows
 * each: row i * (drafts + 1) + j is the target's answer behind the first j drafts
 * of request i, in slot slots[i] (i when NULL).  In FP32, each operation rounded
 * once, for token v of the row:
 *   n = counts[slot][v] + the number of draft[i * draft_stride + t] == v, t < j;
 *   where n > 0 or v is in the slot's prompt: l = l / repetition[slot] if l > 0,
 *     else l * repetition[slot];
 *   where n > 0: l = (l - frequency[slot] * n) - presence[slot];
 *   l = l + the sum, in their order, of the slot's biases for v;
 *   where the row's mask has a 0 for v: l = -inf;
 * and once more to the type of out.
 *   logits [batch * (drafts + 1)][vocab] of `dtype`, out of `out_dtype`, row
 *   strides in elements: BF16 to BF16, BF16 to F32 or F32 to F32; out may be
 *   logits with its type and stride (then only what changes is written), else
 *   they must not overlap.  16-byte accesses where pointers and strides allow.
 *   table: the slots' tokens (vocab as here); NULL: no counts and no prompts,
 *     only the drafts.
 *   draft: device int64 (ids outside [0, vocab) are skipped), or NULL with drafts
 *     = 0 or without penalties; drafts <= DSPARK_ADJUST_MAX_DRAFTS.
 *   repetition, frequency, presence: device FP32 [max_slots], each NULL for none.
 *   bias_start [max_slots + 1], bias_id: device int32, bias: device FP32: slot s
 *     has the entries bias_start[s] .. bias_start[s + 1] - 1, held to [0,
 *     bias_entries]; ids outside [0, vocab) are skipped; all NULL for none.
 *   mask: device int32 [mask_rows][(vocab + 31) / 32], row stride mask_stride: bit
 *     v % 32 of word v / 32 is 1 where v may come; mask_row: device int32, the row
 *     of the mask for each row of logits, -1 (or any outside [0, mask_rows)) for
 *     no mask; mask_row NULL: row r's mask is row r.  mask NULL: none.
 *   max_slots: of the arrays above; equal to the table's if there is one.  A
 *     request whose slot is outside [0, max_slots) gets its masks only.
 * batch, drafts >= 0, vocab 1 to 2^30.  One kernel on `stream`; deterministic.
 */
typedef struct dspark_adjust_args {
  const void *logits;
  int64_t logits_stride;
  void *out;
  int64_t out_stride;
  int32_t dtype;
  int32_t out_dtype;
  int32_t batch;
  int32_t drafts;
  int32_t vocab;
  int32_t max_slots;
  const int32_t *slots;
  const int64_t *draft;
  int64_t draft_stride;
  const float *repetition;
  const float *frequency;
  const float *presence;
  const int32_t *bias_start;
  const int32_t *bias_id;
  const float *bias;
  int64_t bias_entries;
  const int32_t *mask;
  int64_t mask_stride;
  int64_t mask_rows;
  const int32_t *mask_row;
} dspark_adjust_args;

DSPARK_API int dspark_logits_adjust(const dspark_token_table *table, const dspark_adjust_args *args,
                                    cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_LOGITS_H */
