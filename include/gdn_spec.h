/*
 * gdn_spec.h -- C ABI of libgdn_spec.so: the operators of a speculative decode
 * step around the state update of gdn_decode.h, on the GPU from end to end.
 *
 *   gdn_step_maps      index arrays of the step from the requests' lengths
 *   (gdn_decode_update the state update, per-token states written)
 *   gdn_token_probs    logits -> probabilities, a temperature per sequence
 *   gdn_verify_drafts  drafted tokens judged, the next token drawn
 *   gdn_commit_states  the state after the last kept token -> the state pool
 *
 * One packing runs through them.  Sequence i of a step feeds the T_i tokens
 * cu_seqlens[i] .. cu_seqlens[i+1]: its last emitted token, then its
 * T_i - 1 drafted ones.  Row r of the packed range is also the row of the
 * token's logits and of its state in intermediate_states.  num_tokens[i],
 * written by gdn_verify_drafts, counts both the tokens the sequence emits
 * (accepted drafts plus one drawn) and the fed tokens whose state stands,
 * which is what gdn_commit_states reads.
 *
 * Descriptors, status codes, streams and ownership are those of gdn_decode.h:
 * the caller owns all memory, every argument check happens on the host before
 * anything is enqueued, a call launches one kernel on extra->stream, allocates
 * nothing, keeps nothing and can be captured in a CUDA graph.  No written
 * tensor may overlap any other tensor of the call (GDN_ERR_ALIAS; the address
 * ranges are compared, so interleaved views count as overlapping).  In
 * `extra` only stream and device_status are used; every other field must be 0
 * (GDN_ERR_ARG).  flags: GDN_SPEC_CHECK_ONLY, and GDN_LAUNCH_PDL, which every
 * call here implies (the kernel may be scheduled while the previous one on the
 * stream still runs, and waits for it before it touches memory).  The kernels
 * run on the calling thread's current device, which must be the tensors' own.
 *
 * What only the device can see is reported by OR-ing the bits below (and
 * GDN_DEV_* of gdn_decode.h) into *extra->device_status; the offending row or
 * sequence is left out as each entry point says, and nothing traps.
 */
#ifndef GDN_SPEC_H
#define GDN_SPEC_H

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_SPEC_ABI_VERSION 1

#define GDN_DTYPE_I64 4 /* slot_map only */

/* flags beside GDN_LAUNCH_PDL */
#define GDN_SPEC_CHECK_ONLY (1u << 16) /* run the host checks and return their
                                          status; launch nothing */

/* bits OR-ed into *device_status beside GDN_DEV_* */
#define GDN_DEV_BAD_SEQ         (1u << 3) /* a row_seq entry < -1 or past the temperatures */
#define GDN_DEV_BAD_TEMPERATURE (1u << 4) /* negative, infinite or NaN */
#define GDN_DEV_BAD_TOKEN       (1u << 5) /* a drafted token outside -1 .. vocab - 1 */
#define GDN_DEV_BAD_PROBS       (1u << 6) /* a row to draw from without any positive,
                                             finite probability */
#define GDN_DEV_BAD_COUNT       (1u << 7) /* num_tokens[i] outside 0 .. T_i */
#define GDN_DEV_BAD_LENGTH      (1u << 8) /* a length or context < 0, or their sum past
                                             INT32_MAX */
#define GDN_DEV_BAD_BLOCKS      (1u << 9) /* blocks_held outside the table's width or short
                                             of the context, more blocks needed than the
                                             table is wide, or a bad free_head */
#define GDN_DEV_NO_ROOM         (1u << 10) /* the rows or the free blocks ran out */

/* Largest vocabulary of gdn_token_probs. */
#define GDN_SPEC_MAX_VOCAB 393216

/*
 * Probabilities of a step's rows:
 *     probs[r, v] = exp(l[r, v] / t) / sum_w exp(l[r, w] / t),
 *     t = temperature[row_seq[r]]   (1 without temperature, temperature[r]
 *                                    without row_seq)
 *   logits       bf16|fp32  [R, vocab]   vocab contiguous, rows at any stride
 *   temperature  fp32       [S] or NULL  any stride; S = R without row_seq
 *   row_seq      int32      [R] or NULL  contiguous; needs temperature
 *   probs        bf16|fp32  [R, vocab]   vocab contiguous, rows at any stride
 *                                        >= vocab
 * t = 0 is the greedy limit: 1 at the row's largest logit, the lowest index of
 * equals, 0 elsewhere.  A logit of -inf or NaN is masked: probability 0.  A row
 * with every logit masked becomes all zeros, and one with +inf logits shares
 * its mass among them.  row_seq[r] = -1 marks a row behind the last sequence:
 * it is not read and its probabilities are left as they were, as are the rows
 * with GDN_DEV_BAD_SEQ; rows with GDN_DEV_BAD_TEMPERATURE become zeros.
 * Exponentials and sums are fp32.  With GDN_DEV_TIMEOUT rows may be missing in
 * whole or in part; what is written is right.  1 <= vocab <= GDN_SPEC_MAX_VOCAB
 * (GDN_ERR_UNSUPPORTED above); R = 0 is GDN_OK with no launch.
 */
GDN_API int gdn_token_probs(const gdn_tensor *logits, const gdn_tensor *temperature, const gdn_tensor *row_seq,
                            const gdn_tensor *probs, uint32_t flags, const gdn_extra *extra);

/*
 * Drafted tokens judged against the target's probabilities with given random
 * numbers, and the next token drawn.  Sequence i has d = T_i - 1 drafts; draft
 * j (token x_j) is judged by row cu_seqlens[i] + j of the target:
 *     accepted  iff  uniforms[i, j] * q_j(x_j) < p_j(x_j)
 * up to the first that is not; A counts the accepted.  The next token is drawn
 * from w = max(p_A - q_A, 0) after a rejection and w = p_d after d
 * acceptances: the smallest v with w_0 + ... + w_v > u * W, u = uniforms[i, D],
 * W the sum of all w.
 *   target_probs   bf16|fp32  [T_tot, vocab] | [1, T_tot, vocab] (varlen) or
 *                             [N, T, vocab]  vocab contiguous; a row need not
 *                                            sum to 1
 *   draft_tokens   int32      [N, D]         any strides; D may be 0
 *   draft_probs    as target  [N, D, vocab]  vocab contiguous, others any; or
 *                                            NULL: each draft was certain
 *                                            (q = 1 at x_j, 0 elsewhere)
 *   uniforms       fp32       [N, D + 1]     any strides; values in [0, 1)
 *   cu_seqlens     int32      [N + 1] or NULL  contiguous; T_i <= D + 1
 *   state_indices  int32      [N] or NULL    contiguous; a negative one marks a
 *                                            padded sequence
 *   out_tokens     int32      [N, D + 1]     the accepted drafts, the drawn
 *                                            token, then -1
 *   num_tokens     int32      [N]            A + 1
 * A sequence that is padded, empty (T_i = 0) or has bad cu_seqlens
 * (GDN_DEV_BAD_SEQLENS; T_i > D + 1 among them) gets num_tokens 0 and -1 in
 * its whole row of out_tokens.  draft_tokens[i, j] = -1 ends a sequence's
 * drafts early: the token is drawn from p_j itself; so does any other token
 * outside the vocabulary, with GDN_DEV_BAD_TOKEN.  u q < p is compared exactly;
 * p - q, the sums and u W are fp64, added in an order that the arguments fix
 * (weights that are multiples of 2^-52 W are summed exactly).  Where p or p - q
 * is NaN, infinite or not positive it weighs nothing; where that leaves W = 0
 * after a rejection the token is drawn from p_A, and where that is empty too it
 * is -1, with GDN_DEV_BAD_PROBS.  The draw's u counts as 0 when it is below 0,
 * one of 1 or more (or NaN) draws the last (first) token
 * of positive weight.  With GDN_DEV_TIMEOUT a sequence may have num_tokens 0 and
 * an out_tokens row that is not to be read; counts other than 0 stand beside the
 * whole answer.  vocab >= 1; N = 0 is GDN_OK with no launch.
 */
GDN_API int gdn_verify_drafts(const gdn_tensor *target_probs, const gdn_tensor *draft_tokens,
                              const gdn_tensor *draft_probs, const gdn_tensor *uniforms,
                              const gdn_tensor *cu_seqlens, const gdn_tensor *state_indices,
                              const gdn_tensor *out_tokens, const gdn_tensor *num_tokens, uint32_t flags,
                              const gdn_extra *extra);

/*
 * The state after each sequence's last kept token into its slot:
 *     state_pool[state_indices[i]] = intermediate_states[cu_seqlens[i] + n - 1],
 *     n = num_tokens[i]
 * for every sequence with n >= 1 and a slot that is not -1; n = 0 leaves the
 * slot as it was.  For updates run with GDN_WRITE_INTERMEDIATE, normally with
 * GDN_NO_FINAL_WRITEBACK.
 *   intermediate_states  fp32   [T_tot, HV, K, V]
 *   num_tokens           int32  [N]               contiguous
 *   state_pool           fp32   [num_slots, HV, K, V]
 *   state_indices        int32  [N]               contiguous
 *   cu_seqlens           int32  [N + 1] or NULL   contiguous; NULL = T_tot / N
 *                                                 tokens each
 * States are K = V = 128 with the layout rules of gdn_decode.h; those of the
 * pool share no address, slots inside one head stride or heads inside one slot
 * stride (GDN_ERR_SHAPE).  The
 * non-negative state_indices must be distinct.  A sequence with a bad slot,
 * bad cu_seqlens or a count outside 0 .. T_i (GDN_DEV_BAD_SLOT,
 * GDN_DEV_BAD_SEQLENS, GDN_DEV_BAD_COUNT) is skipped.  N = 0 or T_tot = 0 is
 * GDN_OK with no launch.
 */
GDN_API int gdn_commit_states(const gdn_tensor *intermediate_states, const gdn_tensor *num_tokens,
                              const gdn_tensor *state_pool, const gdn_tensor *state_indices,
                              const gdn_tensor *cu_seqlens, uint32_t flags, const gdn_extra *extra);

/*
 * A step's index arrays from its requests' lengths.  Request i runs
 * lengths[i] tokens behind context[i] tokens that it has already; it runs at
 * all when lengths[i] > 0 and slots[i] is not -1.
 *   lengths        int32  [N]      in
 *   context        int32  [N]      in
 *   slots          int32  [N]      in:  the request's slot in the state pool
 *   cu_seqlens     int32  [N + 1]  out: running sum of the lengths that run
 *   state_indices  int32  [N]      out: slots[i], -1 where i does not run
 *   row_seq        int32  [C]      out: the request of each packed row
 *   positions      int32  [C]      out: context[i] + offset in the request
 * Rows behind the last token get -1 in the [C] arrays.  With a cache in blocks
 * of block_size tokens beside the state pool (all of the following, or none):
 *   block_tables     int32  [N, B]  in/out: block of each block_size tokens of
 *                                           request i, row stride >= B
 *   blocks_held      int32  [N]     in:  entries of block_tables[i] in use
 *   free_blocks      int32  [F]     in:  ids of free blocks
 *   free_head        int32  [1]     in:  free_blocks before it are taken
 *   blocks_held_out  int32  [N]     out: entries in use after the step
 *   free_head_out    int32  [1]     out
 *   slot_map         int64  [C]     out: block * block_size + offset, where the
 *                                        row's token goes in the cache
 * Request i takes the blocks it lacks, ceil((context + length) / block_size) -
 * blocks_held[i] when positive, from free_blocks in request order, and they
 * are written behind its entries; the others of its table are left as they
 * were.  All vectors are contiguous.
 *
 * A request with a bad length, context, block count (GDN_DEV_BAD_LENGTH,
 * GDN_DEV_BAD_BLOCKS) or slot < -1 (GDN_DEV_BAD_SLOT) does not run.  Where the
 * C rows or the free blocks run out, the first request that does not fit and
 * every later one do not run (GDN_DEV_NO_ROOM); what does not run takes no
 * block.  Launched even with N = 0 (cu_seqlens = {0}, the rest -1); N is at most
 * INT32_MAX - 1024.
 */
typedef struct gdn_step_maps_call {
    const gdn_tensor *lengths, *context, *slots;
    const gdn_tensor *cu_seqlens, *state_indices, *row_seq, *positions;
    const gdn_tensor *block_tables, *blocks_held, *free_blocks, *free_head;
    const gdn_tensor *blocks_held_out, *free_head_out, *slot_map;
    int32_t block_size; /* >= 1 with a blocked cache, else 0 */
    uint32_t flags;
    const gdn_extra *extra;
} gdn_step_maps_call;

GDN_API int gdn_step_maps(const gdn_step_maps_call *call);

/* GDN_SPEC_ABI_VERSION of the loaded library. */
GDN_API int gdn_spec_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SPEC_H */
