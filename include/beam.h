/*
 * libmamba2 — beam search over recurrent states: the selection over beams and
 * vocabulary, and the reordering of the state pools that follows it. Same
 * conventions as mamba2.h; everything is in device memory, so that a captured
 * CUDA graph can run both calls.
 */
#ifndef MAMBA2_BEAM_H
#define MAMBA2_BEAM_H

#include "mamba2.h"

/* Most beams of a sequence, and most candidates that are kept of it. */
#define MAMBA2_MAX_BEAMS 32
/* Most pools that one call reorders. */
#define MAMBA2_MAX_POOLS 64

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Of every sequence's beams x vocab candidates, whose values are
 *
 *   scores[b][i] + logits[b beams + i][t] - log sum_t' exp(logits[b beams + i][t'])
 *
 * (i the beam, t the token), the `out` largest in descending order; equal ones
 * by ascending i, then t. A value that is not a number counts as -infinity, so
 * a logit of -infinity is a token that may not follow, and a beam whose score
 * is -infinity, whose logits are all -infinity, or hold a NaN or +infinity,
 * has only such candidates. They too are candidates, the last in that order. A
 * finished beam has one other: `eos`, at its score as it is.
 *
 *   scores_out   [batch, out] f32; may not be `scores`
 *   parents      [batch, out] int32: the beam that the candidate continues
 *   tokens       [batch, out] int32
 *   finished_out [batch, out] uint8 or NULL: the parent was finished, or the
 *                token is eos
 *   logits       [batch * beams, vocab] act, row stride ld; the alignment of
 *                an element suffices
 *   scores       [batch, beams] f32, each finite or -infinity
 *   finished     [batch, beams] uint8 or NULL (none is)
 *   eos          a token, or -1: no token ends a beam (then `finished` and
 *                finished_out are NULL)
 *   workspace    of at least mamba2_beam_select_workspace_bytes, 256-byte
 *                aligned
 * 1 <= beams, out <= MAMBA2_MAX_BEAMS, out <= beams * vocab and batch * beams
 * <= 65535. Values are
 * compared in fp64, from an fp32 sum of exponentials. Outputs other than
 * these four are not written; none may overlap an input.
 */
size_t mamba2_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t out, int32_t vocab);

mamba2_status mamba2_beam_select(float* scores_out, int32_t* parents, int32_t* tokens, uint8_t* finished_out,
                                 const void* logits, const float* scores, const uint8_t* finished, int32_t batch,
                                 int32_t beams, int32_t out, int32_t vocab, int64_t ld, int32_t eos,
                                 mamba2_dtype act, void* workspace, size_t workspace_bytes, void* stream);

/*
 * For every sequence b and beam j at once, in every pool:
 *
 *   pool[slots[b][j]] = pool[slots[b][parents[b][j]]]   (as it was before)
 *
 *   pools      host array of num_pools device pointers, each a pool of
 *              num_slots slots of slot_bytes[i] bytes; two that overlap are
 *              refused
 *   slots      [batch, beams] int32, all different
 *   parents    [batch, beams] int32 in [0, beams)
 *   status_dev int32: receives the mamba2_status of what is checked on the
 *              device: MAMBA2_ERR_SLOT_OUT_OF_RANGE, MAMBA2_ERR_SLOT_SHARED,
 *              or MAMBA2_ERR_INVALID_ARGUMENT for a parent out of range; then
 *              no pool is touched
 * batch * beams <= MAMBA2_MAX_SEQS, beams <= MAMBA2_MAX_BEAMS, num_pools <=
 * MAMBA2_MAX_POOLS. Pools that are 16-byte aligned, of slots of a multiple of
 * 16 bytes, are moved at the rate of memory; any other alignment is taken.
 */
mamba2_status mamba2_reorder_states(void* const* pools, const int64_t* slot_bytes, int32_t num_pools,
                                    int32_t num_slots, const int32_t* slots, const int32_t* parents, int32_t batch,
                                    int32_t beams, int32_t* status_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_BEAM_H */
