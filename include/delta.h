/*
 * libmamba2 — the gated delta rule, next to the selective scan of mamba2.h and
 * under the same conventions (caller-owned device buffers, host batch metadata
 * validated before anything is enqueued, asynchronous on `stream`, no device
 * allocation, the same status codes; alignment and row strides as in block.h).
 *
 * Per head h, whose key group is h / (heads / ngroups), with a_t = exp(g_t):
 *
 *   u_t = beta_t (v_t - a_t S_{t-1} k_t)
 *   S_t = a_t S_{t-1} + u_t k_t^T
 *   y_t = scale S_t q_t
 *
 * S is [headdim, d_state] and is kept in fp32. With l2_eps >= 0, q_t and k_t
 * are first divided by sqrt(sum of their squares + l2_eps); a negative l2_eps
 * takes them as they are. The state stays bounded where g <= 0 and
 * 0 <= beta |k|^2 <= 2 (not checked). A g below -10000 is taken as -10000: the
 * state is forgotten, as exp(-104) already leaves nothing of it in fp32.
 *
 * bf16 heads of at most 128 x 128 go by chunks on the tensor cores: operands of
 * the products that end in y alone are bf16, those of the products that end in
 * the state have twice its digits (2-norms of y and of end states are then about
 * 1.4e-3, before y's own rounding, and 2e-6 off). All else is fp32, token by
 * token.
 *
 * Runs do not touch one another, but a value that is not finite may reach the
 * outputs of its run from the beginning of its MAMBA2_DELTA_CHUNK tokens on.
 *
 *   q, k   [rows, ngroups, d_state] act, row strides ld_q, ld_k
 *   v, y   [rows, heads, headdim] act, row strides ld_v, ld_y
 *   g      [rows, heads] f32 or NULL (0: nothing decays)
 *   beta   [rows, heads] f32 or NULL (1)
 *   state  [num_slots, heads, headdim, d_state] f32, updated in place at the
 *          batch's slots (from zero when fresh)
 *   dims   heads a multiple of ngroups; conv_kernel is not used
 *
 * A row's heads are contiguous, rows are 16-byte aligned: d_state, headdim and
 * the row strides are multiples of 8, and the tensors' pointers (those of g and
 * beta too) of 16 bytes. Other sizes, d_state above
 * MAMBA2_MAX_DELTA_STATE and an unaligned stride are
 * MAMBA2_ERR_NOT_IMPLEMENTED.
 */
#ifndef MAMBA2_DELTA_H
#define MAMBA2_DELTA_H

#include "mamba2.h"

#define MAMBA2_DELTA_CHUNK 64
#define MAMBA2_MAX_DELTA_STATE 256

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of `checkpoints`: the sum over runs of ceil(length / MAMBA2_DELTA_CHUNK).
 * -1 for a cu_seqlens that does not start at 0 or decreases, or a bad
 * num_seqs. */
int64_t mamba2_gated_delta_rule_checkpoints(const int32_t* cu_seqlens, int32_t num_seqs);

/* Workspace of the forward (backward = 0) or backward call (backward = 1); 0
 * also for arguments that the call would refuse. 256-byte aligned. */
size_t mamba2_gated_delta_rule_workspace_bytes(const int32_t* cu_seqlens, int32_t num_seqs, const mamba2_dims* dims,
                                               mamba2_dtype act, int32_t backward);

/*
 * Packed runs. A run of no rows zeroes its slot when fresh and leaves it
 * otherwise.
 *   checkpoints [mamba2_gated_delta_rule_checkpoints(...), heads, headdim,
 *               d_state] f32 or NULL: for the backward pass, the state before
 *               each MAMBA2_DELTA_CHUNK tokens of each run, in order
 */
mamba2_status mamba2_gated_delta_rule(void* y, float* checkpoints, const void* q, const void* k, const void* v,
                                      const float* g, const float* beta, float* state, int32_t num_slots,
                                      int32_t rows, int64_t ld_y, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                      const mamba2_dims* dims, float scale, float l2_eps, mamba2_dtype act,
                                      const mamba2_recurrent_batch* rb, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * One token per sequence (row i of the inputs and of y is sequence i's).
 * cu_seqlens of the batch may be NULL; it must be 0..n if given.
 */
mamba2_status mamba2_gated_delta_rule_step(void* y, const void* q, const void* k, const void* v, const float* g,
                                           const float* beta, float* state, int32_t num_slots, int64_t ld_y,
                                           int64_t ld_q, int64_t ld_k, int64_t ld_v, const mamba2_dims* dims,
                                           float scale, float l2_eps, mamba2_dtype act,
                                           const mamba2_recurrent_batch* rb, void* stream);

/*
 * The same with the batch in device memory, for CUDA-graph replay: see
 * mamba2_decode_step_device for slots_dev, fresh_dev, num_seqs_dev, capacity
 * and status_dev, which mean and are checked the same here. fresh_dev may be
 * NULL here: no sequence is fresh.
 */
mamba2_status mamba2_gated_delta_rule_step_device(void* y, const void* q, const void* k, const void* v,
                                                  const float* g, const float* beta, float* state,
                                                  int32_t num_slots, int64_t ld_y, int64_t ld_q, int64_t ld_k,
                                                  int64_t ld_v, const mamba2_dims* dims, float scale, float l2_eps,
                                                  mamba2_dtype act, const int32_t* slots_dev,
                                                  const uint8_t* fresh_dev, const int32_t* num_seqs_dev,
                                                  int32_t capacity, int32_t* status_dev, void* stream);

/*
 * Gradients of the forward call, from the checkpoints that it wrote. With G_t
 * the gradient that reaches S_t: G_t = scale dy_t q_t^T + (a_{t+1} G_{t+1} -
 * a_{t+1} dv_{t+1} k_{t+1}^T), the last one plus dstate_end;
 *   dv_t = beta_t G_t k_t,  dbeta_t = (G_t k_t) . (v_t - a_t S_{t-1} k_t),
 *   dq_t = scale dy_t^T S_t,  dk_t = u_t^T G_t - a_t dv_t^T S_{t-1} (both
 *   summed over the group's heads, and carried through the division by their
 *   lengths),  dg_t = <G_t - dv_t k_t^T, a_t S_{t-1}>,
 *   dstate = a_0 (G_0 - dv_0 k_0^T) (dstate_end itself for a run of no rows).
 * For bf16, with d_state and headdim of at most 128; MAMBA2_ERR_NOT_IMPLEMENTED
 * otherwise. Operands of the products that end in dq, dk, dg and dbeta are
 * rounded to bf16; dv and dstate, and v_t - a_t S_{t-1} k_t, which may be a small
 * difference, come from operands of twice its digits.
 *
 *   dq, dk    [rows, ngroups, d_state] act, row strides ld_dq, ld_dk
 *   dv        [rows, heads, headdim] act, row stride ld_dv
 *   dg, dbeta [rows, heads] act, contiguous, or NULL (also of a g or beta that
 *             is NULL)
 *   dstate    [num_seqs, heads, headdim, d_state] f32 or NULL: of each run's
 *             initial state (also written for fresh runs, whose state was zero)
 *   dy        [rows, heads, headdim] act, row stride ld_dy
 *   dstate_end  as dstate, or NULL (zero)
 */
mamba2_status mamba2_gated_delta_rule_backward(void* dq, void* dk, void* dv, void* dg, void* dbeta, float* dstate,
                                               const void* dy, const float* dstate_end, const void* q, const void* k,
                                               const void* v, const float* g, const float* beta,
                                               const float* checkpoints, int32_t rows, int64_t ld_dq, int64_t ld_dk,
                                               int64_t ld_dv, int64_t ld_dy, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                               const mamba2_dims* dims, float scale, float l2_eps, mamba2_dtype act,
                                               const int32_t* cu_seqlens, int32_t num_seqs, void* workspace,
                                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_DELTA_H */
