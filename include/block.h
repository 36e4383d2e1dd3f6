/*
 * libmamba2 — the operators of a gated-recurrence residual block, next to the
 * Mamba2 layer of mamba2.h and under the same conventions (caller-owned
 * device buffers, host batch metadata validated before anything is enqueued,
 * asynchronous on `stream`, no device allocation, the same status codes):
 *
 *   add + RMS norm      s = x + residual, out = s / rms(s) * weight, in the
 *                       activation type or in 8 bits with a scale per row
 *   linear              out = activation(x . w^T + bias) + residual, from
 *                       bf16 or 8-bit operands
 *   gated recurrence    h_t = f_t h_{t-1} + (1 - f_t) x_t over packed runs
 *
 * each with its backward pass; the recurrence also as a single-token step.
 * Gradients are written, never added to what the buffers held. Sums, states
 * and statistics are fp32; every output is rounded once to its type.
 *
 * Matrices are row-major. Where an argument list has a row stride (ld_*, in
 * elements, >= the row's width), the matrix may be a column range of a wider
 * one; the others are contiguous. Pointers are 16-byte aligned, except those
 * with a row stride, for which the alignment of their element suffices
 * (16-byte aligned rows are fastest); any other misalignment, a null pointer
 * that is not marked optional, a negative size or a row stride below the width
 * is MAMBA2_ERR_INVALID_ARGUMENT, as are more rows or a greater width than
 * MAMBA2_MAX_BLOCK_SIZE. Outputs must not overlap inputs unless said.
 */
#ifndef MAMBA2_BLOCK_H
#define MAMBA2_BLOCK_H

#include "mamba2.h"

/* Most rows, and columns of a matrix, that a call takes: 2^31 less what rounds
 * either up to whole tiles. */
#define MAMBA2_MAX_BLOCK_SIZE 0x7fff0000

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- gated recurrence
 *
 * Per channel, with lo = lower[channel] (0 when lower is NULL):
 *   f_t = lo + (1 - lo) sigmoid(gate_t)
 *   h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t
 * over the rows of each run of the RecurrentBatch, from the run's slot of the
 * state pool (zero when fresh); the slot then holds the last h. A run of no
 * rows zeroes its slot when fresh and leaves it otherwise. 1 - f_t is computed
 * as (1 - lo) sigmoid(-gate_t), which keeps its digits as f_t nears 1.
 *
 *   y     [rows, dim] act, row stride ld_y
 *   x     [rows, dim] act, row stride ld_x;  gate likewise, ld_gate
 *   lower [dim] f32, each in [0, 1] (not checked), or NULL
 *   state [num_slots, dim] f32, updated in place at the named slots
 *   checkpoints [mamba2_gated_recurrence_checkpoints(...), dim] f32 or NULL:
 *         for the backward pass, the state before each
 *         MAMBA2_RECURRENCE_STEP tokens of each run, in order; a run has rows
 *         for whole chunks of MAMBA2_RECURRENCE_CHUNK tokens, and those past
 *         its end are left as they are
 *   workspace 256-byte aligned, of at least the bytes that
 *         mamba2_gated_recurrence_workspace_bytes gives (NULL when 0)
 */
#define MAMBA2_RECURRENCE_CHUNK 128
#define MAMBA2_RECURRENCE_STEP 16

/* Rows of `checkpoints`: chunk / step times the sum over runs of
 * ceil(length / chunk). -1 for a
 * cu_seqlens that does not start at 0 or decreases, or a bad num_seqs. */
int64_t mamba2_gated_recurrence_checkpoints(const int32_t* cu_seqlens, int32_t num_seqs);

/* Workspace of the forward (backward = 0) or backward call (backward = 1); 0
 * also for arguments that the call would refuse. */
size_t mamba2_gated_recurrence_workspace_bytes(const int32_t* cu_seqlens, int32_t num_seqs, int32_t dim,
                                               int32_t backward);

mamba2_status mamba2_gated_recurrence(void* y, float* checkpoints, const void* x, const void* gate,
                                      const float* lower, float* state, int32_t num_slots, int32_t rows,
                                      int32_t dim, int64_t ld_y, int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                      const mamba2_recurrent_batch* rb, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * One token per sequence (row i of x, gate and y is sequence i's).
 * cu_seqlens of the batch may be NULL; it must be 0..n if given.
 */
mamba2_status mamba2_gated_recurrence_step(void* y, const void* x, const void* gate, const float* lower,
                                           float* state, int32_t num_slots, int32_t dim, int64_t ld_y, int64_t ld_x,
                                           int64_t ld_gate, mamba2_dtype act, const mamba2_recurrent_batch* rb,
                                           void* stream);

/*
 * The same with the batch in device memory, for CUDA-graph replay: see
 * mamba2_decode_step_device for slots_dev, fresh_dev, num_seqs_dev, capacity
 * and status_dev, which mean and are checked the same here. fresh_dev may be
 * NULL here: no sequence is fresh.
 */
mamba2_status mamba2_gated_recurrence_step_device(void* y, const void* x, const void* gate, const float* lower,
                                                  float* state, int32_t num_slots, int32_t dim, int64_t ld_y,
                                                  int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                                  const int32_t* slots_dev, const uint8_t* fresh_dev,
                                                  const int32_t* num_seqs_dev, int32_t capacity, int32_t* status_dev,
                                                  void* stream);

/*
 * Gradients of the forward call, from the checkpoints that it wrote. With G_t
 * the gradient that reaches h_t: G_t = dy_t + f_{t+1} G_{t+1}, the last one
 * plus dstate_end;
 *   dx_t = (1 - f_t) G_t,  dgate_t = G_t (h_{t-1} - x_t) (1 - lo) s (1 - s) with
 *   s = sigmoid(gate_t),   dlower = sum_t G_t (h_{t-1} - x_t) (1 - s),
 *   dstate = f_0 G_0 (dstate_end itself for a run of no rows).
 *
 *   dx, dgate  [rows, dim] act, row strides ld_dx, ld_dgate
 *   dlower     [dim] f32 or NULL (must be NULL when lower is); summed in a
 *              fixed order
 *   dstate     [num_seqs, dim] f32 or NULL: of each run's initial state (also
 *              written for fresh runs, whose state was zero)
 *   dy         [rows, dim] act, row stride ld_dy
 *   dstate_end [num_seqs, dim] f32 or NULL (zero)
 */
mamba2_status mamba2_gated_recurrence_backward(void* dx, void* dgate, float* dlower, float* dstate, const void* dy,
                                               const float* dstate_end, const void* x, const void* gate,
                                               const float* lower, const float* checkpoints, int32_t rows,
                                               int32_t dim, int64_t ld_dx, int64_t ld_dgate, int64_t ld_dy,
                                               int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                               const int32_t* cu_seqlens, int32_t num_seqs, void* workspace,
                                               size_t workspace_bytes, void* stream);

/* --------------------------------------------------------- add + RMS norm
 *
 * s = x + residual (x alone when residual is NULL), in fp32;
 * y = s * weight / sqrt(mean(s^2) + eps).
 *
 *   x        [rows, dim] act
 *   residual [rows, dim] sum_type (the activation type or f32) or NULL
 *   sum      [rows, dim] sum_type or NULL: s, rounded to sum_type (may be
 *            `residual` itself; the norm is of the unrounded sum)
 *   out      [rows, dim] out_type: act or MAMBA2_E4M3
 *   scale    [rows] f32, with MAMBA2_E4M3 only: max |y| / 448 over the row (1
 *            for a row of zeros; rounded up where it is below 2^-126); out is
 *            y / scale in e4m3, to nearest even. A row holding a NaN or an
 *            infinity has a NaN scale and NaN outputs.
 *   weight   [dim] f32; eps >= 0
 */
mamba2_status mamba2_add_rmsnorm(void* out, float* scale, void* sum, const void* x, const void* residual,
                                 const float* weight, int32_t rows, int32_t dim, float eps, mamba2_dtype act,
                                 mamba2_dtype sum_type, mamba2_dtype out_type, void* stream);

/* Workspace of the backward call. */
size_t mamba2_add_rmsnorm_backward_workspace_bytes(int32_t rows, int32_t dim);

/*
 * From s (the forward's `sum`, or its x where there was no residual) and the
 * gradients of both outputs: with inv = 1 / sqrt(mean(s^2) + eps),
 *   ds = dsum + inv (weight dy - s inv^2 mean(weight dy s)),
 *   dweight = sum over rows of dy s inv (in a fixed order).
 *
 *   dx        [rows, dim] act or NULL: ds, the gradient of x
 *   dresidual [rows, dim] sum_type or NULL: ds, the gradient of residual (the
 *             same values as dx when the types agree; may be `dsum` itself)
 *   dweight   [dim] f32 or NULL
 *   dy        [rows, dim] act
 *   dsum      [rows, dim] sum_type or NULL (zero)
 *   sum       [rows, dim] sum_type
 */
mamba2_status mamba2_add_rmsnorm_backward(void* dx, void* dresidual, float* dweight, const void* dy,
                                          const void* dsum, const void* sum, const float* weight, int32_t rows,
                                          int32_t dim, float eps, mamba2_dtype act, mamba2_dtype sum_type,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------- linear
 *
 * out = activation(p) + residual, p[m][n] = (sum_k x[m][k] w[n][k]) x_scale[m]
 * w_scale[n] + bias[n], with fp32 accumulation on the tensor cores.
 *
 *   out      [rows, out_features] out_type (bf16 or f32), row stride ld_out
 *   pre      [rows, out_features] bf16 or NULL: p, which the backward pass
 *            takes when there is an activation
 *   x        [rows, in_features] in_type, row stride ld_x; 16-byte aligned rows
 *   w        [out_features, in_features] in_type, the layer's weight as stored
 *   x_scale  [rows] f32, w_scale [out_features] f32: with MAMBA2_E4M3 operands
 *            only, both required (mamba2_add_rmsnorm writes the first)
 *   bias     [out_features] f32 or NULL
 *   residual [rows, out_features] out_type, row stride ld_residual, or NULL;
 *            may be `out` itself (with the same row stride)
 *   in_type  MAMBA2_BF16 or MAMBA2_E4M3
 * in_features and ld_x are multiples of 8 (bf16) or 16 (e4m3), else
 * MAMBA2_ERR_NOT_IMPLEMENTED, as for an in_type of f32.
 */
typedef enum mamba2_activation {
  MAMBA2_ACT_NONE = 0,
  MAMBA2_ACT_RELU = 1, /* max(p, 0); NaN for a NaN, as the others */
  MAMBA2_ACT_SILU = 2, /* p sigmoid(p) */
  MAMBA2_ACT_GELU = 3  /* p Phi(p), Phi the normal distribution function (for p < 0 to a relative (64 + 2 p^2) 2^-24) */
} mamba2_activation;

mamba2_status mamba2_linear(void* out, void* pre, const void* x, const float* x_scale, const void* w,
                            const float* w_scale, const float* bias, const void* residual, int32_t rows,
                            int32_t in_features, int32_t out_features, int64_t ld_out, int64_t ld_x,
                            int64_t ld_residual, mamba2_dtype in_type, mamba2_dtype out_type,
                            mamba2_activation activation, void* stream);

/* Workspace of the backward call. */
size_t mamba2_linear_backward_workspace_bytes(int32_t rows, int32_t in_features, int32_t out_features);

/*
 * Gradients, for bf16 operands: with dp = dy * activation'(pre),
 *   dx = dp . w,  dw = dp^T . x,  dbias = sum over rows of dp (fixed order).
 * The residual's gradient is dy itself. dp is rounded to bf16 where it enters
 * the two products (dbias sums it unrounded); relu'(0) = 0, relu'(NaN) = NaN.
 *
 *   dx    [rows, in_features] bf16 or NULL
 *   dw    [out_features, in_features] bf16 or NULL
 *   dbias [out_features] f32 or NULL
 *   dy    [rows, out_features] bf16, contiguous, also for a forward call with
 *         an f32 out; pre likewise (NULL with MAMBA2_ACT_NONE)
 *   x     [rows, in_features] bf16, row stride ld_x; 16-byte aligned rows
 * in_features and ld_x multiples of 8 (MAMBA2_ERR_NOT_IMPLEMENTED otherwise).
 */
mamba2_status mamba2_linear_backward(void* dx, void* dw, float* dbias, const void* dy, const void* pre,
                                     const void* x, const void* w, int32_t rows, int32_t in_features,
                                     int32_t out_features, int64_t ld_x, mamba2_activation activation,
                                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_BLOCK_H */
