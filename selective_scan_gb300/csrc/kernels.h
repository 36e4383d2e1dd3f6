// Kernel argument blocks and launchers (internal to libmamba2).
//
// Every kernel takes one argument block by value (__grid_constant__), so the
// batch table travels in the launch parameters: no device metadata buffers and
// no host->device copies per call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mamba2.h"

namespace mamba2 {

// Batch table. Sequence i owns rows [cu[i], cu[i+1]); its slot is
// slot_fresh[i] & 0x7fffffff and it is fresh when bit 31 is set. tile[i] is
// the index of the sequence's first work tile (tile[n] = total tiles); each
// kernel defines what a tile is (conv: kConvRows rows; scan: one segment).
struct SeqTable {
  int32_t n;
  int32_t cu[MAMBA2_MAX_SEQS + 1];
  uint32_t slot_fresh[MAMBA2_MAX_SEQS];
  int32_t tile[MAMBA2_MAX_SEQS + 1];
};

// ---------------------------------------------------------------- conv ----
constexpr int kConvThreads = 256;
constexpr int kConvRows = 14;  // rows per work tile (>= kernel - 1)

struct ConvArgs {
  const void* x;
  void* dst;
  const float* weight;
  const float* bias;
  void* conv_state;
  int32_t conv_dim;
  SeqTable tab;
};
cudaError_t launch_conv1d(const ConvArgs& a, mamba2_dtype act, int kernel, cudaStream_t st);

// ---------------------------------------------------------------- scan ----
constexpr int kChunk = 64;  // tokens per chunk of the chunked scan

struct ScanArgs {
  void* dst;
  const void* xbc;
  const void* dt;
  const float* A_log;
  const float* dt_bias;
  const float* D;
  float* ssm_state;
  float* ws_state;  // [segments * state_pieces, heads, P, N] (null when unsegmented)
  float* ws_decay;  // [segments * state_pieces, heads]
  float* dtp;       // [heads, rows] dt' = softplus(dt + dt_bias) (tcgen05 path; null otherwise)
  int32_t heads, headdim, d_state, ngroups, conv_dim;
  int32_t seg_chunks;  // chunks per segment (tile = segment)
  int32_t state_pieces;  // tcgen05 state pass: entries per segment, each over an equal share of its chunks
  SeqTable tab;
};
// True when the chunked tensor-core kernels cover this shape: tcgen05 for
// headdim 64 x d_state 128 (chunks of kChunkTc tokens), mma.sync for 16 x 16.
bool scan_chunked_supported(mamba2_dtype act, int headdim, int d_state);
constexpr int kChunkTc = 128;
inline bool scan_uses_tc(mamba2_dtype act, int headdim, int d_state) {
  return act == MAMBA2_BF16 && headdim == 64 && d_state == 128;
}
inline int scan_chunk_tokens(int headdim, int d_state) {
  return (headdim == 64 && d_state == 128) ? kChunkTc : kChunk;
}
cudaError_t launch_scan_tc(const ScanArgs& a, cudaStream_t st);
unsigned int read_device_timeouts();
// Chunked scan: state pass over all but the last segment of each sequence,
// then the full pass. The serial kernel is the token-at-a-time fallback.
cudaError_t launch_scan_chunked(const ScanArgs& a, cudaStream_t st);
cudaError_t launch_scan_serial(const ScanArgs& a, mamba2_dtype act, cudaStream_t st);
constexpr int kSerialMaxN = 256;
constexpr int kSerialMaxP = 1024;

// ---------------------------------------------------------------- norm ----
struct NormArgs {
  void* dst;
  const void* x;
  const void* z;
  const float* weight;
  int32_t rows;
  int32_t dim;
  int32_t groups;
  float eps;
};
cudaError_t launch_gated_rmsnorm(const NormArgs& a, mamba2_dtype act, cudaStream_t st);

// -------------------------------------------------------------- decode ----
constexpr int kDecodeThreads = 256;
constexpr int kDecodeMaxHeadsPerCta = 8;  // heads per CTA of the state kernel for large batches
constexpr int kDecodeMaxNormGroups = 64;

struct DecodeArgs {
  void* dst;
  const void* xBC;
  const void* z;
  const void* dt;
  const float* conv_w;
  const float* conv_b;
  const float* A_log;
  const float* dt_bias;
  const float* D;
  const float* norm_w;
  void* conv_state;
  float* ssm_state;
  int32_t heads, headdim, d_state, ngroups, conv_kernel;
  int32_t norm_groups;
  float eps;
  int32_t ctas_per_seq;    // CTAs per sequence of the state kernel
  int32_t heads_per_cta;
  SeqTable tab;            // host batch: tab.n sequences; device batch: tab.n = capacity, rest unused
  // Device batch (all null for a host batch): sequence s < *dev_n has slot dev_slots[s]
  // and is fresh when dev_fresh[s] != 0; no CTA touches anything while *dev_status != 0.
  const int32_t* dev_slots;
  const uint8_t* dev_fresh;
  const int32_t* dev_n;
  const int32_t* dev_status;
};
bool decode_supported(mamba2_dtype act, const mamba2_dims& d, int norm_groups);

// ------------------------------------------------------------ GEMM ----
// dst = A[M, K] . B[N, K]^T (bf16, K contiguous in both), bf16 out. Output columns
// [seg_end[i-1], seg_end[i]) go to dst[i] (row stride ld[i], column 0 = seg_end[i-1]);
// every segment boundary is a multiple of 8 columns and every dst row 16-byte aligned.
struct GemmArgs {
  int32_t M, N, K;
  int32_t nseg;
  int32_t seg_end[3];
  void* dst[3];
  int64_t ld[3];
};
cudaError_t launch_gemm_tc(const GemmArgs& g, const void* A, const void* B, cudaStream_t st);
unsigned int read_gemm_timeouts();

// ------------------------------------------------------ recurrent block ----
// Gated recurrence, forward. tab.tile[i] = the sequence's first chunk (chunks of
// MAMBA2_RECURRENCE_CHUNK tokens, ceil(length / chunk) a sequence).
struct RecTensors {
  void* y;
  float* ckpt;  // [chunks * chunk / step, dim] or null
  const void* x;
  const void* gate;
  const float* lower;  // [dim] or null
  float* state;
  int32_t dim;
  int64_t ld_y, ld_x, ld_gate;
};
struct RecArgs : RecTensors {
  SeqTable tab;
};
cudaError_t launch_recurrence(const RecArgs& a, mamba2_dtype act, void* ws, cudaStream_t st);
size_t recurrence_workspace(int64_t chunks, bool chained, int32_t runs, int32_t dim, bool backward);

struct RecStepArgs {
  void* y;
  const void* x;
  const void* gate;
  const float* lower;
  float* state;
  int32_t dim, n;  // n: sequences, or the capacity of a device batch
  int64_t ld_y, ld_x, ld_gate;
  int32_t num_slots;
  const int32_t* dev_slots;  // device batch (null for a host batch), as in DecodeArgs
  const uint8_t* dev_fresh;
  const int32_t* dev_n;
  int32_t* dev_status;
  uint32_t slot_fresh[MAMBA2_MAX_SEQS];
};
// Checks a device batch too (in the kernel, or by launch_check_device_batch).
cudaError_t launch_recurrence_step(const RecStepArgs& a, mamba2_dtype act, cudaStream_t st);

// Gated recurrence, backward (tab.tile as in RecArgs; slots unused).
struct RecBwdTensors {
  void* dx;
  void* dgate;
  float* dlower;
  float* dstate;
  const void* dy;
  const float* dstate_end;
  const void* x;
  const void* gate;
  const float* lower;
  const float* ckpt;
  int32_t dim;
  int64_t ld_dx, ld_dgate, ld_dy, ld_x, ld_gate;
};
struct RecBwdArgs : RecBwdTensors {
  SeqTable tab;
};
cudaError_t launch_recurrence_backward(const RecBwdArgs& a, mamba2_dtype act, void* ws, cudaStream_t st);

struct AddNormArgs {
  void* out;
  float* scale;
  void* sum;
  const void* x;
  const void* residual;
  const float* weight;
  int32_t rows, dim;
  float eps;
};
cudaError_t launch_add_rmsnorm(const AddNormArgs& a, mamba2_dtype act, mamba2_dtype sum_type, mamba2_dtype out_type,
                               cudaStream_t st);

struct AddNormBwdArgs {
  void* dx;
  void* dresidual;
  float* dweight;
  const void* dy;
  const void* dsum;
  const void* sum;
  const float* weight;
  float* partial;  // [add_rmsnorm_backward_parts, dim]
  int32_t rows, dim;
  float eps;
};
int add_rmsnorm_backward_parts(int32_t rows, int32_t dim);
cudaError_t launch_add_rmsnorm_backward(const AddNormBwdArgs& a, mamba2_dtype act, mamba2_dtype sum_type,
                                        cudaStream_t st);

// dst[i] = sum over p < parts of part[p][i], in a fixed order.
cudaError_t launch_column_sum(float* dst, const float* part, int parts, int dim, cudaStream_t st);

struct LinearArgs {
  void* out;
  void* pre;
  const void* x;
  const float* x_scale;
  const void* w;
  const float* w_scale;
  const float* bias;
  const void* residual;
  int32_t rows, in_f, out_f;
  int64_t ld_out, ld_x, ld_res;
};
cudaError_t launch_linear(const LinearArgs& a, mamba2_dtype in, mamba2_dtype out, int act, cudaStream_t st);

struct LinearBwdArgs {
  void* dx;
  void* dw;
  float* dbias;
  const void* dy;
  const void* pre;
  const void* x;
  const void* w;
  int32_t rows, in_f, out_f;
  int64_t ld_x;
  void* dp;        // [rows, ld_dp] bf16, or null where dy serves
  int64_t ld_dp;
  float* partial;  // [linear_bias_parts(rows), out_f] column sums
};
int linear_bias_parts(int32_t rows);
cudaError_t launch_linear_backward(const LinearBwdArgs& a, int act, cudaStream_t st);
unsigned int read_linear_timeouts();
unsigned int read_recurrence_timeouts();

// ------------------------------------------------------ gated delta rule ----
// Packed runs (delta.h). tab.tile[i] = the sequence's first chunk of MAMBA2_DELTA_CHUNK tokens.
struct DeltaTensors {
  void* y;
  float* ckpt;  // [chunks, heads, dv, dk] or null
  const void* q;
  const void* k;
  const void* v;
  const float* g;     // [rows, heads] or null
  const float* beta;  // [rows, heads] or null
  float* state;       // [num_slots, heads, dv, dk]
  int32_t heads, groups, dv, dk;
  int64_t ld_y, ld_q, ld_k, ld_v;
  float scale, l2_eps;
};
struct DeltaMaps;  // delta_tiles.h
struct DeltaArgs : DeltaTensors {
  SeqTable tab;
  uint16_t order[MAMBA2_MAX_SEQS];  // the runs, longest first: a chain that starts late is a short one
};
cudaError_t launch_delta_serial(const DeltaArgs& a, mamba2_dtype act, cudaStream_t st);
// Whether the chunked kernels take this shape; the records of their first pass, which are the forward's workspace.
bool delta_chunked_supported(mamba2_dtype act, int dv, int dk);
unsigned int read_delta_timeouts();
size_t delta_records(int64_t chunks, int heads, bool backward);
cudaError_t launch_delta_chunked(const DeltaArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_delta_records(const DeltaArgs& a, const DeltaMaps& maps, void* ws, cudaStream_t st);  // the backward's

struct DeltaBwdArgs : DeltaArgs {  // (y and state unused, ckpt read; tab's slots unused)
  void* dq;
  void* dk_out;
  void* dv_out;
  void* dg;
  void* dbeta;
  float* dstate;
  const void* dy;
  const float* dstate_end;
  int64_t ld_dq, ld_dk, ld_dv, ld_dy;
};
size_t delta_backward_workspace(int64_t chunks, int heads, int dv, int dk);
unsigned int read_delta_back_timeouts();
cudaError_t launch_delta_backward(const DeltaBwdArgs& a, void* ws, cudaStream_t st);

struct DeltaStepArgs : DeltaTensors {  // (ckpt unused)
  int32_t n;  // sequences, or the capacity of a device batch
  int32_t num_slots;
  const int32_t* dev_slots;  // device batch (null for a host batch), as in DecodeArgs
  const uint8_t* dev_fresh;
  const int32_t* dev_n;
  int32_t* dev_status;
  uint32_t slot_fresh[MAMBA2_MAX_SEQS];
};
// Checks a device batch too (in the kernel, or by launch_check_device_batch).
cudaError_t launch_delta_step(const DeltaStepArgs& a, mamba2_dtype act, cudaStream_t st);

// ------------------------------------------------------------ beams ----
struct BeamArgs {
  float* scores_out;
  int32_t* parents;
  int32_t* tokens;
  uint8_t* finished_out;
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  int32_t batch, beams, out, vocab, eos;
  int64_t ld;
  void* ws;
};
size_t beam_workspace(int64_t rows, int32_t out, int32_t vocab);
cudaError_t launch_beam_select(const BeamArgs& a, mamba2_dtype act, cudaStream_t st);

struct ReorderArgs {
  int32_t num_pools, num_slots, batch, beams;
  const int32_t* slots;
  const int32_t* parents;
  int32_t* status;
  char* pool[64];
  int64_t bytes[64];  // of a slot
  int32_t tile[65];   // first work tile of the pool (kReorderTile bytes of every beam's slot)
};
constexpr int kReorderTile = 4096;
cudaError_t launch_reorder(const ReorderArgs& a, cudaStream_t st);

// ------------------------------------------------------------ mamba3 ----
// Mamba-3 SISO varlen forward (head width 64, Q/K width 128). Sequence i owns
// rows [cu[i], cu[i+1]); order[] lists the sequences longest first (the CTAs
// take (sequence, head) items in that order).
struct Mamba3Args {
  void* out;
  void* final_angle;
  float* final_ssm;
  float* final_k;
  void* final_v;
  const void* q;
  const void* k;
  const void* v;
  const float* adt;
  const float* dt;
  const void* trap;
  const float* q_bias;
  const float* k_bias;
  const void* angles;
  const float* d;
  const void* z;
  int32_t nseq, heads, rot_dim;
  int32_t cu[MAMBA2_MAX_SEQS + 1];
  int32_t order[MAMBA2_MAX_SEQS];
};
cudaError_t launch_m3_forward(const Mamba3Args& a, int num_sms, cudaStream_t st);
unsigned int read_m3_timeouts();

// Failure-detection self-test: one bounded wait on a barrier nothing arrives at.
cudaError_t launch_bounded_wait_probe(int32_t* status, cudaStream_t st);

// ------------------------------------------------------------ pack ----
constexpr int kPackThreads = 256;
// Padded [batch, seqlen, width] <-> packed [cu[batch], width]: sequence b's tokens sit
// at padded positions [first[b], first[b] + cu[b+1] - cu[b]) of row b.
struct PackArgs {
  const void* src;
  void* dst;
  int32_t batch, seqlen, width;  // width in bytes
  int32_t cu[MAMBA2_MAX_SEQS + 1];
  int32_t first[MAMBA2_MAX_SEQS];
};
cudaError_t launch_pack_rows(const PackArgs& a, bool unpack, cudaStream_t st);
// The widest copy unit (16, 4, 2 or 1 bytes) dividing both addresses and the width.
int pack_unit_bytes(const void* dst, const void* src, int width);
cudaError_t launch_decode(const DecodeArgs& a, mamba2_dtype act, cudaStream_t st);
// Checks a device batch (count in [0, capacity], slots in range, no slot twice) and
// writes its mamba2_status to *status.
cudaError_t launch_check_device_batch(const int32_t* slots, const int32_t* n, int32_t capacity, int32_t num_slots,
                                      int32_t* status, cudaStream_t st);

}  // namespace mamba2
