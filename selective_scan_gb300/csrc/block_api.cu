// C entry points of block.h: host-side validation of every argument, then kernel
// launches on the caller's stream. All checks run before the first launch, so a
// refused call leaves every buffer untouched.
#include <algorithm>
#include <cstring>

#include "../../include/block.h"
#include "host.h"
#include "kernels.h"

namespace mamba2 {
namespace {

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// A matrix with a row stride: element-aligned, rows at least `width` apart.
bool strided_ok(const void* p, int64_t ld, int64_t width, size_t elem) {
  return p && aligned_to(p, elem) && ld >= width;
}

// Rows and columns that the kernels can round up to tiles in 32 bits.
bool rows_ok(int32_t n) { return n >= 0 && n <= MAMBA2_MAX_BLOCK_SIZE; }
bool width_ok(int32_t n) { return n > 0 && n <= MAMBA2_MAX_BLOCK_SIZE; }

// cu_seqlens from 0, non-decreasing.
bool cu_ok(const int32_t* cu, int32_t n) {
  if (n < 0 || n > MAMBA2_MAX_SEQS || (n > 0 && !cu)) return false;
  if (n == 0) return true;
  if (cu[0] != 0) return false;
  for (int i = 0; i < n; ++i)
    if (cu[i + 1] < cu[i]) return false;
  return true;
}

int64_t chunks_of(int64_t len) { return (len + MAMBA2_RECURRENCE_CHUNK - 1) / MAMBA2_RECURRENCE_CHUNK; }

int64_t count_chunks(const int32_t* cu, int32_t n, bool* chained) {
  int64_t total = 0;
  *chained = false;
  for (int i = 0; i < n; ++i) {
    const int64_t c = chunks_of((int64_t)cu[i + 1] - cu[i]);
    *chained |= c > 1;
    total += c;
  }
  return total;
}

void fill_chunks(SeqTable& t) {
  t.tile[0] = 0;
  for (int i = 0; i < t.n; ++i) t.tile[i + 1] = t.tile[i] + (int32_t)chunks_of((int64_t)t.cu[i + 1] - t.cu[i]);
}

mamba2_status done(cudaError_t e) { return e == cudaSuccess ? MAMBA2_OK : cuda_fail(e); }

}  // namespace
}  // namespace mamba2

using namespace mamba2;

extern "C" {

int64_t mamba2_gated_recurrence_checkpoints(const int32_t* cu_seqlens, int32_t num_seqs) {
  if (!cu_ok(cu_seqlens, num_seqs)) return -1;
  bool chained;
  return count_chunks(cu_seqlens, num_seqs, &chained) * (MAMBA2_RECURRENCE_CHUNK / MAMBA2_RECURRENCE_STEP);
}

size_t mamba2_gated_recurrence_workspace_bytes(const int32_t* cu_seqlens, int32_t num_seqs, int32_t dim,
                                               int32_t backward) {
  if (!width_ok(dim) || !cu_ok(cu_seqlens, num_seqs)) return 0;
  bool chained;
  const int64_t chunks = count_chunks(cu_seqlens, num_seqs, &chained);
  return recurrence_workspace(chunks, chained, num_seqs, dim, backward != 0);
}

mamba2_status mamba2_gated_recurrence(void* y, float* checkpoints, const void* x, const void* gate,
                                      const float* lower, float* state, int32_t num_slots, int32_t rows,
                                      int32_t dim, int64_t ld_y, int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                      const mamba2_recurrent_batch* rb, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (!act_ok(act) || !rows_ok(rows) || !width_ok(dim) || !rb) return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t e = act_size(act);
  if (rows > 0 && (!strided_ok(y, ld_y, dim, e) || !strided_ok(x, ld_x, dim, e) ||
                   !strided_ok(gate, ld_gate, dim, e) || y == x || y == gate))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (!aligned16(lower) || !aligned16(checkpoints)) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (rb->num_seqs > 0 && (!state || !aligned16(state))) return MAMBA2_ERR_INVALID_ARGUMENT;
  const mamba2_status s = validate_batch(rb, num_slots, rows, true);
  if (s != MAMBA2_OK) return s;
  if (rb->num_seqs == 0) return MAMBA2_OK;
  bool chained;
  const int64_t chunks = count_chunks(rb->cu_seqlens, rb->num_seqs, &chained);
  const size_t need = recurrence_workspace(chunks, chained, rb->num_seqs, dim, false);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  RecArgs a;
  a.y = y;
  a.ckpt = checkpoints;
  a.x = x;
  a.gate = gate;
  a.lower = lower;
  a.state = state;
  a.dim = dim;
  a.ld_y = ld_y;
  a.ld_x = ld_x;
  a.ld_gate = ld_gate;
  fill_table(a.tab, rb);
  fill_chunks(a.tab);
  return done(launch_recurrence(a, act, workspace, static_cast<cudaStream_t>(stream)));
}

namespace {
mamba2_status check_step(const void* y, const void* x, const void* gate, const float* lower, const float* state,
                         int32_t n, int32_t dim, int64_t ld_y, int64_t ld_x, int64_t ld_gate, mamba2_dtype act) {
  if (!act_ok(act) || !width_ok(dim)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t e = act_size(act);
  if (n > 0 && (!strided_ok(y, ld_y, dim, e) || !strided_ok(x, ld_x, dim, e) ||
                !strided_ok(gate, ld_gate, dim, e) || y == x || y == gate || !state || !aligned16(state)))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  return aligned16(lower) ? MAMBA2_OK : MAMBA2_ERR_INVALID_ARGUMENT;
}
}  // namespace

mamba2_status mamba2_gated_recurrence_step(void* y, const void* x, const void* gate, const float* lower,
                                           float* state, int32_t num_slots, int32_t dim, int64_t ld_y, int64_t ld_x,
                                           int64_t ld_gate, mamba2_dtype act, const mamba2_recurrent_batch* rb,
                                           void* stream) {
  if (!rb) return MAMBA2_ERR_INVALID_ARGUMENT;
  const int32_t n = rb->num_seqs;
  mamba2_status s = check_step(y, x, gate, lower, state, n, dim, ld_y, ld_x, ld_gate, act);
  if (s != MAMBA2_OK) return s;
  s = validate_batch(rb, num_slots, n, false);
  if (s != MAMBA2_OK) return s;
  if (rb->cu_seqlens)
    for (int i = 0; i <= n; ++i)
      if (rb->cu_seqlens[i] != i) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (n == 0) return MAMBA2_OK;
  RecStepArgs a = {y, x, gate, lower, state, dim, n, ld_y, ld_x, ld_gate, num_slots, nullptr, nullptr, nullptr, nullptr, {}};
  for (int i = 0; i < n; ++i) a.slot_fresh[i] = (uint32_t)rb->slots[i] | (rb->fresh[i] ? 0x80000000u : 0u);
  return done(launch_recurrence_step(a, act, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_gated_recurrence_step_device(void* y, const void* x, const void* gate, const float* lower,
                                                  float* state, int32_t num_slots, int32_t dim, int64_t ld_y,
                                                  int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                                  const int32_t* slots_dev, const uint8_t* fresh_dev,
                                                  const int32_t* num_seqs_dev, int32_t capacity, int32_t* status_dev,
                                                  void* stream) {
  if (capacity < 1 || capacity > MAMBA2_MAX_SEQS || num_slots < 0 || !slots_dev || !num_seqs_dev || !status_dev ||
      !aligned_to(slots_dev, 4) || !aligned_to(num_seqs_dev, 4) || !aligned_to(status_dev, 4))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const mamba2_status s = check_step(y, x, gate, lower, state, capacity, dim, ld_y, ld_x, ld_gate, act);
  if (s != MAMBA2_OK) return s;
  const RecStepArgs a = {y, x, gate, lower, state, dim, capacity, ld_y, ld_x, ld_gate, num_slots, slots_dev, fresh_dev,
                         num_seqs_dev, status_dev, {}};
  return done(launch_recurrence_step(a, act, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_gated_recurrence_backward(void* dx, void* dgate, float* dlower, float* dstate, const void* dy,
                                               const float* dstate_end, const void* x, const void* gate,
                                               const float* lower, const float* checkpoints, int32_t rows,
                                               int32_t dim, int64_t ld_dx, int64_t ld_dgate, int64_t ld_dy,
                                               int64_t ld_x, int64_t ld_gate, mamba2_dtype act,
                                               const int32_t* cu_seqlens, int32_t num_seqs, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || !rows_ok(rows) || !width_ok(dim) || num_seqs < 0 || num_seqs > MAMBA2_MAX_SEQS ||
      (num_seqs > 0 && !cu_seqlens) || (dlower && !lower))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t e = act_size(act);
  if (rows > 0) {
    const void* out[] = {dx, dgate};
    const void* in[] = {dy, x, gate};
    if (!strided_ok(dx, ld_dx, dim, e) || !strided_ok(dgate, ld_dgate, dim, e) || !strided_ok(dy, ld_dy, dim, e) ||
        !strided_ok(x, ld_x, dim, e) || !strided_ok(gate, ld_gate, dim, e) || !checkpoints || dx == dgate)
      return MAMBA2_ERR_INVALID_ARGUMENT;
    for (const void* o : out)
      for (const void* i : in)
        if (o == i) return MAMBA2_ERR_INVALID_ARGUMENT;
  }
  const void* plain[] = {dlower, dstate, dstate_end, lower, checkpoints};
  for (const void* p : plain)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0) {
    if (rows != 0) return MAMBA2_ERR_RUNS_DONT_COVER_ROWS;
  } else if (!cu_ok(cu_seqlens, num_seqs) || cu_seqlens[num_seqs] != rows) {
    return MAMBA2_ERR_RUNS_DONT_COVER_ROWS;
  }
  bool chained;
  const int64_t chunks = count_chunks(cu_seqlens, num_seqs, &chained);
  const size_t need = recurrence_workspace(chunks, chained, num_seqs, dim, true);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  RecBwdArgs a;
  a.dx = dx;
  a.dgate = dgate;
  a.dlower = dlower;
  a.dstate = dstate;
  a.dy = dy;
  a.dstate_end = dstate_end;
  a.x = x;
  a.gate = gate;
  a.lower = lower;
  a.ckpt = checkpoints;
  a.dim = dim;
  a.ld_dx = ld_dx;
  a.ld_dgate = ld_dgate;
  a.ld_dy = ld_dy;
  a.ld_x = ld_x;
  a.ld_gate = ld_gate;
  a.tab.n = num_seqs;
  for (int i = 0; i <= num_seqs; ++i) a.tab.cu[i] = num_seqs > 0 ? cu_seqlens[i] : 0;
  fill_chunks(a.tab);
  return done(launch_recurrence_backward(a, act, workspace, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_add_rmsnorm(void* out, float* scale, void* sum, const void* x, const void* residual,
                                 const float* weight, int32_t rows, int32_t dim, float eps, mamba2_dtype act,
                                 mamba2_dtype sum_type, mamba2_dtype out_type, void* stream) {
  if (!act_ok(act) || (sum_type != act && sum_type != MAMBA2_F32) || (out_type != act && out_type != MAMBA2_E4M3) ||
      !rows_ok(rows) || !width_ok(dim) || !(eps >= 0.0f) || (out_type == MAMBA2_E4M3 ? (rows > 0 && !scale) : scale != nullptr))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MAMBA2_OK;
  if (!out || !x || !weight || out == x || (residual && out == residual) || (sum && (sum == out || sum == x)))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {out, scale, sum, x, residual, weight};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const AddNormArgs a{out, scale, sum, x, residual, weight, rows, dim, eps};
  return done(launch_add_rmsnorm(a, act, sum_type, out_type, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_add_rmsnorm_backward_workspace_bytes(int32_t rows, int32_t dim) {
  if (rows == 0 || !rows_ok(rows) || !width_ok(dim)) return 0;
  return align256((size_t)add_rmsnorm_backward_parts(rows, dim) * dim * 4);
}

mamba2_status mamba2_add_rmsnorm_backward(void* dx, void* dresidual, float* dweight, const void* dy,
                                          const void* dsum, const void* sum, const float* weight, int32_t rows,
                                          int32_t dim, float eps, mamba2_dtype act, mamba2_dtype sum_type,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || (sum_type != act && sum_type != MAMBA2_F32) || !rows_ok(rows) || !width_ok(dim) ||
      !(eps >= 0.0f))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (!weight || (rows > 0 && (!dy || !sum))) return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* in[] = {dy, sum, dsum};
  for (const void* p : in)
    if (p && (p == dx || (p == dresidual && p != dsum))) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (dx && dx == dresidual) return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {dx, dresidual, dweight, dy, dsum, sum, weight};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t need = dweight ? mamba2_add_rmsnorm_backward_workspace_bytes(rows, dim) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const AddNormBwdArgs a{dx, dresidual, dweight, dy, dsum, sum, weight, static_cast<float*>(workspace), rows, dim, eps};
  return done(launch_add_rmsnorm_backward(a, act, sum_type, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_linear(void* out, void* pre, const void* x, const float* x_scale, const void* w,
                            const float* w_scale, const float* bias, const void* residual, int32_t rows,
                            int32_t in_features, int32_t out_features, int64_t ld_out, int64_t ld_x,
                            int64_t ld_residual, mamba2_dtype in_type, mamba2_dtype out_type,
                            mamba2_activation activation, void* stream) {
  const bool fp8 = in_type == MAMBA2_E4M3;
  if ((!fp8 && !act_ok(in_type)) || !act_ok(out_type) || (int)activation < 0 || activation > MAMBA2_ACT_GELU ||
      !rows_ok(rows) || !width_ok(in_features) || !width_ok(out_features))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const int unit = fp8 ? 16 : 8;  // elements of 16 bytes
  if (in_type == MAMBA2_F32 || in_features % unit != 0 || ld_x % unit != 0) return MAMBA2_ERR_NOT_IMPLEMENTED;
  if (fp8 ? (!w_scale || (rows > 0 && !x_scale)) : (x_scale || w_scale)) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MAMBA2_OK;
  const size_t oe = act_size(out_type);
  if (!strided_ok(out, ld_out, out_features, oe) ||
      (residual && !strided_ok(residual, ld_residual, out_features, oe)) ||
      !x || !w || ld_x < in_features)
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (out == x || out == w || (pre && (pre == out || pre == x || pre == w || pre == residual)) ||
      (residual == out && ld_residual != ld_out))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {pre, x, x_scale, w, w_scale, bias};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const LinearArgs a{out,  pre,         x,            w_scale ? x_scale : nullptr, w,    w_scale,    bias, residual,
                     rows, in_features, out_features, ld_out,                      ld_x, ld_residual};
  return done(launch_linear(a, in_type, out_type, (int)activation, static_cast<cudaStream_t>(stream)));
}

namespace {
// Rows of dp are padded to whole blocks of 64 columns.
int64_t ld_dp(int32_t out_features) { return ((int64_t)out_features + 63) / 64 * 64; }
size_t dp_bytes(int32_t rows, int32_t out_features) { return align256((size_t)rows * ld_dp(out_features) * 2); }
}  // namespace

size_t mamba2_linear_backward_workspace_bytes(int32_t rows, int32_t in_features, int32_t out_features) {
  if (rows == 0 || !rows_ok(rows) || !width_ok(in_features) || !width_ok(out_features)) return 0;
  return dp_bytes(rows, out_features) + align256((size_t)linear_bias_parts(rows) * out_features * 4);
}

mamba2_status mamba2_linear_backward(void* dx, void* dw, float* dbias, const void* dy, const void* pre,
                                     const void* x, const void* w, int32_t rows, int32_t in_features,
                                     int32_t out_features, int64_t ld_x, mamba2_activation activation,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if ((int)activation < 0 || activation > MAMBA2_ACT_GELU || !rows_ok(rows) || !width_ok(in_features) ||
      !width_ok(out_features))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (in_features % 8 != 0 || ld_x % 8 != 0) return MAMBA2_ERR_NOT_IMPLEMENTED;
  if (rows > 0 && (!dy || (activation != MAMBA2_ACT_NONE && !pre) ||
                   (dx && !w) || (dw && (!x || ld_x < in_features))))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* in[] = {dy, pre, x, w};
  for (const void* p : in)
    if (p && (p == dx || p == dw || p == dbias)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {dx, dw, dbias, dy, pre, x, w};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t need = mamba2_linear_backward_workspace_bytes(rows, in_features, out_features);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  LinearBwdArgs a;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dy = dy;
  a.pre = pre;
  a.x = x;
  a.w = w;
  a.rows = rows;
  a.in_f = in_features;
  a.out_f = out_features;
  a.ld_x = ld_x;
  a.dp = workspace;
  a.ld_dp = ld_dp(out_features);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + dp_bytes(rows > 0 ? rows : 0, out_features));
  return done(launch_linear_backward(a, (int)activation, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
