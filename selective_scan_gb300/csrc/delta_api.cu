// C entry points of delta.h and beam.h: host-side validation of every argument, then kernel launches on the caller's
// stream. All checks run before the first launch, so a refused call leaves every buffer untouched.
#include <algorithm>
#include <cmath>

#include "../../include/beam.h"
#include "../../include/block.h"
#include "../../include/delta.h"
#include "host.h"
#include "kernels.h"

namespace mamba2 {
namespace {

mamba2_status done(cudaError_t e) { return e == cudaSuccess ? MAMBA2_OK : cuda_fail(e); }

int64_t chunks_of(int64_t len) { return (len + MAMBA2_DELTA_CHUNK - 1) / MAMBA2_DELTA_CHUNK; }

// cu_seqlens from 0, non-decreasing.
bool cu_ok(const int32_t* cu, int32_t n) {
  if (n < 0 || n > MAMBA2_MAX_SEQS || (n > 0 && !cu)) return false;
  if (n == 0) return true;
  if (cu[0] != 0) return false;
  for (int i = 0; i < n; ++i)
    if (cu[i + 1] < cu[i]) return false;
  return true;
}

int64_t count_chunks(const int32_t* cu, int32_t n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += chunks_of((int64_t)cu[i + 1] - cu[i]);
  return total;
}

void fill_chunks(DeltaArgs& a) {
  SeqTable& t = a.tab;
  t.tile[0] = 0;
  for (int i = 0; i < t.n; ++i) {
    t.tile[i + 1] = t.tile[i] + (int32_t)chunks_of((int64_t)t.cu[i + 1] - t.cu[i]);
    a.order[i] = (uint16_t)i;
  }
  std::sort(a.order, a.order + t.n, [&](int x, int y) {
    const int32_t lx = t.cu[x + 1] - t.cu[x], ly = t.cu[y + 1] - t.cu[y];
    return lx != ly ? lx > ly : x < y;
  });
}

// Sizes that make sense, then those that the kernels take. (Heads are a grid dimension.)
mamba2_status delta_dims(const mamba2_dims* d) {
  if (!d || d->heads <= 0 || d->ngroups <= 0 || d->headdim <= 0 || d->d_state <= 0 || d->heads % d->ngroups != 0 ||
      d->heads > 65535 || (int64_t)d->heads * d->headdim > MAMBA2_MAX_BLOCK_SIZE ||
      (int64_t)d->ngroups * d->d_state > MAMBA2_MAX_BLOCK_SIZE)
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (d->headdim % 8 != 0 || d->d_state % 8 != 0 || d->d_state > MAMBA2_MAX_DELTA_STATE) return MAMBA2_ERR_NOT_IMPLEMENTED;
  return MAMBA2_OK;
}

// What the three forward calls have in common; rows > 0.
mamba2_status delta_tensors(const void* y, const void* q, const void* k, const void* v, const float* g,
                            const float* beta, const float* state, int64_t ld_y, int64_t ld_q, int64_t ld_k,
                            int64_t ld_v, const mamba2_dims* d) {
  const int64_t wide = (int64_t)d->heads * d->headdim, narrow = (int64_t)d->ngroups * d->d_state;
  if (!y || !q || !k || !v || y == q || y == k || y == v || ld_y < wide || ld_v < wide || ld_q < narrow || ld_k < narrow)
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {y, q, k, v, g, beta, state};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (ld_y % 8 != 0 || ld_q % 8 != 0 || ld_k % 8 != 0 || ld_v % 8 != 0) return MAMBA2_ERR_NOT_IMPLEMENTED;
  return MAMBA2_OK;
}

void fill(DeltaTensors& a, void* y, const void* q, const void* k, const void* v, const float* g, const float* beta,
          float* state, int64_t ld_y, int64_t ld_q, int64_t ld_k, int64_t ld_v, const mamba2_dims* d, float scale,
          float l2_eps) {
  a.y = y;
  a.ckpt = nullptr;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.heads = d->heads;
  a.groups = d->ngroups;
  a.dv = d->headdim;
  a.dk = d->d_state;
  a.ld_y = ld_y;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.scale = scale;
  a.l2_eps = l2_eps;
}

}  // namespace
}  // namespace mamba2

using namespace mamba2;

extern "C" {

int64_t mamba2_gated_delta_rule_checkpoints(const int32_t* cu_seqlens, int32_t num_seqs) {
  return cu_ok(cu_seqlens, num_seqs) ? count_chunks(cu_seqlens, num_seqs) : -1;
}

size_t mamba2_gated_delta_rule_workspace_bytes(const int32_t* cu_seqlens, int32_t num_seqs, const mamba2_dims* dims,
                                               mamba2_dtype act, int32_t backward) {
  if (!act_ok(act) || delta_dims(dims) != MAMBA2_OK || !cu_ok(cu_seqlens, num_seqs) ||
      !delta_chunked_supported(act, dims->headdim, dims->d_state))
    return 0;
  const int64_t chunks = count_chunks(cu_seqlens, num_seqs);
  if (backward) return delta_backward_workspace(chunks, dims->heads, dims->headdim, dims->d_state);
  return (delta_records(chunks, dims->heads, false) + 255) / 256 * 256;
}

mamba2_status mamba2_gated_delta_rule(void* y, float* checkpoints, const void* q, const void* k, const void* v,
                                      const float* g, const float* beta, float* state, int32_t num_slots,
                                      int32_t rows, int64_t ld_y, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                      const mamba2_dims* dims, float scale, float l2_eps, mamba2_dtype act,
                                      const mamba2_recurrent_batch* rb, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (!act_ok(act) || !rb || rows < 0 || rows > MAMBA2_MAX_BLOCK_SIZE || std::isnan(scale) || std::isnan(l2_eps))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  mamba2_status s = delta_dims(dims);
  if (s != MAMBA2_OK) return s;
  if (rows > 0) s = delta_tensors(y, q, k, v, g, beta, state, ld_y, ld_q, ld_k, ld_v, dims);
  if (s != MAMBA2_OK) return s;
  if (!aligned16(checkpoints) || (rb->num_seqs > 0 && (!state || !aligned16(state)))) return MAMBA2_ERR_INVALID_ARGUMENT;
  s = validate_batch(rb, num_slots, rows, true);
  if (s != MAMBA2_OK) return s;
  if (rb->num_seqs == 0) return MAMBA2_OK;
  const size_t need = mamba2_gated_delta_rule_workspace_bytes(rb->cu_seqlens, rb->num_seqs, dims, act, 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  DeltaArgs a;
  fill(a, y, q, k, v, g, beta, state, ld_y, ld_q, ld_k, ld_v, dims, scale, l2_eps);
  a.ckpt = checkpoints;
  fill_table(a.tab, rb);
  fill_chunks(a);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(delta_chunked_supported(act, a.dv, a.dk) ? launch_delta_chunked(a, workspace, st) : launch_delta_serial(a, act, st));
}

namespace {
mamba2_status check_delta_step(const void* y, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* state, int32_t n, int64_t ld_y, int64_t ld_q,
                               int64_t ld_k, int64_t ld_v, const mamba2_dims* dims, float scale, float l2_eps,
                               mamba2_dtype act) {
  if (!act_ok(act) || std::isnan(scale) || std::isnan(l2_eps)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const mamba2_status s = delta_dims(dims);
  if (s != MAMBA2_OK || n == 0) return s;
  if (!state) return MAMBA2_ERR_INVALID_ARGUMENT;
  return delta_tensors(y, q, k, v, g, beta, state, ld_y, ld_q, ld_k, ld_v, dims);
}
}  // namespace

mamba2_status mamba2_gated_delta_rule_step(void* y, const void* q, const void* k, const void* v, const float* g,
                                           const float* beta, float* state, int32_t num_slots, int64_t ld_y,
                                           int64_t ld_q, int64_t ld_k, int64_t ld_v, const mamba2_dims* dims,
                                           float scale, float l2_eps, mamba2_dtype act,
                                           const mamba2_recurrent_batch* rb, void* stream) {
  if (!rb || rb->num_seqs < 0 || rb->num_seqs > MAMBA2_MAX_SEQS) return MAMBA2_ERR_INVALID_ARGUMENT;
  const int32_t n = rb->num_seqs;
  mamba2_status s = check_delta_step(y, q, k, v, g, beta, state, n, ld_y, ld_q, ld_k, ld_v, dims, scale, l2_eps, act);
  if (s != MAMBA2_OK) return s;
  s = validate_batch(rb, num_slots, n, false);
  if (s != MAMBA2_OK) return s;
  if (rb->cu_seqlens)
    for (int i = 0; i <= n; ++i)
      if (rb->cu_seqlens[i] != i) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (n == 0) return MAMBA2_OK;
  DeltaStepArgs a = {};
  fill(a, y, q, k, v, g, beta, state, ld_y, ld_q, ld_k, ld_v, dims, scale, l2_eps);
  a.n = n;
  a.num_slots = num_slots;
  for (int i = 0; i < n; ++i) a.slot_fresh[i] = (uint32_t)rb->slots[i] | (rb->fresh[i] ? 0x80000000u : 0u);
  return done(launch_delta_step(a, act, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_gated_delta_rule_step_device(void* y, const void* q, const void* k, const void* v,
                                                  const float* g, const float* beta, float* state,
                                                  int32_t num_slots, int64_t ld_y, int64_t ld_q, int64_t ld_k,
                                                  int64_t ld_v, const mamba2_dims* dims, float scale, float l2_eps,
                                                  mamba2_dtype act, const int32_t* slots_dev,
                                                  const uint8_t* fresh_dev, const int32_t* num_seqs_dev,
                                                  int32_t capacity, int32_t* status_dev, void* stream) {
  if (capacity < 1 || capacity > MAMBA2_MAX_SEQS || num_slots < 0 || !slots_dev || !num_seqs_dev || !status_dev ||
      !aligned_to(slots_dev, 4) || !aligned_to(num_seqs_dev, 4) || !aligned_to(status_dev, 4))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const mamba2_status s = check_delta_step(y, q, k, v, g, beta, state, capacity, ld_y, ld_q, ld_k, ld_v, dims, scale,
                                           l2_eps, act);
  if (s != MAMBA2_OK) return s;
  DeltaStepArgs a = {};
  fill(a, y, q, k, v, g, beta, state, ld_y, ld_q, ld_k, ld_v, dims, scale, l2_eps);
  a.n = capacity;
  a.num_slots = num_slots;
  a.dev_slots = slots_dev;
  a.dev_fresh = fresh_dev;
  a.dev_n = num_seqs_dev;
  a.dev_status = status_dev;
  return done(launch_delta_step(a, act, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_gated_delta_rule_backward(void* dq, void* dk, void* dv, void* dg, void* dbeta, float* dstate,
                                               const void* dy, const float* dstate_end, const void* q, const void* k,
                                               const void* v, const float* g, const float* beta,
                                               const float* checkpoints, int32_t rows, int64_t ld_dq, int64_t ld_dk,
                                               int64_t ld_dv, int64_t ld_dy, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                               const mamba2_dims* dims, float scale, float l2_eps, mamba2_dtype act,
                                               const int32_t* cu_seqlens, int32_t num_seqs, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || rows < 0 || rows > MAMBA2_MAX_BLOCK_SIZE || num_seqs < 0 || num_seqs > MAMBA2_MAX_SEQS ||
      (num_seqs > 0 && !cu_seqlens) || std::isnan(scale) || std::isnan(l2_eps))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  mamba2_status s = delta_dims(dims);
  if (s != MAMBA2_OK) return s;
  if (!delta_chunked_supported(act, dims->headdim, dims->d_state)) return MAMBA2_ERR_NOT_IMPLEMENTED;
  const void* plain[] = {dg, dbeta, dstate, dstate_end, checkpoints};
  for (const void* p : plain)
    if (!aligned16(p)) return MAMBA2_ERR_INVALID_ARGUMENT;
  if (rows > 0) {
    // (dv stands where the forward has y; dq, dk and dy are held to the same; v may be dy)
    s = delta_tensors(dv, q, k, v, g, beta, nullptr, ld_dv, ld_q, ld_k, ld_v, dims);
    if (s == MAMBA2_OK) s = delta_tensors(dy, dq, dk, dv, nullptr, nullptr, nullptr, ld_dy, ld_dq, ld_dk, ld_dv, dims);
    if (s != MAMBA2_OK) return s;
    if (!checkpoints) return MAMBA2_ERR_INVALID_ARGUMENT;
    const void* out[] = {dq, dk, dv, dg, dbeta};
    const void* in[] = {dy, q, k, v, g, beta, checkpoints, dstate_end};
    for (int i = 0; i < 5; ++i) {
      if (!out[i]) continue;
      for (const void* p : in)
        if (p == out[i]) return MAMBA2_ERR_INVALID_ARGUMENT;
      for (int j = 0; j < i; ++j)
        if (out[j] == out[i]) return MAMBA2_ERR_INVALID_ARGUMENT;
    }
  }
  if (num_seqs == 0) {
    if (rows != 0) return MAMBA2_ERR_RUNS_DONT_COVER_ROWS;
    return MAMBA2_OK;
  }
  if (!cu_ok(cu_seqlens, num_seqs) || cu_seqlens[num_seqs] != rows) return MAMBA2_ERR_RUNS_DONT_COVER_ROWS;
  if (dstate && dstate == dstate_end) return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t need = mamba2_gated_delta_rule_workspace_bytes(cu_seqlens, num_seqs, dims, act, 1);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  DeltaBwdArgs a;
  fill(a, nullptr, q, k, v, g, beta, nullptr, 0, ld_q, ld_k, ld_v, dims, scale, l2_eps);
  a.ckpt = const_cast<float*>(checkpoints);
  a.dq = dq;
  a.dk_out = dk;
  a.dv_out = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dstate = dstate;
  a.dy = dy;
  a.dstate_end = dstate_end;
  a.ld_dq = ld_dq;
  a.ld_dk = ld_dk;
  a.ld_dv = ld_dv;
  a.ld_dy = ld_dy;
  a.tab.n = num_seqs;
  for (int i = 0; i <= num_seqs; ++i) a.tab.cu[i] = cu_seqlens[i];
  fill_chunks(a);
  return done(launch_delta_backward(a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t out, int32_t vocab) {
  if (batch <= 0 || beams < 1 || beams > MAMBA2_MAX_BEAMS || out < 1 || out > MAMBA2_MAX_BEAMS || vocab < 1 ||
      vocab > MAMBA2_MAX_BLOCK_SIZE || (int64_t)batch * beams > 65535)
    return 0;
  return (beam_workspace((int64_t)batch * beams, out, vocab) + 255) / 256 * 256;
}

mamba2_status mamba2_beam_select(float* scores_out, int32_t* parents, int32_t* tokens, uint8_t* finished_out,
                                 const void* logits, const float* scores, const uint8_t* finished, int32_t batch,
                                 int32_t beams, int32_t out, int32_t vocab, int64_t ld, int32_t eos,
                                 mamba2_dtype act, void* workspace, size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || batch < 0 || beams < 1 || beams > MAMBA2_MAX_BEAMS || out < 1 || out > MAMBA2_MAX_BEAMS ||
      vocab < 1 || vocab > MAMBA2_MAX_BLOCK_SIZE || (int64_t)batch * beams > 65535 || out > (int64_t)beams * vocab ||
      eos < -1 || eos >= vocab || (eos < 0 && (finished || finished_out)) || ld < vocab)
    return MAMBA2_ERR_INVALID_ARGUMENT;
  if (batch == 0) return MAMBA2_OK;
  if (!scores_out || !parents || !tokens || !logits || !scores || scores_out == scores ||
      (finished_out && finished_out == finished) || !aligned_to(logits, act_size(act)) || !aligned_to(scores_out, 4) ||
      !aligned_to(parents, 4) || !aligned_to(tokens, 4) || !aligned_to(scores, 4))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  const size_t need = mamba2_beam_select_workspace_bytes(batch, beams, out, vocab);
  if (!workspace || workspace_bytes < need) return MAMBA2_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_to(workspace, 256)) return MAMBA2_ERR_INVALID_ARGUMENT;
  const BeamArgs a = {scores_out, parents, tokens, finished_out, logits, scores, finished, batch,
                      beams,      out,     vocab,  eos,          ld,     workspace};
  return done(launch_beam_select(a, act, static_cast<cudaStream_t>(stream)));
}

mamba2_status mamba2_reorder_states(void* const* pools, const int64_t* slot_bytes, int32_t num_pools,
                                    int32_t num_slots, const int32_t* slots, const int32_t* parents, int32_t batch,
                                    int32_t beams, int32_t* status_dev, void* stream) {
  if (num_pools < 0 || num_pools > MAMBA2_MAX_POOLS || (num_pools > 0 && (!pools || !slot_bytes)) || num_slots < 0 ||
      batch < 0 || beams < 1 || beams > MAMBA2_MAX_BEAMS || (int64_t)batch * beams > MAMBA2_MAX_SEQS || !status_dev ||
      !aligned_to(status_dev, 4) || (batch > 0 && (!slots || !parents)) || !aligned_to(slots, 4) || !aligned_to(parents, 4))
    return MAMBA2_ERR_INVALID_ARGUMENT;
  ReorderArgs a = {};
  int64_t tiles = 0;
  for (int i = 0; i < num_pools; ++i) {
    if (slot_bytes[i] < 0 || (slot_bytes[i] > 0 && num_slots > 0 && !pools[i])) return MAMBA2_ERR_INVALID_ARGUMENT;
    a.pool[i] = static_cast<char*>(pools[i]);
    a.bytes[i] = slot_bytes[i];
    a.tile[i] = (int32_t)tiles;
    tiles += (slot_bytes[i] + kReorderTile - 1) / kReorderTile;
    if (tiles > MAMBA2_MAX_BLOCK_SIZE) return MAMBA2_ERR_INVALID_ARGUMENT;
    if (slot_bytes[i] == 0 || num_slots == 0) continue;
    if (num_slots > (int64_t(1) << 48) / slot_bytes[i]) return MAMBA2_ERR_INVALID_ARGUMENT;  // (no memory is as large)
    const uintptr_t p = reinterpret_cast<uintptr_t>(pools[i]), end = p + (uint64_t)slot_bytes[i] * num_slots;
    for (int j = 0; j < i; ++j) {  // what overlaps would be moved twice
      const uintptr_t q = reinterpret_cast<uintptr_t>(pools[j]);
      if (slot_bytes[j] > 0 && p < q + (uint64_t)slot_bytes[j] * num_slots && q < end) return MAMBA2_ERR_INVALID_ARGUMENT;
    }
  }
  for (int i = num_pools; i <= MAMBA2_MAX_POOLS; ++i) a.tile[i] = (int32_t)tiles;
  if (batch == 0) return done(cudaMemsetAsync(status_dev, 0, 4, static_cast<cudaStream_t>(stream)));
  a.num_pools = num_pools;
  a.num_slots = num_slots;
  a.batch = batch;
  a.beams = beams;
  a.slots = slots;
  a.parents = parents;
  a.status = status_dev;
  return done(launch_reorder(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
