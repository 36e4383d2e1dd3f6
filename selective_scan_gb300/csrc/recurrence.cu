// Gated recurrence (block.h): h_t = f_t h_{t-1} + k_t x_t per channel, with
// f = lo + (1 - lo) sigmoid(gate) and k = 1 - f, over packed runs; its backward pass
// and its single-token step.
//
// One thread per (run, channel), token after token.
#include "../../include/block.h"
#include "common.cuh"

namespace mamba2 {
namespace {

constexpr int kThreads = 128;
constexpr int kChunkR = MAMBA2_RECURRENCE_CHUNK;

// sigmoid(g) and sigmoid(-g), each with its own digits: with e = exp(-|g|) they are
// 1 / (1 + e) and e / (1 + e), in the order that g's sign gives.
__device__ __forceinline__ void sigmoids(float g, float& up, float& down) {
  const float e = __expf(-fabsf(g));
  const float r = __fdividef(1.0f, 1.0f + e);
  const float small = e * r;
  up = g >= 0.0f ? r : small;
  down = g >= 0.0f ? small : r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rec_fwd_kernel(const __grid_constant__ RecArgs a) {
  const int ch = blockIdx.x * kThreads + threadIdx.x, i = blockIdx.y;
  if (ch >= a.dim) return;
  const float lo = a.lower ? a.lower[ch] : 0.0f;
  float* st = a.state + (int64_t)seq_slot(a.tab, i) * a.dim + ch;
  float h = seq_fresh(a.tab, i) ? 0.0f : *st;
  const int t0 = a.tab.cu[i], t1 = a.tab.cu[i + 1];
  for (int t = t0; t < t1; ++t) {
    if (a.ckpt && (t - t0) % kChunkR == 0) a.ckpt[(int64_t)(a.tab.tile[i] + (t - t0) / kChunkR) * a.dim + ch] = h;
    const float x = Act<T>::to_f(static_cast<const T*>(a.x)[t * a.ld_x + ch]);
    float up, down;
    sigmoids(Act<T>::to_f(static_cast<const T*>(a.gate)[t * a.ld_gate + ch]), up, down);
    h = fmaf(fmaf(1.0f - lo, up, lo), h, (1.0f - lo) * down * x);
    static_cast<T*>(a.y)[t * a.ld_y + ch] = Act<T>::from_f(h);
  }
  *st = h;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rec_bwd_kernel(const __grid_constant__ RecBwdArgs a, float* part) {
  const int ch = blockIdx.x * kThreads + threadIdx.x, i = blockIdx.y;
  if (ch >= a.dim) return;
  const float lo = a.lower ? a.lower[ch] : 0.0f;
  const int t0 = a.tab.cu[i], t1 = a.tab.cu[i + 1];
  float G = a.dstate_end ? a.dstate_end[(int64_t)i * a.dim + ch] : 0.0f;
  for (int c = a.tab.tile[i + 1] - a.tab.tile[i] - 1; c >= 0; --c) {
    const int c0 = t0 + c * kChunkR, c1 = min(c0 + kChunkR, t1);
    const float start = a.ckpt[(int64_t)(a.tab.tile[i] + c) * a.dim + ch];
    float dlo = 0.0f;
    float hs[kChunkR];
    float h = start;
    for (int t = c0; t < c1; ++t) {
      hs[t - c0] = h;
      const float x = Act<T>::to_f(static_cast<const T*>(a.x)[t * a.ld_x + ch]);
      float up, down;
      sigmoids(Act<T>::to_f(static_cast<const T*>(a.gate)[t * a.ld_gate + ch]), up, down);
      h = fmaf(fmaf(1.0f - lo, up, lo), h, (1.0f - lo) * down * x);
    }
    for (int t = c1 - 1; t >= c0; --t) {
      const float x = Act<T>::to_f(static_cast<const T*>(a.x)[t * a.ld_x + ch]);
      float up, down;
      sigmoids(Act<T>::to_f(static_cast<const T*>(a.gate)[t * a.ld_gate + ch]), up, down);
      const float g = G + Act<T>::to_f(static_cast<const T*>(a.dy)[t * a.ld_dy + ch]);
      const float df = g * (hs[t - c0] - x);
      static_cast<T*>(a.dx)[t * a.ld_dx + ch] = Act<T>::from_f((1.0f - lo) * down * g);
      static_cast<T*>(a.dgate)[t * a.ld_dgate + ch] = Act<T>::from_f(df * (1.0f - lo) * up * down);
      dlo = fmaf(df, down, dlo);
      G = fmaf(1.0f - lo, up, lo) * g;
    }
    if (part) part[(int64_t)(a.tab.tile[i] + c) * a.dim + ch] = dlo;
  }
  if (a.dstate) a.dstate[(int64_t)i * a.dim + ch] = G;
}

// dlower[ch] = sum over the chunks' parts, in order.
__global__ void __launch_bounds__(kThreads) rec_dlower_kernel(float* dlower, const float* part, int chunks, int dim) {
  const int ch = blockIdx.x * kThreads + threadIdx.x;
  if (ch >= dim) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += part[(int64_t)c * dim + ch];
  dlower[ch] = s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rec_step_kernel(const __grid_constant__ RecStepArgs a) {
  const int ch = blockIdx.x * kThreads + threadIdx.x, i = blockIdx.y;
  if (ch >= a.dim) return;
  int slot;
  bool fresh;
  if (a.dev_slots) {
    if (*a.dev_status != MAMBA2_OK || i >= *a.dev_n) return;
    slot = a.dev_slots[i];
    fresh = a.dev_fresh && a.dev_fresh[i];
  } else {
    slot = (int)(a.slot_fresh[i] & 0x7fffffffu);
    fresh = (a.slot_fresh[i] >> 31) != 0u;
  }
  const float lo = a.lower ? a.lower[ch] : 0.0f;
  float* st = a.state + (int64_t)slot * a.dim + ch;
  float h = fresh ? 0.0f : *st;
  float up, down;
  sigmoids(Act<T>::to_f(static_cast<const T*>(a.gate)[i * a.ld_gate + ch]), up, down);
  h = fmaf(fmaf(1.0f - lo, up, lo), h, (1.0f - lo) * down * Act<T>::to_f(static_cast<const T*>(a.x)[i * a.ld_x + ch]));
  static_cast<T*>(a.y)[i * a.ld_y + ch] = Act<T>::from_f(h);
  *st = h;
}

}  // namespace

size_t recurrence_workspace(int64_t chunks, bool, int32_t dim, bool backward) {
  return backward ? ((size_t)chunks * dim * 4 + 255) / 256 * 256 : 0;
}

cudaError_t launch_recurrence(const RecArgs& a, mamba2_dtype act, void*, cudaStream_t st) {
  const dim3 grid((a.dim + kThreads - 1) / kThreads, a.tab.n);
  if (act == MAMBA2_BF16) rec_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
  else rec_fwd_kernel<float><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_recurrence_backward(const RecBwdArgs& a, mamba2_dtype act, void* ws, cudaStream_t st) {
  float* part = a.dlower ? static_cast<float*>(ws) : nullptr;
  if (a.tab.n > 0) {
    const dim3 grid((a.dim + kThreads - 1) / kThreads, a.tab.n);
    if (act == MAMBA2_BF16) rec_bwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, part);
    else rec_bwd_kernel<float><<<grid, kThreads, 0, st>>>(a, part);
  }
  if (a.dlower)
    rec_dlower_kernel<<<(a.dim + kThreads - 1) / kThreads, kThreads, 0, st>>>(a.dlower, part, a.tab.tile[a.tab.n], a.dim);
  return cudaGetLastError();
}

cudaError_t launch_recurrence_step(const RecStepArgs& a, mamba2_dtype act, cudaStream_t st) {
  const dim3 grid((a.dim + kThreads - 1) / kThreads, a.n);
  if (act == MAMBA2_BF16) rec_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
  else rec_step_kernel<float><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mamba2
