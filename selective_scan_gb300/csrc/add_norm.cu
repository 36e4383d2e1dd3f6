// RMS norm with the residual's addition (block.h), its 8-bit output, and its backward pass.
//
// One CTA per row; the row is read twice (the second time from L2).
#include <cuda_fp8.h>

#include "common.cuh"

namespace mamba2 {
namespace {

constexpr int kThreads = 256;
constexpr float kMax8 = 448.0f;  // largest e4m3 value

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}
__device__ __forceinline__ float block_max(float v) {
  __shared__ float part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) s = max_nan(s, part[i]);
  return s;
}

template <typename T, typename S, bool F8>
__global__ void __launch_bounds__(kThreads) add_norm_kernel(const AddNormArgs a) {
  const int64_t base = (int64_t)blockIdx.x * a.dim;
  const T* x = static_cast<const T*>(a.x) + base;
  const S* r = a.residual ? static_cast<const S*>(a.residual) + base : nullptr;
  extern __shared__ float srow[];  // the row's s when it fits
  float ss = 0.0f;
  auto value = [&](int i) { return Act<T>::to_f(x[i]) + (r ? Act<S>::to_f(r[i]) : 0.0f); };
  for (int i = threadIdx.x; i < a.dim; i += kThreads) ss = fmaf(value(i), value(i), ss);
  const float inv = rsqrtf(block_sum(ss) / (float)a.dim + a.eps);
  float top = 0.0f;
  if (F8)
    for (int i = threadIdx.x; i < a.dim; i += kThreads) top = max_nan(top, fabsf(value(i) * inv * a.weight[i]));
  float scale = 1.0f;
  if (F8) {
    top = block_max(top);
    if (!(top == 0.0f)) scale = top / kMax8;
    if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
  }
  for (int i = threadIdx.x; i < a.dim; i += kThreads) {
    const float s = value(i), y = s * inv * a.weight[i];
    if (F8) static_cast<__nv_fp8_e4m3*>(a.out)[base + i] = __nv_fp8_e4m3(y / scale);
    else static_cast<T*>(a.out)[base + i] = Act<T>::from_f(y);
    if (a.sum) static_cast<S*>(a.sum)[base + i] = Act<S>::from_f(s);
  }
}

template <typename T, typename S>
__global__ void __launch_bounds__(kThreads) add_norm_bwd_kernel(const AddNormBwdArgs a, int parts) {
  for (int64_t row = blockIdx.x; row < a.rows; row += parts) {
    const int64_t base = row * a.dim;
    const T* dy = static_cast<const T*>(a.dy) + base;
    const S* s = static_cast<const S*>(a.sum) + base;
    float ss = 0.0f, sd = 0.0f;
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
      const float v = Act<S>::to_f(s[i]);
      ss = fmaf(v, v, ss);
      sd = fmaf(v, a.weight[i] * Act<T>::to_f(dy[i]), sd);
    }
    const float inv = rsqrtf(block_sum(ss) / (float)a.dim + a.eps);
    const float c = inv * inv * (block_sum(sd) / (float)a.dim);
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
      const float v = Act<S>::to_f(s[i]), g = Act<T>::to_f(dy[i]);
      float d = inv * (a.weight[i] * g - v * c);
      if (a.dsum) d += Act<S>::to_f(static_cast<const S*>(a.dsum)[base + i]);
      if (a.dx) static_cast<T*>(a.dx)[base + i] = Act<T>::from_f(d);
      if (a.dresidual) static_cast<S*>(a.dresidual)[base + i] = Act<S>::from_f(d);
      if (a.dweight) {
        float* p = a.partial + (int64_t)blockIdx.x * a.dim + i;  // this thread's own column in every row
        *p = (row == blockIdx.x ? 0.0f : *p) + g * v * inv;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) column_sum_kernel(float* dst, const float* part, int parts, int dim) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= dim) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += part[(int64_t)p * dim + i];
  dst[i] = s;
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, mamba2_dtype act, mamba2_dtype sum_type, mamba2_dtype out_type,
                               cudaStream_t st) {
  using B = __nv_bfloat16;
  const bool f8 = out_type == MAMBA2_E4M3;
  if (act == MAMBA2_F32) {
    if (f8) add_norm_kernel<float, float, true><<<a.rows, kThreads, 0, st>>>(a);
    else add_norm_kernel<float, float, false><<<a.rows, kThreads, 0, st>>>(a);
  } else if (sum_type == MAMBA2_F32) {
    if (f8) add_norm_kernel<B, float, true><<<a.rows, kThreads, 0, st>>>(a);
    else add_norm_kernel<B, float, false><<<a.rows, kThreads, 0, st>>>(a);
  } else {
    if (f8) add_norm_kernel<B, B, true><<<a.rows, kThreads, 0, st>>>(a);
    else add_norm_kernel<B, B, false><<<a.rows, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

int add_rmsnorm_backward_parts(int32_t rows, int32_t) { return rows < 304 ? rows : 304; }

cudaError_t launch_add_rmsnorm_backward(const AddNormBwdArgs& a, mamba2_dtype act, mamba2_dtype sum_type,
                                        cudaStream_t st) {
  using B = __nv_bfloat16;
  const int parts = add_rmsnorm_backward_parts(a.rows, a.dim);
  if (parts > 0) {
    if (act == MAMBA2_F32) add_norm_bwd_kernel<float, float><<<parts, kThreads, 0, st>>>(a, parts);
    else if (sum_type == MAMBA2_F32) add_norm_bwd_kernel<B, float><<<parts, kThreads, 0, st>>>(a, parts);
    else add_norm_bwd_kernel<B, B><<<parts, kThreads, 0, st>>>(a, parts);
  }
  if (a.dweight)
    column_sum_kernel<<<(a.dim + kThreads - 1) / kThreads, kThreads, 0, st>>>(a.dweight, a.partial, parts, a.dim);
  return cudaGetLastError();
}

}  // namespace mamba2
