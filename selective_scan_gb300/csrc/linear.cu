// Matrix product with bias, activation and residual in its epilogue (block.h), from bf16
// or e4m3 operands, and its backward pass.
//
// 64 x 64 output tiles, 16 deep, staged in shared memory, 16 products a thread on the
// CUDA cores.
#include <cuda_fp8.h>

#include "../../include/block.h"
#include "common.cuh"

namespace mamba2 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kDeep = 16;

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__nv_fp8_e4m3 v) { return float(v); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MAMBA2_ACT_RELU: return fmaxf(v, 0.0f);
    case MAMBA2_ACT_SILU: return silu_f(v);
    case MAMBA2_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  }
  return v;
}
__device__ __forceinline__ float slope(float v, int act) {
  switch (act) {
    case MAMBA2_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case MAMBA2_ACT_SILU: {
      const float p = __fdividef(1.0f, 1.0f + __expf(-v));
      return p * fmaf(v, 1.0f - p, 1.0f);
    }
    case MAMBA2_ACT_GELU:
      return fmaf(v * 0.39894228040143268f, __expf(-0.5f * v * v), 0.5f * (1.0f + erff(v * 0.70710678118654752f)));
  }
  return 1.0f;
}

// acc[i][j] of rows m0 + ty + 16 i, columns n0 + tx + 16 j of the product of A(m, k) and B(n, k)
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(int M, int N, int K, FA A, FB B, float (&acc)[4][4]) {
  __shared__ float sa[kDeep][kTile + 1], sb[kDeep][kTile + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int k0 = 0; k0 < K; k0 += kDeep) {
    for (int e = threadIdx.x; e < kTile * kDeep; e += kThreads) {
      const int r = e / kDeep, k = e % kDeep;
      sa[k][r] = m0 + r < M && k0 + k < K ? A(m0 + r, k0 + k) : 0.0f;
      sb[k][r] = n0 + r < N && k0 + k < K ? B(n0 + r, k0 + k) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kDeep; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) linear_kernel(const LinearArgs a, int act) {
  const TI* x = static_cast<const TI*>(a.x);
  const TI* w = static_cast<const TI*>(a.w);
  float acc[4][4];
  tile_product(a.rows, a.out_f, a.in_f, [&](int m, int k) { return to_float(x[m * a.ld_x + k]); },
               [&](int n, int k) { return to_float(w[(int64_t)n * a.in_f + k]); }, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = blockIdx.y * kTile + threadIdx.x / 16 + 16 * i, n = blockIdx.x * kTile + threadIdx.x % 16 + 16 * j;
      if (m >= a.rows || n >= a.out_f) continue;
      float v = acc[i][j];
      if (a.w_scale) v = v * a.x_scale[m] * a.w_scale[n];
      if (a.bias) v += a.bias[n];
      if (a.pre) static_cast<__nv_bfloat16*>(a.pre)[(int64_t)m * a.out_f + n] = __float2bfloat16_rn(v);
      v = activate(v, act);
      if (a.residual) v += Act<TO>::to_f(static_cast<const TO*>(a.residual)[m * a.ld_res + n]);
      static_cast<TO*>(a.out)[m * a.ld_out + n] = Act<TO>::from_f(v);
    }
}

constexpr int kRowsPerPart = 64;

// dp = dy * activation'(pre) in bf16, and the column sums of each kRowsPerPart rows
__global__ void __launch_bounds__(kThreads) dp_kernel(const LinearBwdArgs a, int act) {
  const int n = blockIdx.x * kThreads + threadIdx.x;
  if (n >= a.ld_dp) return;
  const int m1 = min(a.rows, (int)(blockIdx.y + 1) * kRowsPerPart);
  float s = 0.0f;
  for (int m = blockIdx.y * kRowsPerPart; m < m1; ++m) {
    float v = 0.0f;
    if (n < a.out_f) {
      v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.dy)[(int64_t)m * a.out_f + n]);
      if (act) v *= slope(__bfloat162float(static_cast<const __nv_bfloat16*>(a.pre)[(int64_t)m * a.out_f + n]), act);
    }
    s += v;
    static_cast<__nv_bfloat16*>(a.dp)[m * a.ld_dp + n] = __float2bfloat16_rn(v);
  }
  if (n < a.out_f) a.partial[(int64_t)blockIdx.y * a.out_f + n] = s;
}

__global__ void __launch_bounds__(kThreads) bias_sum_kernel(float* dst, const float* part, int parts, int n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += part[(int64_t)p * n + i];
  dst[i] = s;
}

// which = 0: dx[m][k] = sum_n dp[m][n] w[n][k]; 1: dw[n][k] = sum_m dp[m][n] x[m][k]
template <int which>
__global__ void __launch_bounds__(kThreads) grad_kernel(const LinearBwdArgs a) {
  const __nv_bfloat16* dp = static_cast<const __nv_bfloat16*>(a.dp);
  const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(which ? a.x : a.w);
  const int64_t ldb = which ? a.ld_x : a.in_f;
  const int M = which ? a.out_f : a.rows, K = which ? a.rows : a.out_f;
  float acc[4][4];
  tile_product(M, a.in_f, K, [&](int m, int k) { return to_float(which ? dp[k * a.ld_dp + m] : dp[m * a.ld_dp + k]); },
               [&](int n, int k) { return to_float(b[k * ldb + n]); }, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = blockIdx.y * kTile + threadIdx.x / 16 + 16 * i, n = blockIdx.x * kTile + threadIdx.x % 16 + 16 * j;
      if (m < M && n < a.in_f)
        static_cast<__nv_bfloat16*>(which ? a.dw : a.dx)[(int64_t)m * a.in_f + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

dim3 tiles(int m, int n) { return dim3((n + kTile - 1) / kTile, (m + kTile - 1) / kTile); }

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, mamba2_dtype in, mamba2_dtype out, int act, cudaStream_t st) {
  const dim3 g = tiles(a.rows, a.out_f);
  if (in == MAMBA2_BF16) {
    if (out == MAMBA2_BF16) linear_kernel<__nv_bfloat16, __nv_bfloat16><<<g, kThreads, 0, st>>>(a, act);
    else linear_kernel<__nv_bfloat16, float><<<g, kThreads, 0, st>>>(a, act);
  } else {
    if (out == MAMBA2_BF16) linear_kernel<__nv_fp8_e4m3, __nv_bfloat16><<<g, kThreads, 0, st>>>(a, act);
    else linear_kernel<__nv_fp8_e4m3, float><<<g, kThreads, 0, st>>>(a, act);
  }
  return cudaGetLastError();
}

int linear_bias_parts(int32_t rows) { return (rows + kRowsPerPart - 1) / kRowsPerPart; }

cudaError_t launch_linear_backward(const LinearBwdArgs& a, int act, cudaStream_t st) {
  const int parts = linear_bias_parts(a.rows);
  if (parts > 0) dp_kernel<<<dim3((unsigned)((a.ld_dp + kThreads - 1) / kThreads), parts), kThreads, 0, st>>>(a, act);
  if (a.dbias)
    bias_sum_kernel<<<(a.out_f + kThreads - 1) / kThreads, kThreads, 0, st>>>(a.dbias, a.partial, parts, a.out_f);
  if (a.dx && a.rows > 0) grad_kernel<0><<<tiles(a.rows, a.in_f), kThreads, 0, st>>>(a);
  if (a.dw) grad_kernel<1><<<tiles(a.out_f, a.in_f), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mamba2
