// Gated delta rule (delta.h): token by token over packed runs, and the single-token step.
//
// A row of the state (one v channel) does not depend on the others, so 16 lanes hold a row, four adjacent elements of
// every 64 each, and its two sums over d_state (S k before the update, S q after it) are four shuffles each:
//   p = S k,  u = beta (v - a p),  S = a S + u k,  y = S q
// (a S k = a (S k): the decay needs no pass of its own; a key's length divides p and u instead of the key).
#include <type_traits>

#include "../../include/delta.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {
namespace {

#include "batch_check.cuh"

constexpr int kThreads = 256;
constexpr int kLanes = 16;                          // of a row of the state
constexpr int kRowsThread = 2;                      // rows of a thread (adjacent)
constexpr int kRowsCta = kThreads / kLanes * kRowsThread;  // 32

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Four adjacent elements as fp32.
__device__ __forceinline__ void four(const float* p, float* v) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}
__device__ __forceinline__ void four(const __nv_bfloat16* p, float* v) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(w.x << 16);
  v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16);
  v[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void store_two(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store_two(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// One token: the state rows s, the key and query of this lane's elements, the rows' v; gives the rows' y.
template <int E>
__device__ __forceinline__ void token(float (&s)[kRowsThread][E], const float (&k)[E], const float (&q)[E],
                                      const float (&v)[kRowsThread], float g, float beta, float scale, float l2_eps,
                                      float (&y)[kRowsThread]) {
  float p[kRowsThread], kk = 0.0f, qq = 0.0f;
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    p[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) p[r] = fmaf(s[r][e], k[e], p[r]);
  }
  float kn = 1.0f, qn = scale;
  if (l2_eps >= 0.0f) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kk = fmaf(k[e], k[e], kk);
      qq = fmaf(q[e], q[e], qq);
    }
    kn = rsqrtf(sum16(kk) + l2_eps);
    qn = scale * rsqrtf(sum16(qq) + l2_eps);
  }
  const float a = expf(g);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    const float u = beta * (v[r] - a * kn * sum16(p[r])) * kn;
    y[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s[r][e] = fmaf(a, s[r][e], u * k[e]);
      y[r] = fmaf(s[r][e], q[e], y[r]);
    }
    y[r] = qn * sum16(y[r]);
  }
}

// ------------------------------------------------------------------ packed runs

// A CTA takes 32 rows of one head's state over a whole run; the inputs of 16 tokens (8 where they are wide) are copied
// to shared memory while those before them are worked on. Bound by the chain of a token (a product, four shuffles, the update).
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src));
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src));
}

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) delta_serial_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int E = DK / kLanes;
  constexpr int unit = 16 / sizeof(T), kTile = sizeof(T) * DK > 512 ? 8 : 16;
  __shared__ __align__(16) T sk[2][kTile][DK], sq[2][kTile][DK], sv[2][kTile][kRowsCta];
  __shared__ float sg[2][kTile], sb[2][kTile];
  const int i = a.order[blockIdx.z], h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int row0 = blockIdx.x * kRowsCta, lane = threadIdx.x % kLanes;
  const int mine = (int)threadIdx.x / kLanes * kRowsThread, row = row0 + mine;
  const bool live = row < a.dv;  // (dv is even)
  const int first = a.tab.cu[i], len = a.tab.cu[i + 1] - first;
  float s[kRowsThread][E];
  float* st = a.state + (((int64_t)seq_slot(a.tab, i) * a.heads + h) * a.dv + row) * a.dk;
  const bool fresh = seq_fresh(a.tab, i);
  if (len == 0 && !fresh) return;
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int c = 0; c < E; c += 4) {
      const int at = 16 * c + 4 * lane;
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (live && !fresh && at < a.dk) four(st + (int64_t)r * a.dk + at, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][c + e] = f[e];
    }
  // the elements past d_state (and the rows past headdim) that the loops below read are zeros
  for (int e = threadIdx.x; e < 2 * kTile * DK; e += kThreads) (&sk[0][0][0])[e] = (&sq[0][0][0])[e] = Act<T>::from_f(0.0f);
  for (int e = threadIdx.x; e < 2 * kTile * kRowsCta; e += kThreads) (&sv[0][0][0])[e] = Act<T>::from_f(0.0f);
  __syncthreads();
  const T* q = static_cast<const T*>(a.q) + (int64_t)grp * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)grp * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv + row0;
  T* y = static_cast<T*>(a.y) + (int64_t)h * a.dv + row;
  const int wide = a.dk / unit, tall = min(kRowsCta, a.dv - row0) / unit;
  auto fetch = [&](int t0) {
    const int b = (t0 / kTile) & 1, n = min(kTile, len - t0);
    for (int e = threadIdx.x; e < n * wide; e += kThreads) {
      const int t = e / wide, c = (e - t * wide) * unit;
      const int64_t at = (int64_t)first + t0 + t;
      copy16(&sk[b][t][c], k + at * a.ld_k + c);
      copy16(&sq[b][t][c], q + at * a.ld_q + c);
    }
    for (int e = threadIdx.x; e < n * tall; e += kThreads) {
      const int t = e / tall, c = (e - t * tall) * unit;
      copy16(&sv[b][t][c], v + ((int64_t)first + t0 + t) * a.ld_v + c);
    }
    if ((int)threadIdx.x < n) {
      const int64_t at = ((int64_t)first + t0 + threadIdx.x) * a.heads + h;
      if (a.g) copy4(&sg[b][threadIdx.x], a.g + at);
      else sg[b][threadIdx.x] = 0.0f;
      if (a.beta) copy4(&sb[b][threadIdx.x], a.beta + at);
      else sb[b][threadIdx.x] = 1.0f;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (len > 0) fetch(0);
  for (int t0 = 0; t0 < len; t0 += kTile) {
    const int b = (t0 / kTile) & 1, n = min(kTile, len - t0);
    if (t0 + kTile < len) {
      fetch(t0 + kTile);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    if (a.ckpt && t0 % MAMBA2_DELTA_CHUNK == 0 && live) {
      float* o = a.ckpt + (((int64_t)(a.tab.tile[i] + t0 / MAMBA2_DELTA_CHUNK) * a.heads + h) * a.dv + row) * a.dk;
#pragma unroll
      for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
        for (int c = 0; c < E; c += 4)
          if (16 * c + 4 * lane < a.dk)
            *reinterpret_cast<float4*>(o + (int64_t)r * a.dk + 16 * c + 4 * lane) =
                make_float4(s[r][c], s[r][c + 1], s[r][c + 2], s[r][c + 3]);
    }
    for (int t = 0; t < n; ++t) {
      float kv[E], qv[E], vv[kRowsThread], yv[kRowsThread];
#pragma unroll
      for (int c = 0; c < E; c += 4) {
        four(&sk[b][t][16 * c + 4 * lane], kv + c);
        four(&sq[b][t][16 * c + 4 * lane], qv + c);
      }
#pragma unroll
      for (int r = 0; r < kRowsThread; ++r) vv[r] = Act<T>::to_f(sv[b][t][mine + r]);
      token<E>(s, kv, qv, vv, sg[b][t], sb[b][t], a.scale, a.l2_eps, yv);
      if (live && lane == 0) store_two(y + ((int64_t)first + t0 + t) * a.ld_y, yv[0], yv[1]);
    }
    __syncthreads();  // (the next fetch but one overwrites this buffer)
  }
  if (!live) return;
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int c = 0; c < E; c += 4)
      if (16 * c + 4 * lane < a.dk)
        *reinterpret_cast<float4*>(st + (int64_t)r * a.dk + 16 * c + 4 * lane) =
            make_float4(s[r][c], s[r][c + 1], s[r][c + 2], s[r][c + 3]);
}

// ------------------------------------------------------------------ single tokens

// One token of each sequence: a CTA takes 32 rows of one head's state. Bound by HBM: the state is read and written
// once, everything is asked for before anything is waited for.
constexpr int kCheckHere = kThreads;

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(const __grid_constant__ DeltaStepArgs a) {
  constexpr int E = DK / kLanes;
  const int i = blockIdx.z, h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int lane = threadIdx.x % kLanes, row = blockIdx.x * kRowsCta + (int)threadIdx.x / kLanes * kRowsThread;
  int slot, num = a.n, mine = 0;
  bool fresh;
  if (a.dev_slots) {
    num = *a.dev_n;
    slot = a.dev_slots[i];
    fresh = a.dev_fresh && a.dev_fresh[i];
    if (a.n <= kCheckHere && (int)threadIdx.x < a.n) mine = a.dev_slots[threadIdx.x];
  } else {
    slot = (int)(a.slot_fresh[i] & 0x7fffffffu);
    fresh = (a.slot_fresh[i] >> 31) != 0u;
  }
  const bool live = row < a.dv, is_slot = slot >= 0 && slot < a.num_slots;
  float* st = a.state + (((int64_t)(is_slot ? slot : 0) * a.heads + h) * a.dv + row) * a.dk;
  float s[kRowsThread][E], k[E], q[E], v[kRowsThread], y[kRowsThread];
  const T* qp = static_cast<const T*>(a.q) + i * a.ld_q + (int64_t)grp * a.dk;
  const T* kp = static_cast<const T*>(a.k) + i * a.ld_k + (int64_t)grp * a.dk;
#pragma unroll
  for (int c = 0; c < E; c += 4) {
    const int at = 16 * c + 4 * lane;
#pragma unroll
    for (int e = 0; e < 4; ++e) k[c + e] = q[c + e] = 0.0f;
    if (at < a.dk) {
      four(kp + at, k + c);
      four(qp + at, q + c);
    }
#pragma unroll
    for (int r = 0; r < kRowsThread; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][c + e] = 0.0f;
      if (live && is_slot && !fresh && at < a.dk) four(st + (int64_t)r * a.dk + at, s[r] + c);
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
    v[r] = live ? Act<T>::to_f(static_cast<const T*>(a.v)[i * a.ld_v + (int64_t)h * a.dv + row + r]) : 0.0f;
  const float g = a.g ? a.g[(int64_t)i * a.heads + h] : 0.0f, beta = a.beta ? a.beta[(int64_t)i * a.heads + h] : 1.0f;
  if (a.dev_slots) {
    if (a.n <= kCheckHere) {
      const int status = check_batch<kThreads>(num, a.n, a.num_slots, mine);
      if (blockIdx.x == 0 && h == 0 && i == 0 && threadIdx.x == 0) *a.dev_status = status;
      if (status != MAMBA2_OK) return;
    } else if (*a.dev_status != MAMBA2_OK) {
      return;
    }
    if (i >= num) return;
  }
  token<E>(s, k, q, v, g, beta, a.scale, a.l2_eps, y);
  if (!live) return;
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int c = 0; c < E; c += 4)
      if (16 * c + 4 * lane < a.dk)
        *reinterpret_cast<float4*>(st + (int64_t)r * a.dk + 16 * c + 4 * lane) =
            make_float4(s[r][c], s[r][c + 1], s[r][c + 2], s[r][c + 3]);
  if (lane == 0) store_two(static_cast<T*>(a.y) + i * a.ld_y + (int64_t)h * a.dv + row, y[0], y[1]);
}

// Runs f with the padded d_state as a constant.
template <typename F>
cudaError_t with_state(int dk, F f) {
  if (dk <= 64) f(std::integral_constant<int, 64>{});
  else if (dk <= 128) f(std::integral_constant<int, 128>{});
  else f(std::integral_constant<int, 256>{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_serial(const DeltaArgs& a, mamba2_dtype act, cudaStream_t st) {
  const dim3 grid((a.dv + kRowsCta - 1) / kRowsCta, a.heads, a.tab.n);
  return with_state(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    if (act == MAMBA2_BF16) delta_serial_kernel<__nv_bfloat16, DK><<<grid, kThreads, 0, st>>>(a);
    else delta_serial_kernel<float, DK><<<grid, kThreads, 0, st>>>(a);
  });
}

cudaError_t launch_delta_step(const DeltaStepArgs& a, mamba2_dtype act, cudaStream_t st) {
  if (a.dev_slots && a.n > kCheckHere) {
    const cudaError_t e = launch_check_device_batch(a.dev_slots, a.dev_n, a.n, a.num_slots, a.dev_status, st);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((a.dv + kRowsCta - 1) / kRowsCta, a.heads, a.n);
  return with_state(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    if (act == MAMBA2_BF16) delta_step_kernel<__nv_bfloat16, DK><<<grid, kThreads, 0, st>>>(a);
    else delta_step_kernel<float, DK><<<grid, kThreads, 0, st>>>(a);
  });
}

}  // namespace mamba2
