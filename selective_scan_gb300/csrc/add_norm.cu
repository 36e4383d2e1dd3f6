// RMS norm with the residual's addition (block.h), its 8-bit output, and its backward pass.
// Each reads its inputs from HBM once and writes its outputs once, and that bounds it.
//
// A row lives in the registers of `nt` threads, 32 elements each at most (16 in the backward pass, whose threads
// also hold their columns' sums), read and written in units of 8 elements, 16 bytes of bf16. nt is the fewest whole
// warps that hold the row, so all of a row's loads are on the way at once; with fewer rows than SMs a row is spread
// further, up to a thread per unit. Several rows share a CTA up to 256 threads. Sums of squares go warp by warp and
// then over the warps in order, in fp32. Rows wider than 512 threads hold (16 384, or 8 192 in the backward pass) are
// read again from L2 instead (the streamed kernels), an element a thread and access, the backward's sums of dweight kept
// in global memory: 2 000 x 20 000 of bf16 with a residual and its sum takes 144 us (2.2 TB/s), 160 with an 8-bit
// output, backwards 259 (1.2 TB/s). No configuration here has such rows.
//
// Where the width is no multiple of 8, units keep the matrix's boundaries instead of the row's (kShift): a row's
// first and last unit hold other rows' elements too, which are cleared as they arrive and not written. 16 384 x
// 2 047 of bf16 takes 47 us so, 77 in single elements; its backward 71 against 120 (2 046 in pairs of elements: 66
// and 74). Units of a row's own are faster where they fit: 2 048 takes 41 and 51, with one warp fewer to a row.
//
// Measured (GB300): 16 384 x 2 560, bf16 with a 32-bit sum, 74 us (6.8 TB/s, the measured copy rate); backward
// of 16 384 x 2 048, bf16, 51 us (5.3 TB/s; 5 of them the column sums' own kernel), of 16 384 x 2 560 with a
// 32-bit sum 84 us (6.0 TB/s). A backward CTA loads a row, reduces and stores in turn, so the rate follows the
// CTAs that an SM holds: with 32 elements a thread and two of them it was 54 and 118 us, with 8 elements 61; the
// next row's loads in between the stores made it slower (55 and 94).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "host.h"

namespace mamba2 {
namespace {

constexpr int W = 8;          // elements of a unit
constexpr int kHeld = 32;     // elements of a row that a thread holds
constexpr int kBwdHeld = 16;  // the same in the backward pass
constexpr int kCtaThreads = 256;
constexpr int kMaxThreads = 512;
constexpr float kMax8 = 448.0f;  // largest e4m3 value

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The scale of a row whose largest |y| is top: with it as the divisor, top comes to 448. Below the normal numbers, where
// a rounding may be of any size, it is rounded up, so that no quotient passes 448 and none is by zero.
__device__ __forceinline__ float scale_of(float top) {
  if (top == 0.0f) return 1.0f;
  const float scale = top / kMax8;
  return scale < 0x1p-126f ? __fdiv_ru(top, kMax8) : scale;
}
// Many quotients by one scale, each as if divided: with r near 1 / d and q = y r, the remainder q d - y is exact in one
// fma, and q - r (q d - y) is y / d to 2^-47 before its rounding (Markstein's correction). y and d are made 2^100 times as
// large where the reciprocal or the remainder would leave the normal numbers (a y that is still too small for that is
// 0 in 8 bits), and an infinite scale makes them 0 (or NaN, for an infinite y). (16 384 x 2 048 of bf16, with the residual and
// its sum: by division 42 us, by a reciprocal alone, which rounds twice, 38.)
struct Quotients {
  float m, d, r;
  __device__ __forceinline__ explicit Quotients(float scale)
      : m(scale < 0x1p-60f ? 0x1p100f : isinf(scale) ? 0.0f : 1.0f), d(isinf(scale) ? 1.0f : scale * m), r(1.0f / d) {}
  __device__ __forceinline__ float operator()(float y) const {
    const float v = y * m, q = v * r;
    return fmaf(-fmaf(q, d, -v), r, q);  // (with these signs -0 stays -0)
  }
};

// Where a thread's u-th unit lies in its row. With kShift rows start inside a unit of the matrix (dim is no multiple
// of 8): units keep the matrix's boundaries, so the first may begin before the row and the last end after it.
template <bool kShift>
struct At {
  int c;  // its first column
  __device__ __forceinline__ At(int shift, int nt, int u) : c(((int)threadIdx.x + nt * u) * W - (kShift ? shift : 0)) {}
  __device__ __forceinline__ bool has(int j, int dim) const { return !kShift || (unsigned)(c + j) < (unsigned)dim; }
  __device__ __forceinline__ bool whole(int dim) const { return !kShift || (c >= 0 && c + W <= dim); }
};

// How far a row starts behind a boundary.
__device__ __forceinline__ int shift_of(int64_t row, int dim) { return (int)(row * dim & (W - 1)); }

// A unit's values of one matrix. p: its first column's, which may lie outside the row where whole() is false; the
// 16 bytes that hold any of the row's elements are read and the rest are zeros, and only the row's are written.
template <typename T, bool kShift>
struct Unit {
  static constexpr int kWords = W * (int)sizeof(T) / 16, kEach = 16 / (int)sizeof(T);
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p, const At<kShift>& at, int dim) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int c = at.c + i * kEach;
      if (!kShift || kWords == 1 || (c < dim && c + kEach > 0)) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      else w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void store(T* p, const At<kShift>& at, int dim) const {
    if (at.whole(dim)) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (at.has(j, dim)) p[j] = reinterpret_cast<const T*>(w)[j];
    }
  }
  // other rows' elements become zeros
  __device__ __forceinline__ void clear(const At<kShift>& at, int dim) {
#pragma unroll
    for (int i = 0; i < W * (int)sizeof(T) / 4; ++i) {
      uint32_t& v = reinterpret_cast<uint32_t*>(w)[i];
      if constexpr (sizeof(T) == 2) v &= (at.has(2 * i, dim) ? 0xffffu : 0u) | (at.has(2 * i + 1, dim) ? 0xffff0000u : 0u);
      else v = at.has(i, dim) ? v : 0u;
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[W]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint32_t u = reinterpret_cast<const uint32_t*>(w)[i];
        v[2 * i] = __uint_as_float(u << 16);
        v[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = Act<T>::to_f(reinterpret_cast<const T*>(w)[i]);
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[W]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        reinterpret_cast<uint32_t*>(w)[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) reinterpret_cast<T*>(w)[i] = Act<T>::from_f(v[i]);
    }
  }
};
// W e4m3 values from fp32, to nearest even
template <bool kShift>
__device__ __forceinline__ void store8(__nv_fp8_storage_t* p, const float (&v)[W], const At<kShift>& at, int dim) {
  uint16_t h[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  if (at.whole(dim)) {
    *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (at.has(j, dim)) p[j] = (__nv_fp8_storage_t)(h[j / 2] >> (8 * (j & 1)));
  }
}

// The fp32 weights of a unit's columns; anything for columns outside the row. Where they start between two 16-byte words, the same for the whole row, the
// three words that hold them are read and shifted into place.
template <bool kShift>
__device__ __forceinline__ void load_weight(const float* weight, const At<kShift>& at, int dim, float (&w)[W]) {
  constexpr int kRead = kShift ? 12 : 8;
  float v[kRead];
  const int first = kShift ? at.c & ~3 : at.c;
#pragma unroll
  for (int i = 0; i < kRead / 4; ++i) {
    const int c = first + 4 * i;
    const bool in = !kShift || (c >= 0 && c < dim && c < at.c + W);
    const float4 a = in ? __ldg(reinterpret_cast<const float4*>(weight + c)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v[4 * i] = a.x;
    v[4 * i + 1] = a.y;
    v[4 * i + 2] = a.z;
    v[4 * i + 3] = a.w;
  }
  if constexpr (kShift) {
    if (at.c & 1)
#pragma unroll
      for (int j = 0; j < 11; ++j) v[j] = v[j + 1];
    if (at.c & 2)
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = v[j + 2];
  }
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = v[j];
}

// The sums (or NaN-keeping maxima) of n values over the row's nt threads, in a fixed order. part: a place per
// warp of the CTA that no reduction before the last barrier of the row's threads used; they alone meet here.
template <bool kMax, int n>
__device__ __forceinline__ void row_reduce(float (&v)[n], int nt, float (*part)[n]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float u = __shfl_xor_sync(0xffffffffu, v[k], o);
      v[k] = kMax ? max_nan(v[k], u) : v[k] + u;
    }
  if (nt == 32) return;
  const int warps = nt >> 5, row0 = (int)threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < n; ++k) part[row0 + (threadIdx.x >> 5)][k] = v[k];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"(nt) : "memory");
#pragma unroll
  for (int k = 0; k < n; ++k) v[k] = part[row0][k];
  for (int i = 1; i < warps; ++i)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = kMax ? max_nan(v[k], part[row0 + i][k]) : v[k] + part[row0 + i][k];
}

// Launched as a programmatic dependent: nothing of global memory is read or written before this. (The weights too may
// come from the kernel in front, an optimizer's step or a cast, or from one before it that it did not wait for.)
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename T, typename S, bool F8, bool kShift>
__global__ void __launch_bounds__(kMaxThreads)
add_norm_kernel(const AddNormArgs a, const int nt) {
  constexpr int U = kHeld / W;
  __shared__ float part[2][kMaxThreads / 32][1];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const int shift = shift_of(row, a.dim);
  const T* x = static_cast<const T*>(a.x) + row * a.dim;
  const S* r = static_cast<const S*>(a.residual) + row * a.dim;
  wait_for_inputs();
  Unit<T, kShift> xv[U];
  Unit<S, kShift> rv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const At<kShift> at(shift, nt, u);
    if (live && at.c < a.dim) {
      xv[u].load(x + at.c, at, a.dim);
      if (a.residual) rv[u].load(r + at.c, at, a.dim);
    }
  }
  float s[U][W], ss[1] = {0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const At<kShift> at(shift, nt, u);
    if (live && at.c < a.dim) {
      if (!at.whole(a.dim)) {
        xv[u].clear(at, a.dim);
        if (a.residual) rv[u].clear(at, a.dim);
      }
      xv[u].unpack(s[u]);
      if (a.residual) {
        float r1[W];
        rv[u].unpack(r1);
#pragma unroll
        for (int j = 0; j < W; ++j) s[u][j] += r1[j];
      }
#pragma unroll
      for (int j = 0; j < W; ++j) ss[0] = fmaf(s[u][j], s[u][j], ss[0]);
      if (a.sum) {
        rv[u].pack(s[u]);
        rv[u].store(static_cast<S*>(a.sum) + row * a.dim + at.c, at, a.dim);
      }
    }
  }
  row_reduce<false, 1>(ss, nt, part[0]);
  const float inv = rsqrtf(ss[0] / (float)a.dim + a.eps);
  float top[1] = {0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const At<kShift> at(shift, nt, u);
    if (live && at.c < a.dim) {
      float w[W];
      load_weight(a.weight, at, a.dim, w);
#pragma unroll
      for (int j = 0; j < W; ++j) s[u][j] = s[u][j] * inv * w[j];
      if (F8) {
        if (!at.whole(a.dim))  // (what lies behind the last weight may be anything)
#pragma unroll
          for (int j = 0; j < W; ++j) s[u][j] = at.has(j, a.dim) ? s[u][j] : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) top[0] = max_nan(top[0], fabsf(s[u][j]));
      }
      if (!F8) {
        Unit<T, kShift> o;
        o.pack(s[u]);
        o.store(static_cast<T*>(a.out) + row * a.dim + at.c, at, a.dim);
      }
    }
  }
  if (F8) {
    row_reduce<true, 1>(top, nt, part[1]);
    const float scale = scale_of(top[0]);
    const Quotients by(scale);
    if (!live) return;
    if (threadIdx.x == 0) a.scale[row] = scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const At<kShift> at(shift, nt, u);
      if (at.c < a.dim) {
#pragma unroll
        for (int j = 0; j < W; ++j) s[u][j] = by(s[u][j]);
        store8(static_cast<__nv_fp8_storage_t*>(a.out) + row * a.dim + at.c, s[u], at, a.dim);
      }
    }
  }
}

// ------------------------------------------------------------------ backward

// CTAs walk the rows; a thread's columns are the same in every row, so it adds up its share of dweight in registers.
// The CTA's row groups add theirs in order through shared memory, and the CTA writes one row of partial sums.
// (The registers that keep a row's values packed between its two uses: left alone, the compiler unpacks them once,
// and half of the CTAs fit. With kShift what is fastest: 16 bits 71 us with 80, 86 with 64 and 94 with 128, at 16 384
// x 2 047; 32 bits 52 us with 96 and 54 with 112, at 8 192 x 2 047.)
// With kShift a thread's columns repeat every eighth row; the grid takes whole multiples of that. Its weights lie in
// shared memory, shifted once (read with their row's shift from L1 each time: 94 us).
template <typename T, typename S, bool kShift>
constexpr int kBwdRegs = sizeof(S) == 2 ? (kShift ? 80 : 64) : sizeof(T) == 2 ? (kShift ? 96 : 80) : (kShift ? 96 : 112);

template <typename T, typename S, bool kShift>
__global__ void __maxnreg__((kBwdRegs<T, S, kShift>))
add_norm_bwd_kernel(const AddNormBwdArgs a, const int nt) {
  constexpr int U = kBwdHeld / W;
  __shared__ float part[2][kMaxThreads / 32][2];
  // With more than one row to a CTA, the sums of dweight [dim]. Before that, with kShift, a row of weights for each of
  // them, shifted as its units are.
  extern __shared__ __align__(16) float columns[];
  const float4* weights = reinterpret_cast<const float4*>(columns + threadIdx.y * nt * U * W) + threadIdx.x * 2;
  const int shift = shift_of((int64_t)blockIdx.x * blockDim.y + threadIdx.y, a.dim);  // of all of its rows
  wait_for_inputs();
  if constexpr (kShift) {
#pragma unroll
    for (int k = 0; k < U * W; ++k) {
      const int i = (int)threadIdx.x + nt * k, c = i - shift;
      columns[threadIdx.y * nt * U * W + i] = c >= 0 && c < a.dim ? __ldg(a.weight + c) : 0.0f;
    }
    __syncthreads();
  }
  auto unit_weight = [&](int u, int c, float (&w)[W]) {
    const float4* p = kShift ? weights + nt * u * 2 : reinterpret_cast<const float4*>(a.weight + c);
    const float4 lo = kShift ? p[0] : __ldg(p), hi = kShift ? p[1] : __ldg(p + 1);
    w[0] = lo.x;
    w[1] = lo.y;
    w[2] = lo.z;
    w[3] = lo.w;
    w[4] = hi.x;
    w[5] = hi.y;
    w[6] = hi.z;
    w[7] = hi.w;
  };
  float acc[U][W];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < W; ++j) acc[u][j] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + threadIdx.y, base = row * a.dim;
    const bool live = row < a.rows;
    Unit<S, kShift> sv[U], dv[U];
    Unit<T, kShift> gv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const At<kShift> at(shift, nt, u);
      if (live && at.c < a.dim) {
        sv[u].load(static_cast<const S*>(a.sum) + base + at.c, at, a.dim);
        gv[u].load(static_cast<const T*>(a.dy) + base + at.c, at, a.dim);
        if (a.dsum) dv[u].load(static_cast<const S*>(a.dsum) + base + at.c, at, a.dim);
      }
    }
    float sums[2] = {0.0f, 0.0f};  // of s^2, and of s weight dy
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const At<kShift> at(shift, nt, u);
      if (live && at.c < a.dim) {
        if (!at.whole(a.dim)) {
          sv[u].clear(at, a.dim);
          gv[u].clear(at, a.dim);
        }
        float w[W], v[W], g[W];
        unit_weight(u, at.c, w);
        sv[u].unpack(v);
        gv[u].unpack(g);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          sums[0] = fmaf(v[j], v[j], sums[0]);
          sums[1] = fmaf(v[j], w[j] * g[j], sums[1]);
        }
      }
    }
    row_reduce<false, 2>(sums, nt, part[turn ^= 1]);
    const float inv = rsqrtf(sums[0] / (float)a.dim + a.eps);
    const float k = inv * inv * (sums[1] / (float)a.dim);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const At<kShift> at(shift, nt, u);
      if (live && at.c < a.dim) {
        float w[W], v[W], g[W], d[W];
        unit_weight(u, at.c, w);
        sv[u].unpack(v);
        gv[u].unpack(g);
#pragma unroll
        for (int j = 0; j < W; ++j) d[j] = 0.0f;
        if (a.dsum) dv[u].unpack(d);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          d[j] = fmaf(inv, fmaf(w[j], g[j], -v[j] * k), d[j]);
          acc[u][j] = fmaf(g[j] * v[j], inv, acc[u][j]);
        }
        if (a.dx) {
          gv[u].pack(d);
          gv[u].store(static_cast<T*>(a.dx) + base + at.c, at, a.dim);
        }
        if (a.dresidual) {
          sv[u].pack(d);
          sv[u].store(static_cast<S*>(a.dresidual) + base + at.c, at, a.dim);
        }
      }
    }
  }
  if (!a.dweight) return;
  if (kShift) __syncthreads();  // done with the weights
  for (int y = 0; y < (int)blockDim.y; ++y) {
    if ((int)threadIdx.y == y) {
      const bool last = y == (int)blockDim.y - 1;
      float* out = last ? a.partial + (int64_t)blockIdx.x * a.dim : columns;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const At<kShift> at(shift, nt, u);
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (at.c < a.dim && at.has(j, a.dim)) out[at.c + j] = (y > 0 ? columns[at.c + j] : 0.0f) + acc[u][j];
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// dst[i] = sum of part[.][i]: 32 columns a CTA, a warp for every 32nd row, then the warps' sums in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(float* dst, const float* part, int parts, int dim) {
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.0f;
  if (i < dim)
    for (int p = w; p < parts; p += 32) s += part[(int64_t)p * dim + i];
  sum[w][lane] = s;
  __syncthreads();
  s = sum[lane][w];  // column w of this CTA, the warps' sums in the lanes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + w < dim) dst[blockIdx.x * 32 + w] = s;
}

// ------------------------------------------------------------------ rows wider than a CTA holds

__device__ __forceinline__ float block_reduce(float v, bool max) {
  __shared__ float part[kCtaThreads / 32];
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = max ? max_nan(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kCtaThreads / 32; ++i) v = max ? max_nan(v, part[i]) : v + part[i];
  return v;
}

template <typename T, typename S, bool F8>
__global__ void __launch_bounds__(kCtaThreads) add_norm_streamed_kernel(const AddNormArgs a) {
  const int64_t base = (int64_t)blockIdx.x * a.dim;
  const T* x = static_cast<const T*>(a.x) + base;
  const S* r = a.residual ? static_cast<const S*>(a.residual) + base : nullptr;
  auto value = [&](int i) { return Act<T>::to_f(x[i]) + (r ? Act<S>::to_f(r[i]) : 0.0f); };
  float ss = 0.0f, top = 0.0f, scale = 0.0f;
  for (int i = threadIdx.x; i < a.dim; i += kCtaThreads) ss = fmaf(value(i), value(i), ss);
  const float inv = rsqrtf(block_reduce(ss, false) / (float)a.dim + a.eps);
  if (F8) {
    for (int i = threadIdx.x; i < a.dim; i += kCtaThreads) top = max_nan(top, fabsf(value(i) * inv * a.weight[i]));
    scale = scale_of(block_reduce(top, true));
    if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
  }
  for (int i = threadIdx.x; i < a.dim; i += kCtaThreads) {
    const float s = value(i), y = s * inv * a.weight[i];
    if (F8) static_cast<__nv_fp8_storage_t*>(a.out)[base + i] = __nv_cvt_float_to_fp8(y / scale, __NV_SATFINITE, __NV_E4M3);
    else static_cast<T*>(a.out)[base + i] = Act<T>::from_f(y);
    if (a.sum) static_cast<S*>(a.sum)[base + i] = Act<S>::from_f(s);
  }
}

template <typename T, typename S>
__global__ void __launch_bounds__(kCtaThreads) add_norm_bwd_streamed_kernel(const AddNormBwdArgs a, int parts) {
  for (int64_t row = blockIdx.x; row < a.rows; row += parts) {
    const int64_t base = row * a.dim;
    const T* dy = static_cast<const T*>(a.dy) + base;
    const S* s = static_cast<const S*>(a.sum) + base;
    float ss = 0.0f, sd = 0.0f;
    for (int i = threadIdx.x; i < a.dim; i += kCtaThreads) {
      const float v = Act<S>::to_f(s[i]);
      ss = fmaf(v, v, ss);
      sd = fmaf(v, a.weight[i] * Act<T>::to_f(dy[i]), sd);
    }
    const float inv = rsqrtf(block_reduce(ss, false) / (float)a.dim + a.eps);
    const float c = inv * inv * (block_reduce(sd, false) / (float)a.dim);
    for (int i = threadIdx.x; i < a.dim; i += kCtaThreads) {
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

// Elements that a row's units span at most.
int span(int dim) { return dim % W == 0 ? dim : dim + W - 1; }
// Threads of a row, and rows of a CTA.
struct Shape {
  int nt, rows;
};
Shape shape(int64_t rows, int dim, int held) {
  const int fewest = 32 * ((span(dim) + 32 * held - 1) / (32 * held));
  const int most = 32 * ((span(dim) + 32 * W - 1) / (32 * W));
  if (rows <= device_sm_count()) return {std::max(fewest, std::min(most, kCtaThreads)), 1};
  return {fewest, std::max(1, kCtaThreads / fewest)};
}

cudaLaunchConfig_t config(int grid, dim3 block, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return c;
}

template <typename T, typename S, bool F8>
cudaError_t run_norm(const AddNormArgs& a, cudaStream_t st) {
  if (span(a.dim) > kMaxThreads * kHeld) {
    add_norm_streamed_kernel<T, S, F8><<<a.rows, kCtaThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const Shape s = shape(a.rows, a.dim, kHeld);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t c = config((a.rows + s.rows - 1) / s.rows, dim3(s.nt, s.rows), 0, st, &attr);
  if (a.dim % W == 0) return cudaLaunchKernelEx(&c, add_norm_kernel<T, S, F8, false>, a, s.nt);
  return cudaLaunchKernelEx(&c, add_norm_kernel<T, S, F8, true>, a, s.nt);
}

template <typename T, typename S>
cudaError_t run_norm_bwd(const AddNormBwdArgs& a, int* used, cudaStream_t st) {
  const int most = add_rmsnorm_backward_parts(a.rows, a.dim);
  if (span(a.dim) > kMaxThreads * kBwdHeld) {
    *used = most;
    add_norm_bwd_streamed_kernel<T, S><<<most, kCtaThreads, 0, st>>>(a, most);
    return cudaGetLastError();
  }
  const Shape s = shape(a.rows, a.dim, kBwdHeld);
  const size_t smem = a.dim % W ? (size_t)s.rows * s.nt * kBwdHeld * 4 : s.rows > 1 ? (size_t)a.dim * 4 : 0;
  auto run = [&](auto kernel) {  // as many CTAs as the GPU holds: each loads a row while others work on theirs
    int fit = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, s.nt * s.rows, smem);
    if (e != cudaSuccess) return e;
    *used = (int)std::min<int64_t>({(int64_t)most, ((int64_t)a.rows + s.rows - 1) / s.rows,
                                    std::max(1, fit) * (int64_t)device_sm_count()});
    if ((int64_t)*used * s.rows < a.rows) *used &= ~(W - 1);  // a thread's columns are the same in every W-th row
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t c = config(*used, dim3(s.nt, s.rows), smem, st, &attr);
    return cudaLaunchKernelEx(&c, kernel, a, s.nt);
  };
  if (a.dim % W == 0) return run(add_norm_bwd_kernel<T, S, false>);
  return run(add_norm_bwd_kernel<T, S, true>);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, mamba2_dtype act, mamba2_dtype sum_type, mamba2_dtype out_type,
                               cudaStream_t st) {
  using B = __nv_bfloat16;
  const bool f8 = out_type == MAMBA2_E4M3;
  if (act == MAMBA2_F32) return f8 ? run_norm<float, float, true>(a, st) : run_norm<float, float, false>(a, st);
  if (sum_type == MAMBA2_F32) return f8 ? run_norm<B, float, true>(a, st) : run_norm<B, float, false>(a, st);
  return f8 ? run_norm<B, B, true>(a, st) : run_norm<B, B, false>(a, st);
}

// CTAs of the backward kernel at most (each writes one row of partial sums): eight to an SM.
int add_rmsnorm_backward_parts(int32_t rows, int32_t) { return (int)std::min<int64_t>(rows, 8 * (int64_t)device_sm_count()); }

cudaError_t launch_add_rmsnorm_backward(const AddNormBwdArgs& a, mamba2_dtype act, mamba2_dtype sum_type,
                                        cudaStream_t st) {
  using B = __nv_bfloat16;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    if (act == MAMBA2_F32) e = run_norm_bwd<float, float>(a, &parts, st);
    else if (sum_type == MAMBA2_F32) e = run_norm_bwd<B, float>(a, &parts, st);
    else e = run_norm_bwd<B, B>(a, &parts, st);
  }
  if (e != cudaSuccess || !a.dweight) return e;
  return launch_column_sum(a.dweight, a.partial, parts, a.dim, st);
}

cudaError_t launch_column_sum(float* dst, const float* part, int parts, int dim, cudaStream_t st) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t c = config((dim + 31) / 32, dim3(1024), 0, st, &attr);
  return cudaLaunchKernelEx(&c, column_sum_kernel, dst, part, parts, dim);
}

}  // namespace mamba2
