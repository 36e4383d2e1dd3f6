// Gated delta rule (delta.h): token by token over packed runs, and the single-token step.
//
// A row of the state (one v channel) does not depend on the others, so 8 lanes hold a row, four adjacent elements of
// every 32 each, and its two sums over d_state (S k before the update, S q after it) are three shuffles each:
//   p = S k,  u = beta (v - a p),  S = a S + u k,  y = S q
// (a S k = a (S k): the decay needs no pass of its own; a key's length divides p and u instead of the key). Elements are
// worked on in pairs, one instruction for two.
#include <type_traits>

#include "../../include/delta.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {
namespace {

#include "batch_check.cuh"

constexpr int kLanes = 8;       // of a row of the state
constexpr int kRowsThread = 2;  // rows of a thread (adjacent)

__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Two {  // two fp32 numbers
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float both(Two a) {  // their sum
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
  return lo + hi;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Four adjacent elements.
__device__ __forceinline__ void four(const float* p, Two* v) {
  const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(p);
  v[0].v = f.x;
  v[1].v = f.y;
}
__device__ __forceinline__ void four(const __nv_bfloat16* p, Two* v) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = two(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
  v[1] = two(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store_four(float* p, const Two* v) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0].v, v[1].v);
}
__device__ __forceinline__ void store_two(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store_two(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// Sum of products over this lane's 2 N elements, in two chains.
template <int N>
__device__ __forceinline__ float dot(const Two (&a)[N], const Two (&b)[N]) {
  Two s = mul(a[0], b[0]), t = mul(a[1], b[1]);
#pragma unroll
  for (int e = 2; e < N; e += 2) {
    s = fma(a[e], b[e], s);
    t = fma(a[e + 1], b[e + 1], t);
  }
  return both(s) + both(t);
}

// What a token's key, query, decay and beta come to: a; beta / |k|; a / |k|; scale / |q|.
struct Token {
  float a, write, read, qn;
};
template <int N>
__device__ __forceinline__ Token token_of(const Two (&k)[N], const Two (&q)[N], float g, float beta, float scale, float l2_eps) {
  float kn = 1.0f, qn = scale;
  if (l2_eps >= 0.0f) {
    kn = rsqrtf(sum8(dot(k, k)) + l2_eps);
    qn = scale * rsqrtf(sum8(dot(q, q)) + l2_eps);
  }
  const float a = expf(g);
  return {a, beta * kn, a * kn, qn};
}

// One token: the state rows s, the key and query of this lane's elements, the rows' v; gives this lane's part of the
// rows' S q.
template <int N>
__device__ __forceinline__ void advance(Two (&s)[kRowsThread][N], const Two (&k)[N], const Two (&q)[N],
                                        const float (&v)[kRowsThread], const Token& t, float (&y)[kRowsThread]) {
  float p[kRowsThread];
  const Two a = two(t.a, t.a);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) p[r] = dot(s[r], k);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = mul(a, s[r][e]);  // (while the sums go round)
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) p[r] = sum8(p[r]);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    const float u = t.write * fmaf(-t.read, p[r], v[r]);
    const Two uu = two(u, u);
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = fma(uu, k[e], s[r][e]);
  }
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) y[r] = dot(s[r], q);
}

// Two tokens at once, from the state S before them, so that all of S's sums go round together and S is scaled once: with
// a and u of each, and S' the state between,
//   S' k1 = a0 (S k1) + u0 (k0 . k1),  S'' = a0 a1 S + a1 u0 k0 + u1 k1,
//   S' q0 = a0 (S q0) + u0 (k0 . q0),  S'' q1 = a0 a1 (S q1) + a1 u0 (k0 . q1) + u1 (k1 . q1)
struct Products {
  float kk, kq00, kq01, kq11;
};
// Gives this lane's parts of S q0 and S q1, and what u0 and u1 add to them.
template <int N>
__device__ __forceinline__ void advance_two(Two (&s)[kRowsThread][N], const Two (&k0)[N], const Two (&k1)[N], const Two (&q0)[N],
                                            const Two (&q1)[N], const float (&v0)[kRowsThread], const float (&v1)[kRowsThread],
                                            const Token& t0, const Token& t1, const Products& c, float (&y0)[kRowsThread],
                                            float (&y1)[kRowsThread], float (&add0)[kRowsThread], float (&add1)[kRowsThread]) {
  float p0[kRowsThread], p1[kRowsThread];
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    p0[r] = dot(s[r], k0);
    p1[r] = dot(s[r], k1);
  }
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    p0[r] = sum8(p0[r]);
    p1[r] = sum8(p1[r]);
  }
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {  // (while the sums go round)
    y0[r] = dot(s[r], q0);
    y1[r] = dot(s[r], q1);
  }
  const Two a = two(t0.a * t1.a, t0.a * t1.a);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = mul(a, s[r][e]);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) {
    const float u0 = t0.write * fmaf(-t0.read, p0[r], v0[r]);
    const float u1 = t1.write * fmaf(-t1.read, fmaf(u0, c.kk, t0.a * p1[r]), v1[r]);
    const float u = t1.a * u0;
    add0[r] = u0 * c.kq00;
    add1[r] = fmaf(u, c.kq01, u1 * c.kq11);
    const Two w0 = two(u, u), w1 = two(u1, u1);
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = fma(w1, k1[e], fma(w0, k0[e], s[r][e]));
  }
}

// ------------------------------------------------------------------ packed runs

// A CTA takes 32 rows of one head's state over a whole run; the inputs of 16 tokens (8 where they are wide) are copied to
// shared memory while those before them are worked on, and what depends on a token's key and query alone is made for all
// 16 at once. Bound by the chain of two tokens, a product, three shuffles and the update, and the issue of their
// instructions: 13 runs of fp32, 3 109 tokens, 6 heads of 104 x 72, take 95 us, about 200 ns a token of the longest (one
// token at a time 108). A row to eight lanes instead of two takes 119, as every warp reads the keys and queries.
constexpr int kSerialThreads = 128, kSerialRows = kSerialThreads / kLanes * kRowsThread;

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src));
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src));
}

template <typename T, int DK>
__global__ void __launch_bounds__(kSerialThreads) delta_serial_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int N = DK / kLanes / 2;  // pairs of a lane
  constexpr int unit = 16 / sizeof(T), kTile = sizeof(T) * DK > 512 ? 8 : 16;
  __shared__ __align__(16) T sk[2][kTile][DK], sq[2][kTile][DK], sv[2][kTile][kSerialRows];
  __shared__ float sg[2][kTile], sb[2][kTile];
  __shared__ __align__(16) Token tokens[kTile];
  __shared__ __align__(16) Products products[kTile / 2];
  const int i = a.order[blockIdx.z], h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int row0 = blockIdx.x * kSerialRows, lane = threadIdx.x % kLanes;
  const int mine = (int)threadIdx.x / kLanes * kRowsThread, row = row0 + mine;
  const bool live = row < a.dv;  // (dv is even)
  const int first = a.tab.cu[i], len = a.tab.cu[i + 1] - first;
  const bool fresh = seq_fresh(a.tab, i);
  if (len == 0 && !fresh) return;
  Two s[kRowsThread][N];
  float* st = a.state + (((int64_t)seq_slot(a.tab, i) * a.heads + h) * a.dv + row) * a.dk;
  auto each = [&](auto f) {  // f(pairs, offset) of this thread's fours
    if (!live) return;
#pragma unroll
    for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
      for (int c = 0; c < N; c += 2)
        if (16 * c + 4 * lane < a.dk) f(s[r] + c, (int64_t)r * a.dk + 16 * c + 4 * lane);
  };
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int e = 0; e < N; ++e) s[r][e] = two(0.0f, 0.0f);
  if (!fresh) each([&](Two* v, int64_t at) { four(st + at, v); });
  // the elements past d_state (and the rows past headdim) that the loops below read are zeros
  for (int e = threadIdx.x; e < 2 * kTile * DK; e += kSerialThreads) (&sk[0][0][0])[e] = (&sq[0][0][0])[e] = Act<T>::from_f(0.0f);
  for (int e = threadIdx.x; e < 2 * kTile * kSerialRows; e += kSerialThreads) (&sv[0][0][0])[e] = Act<T>::from_f(0.0f);
  __syncthreads();
  const T* q = static_cast<const T*>(a.q) + (int64_t)grp * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)grp * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv + row0;
  T* y = static_cast<T*>(a.y) + (int64_t)h * a.dv + row;
  const int tall = min(kSerialRows, a.dv - row0);
  auto fetch = [&](int t0) {  // (eight threads a token)
    const int b = (t0 / kTile) & 1, n = min(kTile, len - t0), t = (int)threadIdx.x / kLanes;
    if (t < n) {
      const int64_t at = (int64_t)first + t0 + t;
      const T *kt = k + at * a.ld_k, *qt = q + at * a.ld_q, *vt = v + at * a.ld_v;
#pragma unroll
      for (int c = lane * unit; c < DK; c += kLanes * unit)
        if (c < a.dk) {
          copy16(&sk[b][t][c], kt + c);
          copy16(&sq[b][t][c], qt + c);
        }
      if (lane * unit < tall) copy16(&sv[b][t][lane * unit], vt + lane * unit);
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
  auto load = [&](const T* p, Two (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 2) four(p + 16 * c + 4 * lane, v + c);
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
    if (a.ckpt && t0 % MAMBA2_DELTA_CHUNK == 0) {
      float* o = a.ckpt + (((int64_t)(a.tab.tile[i] + t0 / MAMBA2_DELTA_CHUNK) * a.heads + h) * a.dv + row) * a.dk;
      each([&](Two* w, int64_t at) { store_four(o + at, w); });
    }
    {  // (what is computed of tokens behind the last is not used)
      const int t = min((int)threadIdx.x / kLanes, kTile - 1);
      Two kv[N], qv[N];
      load(sk[b][t], kv);
      load(sq[b][t], qv);
      const Token tok = token_of(kv, qv, sg[b][t], sb[b][t], a.scale, a.l2_eps);
      if (lane == 0) tokens[t] = tok;
      const float own = sum8(dot(kv, qv));
      load(sk[b][t ^ 1], qv);
      const float kk = sum8(dot(kv, qv));
      load(sq[b][t ^ 1], qv);
      const float across = sum8(dot(kv, qv));
      if (lane == 0) {  // (an odd token's own product alone)
        if (t & 1) products[t >> 1].kq11 = own;
        else products[t >> 1].kk = kk, products[t >> 1].kq00 = own, products[t >> 1].kq01 = across;
      }
    }
    __syncthreads();
    auto one = [&](int t, float (&yp)[kRowsThread]) {
      Two kv[N], qv[N];
      float vv[kRowsThread];
      load(sk[b][t], kv);
      load(sq[b][t], qv);
#pragma unroll
      for (int r = 0; r < kRowsThread; ++r) vv[r] = Act<T>::to_f(sv[b][t][mine + r]);
      advance(s, kv, qv, vv, tokens[t], yp);
    };
    int t = row0 + (int)(threadIdx.x & ~31u) / kLanes * kRowsThread < a.dv ? 0 : n;  // (a warp without rows has no work)
    for (; t + 8 <= n; t += 8) {
      // eight tokens' parts are summed at once, so that no token waits for another's output: 7 shuffles a row that leave
      // lane j with token j's
      float yp[8][kRowsThread], add[kRowsThread] = {};
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        Two k0[N], k1[N], q0[N], q1[N];
        float v0[kRowsThread], v1[kRowsThread], add0[kRowsThread], add1[kRowsThread];
        load(sk[b][t + j], k0);
        load(sk[b][t + j + 1], k1);
        load(sq[b][t + j], q0);
        load(sq[b][t + j + 1], q1);
#pragma unroll
        for (int r = 0; r < kRowsThread; ++r) {
          v0[r] = Act<T>::to_f(sv[b][t + j][mine + r]);
          v1[r] = Act<T>::to_f(sv[b][t + j + 1][mine + r]);
        }
        advance_two(s, k0, k1, q0, q1, v0, v1, tokens[t + j], tokens[t + j + 1], products[(t + j) >> 1], yp[j], yp[j + 1], add0, add1);
#pragma unroll
        for (int r = 0; r < kRowsThread; ++r) add[r] = lane == j ? add0[r] : lane == j + 1 ? add1[r] : add[r];
      }
      float out[kRowsThread];
      const float left = lane & 1 ? tokens[t + lane - 1].a * tokens[t + lane].a : tokens[t + lane].a;
#pragma unroll
      for (int r = 0; r < kRowsThread; ++r) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < o) {
              const bool up = (lane & o) != 0;
              const float keep = up ? yp[j + o][r] : yp[j][r], send = up ? yp[j][r] : yp[j + o][r];
              yp[j][r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        out[r] = tokens[t + lane].qn * fmaf(left, yp[0][r], add[r]);
      }
      if (live) store_two(y + ((int64_t)first + t0 + t + lane) * a.ld_y, out[0], out[1]);
    }
    for (; t < n; ++t) {
      float yp[kRowsThread];
      one(t, yp);
#pragma unroll
      for (int r = 0; r < kRowsThread; ++r) yp[r] = tokens[t].qn * sum8(yp[r]);
      if (live && lane == 0) store_two(y + ((int64_t)first + t0 + t) * a.ld_y, yp[0], yp[1]);
    }
    __syncthreads();  // (the next fetch but one overwrites this buffer)
  }
  each([&](Two* w, int64_t at) { store_four(st + at, w); });
}

// ------------------------------------------------------------------ single tokens

// One token of each sequence: a CTA takes 64 rows of one head's state. Bound by HBM: the state is read and written once,
// everything is asked for before anything is waited for. 256 sequences of 16 heads of 128 x 128: 92 us, 5.8 TB/s.
constexpr int kStepThreads = 256, kStepRows = kStepThreads / kLanes * kRowsThread;
constexpr int kCheckHere = kStepThreads;

template <typename T, int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ DeltaStepArgs a) {
  constexpr int N = DK / kLanes / 2;
  const int i = blockIdx.z, h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int lane = threadIdx.x % kLanes, row = blockIdx.x * kStepRows + (int)threadIdx.x / kLanes * kRowsThread;
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
  Two s[kRowsThread][N], k[N], q[N];
  float v[kRowsThread], y[kRowsThread];
  const T* qp = static_cast<const T*>(a.q) + i * a.ld_q + (int64_t)grp * a.dk;
  const T* kp = static_cast<const T*>(a.k) + i * a.ld_k + (int64_t)grp * a.dk;
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const int at = 16 * c + 4 * lane;
#pragma unroll
    for (int r = 0; r < kRowsThread; ++r) {
      s[r][c] = s[r][c + 1] = two(0.0f, 0.0f);
      if (live && is_slot && !fresh && at < a.dk) four(st + (int64_t)r * a.dk + at, s[r] + c);
    }
  }
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const int at = 16 * c + 4 * lane;
    k[c] = k[c + 1] = q[c] = q[c + 1] = two(0.0f, 0.0f);
    if (at < a.dk) {
      four(kp + at, k + c);
      four(qp + at, q + c);
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
    v[r] = live ? Act<T>::to_f(static_cast<const T*>(a.v)[i * a.ld_v + (int64_t)h * a.dv + row + r]) : 0.0f;
  const float g = a.g ? a.g[(int64_t)i * a.heads + h] : 0.0f, beta = a.beta ? a.beta[(int64_t)i * a.heads + h] : 1.0f;
  if (a.dev_slots) {
    if (a.n <= kCheckHere) {
      const int status = check_batch<kStepThreads>(num, a.n, a.num_slots, mine);
      if (blockIdx.x == 0 && h == 0 && i == 0 && threadIdx.x == 0) *a.dev_status = status;
      if (status != MAMBA2_OK) return;
    } else if (*a.dev_status != MAMBA2_OK) {
      return;
    }
    if (i >= num) return;
  }
  const Token t = token_of(k, q, g, beta, a.scale, a.l2_eps);
  advance(s, k, q, v, t, y);
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r) y[r] = t.qn * sum8(y[r]);
  if (!live) return;
#pragma unroll
  for (int r = 0; r < kRowsThread; ++r)
#pragma unroll
    for (int c = 0; c < N; c += 2)
      if (16 * c + 4 * lane < a.dk) store_four(st + (int64_t)r * a.dk + 16 * c + 4 * lane, s[r] + c);
  if (lane == 0) store_two(static_cast<T*>(a.y) + i * a.ld_y + (int64_t)h * a.dv + row, y[0], y[1]);
}

// Runs f with the padded d_state as a constant.
template <typename F>
cudaError_t with_state(int dk, F f) {
  if (dk <= 32) f(std::integral_constant<int, 32>{});
  else if (dk <= 64) f(std::integral_constant<int, 64>{});
  else if (dk <= 96) f(std::integral_constant<int, 96>{});
  else if (dk <= 128) f(std::integral_constant<int, 128>{});
  else f(std::integral_constant<int, 256>{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_serial(const DeltaArgs& a, mamba2_dtype act, cudaStream_t st) {
  const dim3 grid((a.dv + kSerialRows - 1) / kSerialRows, a.heads, a.tab.n);
  return with_state(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    if (act == MAMBA2_BF16) delta_serial_kernel<__nv_bfloat16, DK><<<grid, kSerialThreads, 0, st>>>(a);
    else delta_serial_kernel<float, DK><<<grid, kSerialThreads, 0, st>>>(a);
  });
}

cudaError_t launch_delta_step(const DeltaStepArgs& a, mamba2_dtype act, cudaStream_t st) {
  if (a.dev_slots && a.n > kCheckHere) {
    const cudaError_t e = launch_check_device_batch(a.dev_slots, a.dev_n, a.n, a.num_slots, a.dev_status, st);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((a.dv + kStepRows - 1) / kStepRows, a.heads, a.n);
  return with_state(a.dk, [&](auto dk) {
    constexpr int DK = decltype(dk)::value;
    if (act == MAMBA2_BF16) delta_step_kernel<__nv_bfloat16, DK><<<grid, kStepThreads, 0, st>>>(a);
    else delta_step_kernel<float, DK><<<grid, kStepThreads, 0, st>>>(a);
  });
}

}  // namespace mamba2
