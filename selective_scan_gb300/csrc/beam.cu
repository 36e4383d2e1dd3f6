// Beam search over recurrent states (beam.h): selection over beams and vocabulary, and the reordering of state pools.
#include <algorithm>

#include "../../include/beam.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {
namespace {

#include "batch_check.cuh"

// ------------------------------------------------------------------ selection
//
// Two kernels. The first reads the logits, once: a CTA takes a part of a row into registers and leaves its maximum, the
// sum of exp(x - maximum) and its `out` largest logits; a row's order is that of its logits, so the log-sum-exp is not
// needed to choose among them. The second joins a row's parts, forms the values in fp64 and ranks a sequence's
// candidates by counting how many come before each.
//
// In a part, the threads fall into 8, 16 or 32 groups (at least `out` of them) by their lane, and the least of the
// groups' maxima has `out` logits at or above it: a bound below which nothing counts. The few logits that reach it (22,
// 54 or 130 of a part in random order) are collected and ranked by counting. Where more reach it than are held (many
// ties), the warps take them one by one instead.
//
// The first is bound by issue and latency between a part's loads and its end: 512 rows of 131 072 bf16 logits 29 us,
// 4.6 TB/s. The second waits for its own steps: 64 sequences of 8 beams about 5 us behind the first.
constexpr int kScanThreads = 256, kScanWarps = kScanThreads / 32;
constexpr int kMost = MAMBA2_MAX_BEAMS;  // candidates of a list: one to a lane
constexpr int kHeld = 1024;              // logits that are collected
// 16-byte vectors of a thread. Half as many doubles the parts that a row's lists are joined from, and is no faster even
// where the parts are fewer than the SMs (scan and join, us, of 8, 4 and 2 vectors: 4 rows of 131 072 fp32 logits
// 3.6 + 6.8, 3.5 + 10.1, 3.6 + 14.5; 80 of 32 001 5.2 + 6.7, 6.1 + 7.8, 8.3 + 13.6; 512 of 131 072 bf16 41 + 13, 62 + 16,
// 87 + 18).
constexpr int kVectors = 8;

__device__ __forceinline__ float ex2(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
constexpr float kLog2e = 1.4426950408889634f;

struct Two {  // of packed instructions
  unsigned long long v;
  __device__ __forceinline__ Two(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
// sum += exp(x + off). (One product and sum, x log2(e) + off log2(e), would round what all terms share: 4e-5 of the sum at
// logits of 1 000, all of it above 1e10.)
__device__ __forceinline__ void add_exp(Two& sum, Two x, Two off) {
  asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(x.v) : "l"(off.v));
  asm volatile("mul.rn.f32x2 %0, %0, %1;" : "+l"(x.v) : "l"(Two(kLog2e, kLog2e).v));
  const float2 f = x.get();
  const Two e(ex2(f.x), ex2(f.y));
  asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(sum.v) : "l"(e.v));
}

// The largest logits that a warp has met, a lane each, descending, equal ones by index: lane r holds the r-th. What it
// is offered comes with ascending indices, so an equal one always goes behind. -infinity is never taken.
struct Best {
  float x, least;  // least: of the `out`-th, in every lane
  int at;
  __device__ __forceinline__ void clear() {
    x = least = -INFINITY;
    at = -1;
  }
  __device__ __forceinline__ void add(float v, int index, int out, int lane) {  // v > least, the same for the warp
    const int pos = __popc(__ballot_sync(0xffffffffu, x >= v));
    const float px = __shfl_up_sync(0xffffffffu, x, 1);
    const int pa = __shfl_up_sync(0xffffffffu, at, 1);
    if (lane > pos) {
      x = px;
      at = pa;
    }
    if (lane == pos) {
      x = v;
      at = index;
    }
    least = __shfl_sync(0xffffffffu, x, out - 1);
  }
};

struct PartOut {  // of one part of one row
  float* m;
  float* s;
  float* x;  // [out], descending; -infinity behind the last
  int* at;
};
__host__ __device__ inline size_t part_words(int out) { return 2 + 2 * (size_t)out; }
__device__ __forceinline__ PartOut part_at(void* ws, int64_t i, int out) {
  float* p = static_cast<float*>(ws) + i * (int64_t)part_words(out);
  return {p, p + 1, p + 2, reinterpret_cast<int*>(p + 2 + out)};
}
template <typename T>
constexpr int kPartLogits = kScanThreads * kVectors * Vec16<T>::n;

// An order-preserving image of a float (-0 as 0), and with it a logit and its index as one number: larger is better.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ uint64_t key_of(float v, int index) { return (uint64_t)ordered(v) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float key_logit(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ int64_t ordered(double v) {  // (v is a number or an infinity)
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ (b < 0 ? 0x7fffffffffffffffll : 0);
}
__device__ __forceinline__ double unordered(int64_t k) { return __longlong_as_double(k ^ (k < 0 ? 0x7fffffffffffffffll : 0)); }

// A thread's vector of logits and their maximum.
template <typename T> struct Logits;
template <> struct Logits<float> {
  static constexpr int n = 4;
  float v[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
  __device__ __forceinline__ void load_some(const float* p, int64_t left) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : -INFINITY;
  }
  __device__ __forceinline__ float at(int j) const { return v[j]; }
  __device__ __forceinline__ float top() const { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }  // (passes over a NaN)
  // sets the bits of vector u's logits that reach `least`: element j's is 4 u + j
  __device__ __forceinline__ void reach(float least, int u, uint32_t (&bits)[2]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v[j] >= least) bits[0] |= 1u << (4 * u + j);
  }
  __device__ static __forceinline__ int element(int half, int bit) { return bit; }  // 4 u + j of a bit
};
template <> struct Logits<__nv_bfloat16> {
  static constexpr int n = 8;
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int64_t left) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = 2 * j < left ? *reinterpret_cast<const uint16_t*>(p + 2 * j) : 0xff80u;
      const uint32_t hi = 2 * j + 1 < left ? *reinterpret_cast<const uint16_t*>(p + 2 * j + 1) : 0xff80u;
      w[j] = hi << 16 | lo;
    }
  }
  __device__ __forceinline__ float at(int j) const { return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16); }
  __device__ __forceinline__ float top() const {
    auto h = [&](int j) { return *reinterpret_cast<const __nv_bfloat162*>(&w[j]); };
    const __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  // word 4 u + i, of elements 2 i and 2 i + 1, has bits (4 u + i) % 16 and that + 16 of bits[(4 u + i) / 16]
  __device__ __forceinline__ void reach(float least, int u, uint32_t (&bits)[2]) const {
    const __nv_bfloat162 l = __float2bfloat162_rn(least);  // (a logit itself, or the lowest number)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 4 * u + i;
      bits[k >> 4] |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), l) & (0x00010001u << (k & 15));
    }
  }
  __device__ static __forceinline__ int element(int half, int bit) { return 2 * (16 * half + (bit & 15)) + (bit >> 4); }
};

// The part's last vector may pass the row's end, and the row's first logits up to a 16-byte boundary (`head`) are part
// 0's besides.
template <typename T>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int V = Logits<T>::n;
  __shared__ __align__(16) uint64_t key[kHeld + 2];
  __shared__ float tops[kScanWarps][32], wsum[kScanWarps];
  __shared__ int held;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.y;
  if (a.finished && a.finished[row]) return;  // (its logits are not candidates)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  const int head = min(a.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
  const int rest = a.vocab - head;
  const int64_t lo = (int64_t)blockIdx.x * kPartLogits<T>;
  auto first = [&](int u) { return lo + ((int64_t)u * kScanThreads + threadIdx.x) * V; };  // behind the head
  Logits<T> x[kVectors];
  auto load = [&](Logits<T>& to, int u) {
    if (first(u) + V <= rest) to.load(p + head + first(u));
    else to.load_some(p + head + first(u), rest - first(u));
  };
  if (lo + kPartLogits<T> <= rest) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u].load(p + head + first(u));
  } else {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) load(x[u], u);
  }
  // a logit of the head (warp 0's lanes)
  const float extra = blockIdx.x == 0 && (int)threadIdx.x < head ? Act<T>::to_f(p[threadIdx.x]) : -INFINITY;
  float top = extra;
#pragma unroll
  for (int u = 0; u < kVectors; ++u) top = fmaxf(top, x[u].top());
  if (!(top > -INFINITY)) top = -INFINITY;  // (nothing but NaNs)
  tops[warp][lane] = top;
  if (threadIdx.x == 0) held = 0;
  __syncthreads();
  float group = tops[0][lane];
#pragma unroll
  for (int w = 1; w < kScanWarps; ++w) group = fmaxf(group, tops[w][lane]);
  if (a.out <= 16) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, 16));
  if (a.out <= 8) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, 8));
  const float m = unordered(__reduce_max_sync(0xffffffffu, ordered(group)));
  float least = unordered(__reduce_min_sync(0xffffffffu, ordered(group)));
  auto collect = [&](float v, int index) {
    const int to = atomicAdd(&held, 1);
    if (to < kHeld) key[to] = key_of(v, index);
  };
  if (least == -INFINITY) least = sizeof(T) == 4 ? -3.402823466e38f : -3.389531390e38f;  // the type's lowest number
  if (top >= least) {  // which of this thread's logits they are; they are few, and read again
    if (extra >= least) collect(extra, (int)threadIdx.x);
    uint32_t bits[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u].reach(least, u, bits);
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
#pragma unroll 1
      for (uint32_t todo = bits[half]; todo; todo &= todo - 1) {
        const int e = Logits<T>::element(half, __ffs(todo) - 1), at = (int)(first(e / V) + e % V);
        collect(Act<T>::to_f(p[head + at]), head + at);
      }
  }
  const float off = m == -INFINITY ? 0.0f : -m;
  Two part(ex2((extra + off) * kLog2e), 0.0f);
#pragma unroll
  for (int u = 0; u < kVectors; ++u)
#pragma unroll
    for (int j = 0; j < V; j += 2) add_exp(part, {x[u].at(j), x[u].at(j + 1)}, {off, off});
  float sum = part.get().x + part.get().y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) wsum[warp] = sum;
  __syncthreads();
  const PartOut o = part_at(a.ws, row * gridDim.x + blockIdx.x, a.out);
  int n = held;
  if (n > kHeld) {  // warp by warp, in the order of their indices: each its own logits, a vector of all lanes at a time
    Best best;
    best.clear();
    for (uint32_t todo = __ballot_sync(0xffffffffu, extra > best.least); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const float c = __shfl_sync(0xffffffffu, extra, from);
      if (c > best.least) best.add(c, from, a.out, lane);
    }
#pragma unroll 1
    for (int u = 0; u < kVectors; ++u) {  // (read again, so that they need not be held until here)
      Logits<T> again;
      load(again, u);
      for (uint32_t todo = __ballot_sync(0xffffffffu, again.top() > best.least); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float c = __shfl_sync(0xffffffffu, again.at(j), from);
          if (c > best.least)
            best.add(c, (int)(head + lo + ((int64_t)u * kScanThreads + warp * 32 + from) * V + j), a.out, lane);
        }
      }
    }
    __syncthreads();  // everyone has read `held`
    if (threadIdx.x == 0) held = 0;
    __syncthreads();
    if (best.at >= 0) key[atomicAdd(&held, 1)] = key_of(best.x, best.at);
    __syncthreads();
    n = held;
  }
  if (threadIdx.x == 0) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) total += wsum[w];
    *o.m = m;
    *o.s = total;
    key[n] = key[n + 1] = 0;  // (no key is as small)
  }
  for (int e = threadIdx.x + n; e < a.out; e += kScanThreads) {  // fewer logits than are asked for
    o.x[e] = -INFINITY;
    o.at[e] = -1;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kScanThreads) {
    const uint64_t mine = key[e];
    int before = 0;
#pragma unroll 4
    for (int c = 0; c < n; c += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(key + c);
      before += (two.x > mine ? 1 : 0) + (two.y > mine ? 1 : 0);
    }
    if (before < a.out) {
      o.x[before] = key_logit(mine);
      o.at[before] = key_index(mine);
    }
  }
}

// A warp a beam, a CTA a sequence. kNear entries of a part's list are held in shared memory; it is rare that more of one
// are among the largest of the row.
constexpr int kNear = 8;
constexpr int kRankSmem = 31 * kNear * (int)sizeof(uint64_t);  // of a beam

__global__ void __launch_bounds__(32 * kMost) beam_rank_kernel(const __grid_constant__ BeamArgs a, int parts) {
  extern __shared__ __align__(16) uint64_t near_keys[];  // [beams][31][kNear]
  __shared__ int64_t value[kMost * kMost];  // (compared as integers: a warp takes 16 cycles to compare doubles)
  __shared__ int token[kMost * kMost];
  __shared__ int before[kMost * kMost];
  __shared__ double lses[kMost];
  __shared__ float tops[kMost], totals[kMost];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int beam = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * a.beams + beam;
  const float score = a.scores[row];
  const bool done = a.finished && a.finished[row];
  uint64_t* near = near_keys + beam * (31 * kNear);
  const int held = min(a.out, kNear);
  uint64_t list = 0;  // the row's `lane`-th largest logit; 0: none
  float m = -INFINITY, total = 0.0f;
  if (!done) {
    // parts 31 at a time, a lane each, merged with what the row has so far: the largest head is taken `out` times
    for (int p0 = 0; p0 < parts; p0 += 31) {
      const int count = min(31, parts - p0);
      auto entry = [&](int p, int e) {
        const PartOut q = part_at(a.ws, row * parts + p0 + p, a.out);
        const int at = q.at[e];
        const float x = q.x[e];
        return at >= 0 ? key_of(x, at) : 0;
      };
      const bool mine = lane < count;
      const PartOut q = part_at(a.ws, row * parts + p0 + (mine ? lane : 0), a.out);
      const float pm = mine ? *q.m : -INFINITY, ps = mine ? *q.s : 0.0f;
      for (int e = lane; e < count * held; e += 32) near[e / held * kNear + e % held] = entry(e / held, e % held);
      __syncwarp();
      float to = pm;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
      to = fmaxf(to, m);
      float s = pm == -INFINITY ? ps : ps * ex2((pm - to) * kLog2e);  // (an empty part's sum is 0, or NaN)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      total = (m == -INFINITY ? total : total * ex2((m - to) * kLog2e)) + s;
      m = to;
      // (what the row has so far stands in lane 31)
      const uint64_t so_far = list;
      const uint64_t first = __shfl_sync(0xffffffffu, so_far, 0);
      uint64_t head = mine ? near[lane * kNear] : lane == 31 ? first : 0;
      int next = 1;
      for (int r = 0; r < a.out; ++r) {
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32));
        const uint32_t low = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32) == hi ? (uint32_t)head : 0u);
        const uint64_t best = (uint64_t)hi << 32 | low;
        if (lane == r) list = best;
        const int from = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
        const uint64_t follow = __shfl_sync(0xffffffffu, so_far, min(__shfl_sync(0xffffffffu, next, 31), 31));
        if (lane == from && best != 0) {
          if (lane == 31) head = next < a.out ? follow : 0;
          else head = next >= a.out ? 0 : next < kNear ? near[lane * kNear + next] : entry(lane, next);
          ++next;
        }
      }
      __syncwarp();
    }
  }
  for (int c = threadIdx.x; c < a.beams * a.out; c += blockDim.x) before[c] = 0;
  if (lane == 0) {
    tops[beam] = m;
    totals[beam] = total;
  }
  __syncthreads();
  if (beam == 0 && lane < a.beams) lses[lane] = (double)tops[lane] + log((double)totals[lane]);
  __syncthreads();
  const double lse = lses[beam];
  double v = -INFINITY;
  int at = -1;
  if (done) {
    if (lane == 0) {
      v = score;
      at = a.eos;
    }
  } else if (list != 0 && lane < a.out) {
    v = (double)score + ((double)key_logit(list) - lse);
    at = key_index(list);
  }
  // what is not a number, or -infinity, is no better than any token: the row goes on with its lowest ones that are not
  // in the list already (a dead row's list counts as empty)
  if (!(v > -INFINITY)) at = -1;
  const int real = __popc(__ballot_sync(0xffffffffu, at >= 0));
  if (lane >= real) v = -INFINITY;
  int free_at = lane - real;
  for (int pass = 0; pass < real && real < a.out; ++pass) {  // the number of listed tokens at or below it settles it
    int below = 0;
    for (int r = 0; r < real; ++r) below += __shfl_sync(0xffffffffu, at, r) <= free_at ? 1 : 0;
    free_at = lane - real + below;
  }
  if (lane >= real) at = lane < a.out && free_at < a.vocab ? free_at : -1;
  if (lane < a.out) {
    value[beam * a.out + lane] = ordered(v);
    token[beam * a.out + lane] = at;
  }
  __syncthreads();
  // Of each beam's list, which is in order, what comes before a candidate is counted by bisection: a thread a candidate
  // and a list.
  const int all = a.beams * a.out;
  for (int i = threadIdx.x; i < all * a.beams; i += blockDim.x) {
    const int c = i % all, ob = i / all, b = c / a.out;
    const int64_t mine = value[c];
    auto ahead = [&](int r) {  // is entry r of that list there, and before this candidate?
      if (r >= a.out || token[ob * a.out + r] < 0) return false;
      const int64_t ov = value[ob * a.out + r];
      return ov > mine || (ov == mine && ob < b);
    };
    int n = 0;
#pragma unroll
    for (int step = kMost / 2; step > 0; step >>= 1)
      if (ahead(n + step - 1)) n += step;
    n += ahead(n) ? 1 : 0;  // (31 is the most that the steps add up to)
    atomicAdd(&before[c], ob == b ? c - b * a.out : n);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < all; c += blockDim.x) {
    const int t = token[c], b = c / a.out;
    if (t < 0 || before[c] >= a.out) continue;  // (no token: a vocabulary smaller than `out`)
    const int64_t to = (int64_t)blockIdx.x * a.out + before[c];
    a.scores_out[to] = (float)unordered(value[c]);
    a.parents[to] = b;
    a.tokens[to] = t;
    if (a.finished_out)
      a.finished_out[to] = (a.finished && a.finished[(int64_t)blockIdx.x * a.beams + b]) || t == a.eos ? 1 : 0;
  }
}

// Parts of a row.
int beam_parts(int vocab, mamba2_dtype act) {
  const int64_t part = act == MAMBA2_F32 ? kPartLogits<float> : kPartLogits<__nv_bfloat16>;
  return (int)((vocab + part - 1) / part);
}

// ------------------------------------------------------------------ reordering

// A CTA takes kReorderTile bytes of the slots of one sequence's beams, a thread the same bytes of every beam: it has
// read what it moves before it writes, so beams may take one another's places in any order. Bound by HBM: each state
// that moves is read and written once (one that several beams take comes from L1 after the first): 16 sequences of 4
// beams, 12 pools of 1 MB a slot, 163 to 171 us, 6.3 to 6.6 TB/s.
constexpr int kReorderThreads = 256;
constexpr int kReorderCheck = kReorderThreads;

template <typename U, int kBeams>
__device__ __forceinline__ void move_bytes(char* pool, int64_t bytes, int64_t begin, int64_t end, int beams,
                                           const int* slot, const int* parent) {
  for (int64_t at = begin + (int64_t)threadIdx.x * sizeof(U); at < end; at += (int64_t)kReorderThreads * sizeof(U)) {
    U v[kBeams];
#pragma unroll
    for (int j = 0; j < kBeams; ++j)
      if (j < beams && parent[j] != j) v[j] = *reinterpret_cast<const U*>(pool + slot[parent[j]] * bytes + at);
#pragma unroll
    for (int j = 0; j < kBeams; ++j)
      if (j < beams && parent[j] != j) *reinterpret_cast<U*>(pool + slot[j] * bytes + at) = v[j];
  }
}

template <int kBeams>
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int slot[kBeams], parent[kBeams];
  const int b = blockIdx.y, n = a.batch * a.beams, me = threadIdx.x;
  if (n <= kReorderCheck) {
    const int mine = me < n ? a.slots[me] : 0, up = me < n ? a.parents[me] : 0;
    int status = check_batch<kReorderThreads>(n, n, a.num_slots, mine);
    const int off = __syncthreads_or(up < 0 || up >= a.beams ? 1 : 0);
    if (status == MAMBA2_OK && off) status = MAMBA2_ERR_INVALID_ARGUMENT;
    if (blockIdx.x == 0 && b == 0 && me == 0) *a.status = status;
    if (status != MAMBA2_OK) return;
  } else if (*a.status != MAMBA2_OK) {
    return;
  }
  if (me < a.beams) {
    slot[me] = a.slots[b * a.beams + me];
    parent[me] = a.parents[b * a.beams + me];
  }
  __syncthreads();
  if (a.tile[a.num_pools] == 0) return;  // (launched for the check alone)
  int lo = 0, hi = a.num_pools - 1;
  while (lo < hi) {  // the pool that this tile is of
    const int mid = (lo + hi + 1) >> 1;
    if (a.tile[mid] <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  char* pool = a.pool[lo];
  const int64_t bytes = a.bytes[lo], begin = (int64_t)((int)blockIdx.x - a.tile[lo]) * kReorderTile;
  const int64_t end = min(bytes, begin + kReorderTile);
  const uint64_t odd = (reinterpret_cast<uintptr_t>(pool) | (uint64_t)bytes) & 15;
  if (odd == 0) move_bytes<uint4, kBeams>(pool, bytes, begin, end, a.beams, slot, parent);
  else if ((odd & 3) == 0) move_bytes<uint32_t, kBeams>(pool, bytes, begin, end, a.beams, slot, parent);
  else move_bytes<uint8_t, kBeams>(pool, bytes, begin, end, a.beams, slot, parent);
}

// The check of more slots than a CTA has threads.
__global__ void __launch_bounds__(MAMBA2_MAX_SEQS) reorder_check_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int seen[MAMBA2_MAX_SEQS];
  const int n = a.batch * a.beams, me = threadIdx.x;
  const int mine = me < n ? a.slots[me] : -1, up = me < n ? a.parents[me] : 0;
  seen[me] = mine;
  const int range = __syncthreads_or(me < n && (mine < 0 || mine >= a.num_slots) ? 1 : 0);
  int twice = 0;
  if (me < n)
    for (int j = 0; j < me; ++j) twice |= seen[j] == mine ? 1 : 0;
  twice = __syncthreads_or(twice);
  const int off = __syncthreads_or(up < 0 || up >= a.beams ? 1 : 0);
  if (me == 0)
    *a.status = range ? MAMBA2_ERR_SLOT_OUT_OF_RANGE : twice ? MAMBA2_ERR_SLOT_SHARED
                : off ? MAMBA2_ERR_INVALID_ARGUMENT : MAMBA2_OK;
}

cudaError_t start(const void* kernel, dim3 grid, int threads, size_t smem, void** args, cudaStream_t st) {
  if (smem > 30 * 1024) {  // (one value for every call: another thread's may be between this and its launch)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRankSmem * kMost);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

// (of fp32 logits, whose parts are the more)
size_t beam_workspace(int64_t rows, int32_t out, int32_t vocab) {
  return (size_t)rows * beam_parts(vocab, MAMBA2_F32) * part_words(out) * 4;
}

cudaError_t launch_beam_select(const BeamArgs& args, mamba2_dtype act, cudaStream_t st) {
  BeamArgs a = args;
  const int64_t rows = (int64_t)a.batch * a.beams;
  int parts = beam_parts(a.vocab, act);
  const void* scan = act == MAMBA2_BF16 ? reinterpret_cast<const void*>(beam_scan_kernel<__nv_bfloat16>)
                                        : reinterpret_cast<const void*>(beam_scan_kernel<float>);
  void* first[] = {&a};
  cudaError_t e = start(scan, dim3((unsigned)parts, (unsigned)rows), kScanThreads, 0, first, st);
  if (e != cudaSuccess) return e;
  void* second[] = {&a, &parts};
  return start(reinterpret_cast<const void*>(beam_rank_kernel), dim3((unsigned)a.batch), 32 * a.beams,
               (size_t)a.beams * kRankSmem, second, st);
}

cudaError_t launch_reorder(const ReorderArgs& a, cudaStream_t st) {
  if (a.batch * a.beams > kReorderCheck) {
    reorder_check_kernel<<<1, MAMBA2_MAX_SEQS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)std::max(1, a.tile[a.num_pools]), (unsigned)a.batch);
  if (a.beams <= 4) reorder_kernel<4><<<grid, kReorderThreads, 0, st>>>(a);
  else if (a.beams <= 8) reorder_kernel<8><<<grid, kReorderThreads, 0, st>>>(a);
  else if (a.beams <= 16) reorder_kernel<16><<<grid, kReorderThreads, 0, st>>>(a);
  else reorder_kernel<32><<<grid, kReorderThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mamba2
