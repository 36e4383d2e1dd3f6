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
// Two kernels. The first reads the logits, once: a CTA takes a part of a row and leaves its maximum, the sum of
// exp(x - maximum) and its `out` largest logits; a row's order is that of its logits, so the log-sum-exp is not
// needed to choose among them. The second joins a row's parts, forms the values in fp64 and ranks a sequence's
// candidates by counting how many come before each. Bound by HBM, and for few rows by the two launches.
constexpr int kScanThreads = 256, kScanWarps = kScanThreads / 32;
constexpr int kMost = MAMBA2_MAX_BEAMS;  // candidates of a list: one to a lane
constexpr int kPartMin = 2048;           // logits of a part at least: 256 a warp

__device__ __forceinline__ float ex2(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
constexpr float kLog2e = 1.4426950408889634f;

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

// Maximum and sum of exponentials below it; nothing yet is (-infinity, 0).
struct Soft {
  float m, s;
  // n values in one go (a NaN makes the sum NaN, an infinity too)
  template <int n>
  __device__ __forceinline__ void add(const float (&v)[n], float top) {
    const float to = fmaxf(m, top), base = to == -INFINITY ? 0.0f : to;
    if (to > m) s = m == -INFINITY ? s : s * ex2((m - base) * kLog2e);
    m = to;
    const float off = -base * kLog2e;
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < n; ++j) t += ex2(fmaf(v[j], kLog2e, off));
    s += t;
  }
  __device__ __forceinline__ void join(float om, float os) {
    const float to = fmaxf(m, om);
    if (to == -INFINITY) {
      s += os;
      return;
    }
    s = (m == -INFINITY ? s : s * ex2((m - to) * kLog2e)) + (om == -INFINITY ? os : os * ex2((om - to) * kLog2e));
    m = to;
  }
};

struct PartOut {  // of one part of one row
  float* m;
  float* s;
  float* x;  // [out]
  int* at;
};
__host__ __device__ inline size_t part_words(int out) { return 2 + 2 * (size_t)out; }
__device__ __forceinline__ PartOut part_at(void* ws, int64_t i, int out) {
  float* p = static_cast<float*>(ws) + i * (int64_t)part_words(out);
  return {p, p + 1, p + 2, reinterpret_cast<int*>(p + 2 + out)};
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamArgs a, int part) {
  constexpr int V = Vec16<T>::n;
  __shared__ float wm[kScanWarps], wsum[kScanWarps], wx[kScanWarps][kMost];
  __shared__ int wat[kScanWarps][kMost];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.y;
  if (a.finished && a.finished[row]) return;  // (its logits are not candidates)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  // elements before the row's first 16-byte boundary; parts and warps begin whole vectors behind it
  const int head = min(a.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T));
  const int64_t lo = (int64_t)blockIdx.x * part, hi = min((int64_t)a.vocab - head, lo + part);  // behind the head
  const int each = part / kScanWarps;
  const int64_t w0 = lo + (int64_t)warp * each, w1 = min(hi, w0 + each);
  Best best;
  best.clear();
  Soft soft = {-INFINITY, 0.0f};
  auto one = [&](float v, bool in, int index) {  // an element a lane (-infinity where there is none)
    const float u[1] = {in ? v : -INFINITY};
    soft.add(u, u[0]);
    for (uint32_t todo = __ballot_sync(0xffffffffu, u[0] > best.least); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const float c = __shfl_sync(0xffffffffu, u[0], from);
      const int at = __shfl_sync(0xffffffffu, index, from);
      if (c > best.least) best.add(c, at, a.out, lane);
    }
  };
  if (blockIdx.x == 0 && warp == 0 && head > 0) one(lane < head ? Act<T>::to_f(p[lane]) : 0.0f, lane < head, lane);
  p += head;
  int64_t i = w0;
  constexpr int kAhead = 4;  // vectors of a lane that are on their way
  auto vector = [&](const float (&v)[V], int64_t from) {
    float top = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, v[j]);
    soft.add(v, top);
    for (uint32_t todo = __ballot_sync(0xffffffffu, top > best.least); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float c = __shfl_sync(0xffffffffu, v[j], l);
        if (c > best.least) best.add(c, (int)(head + from + l * V + j), a.out, lane);
      }
    }
  };
  for (; i + kAhead * 32 * V <= w1; i += kAhead * 32 * V) {
    float v[kAhead][V];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) Vec16<T>::load_stream(p + i + (u * 32 + lane) * V, v[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) vector(v[u], i + u * 32 * V);
  }
  for (; i + 32 * V <= w1; i += 32 * V) {
    float v[V];
    Vec16<T>::load_stream(p + i + lane * V, v);
    vector(v, i);
  }
  for (; i < w1; i += 32) one(i + lane < w1 ? Act<T>::to_f(p[i + lane]) : 0.0f, i + lane < w1, (int)(head + i + lane));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    soft.join(__shfl_xor_sync(0xffffffffu, soft.m, o), __shfl_xor_sync(0xffffffffu, soft.s, o));
  wx[warp][lane] = best.x;
  wat[warp][lane] = best.at;
  if (lane == 0) {
    wm[warp] = soft.m;
    wsum[warp] = soft.s;
  }
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < kScanWarps; ++w) {
    soft.join(wm[w], wsum[w]);
    const float x = wx[w][lane];
    const int at = wat[w][lane];
    for (int r = 0; r < a.out; ++r) {
      const float c = __shfl_sync(0xffffffffu, x, r);
      if (!(c > best.least)) break;
      best.add(c, __shfl_sync(0xffffffffu, at, r), a.out, lane);
    }
  }
  const PartOut o = part_at(a.ws, row * gridDim.x + blockIdx.x, a.out);
  if (lane == 0) {
    *o.m = soft.m;
    *o.s = soft.s;
  }
  if (lane < a.out) {
    o.x[lane] = best.x;
    o.at[lane] = best.at;
  }
}

// A warp a beam, a CTA a sequence.
__global__ void __launch_bounds__(32 * kMost) beam_rank_kernel(const __grid_constant__ BeamArgs a, int parts) {
  __shared__ double value[kMost * kMost];
  __shared__ int token[kMost * kMost];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int beam = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * a.beams + beam;
  const float score = a.scores[row];
  const bool done = a.finished && a.finished[row];
  Best best;
  best.clear();
  double total = 0.0, m = -INFINITY;
  if (!done) {
    for (int p = lane; p < parts; p += 32) m = fmax(m, (double)*part_at(a.ws, row * parts + p, a.out).m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int p = lane; p < parts; p += 32) {
      const PartOut q = part_at(a.ws, row * parts + p, a.out);
      const float pm = *q.m, ps = *q.s;
      total += pm == -INFINITY ? (double)ps : (double)ps * exp((double)pm - m);  // (an empty part's sum is 0, or NaN)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    for (int p = 0; p < parts; ++p) {  // ascending, so ties stay in order
      const PartOut q = part_at(a.ws, row * parts + p, a.out);
      const float x = lane < a.out ? q.x[lane] : -INFINITY;
      const int at = lane < a.out ? q.at[lane] : -1;
      for (int r = 0; r < a.out; ++r) {
        const float c = __shfl_sync(0xffffffffu, x, r);
        if (!(c > best.least)) break;
        best.add(c, __shfl_sync(0xffffffffu, at, r), a.out, lane);
      }
    }
  }
  const double lse = m + log(total);
  double v = -INFINITY;
  int at = -1;
  if (done) {
    if (lane == 0) {
      v = score;
      at = a.eos;
    }
  } else if (lane < a.out && best.x > -INFINITY) {
    v = (double)score + ((double)best.x - lse);
    at = best.at;
  }
  // what is not a number, or -infinity, is no better than any token: the row goes on with its lowest ones that are not
  // in the list already (a dead row's list counts as empty)
  if (!(v > -INFINITY)) at = -1;
  const int real = __popc(__ballot_sync(0xffffffffu, at >= 0));
  if (lane >= real) {  // the (lane - real + 1)-th token that is not among the first `real`
    v = -INFINITY;
    at = -1;
  }
  int free_at = lane - real;
  for (int pass = 0; pass < real; ++pass) {  // the number of listed tokens at or below the candidate settles it
    int below = 0;
    for (int r = 0; r < real; ++r) below += __shfl_sync(0xffffffffu, at, r) <= free_at ? 1 : 0;
    free_at = lane - real + below;
  }
  if (lane >= real && lane < a.out && free_at < a.vocab) at = free_at;
  if (lane < a.out) {
    value[beam * a.out + lane] = v;
    token[beam * a.out + lane] = at;
  }
  __syncthreads();
  const int all = a.beams * a.out;
  for (int c = threadIdx.x; c < all; c += blockDim.x) {
    const double mine = value[c];
    const int t = token[c], b = c / a.out;
    if (t < 0) continue;  // (a vocabulary smaller than `out`)
    int before = 0;
    for (int o = 0; o < all; ++o) {
      const int ot = token[o], ob = o / a.out;
      const double ov = value[o];
      before += ot >= 0 && (ov > mine || (ov == mine && (ob < b || (ob == b && ot < t)))) ? 1 : 0;
    }
    if (before < a.out) {
      const int64_t to = (int64_t)blockIdx.x * a.out + before;
      a.scores_out[to] = (float)mine;
      a.parents[to] = b;
      a.tokens[to] = t;
      if (a.finished_out)
        a.finished_out[to] = (a.finished && a.finished[(int64_t)blockIdx.x * a.beams + b]) || t == a.eos ? 1 : 0;
    }
  }
}

// Parts of a row: as many as give every SM four CTAs, of kPartMin logits at least.
int beam_parts(int64_t rows, int vocab) {
  const int64_t want = std::max<int64_t>(1, 4 * (int64_t)device_sm_count() / std::max<int64_t>(rows, 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, (vocab + kPartMin - 1) / kPartMin));
}
int part_size(int parts, int vocab) {  // whole vectors of every warp
  const int64_t unit = kScanWarps * 32 * 8;
  return (int)(((int64_t)vocab + parts * unit - 1) / (parts * unit) * unit);
}

// ------------------------------------------------------------------ reordering

// A CTA takes kReorderTile bytes of the slots of one sequence's beams, a thread the same bytes of every beam: it has
// read what it moves before it writes, so beams may take one another's places in any order. Bound by HBM: each state
// that moves is read and written once (one that several beams take comes from L1 after the first).
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

cudaError_t start(const void* kernel, dim3 grid, int threads, void** args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
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

size_t beam_workspace(int64_t rows, int32_t out, int32_t vocab) {
  return (size_t)rows * beam_parts(rows, vocab) * part_words(out) * 4;
}

cudaError_t launch_beam_select(const BeamArgs& args, mamba2_dtype act, cudaStream_t st) {
  BeamArgs a = args;
  const int64_t rows = (int64_t)a.batch * a.beams;
  int parts = beam_parts(rows, a.vocab), part = part_size(parts, a.vocab);
  const void* scan = act == MAMBA2_BF16 ? reinterpret_cast<const void*>(beam_scan_kernel<__nv_bfloat16>)
                                        : reinterpret_cast<const void*>(beam_scan_kernel<float>);
  void* first[] = {&a, &part};
  cudaError_t e = start(scan, dim3((unsigned)parts, (unsigned)rows), kScanThreads, first, st);
  if (e != cudaSuccess) return e;
  void* second[] = {&a, &parts};
  return start(reinterpret_cast<const void*>(beam_rank_kernel), dim3((unsigned)a.batch), 32 * a.beams, second, st);
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
