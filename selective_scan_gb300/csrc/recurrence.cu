// Gated recurrence (block.h): h_t = f_t h_{t-1} + k_t x_t per channel, with
// f = lo + (1 - lo) sigmoid(gate) and k = 1 - f, over packed runs; its backward pass
// and its single-token step. All of them are bound by HBM: two exponentials' worth of
// arithmetic for every 6 (forward) or 10 (backward) bytes in bf16.
//
// One pass over the data, split over time. A step of the recurrence is the affine map
// h -> f h + b, and maps compose: (A, B) after (A', B') is (A A', A B' + B). A tile is one
// chunk of MAMBA2_RECURRENCE_CHUNK = 128 tokens by 128 bytes of channels; eight warps take
// 16 tokens each, a lane 4 bytes of channels. Per tile:
//   1. each warp scans its tokens from zero, keeping h_t and the product of the f's in
//      registers, and posts its map; the eight maps compose to the tile's
//   2. the tile publishes its map in the workspace; a ninth warp meanwhile fetches what
//      precedes the tile and folds it into the state that enters it
//   3. each warp adds (product of f's) x (its own entering state) to its tokens and stores
// Inputs stream through a ring in shared memory by cp.async: a warp copies only the rows
// that it will read, so the copies need no barrier, and those of the next tiles are in
// flight while a tile waits for its predecessors.
//
// What precedes chunk l of a run, the same for any timing (so results repeat bit for bit):
// every 16th chunk (0, 16, 32, ...) publishes the state after it, the others their maps.
// Chunk l takes the state after chunk 16 floor((l - 1) / 16) and folds the maps of the
// chunks between in order: maps are published without waiting for anything, so the
// serial part is one hop every 2 048 tokens. Chunk 0 alone reads the pool, so the run's last
// chunk may overwrite the slot.
//
// Tiles are taken by ticket in an order in which a tile's predecessors come first, so a
// waiting tile's predecessors are always held by CTAs that run. Waits are bounded; one that
// gives up raises an abort flag in the workspace that ends every other wait, and is counted
// in g_recurrence_timeouts.
//
// The backward pass runs the same machinery from the end: with R_t = f_t (dy_t + R_{t+1})
// the map of a token is R -> f R + f dy. A tile recomputes its states from the checkpoint
// that the forward pass kept (4 bytes per 128 tokens and channel instead of reading y, and
// unrounded), keeps each token's gate as the smaller of sigmoid(g) and sigmoid(-g) with
// the sign of g (the other is one minus it, to the last digit), and makes dx and dgate in
// one more sweep. dlower is summed per tile and then over the tiles, in order.
#include "../../include/block.h"
#include "common.cuh"

#include <algorithm>

namespace mamba2 {

__device__ unsigned int g_recurrence_timeouts = 0;

namespace {

constexpr int kChunkR = MAMBA2_RECURRENCE_CHUNK;
constexpr int kWarps = 8;                      // that scan; one more looks back
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kTok = kChunkR / kWarps;         // tokens of a warp
constexpr int kGroup = 16;                     // chunks between two published states
constexpr int kInfos = 4;
constexpr uint32_t kPollLimit = 1u << 21;      // polls before giving up (seconds)

// A lane's channels: 4 bytes of them.
template <typename T> constexpr int kCh = 4 / (int)sizeof(T);
template <typename T> constexpr int kTileCh = 32 * kCh<T>;

// Row of a staged matrix: 32 words, or 33 where rows start between two words.
template <bool kVec> constexpr int kPitch = kVec ? 128 : 132;

// sigmoid(g) and sigmoid(-g), each with its own digits: with e = exp(-|g|) they are
// 1 / (1 + e) and e / (1 + e), in the order that g's sign gives. small: the second.
__device__ __forceinline__ float small_sigmoid(float g) {
  const float e = __expf(-fabsf(g));
  return __fdividef(e, 1.0f + e);
}
__device__ __forceinline__ void sigmoids(float g, float& up, float& down) {
  const float s = small_sigmoid(g), r = 1.0f - s;
  up = g >= 0.0f ? r : s;
  down = g >= 0.0f ? s : r;
}

template <typename T>
__device__ __forceinline__ void unpack_word(uint32_t w, float (&v)[kCh<T>]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w);
  } else {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes16) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(n) : "memory"); }

// Is the first of this row's channels in the upper half of its word? (The word is inside the
// allocation all the same: allocations begin and end on words.)
template <typename T>
__device__ __forceinline__ int odd_start(const T* row) {
  return sizeof(T) == 2 ? (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 1) : 0;
}

// This warp's rows [r0, r0 + nt) of the tile at `tile` (row stride ld, m channels from there) into dst.
template <typename T, bool kVec>
__device__ __forceinline__ void load_rows(uint32_t dst, const T* tile, int64_t ld, int r0, int nt, int m, int lane) {
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kTok / 4; ++i) {
      const int r = 4 * i + (lane >> 3), c = lane & 7;
      const int bytes = min(16, m * (int)sizeof(T) - 16 * c);
      if (r < nt && bytes > 0)
        cp_async(dst + (uint32_t)((r0 + r) * 128 + 16 * c), tile + (int64_t)(r0 + r) * ld + c * (16 / (int)sizeof(T)), bytes);
    }
  } else {
    for (int r = 0; r < nt; ++r) {
      const T* row = tile + (int64_t)(r0 + r) * ld;
      const int odd = odd_start(row);
      const int words = (m * (int)sizeof(T) + 2 * odd + 3) / 4;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(row - odd);
      const uint32_t d = dst + (uint32_t)((r0 + r) * 132);
      if (lane < words) cp_async4(d + 4 * lane, src + lane);
      if (lane == 0 && words > 32) cp_async4(d + 128, src + 32);
    }
  }
}

// The lane's word of a staged row.
template <typename T, bool kVec>
__device__ __forceinline__ uint32_t staged(const unsigned char* stage, int r, int lane, const T* tile, int64_t ld) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(stage + r * kPitch<kVec>) + lane;
  if constexpr (kVec || sizeof(T) == 4) {
    return *w;
  } else {
    return odd_start(tile + (int64_t)r * ld) ? __funnelshift_r(w[0], w[1], 16) : w[0];
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_row(T* p, const float (&v)[kCh<T>], int left) {  // left: channels from p on
  if constexpr (sizeof(T) == 4) {
    if (left > 0) *p = v[0];
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    if (left >= 2 && (kVec || !odd_start(p))) {
      *reinterpret_cast<__nv_bfloat162*>(p) = h;
    } else {
      if (left > 0) p[0] = h.x;
      if (left > 1) p[1] = h.y;
    }
  }
}

// ---- workspace: a header, a flag per (chunk, channel group), a record of one (A, B) per channel beside it
struct Chain {
  uint32_t* head;   // ticket, abort
  uint32_t* flags;  // [chunks, groups]
  float* records;   // [chunks, groups, tile channels, 2]
};
constexpr size_t kHead = 256;
size_t chain_bytes(int64_t chunks, int32_t dim) {  // for the narrower groups of f32
  const size_t g = (size_t)chunks * ((dim + 31) / 32);
  return (kHead + g * 4 + 255) / 256 * 256 + (g * 32 * 8 + 255) / 256 * 256;
}
size_t flag_bytes(int64_t chunks, int groups) { return kHead + (size_t)chunks * groups * 4; }
Chain chain_at(void* ws, int64_t chunks, int groups) {
  char* p = static_cast<char*>(ws);
  return {reinterpret_cast<uint32_t*>(p), reinterpret_cast<uint32_t*>(p + kHead),
          reinterpret_cast<float*>(p + (kHead + (size_t)chunks * groups * 4 + 255) / 256 * 256)};
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// A whole warp's record, then its flag.
template <typename T>
__device__ __forceinline__ void publish(const Chain& ch, int64_t at, const float (&A)[kCh<T>], const float (&B)[kCh<T>],
                                        int lane) {
  float* r = ch.records + (at * kTileCh<T> + lane * kCh<T>) * 2;
  if constexpr (kCh<T> == 2) __stcg(reinterpret_cast<float4*>(r), make_float4(A[0], B[0], A[1], B[1]));
  else __stcg(reinterpret_cast<float2*>(r), make_float2(A[0], B[0]));
  __threadfence();
  __syncwarp();
  if (lane == 0) store_release(ch.flags + at, 1u);
}
template <typename T>
__device__ __forceinline__ void fetch(const Chain& ch, int64_t at, float (&A)[kCh<T>], float (&B)[kCh<T>], int lane) {
  const float* r = ch.records + (at * kTileCh<T> + lane * kCh<T>) * 2;
  if constexpr (kCh<T> == 2) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(r));
    A[0] = v.x;
    B[0] = v.y;
    A[1] = v.z;
    B[1] = v.w;
  } else {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(r));
    A[0] = v.x;
    B[0] = v.y;
  }
}

// What a CTA knows of a tile. Chunks count from the end that the pass starts at.
struct Info {
  int item;    // -1: none left
  int seq;
  int chunk;   // of the whole batch, in order of rows
  int group;   // of channels
  int row, n;  // first row, tokens
  int l, last; // chunks of the run before this one (in the pass's order), and whether none follows
};

template <bool kReverse>
__device__ __forceinline__ void tile_info(Info& f, const SeqTable& t, int item, int items, int groups) {
  if (item >= items) {
    f.item = -1;
    return;
  }
  f.item = item;
  const int chunks = t.tile[t.n];
  const int pos = item / groups;
  f.group = item - pos * groups;
  f.chunk = kReverse ? chunks - 1 - pos : pos;
  const int s = find_tile_seq(t, f.chunk);
  f.seq = s;
  const int c = f.chunk - t.tile[s], of = t.tile[s + 1] - t.tile[s];
  f.row = t.cu[s] + c * kChunkR;
  f.n = min(kChunkR, t.cu[s + 1] - f.row);
  f.l = kReverse ? of - 1 - c : c;
  f.last = f.l == of - 1;
}

// Folds what precedes chunk l of this tile's run into the value that enters it (a whole warp; all lanes
// get theirs). base: the index of a record that lies d chunks before this one.
template <typename T, bool kReverse>
__device__ __forceinline__ void look_back(const Chain& ch, const Info& f, int groups, float (&h)[kCh<T>], int lane) {
  auto at = [&](int d) {  // record of the chunk d before this one in the pass's order
    return (int64_t)(kReverse ? f.chunk + d : f.chunk - d) * groups + f.group;
  };
  const int k = (f.l - 1) % kGroup;  // maps between the last published state and this chunk
  // lane i < k watches the i-th map after the state, lane k the state
  bool ready = lane > k;
  const uint32_t* flag = ch.flags + at(lane == k ? k + 1 : k - lane > 0 ? k - lane : 1);
  float A[kCh<T>], B[kCh<T>];
  for (uint32_t it = 0; !__all_sync(0xffffffffu, ready); ++it) {
    if (!ready) ready = load_acquire(flag) != 0u;
    if ((it & 63u) == 63u) {
      __nanosleep(40);
      uint32_t stop = 0;
      if (lane == 0) {
        stop = load_acquire(ch.head + 1);
        if (!stop && it >= kPollLimit) {
          store_release(ch.head + 1, 1u);
          atomicAdd(&g_recurrence_timeouts, 1u);
          stop = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) break;
    }
  }
  __syncwarp();
  fetch<T>(ch, at(k + 1), A, B, lane);
#pragma unroll
  for (int c = 0; c < kCh<T>; ++c) h[c] = B[c];
  for (int d = k; d > 0; d -= 5) {  // five records on the way at a time
    float ra[5][kCh<T>], rb[5][kCh<T>];
#pragma unroll
    for (int j = 0; j < 5; ++j)
      if (d - j > 0) fetch<T>(ch, at(d - j), ra[j], rb[j], lane);
#pragma unroll
    for (int j = 0; j < 5; ++j)
      if (d - j > 0)
#pragma unroll
        for (int c = 0; c < kCh<T>; ++c) h[c] = fmaf(ra[j][c], h[c], rb[j][c]);
  }
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
constexpr int kBarMaps = 1, kBarEnter = 2;

// Takes the next tile: by ticket where tiles wait for one another, else by turns. A CTA takes tickets
// `stages` tiles ahead; where that would be more than an even share, it takes the share and no more, so that
// a CTA that starts late still finds its own.
template <bool kReverse, int stages>
__device__ __forceinline__ void take(Info& f, const Chain& ch, const SeqTable& t, int turn, int items, int groups) {
  int item = items;
  if (!ch.head) {
    item = (int)min((int64_t)blockIdx.x + (int64_t)turn * gridDim.x, (int64_t)items);
  } else {
    const int share = (items + (int)gridDim.x - 1) / (int)gridDim.x;
    if (share > stages || turn < share) item = (int)min(atomicAdd(ch.head, 1u), (uint32_t)items);
  }
  tile_info<kReverse>(f, t, item, items, groups);
}

// ------------------------------------------------------------------ forward

constexpr int kFwdStages = 3;
template <bool kVec> constexpr int kFwdStage = 2 * kChunkR * kPitch<kVec>;

template <typename T>
struct FwdShared {
  Info info[kInfos];
  float A[kWarps][kTileCh<T>], B[kWarps][kTileCh<T>];
  float enter[2][kTileCh<T>];
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
rec_fwd_kernel(const __grid_constant__ RecArgs a, const __grid_constant__ Chain ch, const int items, const int groups) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ FwdShared<T> s;
  constexpr int C = kCh<T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // runs of no token: a fresh one zeroes its slot
  for (int i = blockIdx.x; i < a.tab.n; i += gridDim.x)
    if (a.tab.cu[i] == a.tab.cu[i + 1] && seq_fresh(a.tab, i))
      for (int c = threadIdx.x; c < a.dim; c += kThreads) a.state[(int64_t)seq_slot(a.tab, i) * a.dim + c] = 0.0f;

  auto load = [&](int i) {  // this warp's rows of tile i, if there is one; always a group
    const Info& f = s.info[i % kInfos];
    if (f.item >= 0) {
      const int ch0 = f.group * kTileCh<T>, m = min(kTileCh<T>, a.dim - ch0);
      const int nt = min(kTok, f.n - warp * kTok);
      const uint32_t st = smem_addr(stages) + (uint32_t)(i % kFwdStages) * kFwdStage<kVec>;
      load_rows<T, kVec>(st, static_cast<const T*>(a.x) + f.row * a.ld_x + ch0, a.ld_x, warp * kTok, nt, m, lane);
      load_rows<T, kVec>(st + kChunkR * kPitch<kVec>, static_cast<const T*>(a.gate) + f.row * a.ld_gate + ch0,
                         a.ld_gate, warp * kTok, nt, m, lane);
    }
    cp_commit();
  };
  if (warp == kWarps && lane == 0)
    for (int i = 0; i < kFwdStages; ++i) take<false, kFwdStages>(s.info[i], ch, a.tab, i, items, groups);
  __syncthreads();
  if (warp < kWarps)
    for (int i = 0; i < kFwdStages; ++i) load(i);

  for (int i = 0;; ++i) {
    const Info f = s.info[i % kInfos];
    if (f.item < 0) break;
    const int ch0 = f.group * kTileCh<T> + lane * C;
    const int left = a.dim - ch0;  // channels of this lane and those after it
    if (warp == kWarps) {
      // ---- the next ticket, then what enters this tile
      if (lane == 0) take<false, kFwdStages>(s.info[(i + kFwdStages) % kInfos], ch, a.tab, i + kFwdStages, items, groups);
      __syncwarp();
      bar_arrive(kBarMaps, kThreads);
      float h[C];
      if (f.l == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          h[c] = c < left && !seq_fresh(a.tab, f.seq) ? a.state[(int64_t)seq_slot(a.tab, f.seq) * a.dim + ch0 + c] : 0.0f;
      } else {
        look_back<T, false>(ch, f, groups, h, lane);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        s.enter[i & 1][lane * C + c] = h[c];
        if (a.ckpt && c < left) a.ckpt[(int64_t)f.chunk * a.dim + ch0 + c] = h[c];
      }
      bar_sync(kBarEnter, kThreads);
      continue;
    }
    // ---- scan from zero
    const unsigned char* st = stages + (i % kFwdStages) * kFwdStage<kVec>;
    const T* tx = static_cast<const T*>(a.x) + f.row * a.ld_x + f.group * kTileCh<T>;
    const T* tg = static_cast<const T*>(a.gate) + f.row * a.ld_gate + f.group * kTileCh<T>;
    float lo[C], un[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lo[c] = a.lower && c < left ? a.lower[ch0 + c] : 0.0f;
      un[c] = 1.0f - lo[c];
    }
    const int nt = min(kTok, f.n - warp * kTok);
    cp_wait<kFwdStages - 1>();
    __syncwarp();
    float hs[kTok][C], ps[kTok][C], h[C], p[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      h[c] = 0.0f;
      p[c] = 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (j < nt) {
        const int r = warp * kTok + j;
        float x[C], g[C];
        unpack_word<T>(staged<T, kVec>(st, r, lane, tx, a.ld_x), x);
        unpack_word<T>(staged<T, kVec>(st + kChunkR * kPitch<kVec>, r, lane, tg, a.ld_gate), g);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float up, down;
          sigmoids(g[c], up, down);
          const float ft = fmaf(un[c], up, lo[c]);
          h[c] = fmaf(ft, h[c], un[c] * down * x[c]);
          p[c] *= ft;
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        hs[j][c] = h[c];
        ps[j][c] = p[c];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s.A[warp][lane * C + c] = p[c];
      s.B[warp][lane * C + c] = h[c];
    }
    bar_sync(kBarMaps, kThreads);
    __syncwarp();  // every lane has read this stage
    load(i + kFwdStages);
    // the map before this warp (ex), and the tile's (warp 0 publishes it)
    float ea[C], eb[C], A[C], B[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ea[c] = A[c] = 1.0f;
      eb[c] = B[c] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          ea[c] = A[c];
          eb[c] = B[c];
        }
      if (w < warp || warp == 0)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float wa = s.A[w][lane * C + c], wb = s.B[w][lane * C + c];
          B[c] = fmaf(wa, B[c], wb);
          A[c] *= wa;
        }
    }
    const int64_t at = (int64_t)f.chunk * groups + f.group;
    if (warp == 0 && !f.last && f.l % kGroup != 0) publish<T>(ch, at, A, B, lane);
    bar_sync(kBarEnter, kThreads);
    float in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = s.enter[i & 1][lane * C + c];
    if (warp == 0) {
      float end[C];
#pragma unroll
      for (int c = 0; c < C; ++c) end[c] = fmaf(A[c], in[c], B[c]);
      if (f.last) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < left) a.state[(int64_t)seq_slot(a.tab, f.seq) * a.dim + ch0 + c] = end[c];
      } else if (f.l % kGroup == 0) {
        publish<T>(ch, at, end, end, lane);
      }
    }
    T* ty = static_cast<T*>(a.y) + f.row * a.ld_y + ch0;
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = fmaf(ea[c], in[c], eb[c]);
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < nt) {
        float y[C];
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = fmaf(ps[j][c], in[c], hs[j][c]);
        store_row<T, kVec>(ty + (int64_t)(warp * kTok + j) * a.ld_y, y, left);
      }
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ backward

constexpr int kBwdStages = 2;
template <bool kVec> constexpr int kBwdStage = 3 * kChunkR * kPitch<kVec>;

template <typename T>
struct BwdShared {
  Info info[kInfos];
  float A[kWarps][kTileCh<T>], F[kWarps][kTileCh<T>], R[kWarps][kTileCh<T>];
  float enter[2][kTileCh<T>];
  float dlo[2][kWarps][kTileCh<T>];
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
rec_bwd_kernel(const __grid_constant__ RecBwdArgs a, const __grid_constant__ Chain ch, float* part, const int items,
               const int groups) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ BwdShared<T> s;
  constexpr int C = kCh<T>;
  constexpr uint32_t kMat = kChunkR * kPitch<kVec>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (a.dstate)  // a run of no token hands its gradient on
    for (int i = blockIdx.x; i < a.tab.n; i += gridDim.x)
      if (a.tab.cu[i] == a.tab.cu[i + 1])
        for (int c = threadIdx.x; c < a.dim; c += kThreads)
          a.dstate[(int64_t)i * a.dim + c] = a.dstate_end ? a.dstate_end[(int64_t)i * a.dim + c] : 0.0f;

  auto load = [&](int i) {
    const Info& f = s.info[i % kInfos];
    if (f.item >= 0) {
      const int ch0 = f.group * kTileCh<T>, m = min(kTileCh<T>, a.dim - ch0);
      const int nt = min(kTok, f.n - warp * kTok);
      const uint32_t st = smem_addr(stages) + (uint32_t)(i % kBwdStages) * kBwdStage<kVec>;
      load_rows<T, kVec>(st, static_cast<const T*>(a.x) + f.row * a.ld_x + ch0, a.ld_x, warp * kTok, nt, m, lane);
      load_rows<T, kVec>(st + kMat, static_cast<const T*>(a.gate) + f.row * a.ld_gate + ch0, a.ld_gate, warp * kTok, nt,
                         m, lane);
      load_rows<T, kVec>(st + 2 * kMat, static_cast<const T*>(a.dy) + f.row * a.ld_dy + ch0, a.ld_dy, warp * kTok, nt, m,
                         lane);
    }
    cp_commit();
  };
  // the sum of a finished tile's eight parts of dlower (one warp, a tile later)
  auto sum_part = [&](int i) {
    const Info& f = s.info[i % kInfos];
    const int ch0 = f.group * kTileCh<T> + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s.dlo[i & 1][w][lane * C + c];
      if (ch0 + c < a.dim) part[(int64_t)f.chunk * a.dim + ch0 + c] = v;
    }
  };
  if (warp == kWarps && lane == 0)
    for (int i = 0; i < kBwdStages; ++i) take<true, kBwdStages>(s.info[i], ch, a.tab, i, items, groups);
  __syncthreads();
  if (warp < kWarps)
    for (int i = 0; i < kBwdStages; ++i) load(i);

  int i = 0;
  for (;; ++i) {
    const Info f = s.info[i % kInfos];
    if (f.item < 0) break;
    const int ch0 = f.group * kTileCh<T> + lane * C;
    const int left = a.dim - ch0;
    if (warp == kWarps) {
      // info[i + 2] takes the place of the tile before the last, whose part is summed by now
      if (lane == 0) take<true, kBwdStages>(s.info[(i + kBwdStages) % kInfos], ch, a.tab, i + kBwdStages, items, groups);
      __syncwarp();
      bar_arrive(kBarMaps, kThreads);
      float h[C];
      if (f.l == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          h[c] = c < left && a.dstate_end ? a.dstate_end[(int64_t)f.seq * a.dim + ch0 + c] : 0.0f;
      } else {
        look_back<T, true>(ch, f, groups, h, lane);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) s.enter[i & 1][lane * C + c] = h[c];
      bar_sync(kBarEnter, kThreads);
      continue;
    }
    const unsigned char* st = stages + (i % kBwdStages) * kBwdStage<kVec>;
    const T* tx = static_cast<const T*>(a.x) + f.row * a.ld_x + f.group * kTileCh<T>;
    const T* tg = static_cast<const T*>(a.gate) + f.row * a.ld_gate + f.group * kTileCh<T>;
    const T* td = static_cast<const T*>(a.dy) + f.row * a.ld_dy + f.group * kTileCh<T>;
    float lo[C], un[C], hp[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lo[c] = a.lower && c < left ? a.lower[ch0 + c] : 0.0f;
      un[c] = 1.0f - lo[c];
      hp[c] = c < left ? a.ckpt[(int64_t)f.chunk * a.dim + ch0 + c] : 0.0f;
    }
    const int nt = min(kTok, f.n - warp * kTok);
    cp_wait<kBwdStages - 1>();
    __syncwarp();
    // ---- both scans from zero: h's map (A, F) and R's map (A, R)
    float sg[kTok][C];  // the smaller sigmoid, signed as the gate
    float A[C], F[C], R[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      A[c] = 1.0f;
      F[c] = R[c] = 0.0f;
    }
    auto gates = [&](float v, int c, float& up, float& down, float& ft) {
      const float sm = fabsf(v), big = 1.0f - sm;
      const bool neg = __float_as_int(v) < 0;
      up = neg ? sm : big;
      down = neg ? big : sm;
      ft = fmaf(un[c], up, lo[c]);
    };
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < nt) {
        const int r = warp * kTok + j;
        float x[C], g[C], d[C];
        unpack_word<T>(staged<T, kVec>(st, r, lane, tx, a.ld_x), x);
        unpack_word<T>(staged<T, kVec>(st + kMat, r, lane, tg, a.ld_gate), g);
        unpack_word<T>(staged<T, kVec>(st + 2 * kMat, r, lane, td, a.ld_dy), d);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          sg[j][c] = copysignf(small_sigmoid(g[c]), g[c]);
          float up, down, ft;
          gates(sg[j][c], c, up, down, ft);
          F[c] = fmaf(ft, F[c], un[c] * down * x[c]);
          A[c] *= ft;
          R[c] = fmaf(A[c], d[c], R[c]);
        }
      }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s.A[warp][lane * C + c] = A[c];
      s.F[warp][lane * C + c] = F[c];
      s.R[warp][lane * C + c] = R[c];
    }
    bar_sync(kBarMaps, kThreads);
    if (warp == 1 && i > 0 && part) sum_part(i - 1);
    // the state that enters this warp; the map of R after it; the tile's map of R
    float ea[C], eb[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ea[c] = A[c] = 1.0f;
      eb[c] = R[c] = 0.0f;
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp)
#pragma unroll
        for (int c = 0; c < C; ++c) hp[c] = fmaf(s.A[w][lane * C + c], hp[c], s.F[w][lane * C + c]);
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      if (w == warp)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          ea[c] = A[c];
          eb[c] = R[c];
        }
      if (w > warp || warp == 0)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float wa = s.A[w][lane * C + c];
          R[c] = fmaf(wa, R[c], s.R[w][lane * C + c]);
          A[c] *= wa;
        }
    }
    const int64_t at = (int64_t)f.chunk * groups + f.group;
    if (warp == 0 && !f.last && f.l % kGroup != 0) publish<T>(ch, at, A, R, lane);
    // ---- the state before each token
    float hs[kTok][C];
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < nt) {
        float x[C];
        unpack_word<T>(staged<T, kVec>(st, warp * kTok + j, lane, tx, a.ld_x), x);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float up, down, ft;
          gates(sg[j][c], c, up, down, ft);
          hs[j][c] = hp[c];
          hp[c] = fmaf(ft, hp[c], un[c] * down * x[c]);
        }
      }
    bar_sync(kBarEnter, kThreads);
    float in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = s.enter[i & 1][lane * C + c];
    if (warp == 0) {
      float end[C];
#pragma unroll
      for (int c = 0; c < C; ++c) end[c] = fmaf(A[c], in[c], R[c]);
      if (f.last) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (a.dstate && c < left) a.dstate[(int64_t)f.seq * a.dim + ch0 + c] = end[c];
      } else if (f.l % kGroup == 0) {
        publish<T>(ch, at, end, end, lane);
      }
    }
    // ---- backwards over the tokens
    T* ox = static_cast<T*>(a.dx) + f.row * a.ld_dx + ch0;
    T* og = static_cast<T*>(a.dgate) + f.row * a.ld_dgate + ch0;
    float dlo[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      in[c] = fmaf(ea[c], in[c], eb[c]);
      dlo[c] = 0.0f;
    }
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j)
      if (j < nt) {
        const int r = warp * kTok + j;
        float x[C], d[C], vx[C], vg[C];
        unpack_word<T>(staged<T, kVec>(st, r, lane, tx, a.ld_x), x);
        unpack_word<T>(staged<T, kVec>(st + 2 * kMat, r, lane, td, a.ld_dy), d);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float up, down, ft;
          gates(sg[j][c], c, up, down, ft);
          const float G = in[c] + d[c], k = un[c] * down;
          const float dd = G * (hs[j][c] - x[c]) * down;  // df sigmoid(-g)
          vx[c] = k * G;
          vg[c] = dd * un[c] * up;
          dlo[c] += dd;
          in[c] = ft * G;
        }
        store_row<T, kVec>(ox + (int64_t)r * a.ld_dx, vx, left);
        store_row<T, kVec>(og + (int64_t)r * a.ld_dgate, vg, left);
      }
#pragma unroll
    for (int c = 0; c < C; ++c) s.dlo[i & 1][warp][lane * C + c] = dlo[c];
    __syncwarp();  // every lane is done with this stage
    load(i + kBwdStages);
  }
  __syncthreads();
  if (warp == 1 && i > 0 && part) sum_part(i - 1);
  cp_wait<0>();
}

// dlower[ch] = sum of the tiles' parts: 32 channels a CTA, eight threads a channel over every
// eighth tile, then their sums in order.
__global__ void __launch_bounds__(256) rec_dlower_kernel(float* dlower, const float* part, int chunks, int dim) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < dim)
    for (int t = w; t < chunks; t += 8) s += part[(int64_t)t * dim + c];
  sum[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < dim) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sum[j][lane];
    dlower[c] = s;
  }
}

// ------------------------------------------------------------------ single tokens

constexpr int kStepThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kStepThreads) rec_step_kernel(const __grid_constant__ RecStepArgs a) {
  const int ch = blockIdx.x * kStepThreads + threadIdx.x, i = blockIdx.y;
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

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return sms;
}

bool rows16(const void* p, int64_t ld, size_t e) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (size_t)ld * e % 16 == 0;
}

// CTAs of a launch: two to an SM, no more than tiles; empty runs need one.
int ctas(int64_t items) { return (int)std::max<int64_t>(1, std::min<int64_t>(items, 2 * (int64_t)sm_count())); }

template <typename T, bool kVec>
cudaError_t run_fwd(const RecArgs& a, const Chain& ch, int items, int groups, cudaStream_t st) {
  constexpr int smem = kFwdStages * kFwdStage<kVec>;
  const cudaError_t e = cudaFuncSetAttribute(rec_fwd_kernel<T, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  rec_fwd_kernel<T, kVec><<<ctas(items), kThreads, smem, st>>>(a, ch, items, groups);
  return cudaGetLastError();
}
template <typename T, bool kVec>
cudaError_t run_bwd(const RecBwdArgs& a, const Chain& ch, float* part, int items, int groups, cudaStream_t st) {
  constexpr int smem = kBwdStages * kBwdStage<kVec>;
  const cudaError_t e = cudaFuncSetAttribute(rec_bwd_kernel<T, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  rec_bwd_kernel<T, kVec><<<ctas(items), kThreads, smem, st>>>(a, ch, part, items, groups);
  return cudaGetLastError();
}

// The plan that both passes share: tiles, and the chain (cleared on the stream) when a run has several.
struct Tiles {
  int groups, items;
  Chain chain;
  cudaError_t status;
};
Tiles plan(const SeqTable& t, mamba2_dtype act, int32_t dim, void* ws, cudaStream_t st) {
  Tiles p = {};
  const int width = act == MAMBA2_BF16 ? kTileCh<__nv_bfloat16> : kTileCh<float>;
  p.groups = (dim + width - 1) / width;
  const int64_t chunks = t.tile[t.n], items = chunks * p.groups;
  if (items > 0x3fffffff) {
    p.status = cudaErrorInvalidValue;
    return p;
  }
  p.items = (int)items;
  bool chained = false;
  for (int i = 0; i < t.n; ++i) chained |= t.tile[i + 1] - t.tile[i] > 1;
  if (chained) {
    p.chain = chain_at(ws, chunks, p.groups);
    p.status = cudaMemsetAsync(ws, 0, flag_bytes(chunks, p.groups), st);
  }
  return p;
}

}  // namespace

size_t recurrence_workspace(int64_t chunks, bool chained, int32_t dim, bool backward) {
  const size_t part = backward ? ((size_t)chunks * dim * 4 + 255) / 256 * 256 : 0;
  return part + (chained ? chain_bytes(chunks, dim) : 0);
}

unsigned int read_recurrence_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_recurrence_timeouts, sizeof v) != cudaSuccess) return 0xffffffffu;
  return v;
}

cudaError_t launch_recurrence(const RecArgs& a, mamba2_dtype act, void* ws, cudaStream_t st) {
  const Tiles p = plan(a.tab, act, a.dim, ws, st);
  if (p.status != cudaSuccess) return p.status;
  const size_t e = act == MAMBA2_BF16 ? 2 : 4;
  const bool vec = rows16(a.x, a.ld_x, e) && rows16(a.gate, a.ld_gate, e) && rows16(a.y, a.ld_y, e);
  if (act == MAMBA2_BF16)
    return vec ? run_fwd<__nv_bfloat16, true>(a, p.chain, p.items, p.groups, st)
               : run_fwd<__nv_bfloat16, false>(a, p.chain, p.items, p.groups, st);
  return vec ? run_fwd<float, true>(a, p.chain, p.items, p.groups, st)
             : run_fwd<float, false>(a, p.chain, p.items, p.groups, st);
}

cudaError_t launch_recurrence_backward(const RecBwdArgs& a, mamba2_dtype act, void* ws, cudaStream_t st) {
  const int64_t chunks = a.tab.tile[a.tab.n];
  float* part = a.dlower ? static_cast<float*>(ws) : nullptr;
  const Tiles p = plan(a.tab, act, a.dim, static_cast<char*>(ws) + recurrence_workspace(chunks, false, a.dim, true), st);
  if (p.status != cudaSuccess) return p.status;
  const size_t es = act == MAMBA2_BF16 ? 2 : 4;
  const bool vec = rows16(a.x, a.ld_x, es) && rows16(a.gate, a.ld_gate, es) && rows16(a.dy, a.ld_dy, es) &&
                   rows16(a.dx, a.ld_dx, es) && rows16(a.dgate, a.ld_dgate, es);
  cudaError_t e;
  if (act == MAMBA2_BF16)
    e = vec ? run_bwd<__nv_bfloat16, true>(a, p.chain, part, p.items, p.groups, st)
            : run_bwd<__nv_bfloat16, false>(a, p.chain, part, p.items, p.groups, st);
  else
    e = vec ? run_bwd<float, true>(a, p.chain, part, p.items, p.groups, st)
            : run_bwd<float, false>(a, p.chain, part, p.items, p.groups, st);
  if (e == cudaSuccess && a.dlower) {
    rec_dlower_kernel<<<(a.dim + 31) / 32, 256, 0, st>>>(a.dlower, part, (int)chunks, a.dim);
    e = cudaGetLastError();
  }
  return e;
}

cudaError_t launch_recurrence_step(const RecStepArgs& a, mamba2_dtype act, cudaStream_t st) {
  const dim3 grid((a.dim + kStepThreads - 1) / kStepThreads, a.n);
  if (act == MAMBA2_BF16) rec_step_kernel<__nv_bfloat16><<<grid, kStepThreads, 0, st>>>(a);
  else rec_step_kernel<float><<<grid, kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mamba2
