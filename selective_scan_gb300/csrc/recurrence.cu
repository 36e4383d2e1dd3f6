// Gated recurrence (block.h): h_t = f_t h_{t-1} + k_t x_t per channel, with
// f = lo + (1 - lo) sigmoid(gate) and k = 1 - f, over packed runs; its backward pass
// and its single-token step. HBM has to move 6 bytes a token and channel forward (bf16) and
// 10 backward.
//
// One pass over the data, split over time. A step of the recurrence is the affine map
// h -> f h + b, and maps compose: (A, B) after (A', B') is (A A', A B' + B). A tile is one
// chunk of MAMBA2_RECURRENCE_CHUNK = 128 tokens by 128 bytes of channels; eight warps take
// 16 tokens each, a lane 4 bytes of channels. Per tile:
//   1. each warp scans its tokens from zero, keeping h_t in registers and the product of
//      the f's in shared memory, and posts its map; the eight maps compose to the tile's
//   2. the tile publishes its map in the workspace, and each warp fetches up to four of the
//      maps that precede the tile; folded, they give the state that enters it
//   3. each warp adds (product of f's) x (its own entering state) to its tokens and stores
// Inputs stream through a ring in shared memory by TMA, or by cp.async where rows are not 16-byte
// aligned: a warp fetches only the rows that it will read, so a stage is handed over without the
// other warps, and the next tile's copies are in flight while a tile waits for its predecessors
// (with one stage, while the others finish). Unaligned rows are shifted into place as they are
// read, at a third more instructions: eight runs of 32 768 tokens in all by 2 047 channels of
// bf16 take 121 us forwards and 207 backwards (by 2 048: 81 and 140).
//
// What precedes chunk l of a run, the same for any timing (so results repeat bit for bit):
// every chunk publishes its map, and every 16th (0, 16, 32, ...) the state after it too (the
// first the state alone, which it has as early as its map); every 8th or 4th where many runs or
// channels are under way at a time. Chunk l takes the state that lies one such step further
// back than the nearest, and folds the maps of the up to 31 (15, 7) chunks between in order.
// Maps are published without waiting for anything, and a state is used 16 (8, 4) chunks later
// at the earliest: later than the tiles that the GPU holds at one time for wide matrices, so a
// tile waits for maps alone. (With the nearest state it waited for the maps and
// then for the state made from them: 9 % more time for one run of 65 536 tokens by 2 048 channels
// when this was chosen.) Chunk 0 alone reads the pool, so the run's last chunk may overwrite the slot.
//
// Tiles are taken by ticket in an order in which a tile's predecessors come first, so a
// waiting tile's predecessors are always held by CTAs that run. Waits are bounded; one that
// gives up raises an abort flag in the workspace that ends every other wait, and is counted
// in g_recurrence_timeouts.
//
// The backward pass runs the same machinery from the end: with R_t = f_t (dy_t + R_{t+1})
// the map of a token is R -> f R + f dy. A warp recomputes its states from the checkpoint
// that the forward pass kept for it (4 bytes per 16 tokens and channel: an eighth of reading
// y, and unrounded), and makes dx and dgate in one more sweep over its tokens. dlower is
// summed per tile and then over the tiles, in order.
//
// Measured (GB300, 65 536 tokens x 2 048 channels, bf16, with lower bounds and, forward, checkpoints): one run 189 us
// forward (185 without checkpoints: 4.4 TB/s, 64 % of the measured copy rate) and 289 backward (4.8 TB/s); eight runs
// 154 and 263, 64 runs 155 and 266; 512 runs, where nothing waits, 156 and 270. fp32, 65 536 x 1 024: 5.3 TB/s forward
// and 5.6 backward for one run, 6.3 and 6.2 for 512. What bounds bf16 is latency: 54 % of the issue slots and 48 % of
// HBM are active, and the largest share of a warp's time goes to a tile's two barriers of the whole CTA (3.1 of about 9
// cycles an instruction for one run, where they cover the look-back; 2.0 where nothing is looked back at).
#include <cuda.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "../../include/block.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {

__device__ unsigned int g_recurrence_timeouts = 0;

namespace {

#include "batch_check.cuh"
#include "tc.cuh"

constexpr int kChunkR = MAMBA2_RECURRENCE_CHUNK;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = kChunkR / kWarps;         // tokens of a warp
constexpr int kMostShift = 4, kLeastShift = 2; // log2 of the chunks between two published states
constexpr int kBack = (2 << kMostShift) / kWarps;  // maps that a warp looks back at, at most
constexpr int kInfos = 4;
// The thread that takes the next tile: of a warp that often has no maps to fetch (of the first one, with the nearest
// maps, eight runs of 65 536 x 2 048 took 3 % longer, backwards 4 %).
constexpr int kTaker = 32 * 5;
constexpr uint32_t kPollLimit = 1u << 21;      // polls before giving up (about a second)

// A lane's channels: 4 bytes of them.
template <typename T> constexpr int kCh = 4 / (int)sizeof(T);
template <typename T> constexpr int kTileCh = 32 * kCh<T>;

// Row of a staged matrix: 128 bytes, or with the up to 14 before them that share their first 16.
template <bool kVec> constexpr int kPitch = kVec ? 128 : 144;

// sigmoid(g) and sigmoid(-g), each with its own digits: with e = exp(-|g|) they are
// 1 / (1 + e) and e / (1 + e), in the order that g's sign gives; the first is also one minus the
// second, to the last digit.
__device__ __forceinline__ float recip(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// 2^v. (The instruction's flushing form: what it flushes is below 2^-126; the other form scales around that
// at four more instructions.)
__device__ __forceinline__ float exp2_ftz(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
__device__ __forceinline__ float exp_neg_abs(float g) { return exp2_ftz(fabsf(g) * -1.4426950408889634f); }
__device__ __forceinline__ void sigmoids(float g, float& up, float& down) {
  const float e = exp_neg_abs(g), s = e * recip(1.0f + e), r = 1.0f - s;
  up = g >= 0.0f ? r : s;
  down = g >= 0.0f ? s : r;
}

// A lane's channels as one value: a float, or a pair that the packed fp32 instructions take whole (half
// the issue slots, the same roundings).
template <int C> struct Pack;
template <> struct Pack<1> {
  using V = float;
  __device__ __forceinline__ static V make(const float (&v)[1]) { return v[0]; }
  __device__ __forceinline__ static V all(float v) { return v; }
  __device__ __forceinline__ static void split(V v, float (&o)[1]) { o[0] = v; }
  __device__ __forceinline__ static V fma(V a, V b, V c) { return fmaf(a, b, c); }
  __device__ __forceinline__ static V mul(V a, V b) { return a * b; }
  __device__ __forceinline__ static V add(V a, V b) { return a + b; }
};
template <> struct Pack<2> {
  using V = uint64_t;
  __device__ __forceinline__ static V make(const float (&v)[2]) {
    V r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v[0]), "f"(v[1]));
    return r;
  }
  __device__ __forceinline__ static V all(float v) {
    const float t[2] = {v, v};
    return make(t);
  }
  __device__ __forceinline__ static void split(V v, float (&o)[2]) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o[0]), "=f"(o[1]) : "l"(v));
  }
  __device__ __forceinline__ static V fma(V a, V b, V c) {
    V r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
  }
  __device__ __forceinline__ static V mul(V a, V b) {
    V r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
  }
  __device__ __forceinline__ static V add(V a, V b) {
    V r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
  }
};

template <typename T>
__device__ __forceinline__ void unpack_word(uint32_t w, float (&v)[kCh<T>]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w);
  } else {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
}

// sigmoid(g) and sigmoid(-g) of each channel, each with its own digits: with a = exp(-g) they are 1 / (1 + a) and
// a / (1 + a). a is kept at 2^126 at most, whose reciprocal is the least that is not flushed and stands for 0: `up`
// is too large by that (below 2^-102 it counts), which what uses it takes off. (Of two exponentials and reciprocals a
// channel instead: 6 % more time for one run of 65 536 tokens by 2 048 channels, backwards 7 %, when this was chosen.)
constexpr float kLeast = 0x1p-126f;
template <int C>
__device__ __forceinline__ void both_sigmoids(const float (&g)[C], typename Pack<C>::V& up, typename Pack<C>::V& down) {
  using P = Pack<C>;
  float a[C], r[C];
  P::split(P::mul(P::make(g), P::all(-1.4426950408889634f)), a);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a[c]) : "f"(126.0f));
    a[c] = exp2_ftz(a[c]);
  }
  const typename P::V a2 = P::make(a);
  P::split(P::add(a2, P::all(1.0f)), r);
#pragma unroll
  for (int c = 0; c < C; ++c) r[c] = recip(r[c]);
  up = P::make(r);
  down = P::mul(a2, up);
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

// The runs of a call. They are launch parameters, which take time to hand over by the byte, so there is a short form:
// a call for 300 tokens by 1 536 channels took 1 us less forwards with it and 3 backwards (7.1 and 10.4 in a graph).
//
// Also the order in which the chunks of several runs are taken: runs in turns, each one's first chunk, then each
// one's second, and so on, so that a chunk's predecessors are some time ago and few of them have to be waited for
// (each run by itself, as the rows lie: 1.27 times the time for 64 runs of 65 536 tokens in all by 2 048 channels,
// 1.20 times for eight, when this was chosen). Not more runs at a time than that takes, the longest first: what was published longer
// ago has left L2.
template <int kMost>
struct Runs {
  int32_t n;
  int32_t sorted;             // runs that have chunks; 0: chunks in order of rows
  int32_t turn;               // so many at a time
  int32_t cu[kMost + 1];      // first rows
  int32_t tile[kMost + 1];    // first chunks
  int32_t before[kMost];      // [k turn]: chunks before the k-th of those sets; [k turn + c]: of those in it,
                              // how many are taken before its c longest runs are alone
  uint32_t slot_fresh[kMost];
  uint16_t run[kMost];        // the longest first
};
constexpr int kFewRuns = 64;
template <int kMost>
void fill_runs(Runs<kMost>& o, const SeqTable& t, int turn) {
  o.n = t.n;
  o.sorted = 0;
  o.turn = turn;
  std::copy(t.cu, t.cu + t.n + 1, o.cu);
  std::copy(t.tile, t.tile + t.n + 1, o.tile);
  std::copy(t.slot_fresh, t.slot_fresh + t.n, o.slot_fresh);
  if (turn == 0) return;
  auto chunks = [&](int r) { return t.tile[r + 1] - t.tile[r]; };
  for (int i = 0; i < t.n; ++i)
    if (chunks(i) > 0) o.run[o.sorted++] = (uint16_t)i;
  std::stable_sort(o.run, o.run + o.sorted, [&](int a, int b) { return chunks(a) > chunks(b); });
  int start = 0;
  for (int k = 0; k < o.sorted; k += turn) {
    int shorter = 0;  // chunks of the set's runs after the first c
    for (int c = std::min(turn, o.sorted - k) - 1; c >= 1; --c) {
      shorter += chunks(o.run[k + c]);
      o.before[k + c] = shorter + c * chunks(o.run[k + c]);
    }
    o.before[k] = start;
    start += shorter + chunks(o.run[k]);
  }
}

template <bool kReverse, int kMost>
__device__ __forceinline__ void tile_info(Info& f, const Runs<kMost>& t, int item, int items, int groups) {
  if (item >= items) {
    f.item = -1;
    return;
  }
  f.item = item;
  const int pos = item / groups;
  f.group = item - pos * groups;
  int s, of;
  if (t.sorted > 0) {
    int set = 0, last = (t.sorted - 1) / t.turn;
    while (set < last) {
      const int mid = (set + last + 1) >> 1;
      if (t.before[mid * t.turn] <= pos) set = mid; else last = mid - 1;
    }
    set *= t.turn;
    const int in_set = pos - t.before[set], most = min(t.turn, t.sorted - set);
    int c = 1, hi = most;  // the fewest runs left that in_set allows
    while (c < hi) {
      const int mid = (c + hi) >> 1;
      if (t.before[set + mid] <= in_set) hi = mid; else c = mid + 1;
    }
    const int next = c < most ? t.run[set + c] : 0;
    const int in = in_set - (c < most ? t.before[set + c] : 0), ended = c < most ? t.tile[next + 1] - t.tile[next] : 0;
    s = t.run[set + in % c];
    of = t.tile[s + 1] - t.tile[s];
    f.l = ended + in / c;
    f.chunk = t.tile[s] + (kReverse ? of - 1 - f.l : f.l);
  } else {
    f.chunk = kReverse ? t.tile[t.n] - 1 - pos : pos;
    s = find_tile_seq(t, f.chunk);
    of = t.tile[s + 1] - t.tile[s];
    f.l = kReverse ? of - 1 - (f.chunk - t.tile[s]) : f.chunk - t.tile[s];
  }
  f.seq = s;
  const int c = f.chunk - t.tile[s];
  f.row = t.cu[s] + c * kChunkR;
  f.n = min(kChunkR, t.cu[s + 1] - f.row);
  f.last = f.l == of - 1;
}

// A matrix that is streamed through the ring.
template <typename T>
struct Stream {
  const T* p;
  int64_t ld;
  const CUtensorMap* map;  // boxes of 128 bytes x kTok rows
};
// This warp's rows of tile f of k matrices, kMat bytes apart, into the stage at st (wait_tile waits for them, with bar).
// Where rows are 16-byte aligned, by TMA: rows past the run's end are other runs', or zeros, and nothing uses them. Else
// 16 bytes a lane, each row from the 16-byte boundary before it to the one after it: what that adds shares its 16 bytes
// with the row, so it can be read, and nothing uses it either. (8 runs, 32 768 x 2 046 bf16: 118 us; a bulk copy a row
// took 6 % longer from all lanes and 19 % from one; 4 bytes a lane, which can place a row at its word, longer still.)
template <typename T, bool kVec, int k>
__device__ __forceinline__ void load_tile(const Info& f, const Stream<T> (&m)[k], uint32_t st, uint32_t bar, int dim,
                                          int warp, int lane) {
  constexpr uint32_t kMat = kChunkR * kPitch<kVec>;
  const int ch0 = f.group * kTileCh<T>, nt = f.item >= 0 ? min(kTok, f.n - warp * kTok) : 0;
  if (nt <= 0) return;
  if constexpr (kVec) {
    if (lane == 0) {
      fence_async_smem();  // what this warp read and wrote there before comes first
      mbar_expect_tx(bar, k * kTok * 128);
#pragma unroll
      for (int i = 0; i < k; ++i) tma_load_2d(st + i * kMat + warp * kTok * 128, m[i].map, ch0, f.row + warp * kTok, bar);
    }
  } else {
    constexpr int kUnits = kPitch<false> / 16;  // of a row: where unit u of row r goes is 16 (kUnits r + u) bytes on
    const uint32_t valid = (uint32_t)min(kTileCh<T>, dim - ch0) * (uint32_t)sizeof(T);
#pragma unroll
    for (int c = 0; c < kTok * kUnits; c += 32) {
      const int r = (c + lane) / kUnits, u = c + lane - r * kUnits;
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const uint64_t p = reinterpret_cast<uint64_t>(m[i].p + (int64_t)(f.row + warp * kTok + r) * m[i].ld + ch0);
        if (r < nt && 16u * (uint32_t)u < (uint32_t)(p & 15) + valid)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                       :: "r"(st + i * kMat + (uint32_t)(warp * kTok) * kPitch<kVec> + 16u * (uint32_t)(c + lane)),
                          "l"((p & ~(uint64_t)15) + 16u * (uint32_t)u) : "memory");
      }
    }
  }
}
// Waits for this warp's rows (of its next load).
template <bool kVec>
__device__ __forceinline__ void wait_tile(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if constexpr (kVec) {
    warp_wait(bar, parity, abort);
  } else {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
}

// A lane's words of this warp's staged rows of the k matrices.
template <typename T, bool kVec, int k>
struct Reader {
  unsigned char* base;  // the lane's in row 0 of the first matrix
  uint32_t at = 0, step = 0;  // a byte to a matrix: its first row's address and its stride modulo 16

  __device__ __forceinline__ Reader(unsigned char* st, const Info& f, const Stream<T> (&m)[k], int warp, int lane)
      : base(st + warp * kTok * kPitch<kVec> + 4 * lane) {
    static_assert(kTok <= 16, "a row's sum stays inside its byte");
    if constexpr (!kVec)
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const uint32_t ld = (uint32_t)m[i].ld, row = (uint32_t)(f.row + warp * kTok), e = sizeof(T);
        at |= (((uint32_t)reinterpret_cast<uintptr_t>(m[i].p) + e * (row * ld + f.group * kTileCh<T>)) & 15u) << (8 * i);
        step |= (e * ld & 15u) << (8 * i);
      }
  }
  // the lane's word of row j, or at the row's offset the one or two that hold its channels, shifted into place
  // (by their address's low bits: bit 0 is 0, and a shift counts modulo 32)
  __device__ __forceinline__ uint32_t word(int i, int j) const {
    const uint32_t off = at_row(j);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row(i, j) + (kVec ? 0u : off >> (8 * i) & 12u));
    if constexpr (kVec || sizeof(T) == 4) return w[0];
    else return __funnelshift_r(w[0], w[1], i == 0 ? off << 3 : off >> (8 * i - 3));
  }
  // where row j starts: four bytes there are the lane's once the warp has read the row
  __device__ __forceinline__ unsigned char* row(int i, int j) const {
    return base + i * kChunkR * kPitch<kVec> + j * kPitch<kVec>;
  }

 private:
  __device__ __forceinline__ uint32_t at_row(int j) const { return (at + j * step) & 0x0f0f0f0fu; }
};

// A lane's channels to the output. kInside: all of them are inside the matrix, else `left` are from p on; kWords: p is
// on a word.
template <typename T, bool kInside, bool kWords>
__device__ __forceinline__ void store_row(T* p, const float (&v)[kCh<T>], int left) {
  if constexpr (sizeof(T) == 4) {
    if (kInside || left > 0) *p = v[0];
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    if ((kInside || left > 1) && (kWords || (reinterpret_cast<uintptr_t>(p) & 2) == 0)) {
      *reinterpret_cast<__nv_bfloat162*>(p) = h;
    } else {
      if (kInside || left > 0) p[0] = h.x;
      if (kInside || left > 1) p[1] = h.y;
    }
  }
}

// ---- workspace: a header, then a record of one (A, B) per channel for each (chunk, channel group), then a
// record of one state per channel for every (1 << shift)-th chunk of a run (and group).
// All of it is set to 0xff bytes first. A record's words are their own flags: every word that a tile
// publishes is the result of an fp32 operation, which no NaN makes 0xffffffff, so a reader polls the
// record until that pattern is gone from it, and needs no fence and no second round trip.
struct Chain {
  uint32_t* head;  // tickets taken, less one; abort when it is no longer 0xffffffff
  float* maps;     // [chunks, groups, tile channels, 2]
  float* states;   // [state_rows, groups, tile channels]
  int shift;
};
constexpr size_t kHead = 256;
constexpr uint32_t kUnset = 0xffffffffu;
// Row of the state after chunk l of run i, whose first chunk is t: the runs' rows do not overlap.
__host__ __device__ constexpr int64_t state_row(int64_t t, int i, int l, int shift) {
  return (t >> shift) + i + (l >> shift);
}
size_t chain_bytes(int64_t chunks, int runs, int64_t channels, int shift) {
  return kHead + (size_t)chunks * channels * 8 + (size_t)state_row(chunks, runs, 0, shift) * channels * 4;
}
Chain chain_at(void* ws, int64_t chunks, int64_t channels, int shift) {
  float* maps = reinterpret_cast<float*>(static_cast<char*>(ws) + kHead);
  return {static_cast<uint32_t*>(ws), maps, maps + chunks * channels * 2, shift};
}

// A lane's share of a record: (A, B) of each of its channels.
template <int C>
__device__ __forceinline__ void load_record(const float* p, float (&v)[2 * C]) {
  if constexpr (C == 2)
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p) : "memory");
  else
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p) : "memory");
}
template <int C>
__device__ __forceinline__ void store_record(float* p, const float (&v)[2 * C]) {
  if constexpr (C == 2)
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};"
                 ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
  else
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(v[0]), "f"(v[1]) : "memory");
}
template <int C>
__device__ __forceinline__ void load_state(const float* p, float (&v)[C]) {
  if constexpr (C == 2)
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p) : "memory");
  else
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v[0]) : "l"(p) : "memory");
}
template <int n>
__device__ __forceinline__ bool is_set(const float (&v)[n]) {
  bool set = true;
#pragma unroll
  for (int c = 0; c < n; ++c) set = set && __float_as_uint(v[c]) != kUnset;
  return set;
}
template <typename T>
__device__ __forceinline__ float* map_at(const Chain& ch, int64_t chunk, int groups, int group, int lane) {
  return ch.maps + ((chunk * groups + group) * kTileCh<T> + lane * kCh<T>) * 2;
}
template <typename T>
__device__ __forceinline__ float* state_at(const Chain& ch, const Info& f, int first, int l, int groups, int lane) {
  return ch.states + (state_row(first, f.seq, l, ch.shift) * groups + f.group) * kTileCh<T> + lane * kCh<T>;
}
template <typename T>
__device__ __forceinline__ void publish_map(const Chain& ch, const Info& f, int groups, const float (&A)[kCh<T>],
                                            const float (&B)[kCh<T>], int lane) {
  float v[2 * kCh<T>];
#pragma unroll
  for (int c = 0; c < kCh<T>; ++c) {
    v[2 * c] = A[c];
    v[2 * c + 1] = B[c];
  }
  store_record<kCh<T>>(map_at<T>(ch, f.chunk, groups, f.group, lane), v);
}
template <typename T>
__device__ __forceinline__ void publish_state(const Chain& ch, const Info& f, int first, int groups,
                                              const float (&h)[kCh<T>], int lane) {
  float* p = state_at<T>(ch, f, first, f.l, groups, lane);
  if constexpr (kCh<T> == 2)
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(h[0]), "f"(h[1]) : "memory");
  else
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(h[0]) : "memory");
}

// Chunks between chunk l > 0 and the published state that it starts from.
__device__ __forceinline__ int maps_before(int l, int shift) {
  const int g = (l - 1) >> shift;
  return l - 1 - ((g > 0 ? g - 1 : 0) << shift);
}

// Tells a waiting warp to give up: when another one has, or after kPollLimit polls.
__device__ __forceinline__ bool gave_up(const Chain& ch, uint32_t it, int lane) {
  if ((it & 63u) != 63u) return false;
  uint32_t stop = 0;
  if (lane == 0) {
    stop = *(volatile uint32_t*)(ch.head + 1) != kUnset;
    if (!stop && it >= kPollLimit) {
      atomicExch(ch.head + 1, 0u);
      atomicAdd(&g_recurrence_timeouts, 1u);
      stop = 1;
    }
  }
  return __shfl_sync(0xffffffffu, stop, 0) != 0u;
}

// What enters a tile, in shared memory: the state it starts from, and a map from each warp, the oldest last.
template <typename T>
struct Before {
  float state[kTileCh<T>];
  float A[kWarps][kTileCh<T>], B[kWarps][kTileCh<T>];
};
// This warp's share: the maps of the chunks kBack warp + 1 .. kBack (warp + 1) before the tile as far as there
// are k, composed; and the state: a warp that has no maps where states are frequent, else the first (eight runs
// of 65 536 tokens by 2 048 channels took 1 % longer with the first, one run 3 % longer with the other).
template <typename T, bool kReverse>
__device__ __forceinline__ void look_back(const Chain& ch, const Info& f, int first, int groups, int k,
                                          Before<T>& out, int warp, int lane) {
  constexpr int C = kCh<T>;
  const int d0 = kBack * warp + 1, n = min(kBack, max(0, k - d0 + 1));
  const int64_t step = (int64_t)(kReverse ? groups : -groups) * kTileCh<T> * 2;
  const float* p = map_at<T>(ch, kReverse ? f.chunk + d0 : f.chunk - d0, groups, f.group, lane);
  float r[kBack][2 * C], h[C];
#pragma unroll
  for (int j = 0; j < kBack; ++j)
    if (j < n) load_record<C>(p + j * step, r[j]);
  if (warp == (ch.shift == kMostShift ? 0 : kWarps - 2) && f.l > 0) {  // (the first chunk's is read where its map is made)
    const float* q = state_at<T>(ch, f, first, f.l - 1 - k, groups, lane);
    load_state<C>(q, h);
#pragma unroll 1
    for (uint32_t it = 0; !__all_sync(0xffffffffu, is_set(h)) && !gave_up(ch, it, lane); ++it) load_state<C>(q, h);
#pragma unroll
    for (int c = 0; c < C; ++c) out.state[lane * C + c] = h[c];
  }
#pragma unroll 1
  for (uint32_t it = 0;; ++it) {
    bool set = true;
#pragma unroll
    for (int j = 0; j < kBack; ++j) set = set && (j >= n || is_set(r[j]));
    if (__all_sync(0xffffffffu, set) || gave_up(ch, it, lane)) break;
#pragma unroll
    for (int j = 0; j < kBack; ++j)
      if (j < n) load_record<C>(p + j * step, r[j]);
  }
  if (n == 0) return;  // (nothing reads its share)
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float A = 1.0f, B = 0.0f;
#pragma unroll
    for (int j = kBack - 1; j >= 0; --j)
      if (j < n) {
        B = fmaf(r[j][2 * c], B, r[j][2 * c + 1]);
        A *= r[j][2 * c];
      }
    out.A[warp][lane * C + c] = A;
    out.B[warp][lane * C + c] = B;
  }
}
// After a barrier: what enters the tile.
template <typename T>
__device__ __forceinline__ void fold_before(const Before<T>& in, int k, float (&v)[kCh<T>], int lane) {
#pragma unroll
  for (int c = 0; c < kCh<T>; ++c) v[c] = in.state[lane * kCh<T> + c];
  for (int w = (k + kBack - 1) / kBack - 1; w >= 0; --w)
#pragma unroll
    for (int c = 0; c < kCh<T>; ++c) v[c] = fmaf(in.A[w][lane * kCh<T> + c], v[c], in.B[w][lane * kCh<T> + c]);
}

// The next tile: by ticket where tiles wait for one another, else by turns. A CTA takes tickets `stages`
// tiles ahead; where that would be more than an even share, it takes the share and no more, so that a CTA
// that starts late still finds its own.
template <int stages>
__device__ __forceinline__ int take(const Chain& ch, int turn, int items) {
  if (!ch.head) return (int)min((int64_t)blockIdx.x + (int64_t)turn * gridDim.x, (int64_t)items);
  const int share = (items + (int)gridDim.x - 1) / (int)gridDim.x;
  return share > stages || turn < share ? (int)min(atomicAdd(ch.head, 1u) + 1u, (uint32_t)items) : items;
}

// ------------------------------------------------------------------ forward

// Three CTAs to an SM, with as many stages as they leave room for.
template <bool kVec> constexpr int kFwdStages = kVec ? 2 : 1;
template <bool kVec> constexpr int kFwdStage = 2 * kChunkR * kPitch<kVec>;
constexpr int kCtas = 3;

template <typename T, bool kVec>
struct FwdShared {
  Info info[kInfos];
  float A[kWarps][kTileCh<T>], B[kWarps][kTileCh<T>];      // the warps' maps, then of all the warps before each
  Before<T> before;
  alignas(8) uint64_t full[kFwdStages<kVec>][kWarps];
  uint32_t abort;
};

// The products of the f's go into shared memory, over the inputs that the lane has consumed (the same 8 bytes
// a pair of channels), so that three CTAs fit an SM's registers.
template <typename T, bool kVec, int kMost>
__global__ void __launch_bounds__(kThreads, kCtas)
rec_fwd_kernel(const __grid_constant__ RecTensors a, const __grid_constant__ Runs<kMost> t, const __grid_constant__ CUtensorMap mx,
               const __grid_constant__ CUtensorMap mg, const __grid_constant__ Chain ch, const int items,
               const int groups) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ FwdShared<T, kVec> s;
  constexpr int C = kCh<T>;
  using P = Pack<C>;
  using V = typename P::V;
  constexpr uint32_t kMat = kChunkR * kPitch<kVec>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // runs of no token: a fresh one zeroes its slot
  for (int i = blockIdx.x; i < t.n; i += gridDim.x)
    if (t.cu[i] == t.cu[i + 1] && seq_fresh(t, i))
      for (int c = threadIdx.x; c < a.dim; c += kThreads) a.state[(int64_t)seq_slot(t, i) * a.dim + c] = 0.0f;

  const Stream<T> in_streams[2] = {{static_cast<const T*>(a.x), a.ld_x, &mx}, {static_cast<const T*>(a.gate), a.ld_gate, &mg}};
  auto load = [&](int i) {  // this warp's rows of tile i, if there is one
    load_tile<T, kVec, 2>(s.info[i % kInfos], in_streams, su32(stages) + (uint32_t)(i % kFwdStages<kVec>) * kFwdStage<kVec>,
                          su32(&s.full[i % kFwdStages<kVec>][warp]), a.dim, warp, lane);
  };
  if (threadIdx.x < kFwdStages<kVec> * kWarps) {
    mbar_init(su32(&s.full[0][0] + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s.abort = 0u;
  }
  if (threadIdx.x == 0)
    for (int i = 0; i < kFwdStages<kVec>; ++i)
      tile_info<false>(s.info[i], t, take<kFwdStages<kVec>>(ch, i, items), items, groups);
  __syncthreads();
  for (int i = 0; i < kFwdStages<kVec>; ++i) load(i);

  uint32_t phases = 0;  // bit s: the parity of stage s's next load
  for (int i = 0;; ++i) {
    const Info f = s.info[i % kInfos];
    if (f.item < 0) break;
    const int ch0 = f.group * kTileCh<T> + lane * C;
    const int left = a.dim - ch0;  // channels of this lane and those after it
    int next = 0;
    if (threadIdx.x == kTaker) next = take<kFwdStages<kVec>>(ch, i + kFwdStages<kVec>, items);
    const int first = t.tile[f.seq];
    const int before = f.l > 0 ? maps_before(f.l, ch.shift) : 0;
    float h0[C];  // what the run starts from: asked for early, the run's other tiles wait for it
    if (warp == kWarps - 1 && f.l == 0)
#pragma unroll
      for (int c = 0; c < C; ++c)
        h0[c] = c < left && !seq_fresh(t, f.seq) ? a.state[(int64_t)seq_slot(t, f.seq) * a.dim + ch0 + c] : 0.0f;
    // ---- scan from zero
    unsigned char* st = stages + (i % kFwdStages<kVec>) * kFwdStage<kVec>;
    const Reader<T, kVec, 2> rd(st, f, in_streams, warp, lane);
    float lo[C], un[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lo[c] = a.lower && c < left ? a.lower[ch0 + c] : 0.0f;
      un[c] = 1.0f - lo[c];
    }
    const V un2 = P::make(un), lo2 = P::fma(un2, P::all(-kLeast), P::make(lo));  // (f = up un + lo)
    const int nt = min(kTok, f.n - warp * kTok);
    if (nt > 0) {
      wait_tile<kVec>(su32(&s.full[i % kFwdStages<kVec>][warp]), phases >> (i % kFwdStages<kVec>) & 1u, &s.abort);
      phases ^= 1u << (i % kFwdStages<kVec>);
    }
    V hs[kTok], h2 = P::all(0.0f), p2 = P::all(1.0f);
    auto scan = [&](auto whole) {  // rows past the run's end count as the identity
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (decltype(whole)::value || j < nt) {
          float x[C], g[C];
          unpack_word<T>(rd.word(0, j), x);
          unpack_word<T>(rd.word(1, j), g);
          V up, down;
          both_sigmoids<C>(g, up, down);
          const V f2 = P::fma(un2, up, lo2);
          h2 = P::fma(f2, h2, P::mul(P::mul(un2, down), P::make(x)));
          p2 = P::mul(p2, f2);
        }
        hs[j] = h2;
        float v[C];
        P::split(p2, v);
        if constexpr (!kVec) __syncwarp();  // (the row is read)
        *reinterpret_cast<float*>(rd.row(0, j)) = v[0];
        if constexpr (C == 2) *reinterpret_cast<float*>(rd.row(1, j)) = v[1];
      }
    };
    if (nt == kTok) scan(std::true_type{});
    else scan(std::false_type{});
    float A[C], B[C];
    P::split(p2, A);
    P::split(h2, B);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s.A[warp][lane * C + c] = A[c];
      s.B[warp][lane * C + c] = B[c];
    }
    __syncthreads();
    if (warp == kWarps - 1) {
      // for each warp the map of those before it; after the last, the tile's
#pragma unroll
      for (int c = 0; c < C; ++c) {
        A[c] = 1.0f;
        B[c] = 0.0f;
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float wa = s.A[w][lane * C + c], wb = s.B[w][lane * C + c];
          s.A[w][lane * C + c] = A[c];
          s.B[w][lane * C + c] = B[c];
          B[c] = fmaf(wa, B[c], wb);
          A[c] *= wa;
        }
      if (f.l == 0) {  // nothing to wait for: the state after the first chunk is out as early as the maps
        float end[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          s.before.state[lane * C + c] = h0[c];
          end[c] = fmaf(A[c], h0[c], B[c]);
        }
        if (!f.last) publish_state<T>(ch, f, first, groups, end, lane);
      } else if (!f.last) {
        publish_map<T>(ch, f, groups, A, B, lane);
      }
    }
    if (threadIdx.x == kTaker) tile_info<false>(s.info[(i + kFwdStages<kVec>) % kInfos], t, next, items, groups);
    look_back<T, false>(ch, f, first, groups, before, s.before, warp, lane);
    __syncthreads();
    float in[C];
    fold_before(s.before, before, in, lane);
    if (warp == kWarps - 1) {
      float end[C];
#pragma unroll
      for (int c = 0; c < C; ++c) end[c] = fmaf(A[c], in[c], B[c]);
      if (f.last) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < left) a.state[(int64_t)seq_slot(t, f.seq) * a.dim + ch0 + c] = end[c];
      } else if (f.l > 0 && (f.l & ((1 << ch.shift) - 1)) == 0) {
        publish_state<T>(ch, f, first, groups, end, lane);
      }
    }
    // the state that enters this warp
#pragma unroll
    for (int c = 0; c < C; ++c) {
      in[c] = fmaf(s.A[warp][lane * C + c], in[c], s.B[warp][lane * C + c]);
      if (a.ckpt && c < left && nt > 0) a.ckpt[((int64_t)f.chunk * kWarps + warp) * a.dim + ch0 + c] = in[c];
    }
    T* ty = static_cast<T*>(a.y) + (f.row + warp * kTok) * a.ld_y + ch0;
    const V in2 = P::make(in);
    auto emit = [&](auto whole) {
#pragma unroll
      for (int j = 0; j < kTok; ++j, ty += a.ld_y)
        if (decltype(whole)::value || j < nt) {
          float y[C], v[C];
          v[0] = *reinterpret_cast<const float*>(rd.row(0, j));
          if constexpr (C == 2) v[1] = *reinterpret_cast<const float*>(rd.row(1, j));
          P::split(P::fma(P::make(v), in2, hs[j]), y);
          store_row<T, decltype(whole)::value, kVec>(ty, y, left);
        }
    };
    if (nt == kTok && (f.group + 1) * kTileCh<T> <= a.dim) emit(std::true_type{});
    else emit(std::false_type{});
    __syncwarp();  // every lane is done with this stage
    load(i + kFwdStages<kVec>);
  }
  __syncthreads();
  if (threadIdx.x == 0 && s.abort) atomicAdd(&g_recurrence_timeouts, 1u);
}

// ------------------------------------------------------------------ backward

// One stage, so that three CTAs fit an SM (the gates are made twice for that, too: kept, they take the registers of
// the third). Against two stages and two CTAs, 65 536 tokens by 2 048 channels: one run 289 us and 305, eight 263 and 266,
// 512 270 and 262. (A tile taken further ahead is waited for longer: with the next tile's ticket taken and its rows fetched
// into L2 meanwhile one run took a fifth longer.)
constexpr int kBwdStages = 1;
template <bool kVec> constexpr int kBwdStage = 3 * kChunkR * kPitch<kVec>;

template <typename T>
struct BwdShared {
  Info info[kInfos];
  float A[kWarps][kTileCh<T>], R[kWarps][kTileCh<T>];
  Before<T> before;
  float dlo[kWarps][kTileCh<T>];
  alignas(8) uint64_t full[kBwdStages][kWarps];
  uint32_t abort;
};

template <typename T, bool kVec, int kMost>
__global__ void __launch_bounds__(kThreads, kCtas)
rec_bwd_kernel(const __grid_constant__ RecBwdTensors a, const __grid_constant__ Runs<kMost> t, const __grid_constant__ CUtensorMap mx,
               const __grid_constant__ CUtensorMap mg, const __grid_constant__ CUtensorMap md,
               const __grid_constant__ Chain ch, float* part, const int items, const int groups) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ BwdShared<T> s;
  constexpr int C = kCh<T>;
  using P = Pack<C>;
  using V = typename P::V;
  constexpr uint32_t kMat = kChunkR * kPitch<kVec>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (a.dstate)  // a run of no token hands its gradient on
    for (int i = blockIdx.x; i < t.n; i += gridDim.x)
      if (t.cu[i] == t.cu[i + 1])
        for (int c = threadIdx.x; c < a.dim; c += kThreads)
          a.dstate[(int64_t)i * a.dim + c] = a.dstate_end ? a.dstate_end[(int64_t)i * a.dim + c] : 0.0f;

  const Stream<T> in_streams[3] = {{static_cast<const T*>(a.x), a.ld_x, &mx},
                                   {static_cast<const T*>(a.gate), a.ld_gate, &mg},
                                   {static_cast<const T*>(a.dy), a.ld_dy, &md}};
  auto load = [&](int i) {
    load_tile<T, kVec, 3>(s.info[i % kInfos], in_streams, su32(stages) + (uint32_t)(i % kBwdStages) * kBwdStage<kVec>,
                          su32(&s.full[i % kBwdStages][warp]), a.dim, warp, lane);
  };
  if (threadIdx.x < kBwdStages * kWarps) {
    mbar_init(su32(&s.full[0][0] + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s.abort = 0u;
  }
  // the sum of a finished tile's eight parts of dlower (one warp, a tile later)
  auto sum_part = [&](int i) {
    const Info& f = s.info[i % kInfos];
    const int ch0 = f.group * kTileCh<T> + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s.dlo[w][lane * C + c];
      if (ch0 + c < a.dim) part[(int64_t)f.chunk * a.dim + ch0 + c] = v;
    }
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < kBwdStages; ++i)
      tile_info<true>(s.info[i], t, take<kBwdStages>(ch, i, items), items, groups);
  __syncthreads();
  for (int i = 0; i < kBwdStages; ++i) load(i);

  uint32_t phases = 0;
  int i = 0;
  for (;; ++i) {
    const Info f = s.info[i % kInfos];
    if (f.item < 0) break;
    const int ch0 = f.group * kTileCh<T> + lane * C;
    const int left = a.dim - ch0;
    int next = 0;
    if (threadIdx.x == kTaker) next = take<kBwdStages>(ch, i + kBwdStages, items);
    const int first = t.tile[f.seq];
    const int before = f.l > 0 ? maps_before(f.l, ch.shift) : 0;
    float h0[C];
    if (warp == 0 && f.l == 0)
#pragma unroll
      for (int c = 0; c < C; ++c)
        h0[c] = c < left && a.dstate_end ? a.dstate_end[(int64_t)f.seq * a.dim + ch0 + c] : 0.0f;
    unsigned char* st = stages + (i % kBwdStages) * kBwdStage<kVec>;
    const Reader<T, kVec, 3> rd(st, f, in_streams, warp, lane);
    float lo[C], un[C], hp[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      lo[c] = a.lower && c < left ? a.lower[ch0 + c] : 0.0f;
      un[c] = 1.0f - lo[c];
      hp[c] = c < left && warp * kTok < f.n ? a.ckpt[((int64_t)f.chunk * kWarps + warp) * a.dim + ch0 + c] : 0.0f;
    }
    const V un2 = P::make(un), lo2 = P::fma(un2, P::all(-kLeast), P::make(lo));  // (f = up un + lo)
    const int nt = min(kTok, f.n - warp * kTok);
    if (nt > 0) {
      wait_tile<kVec>(su32(&s.full[i % kBwdStages][warp]), phases >> (i % kBwdStages) & 1u, &s.abort);
      phases ^= 1u << (i % kBwdStages);
    }
    // ---- the states from the checkpoint on, and R's map (A, R)
    V hs[kTok];  // the state before the token
    V A2 = P::all(1.0f), R2 = P::all(0.0f), hp2 = P::make(hp);
    auto scan = [&](auto whole) {
#pragma unroll
      for (int j = 0; j < kTok; ++j)
        if (decltype(whole)::value || j < nt) {
          float x[C], g[C], d[C];
          unpack_word<T>(rd.word(0, j), x);
          unpack_word<T>(rd.word(1, j), g);
          unpack_word<T>(rd.word(2, j), d);
          V up, down;
          both_sigmoids<C>(g, up, down);
          const V ft = P::fma(un2, up, lo2);
          hs[j] = hp2;
          hp2 = P::fma(ft, hp2, P::mul(P::mul(un2, down), P::make(x)));
          A2 = P::mul(A2, ft);
          R2 = P::fma(A2, P::make(d), R2);
        }
    };
    if (nt == kTok) scan(std::true_type{});
    else scan(std::false_type{});
    float A[C], R[C], ea[C], eb[C];
    P::split(A2, A);
    P::split(R2, R);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s.A[warp][lane * C + c] = A[c];
      s.R[warp][lane * C + c] = R[c];
    }
    __syncthreads();
    if (warp == 1 && i > 0 && part) sum_part(i - 1);
    // the map of R after this warp, and of the tile (warp 0)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ea[c] = 1.0f;
      eb[c] = 0.0f;
    }
    for (int w = kWarps - 1; w > warp; --w)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float wa = s.A[w][lane * C + c];
        eb[c] = fmaf(wa, eb[c], s.R[w][lane * C + c]);
        ea[c] *= wa;
      }
    if (warp == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {  // its own tokens are the last of the pass
        R[c] = fmaf(A[c], eb[c], R[c]);
        A[c] *= ea[c];
      }
      if (f.l == 0) {
        float end[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          s.before.state[lane * C + c] = h0[c];
          end[c] = fmaf(A[c], h0[c], R[c]);
        }
        if (!f.last) publish_state<T>(ch, f, first, groups, end, lane);
      } else if (!f.last) {
        publish_map<T>(ch, f, groups, A, R, lane);
      }
    }
    // info[i + 2] takes the place of tile i - 2, whose part of dlower has been summed
    if (threadIdx.x == kTaker) tile_info<true>(s.info[(i + kBwdStages) % kInfos], t, next, items, groups);
    look_back<T, true>(ch, f, first, groups, before, s.before, warp, lane);
    __syncthreads();
    float in[C];
    fold_before(s.before, before, in, lane);
    if (warp == 0) {
      float end[C];
#pragma unroll
      for (int c = 0; c < C; ++c) end[c] = fmaf(A[c], in[c], R[c]);
      if (f.last) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (a.dstate && c < left) a.dstate[(int64_t)f.seq * a.dim + ch0 + c] = end[c];
      } else if (f.l > 0 && (f.l & ((1 << ch.shift) - 1)) == 0) {
        publish_state<T>(ch, f, first, groups, end, lane);
      }
    }
    // ---- backwards over the tokens
    T* ox = static_cast<T*>(a.dx) + (f.row + warp * kTok + kTok - 1) * a.ld_dx + ch0;
    T* og = static_cast<T*>(a.dgate) + (f.row + warp * kTok + kTok - 1) * a.ld_dgate + ch0;
    V in2 = P::fma(P::make(ea), P::make(in), P::make(eb)), dlo2 = P::all(0.0f);
    auto emit = [&](auto whole) {
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j, ox -= a.ld_dx, og -= a.ld_dgate)
        if (decltype(whole)::value || j < nt) {
          float x[C], g[C], d[C], vx[C], vg[C];
          unpack_word<T>(rd.word(0, j), x);
          unpack_word<T>(rd.word(1, j), g);
          unpack_word<T>(rd.word(2, j), d);
          V up, down;
          both_sigmoids<C>(g, up, down);
          const V ft = P::fma(un2, up, lo2);
          const V G = P::add(in2, P::make(d));
          // df sigmoid(-g), with df = G (h - x)
          const V dd = P::mul(P::mul(G, P::fma(P::make(x), P::all(-1.0f), hs[j])), down);
          P::split(P::mul(P::mul(un2, down), G), vx);
          P::split(P::mul(P::mul(dd, un2), P::add(up, P::all(-kLeast))), vg);
          dlo2 = P::add(dlo2, dd);
          in2 = P::mul(ft, G);
          store_row<T, decltype(whole)::value, kVec>(ox, vx, left);
          store_row<T, decltype(whole)::value, kVec>(og, vg, left);
        }
    };
    if (nt == kTok && (f.group + 1) * kTileCh<T> <= a.dim) emit(std::true_type{});
    else emit(std::false_type{});
    float dlo[C];
    P::split(dlo2, dlo);
#pragma unroll
    for (int c = 0; c < C; ++c) s.dlo[warp][lane * C + c] = dlo[c];
    __syncwarp();  // every lane is done with this stage
    load(i + kBwdStages);
  }
  __syncthreads();
  if (warp == 1 && i > 0 && part) sum_part(i - 1);
  if (threadIdx.x == 0 && s.abort) atomicAdd(&g_recurrence_timeouts, 1u);
}

// ------------------------------------------------------------------ single tokens

// One token of each sequence: a CTA takes 1 024 channels of a sequence, a thread four (adjacent ones where rows
// are aligned for them, else every 256th). At most 8 bytes of state and 3 elements a channel: a full batch is
// bound by HBM, a small one by the launch, so a device batch of up to kCheckHere sequences is checked by every
// CTA itself before it touches anything, instead of by a kernel of its own.
constexpr int kStepThreads = 256;
constexpr int kCheckHere = kStepThreads;

template <typename T, bool kVec>
__global__ void __launch_bounds__(kStepThreads) rec_step_kernel(const __grid_constant__ RecStepArgs a) {
  const int i = blockIdx.y;
  // everything is asked for before anything is waited for: the batch, the inputs, and, as soon as the slot is known
  // to be one, its state (a batch that turns out bad is not written)
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
  const int c0 = blockIdx.x * 4 * kStepThreads;
  auto channel = [&](int j) { return c0 + (kVec ? 4 * (int)threadIdx.x + j : (int)threadIdx.x + j * kStepThreads); };
  const T* x = static_cast<const T*>(a.x) + i * a.ld_x;
  const T* gate = static_cast<const T*>(a.gate) + i * a.ld_gate;
  float xv[4], gv[4], h[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) xv[j] = gv[j] = h[j] = lo[j] = 0.0f;
  auto four = [](const auto* p, float (&v)[4]) {
    if constexpr (sizeof(*p) == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xffff0000u);
    }
  };
  const bool any = channel(0) < a.dim;  // (kVec: all four or none)
  if constexpr (kVec) {
    if (any) {
      four(x + channel(0), xv);
      four(gate + channel(0), gv);
      if (a.lower) four(a.lower + channel(0), lo);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (channel(j) < a.dim) {
        xv[j] = Act<T>::to_f(x[channel(j)]);
        gv[j] = Act<T>::to_f(gate[channel(j)]);
        if (a.lower) lo[j] = a.lower[channel(j)];
      }
  }
  const bool is_slot = slot >= 0 && slot < a.num_slots;
  float* st = a.state + (int64_t)(is_slot ? slot : 0) * a.dim;
  if (is_slot && !fresh) {
    if constexpr (kVec) {
      if (any) four(st + channel(0), h);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (channel(j) < a.dim) h[j] = st[channel(j)];
    }
  }
  if (a.dev_slots) {
    if (a.n <= kCheckHere) {
      const int status = check_batch<kStepThreads>(num, a.n, a.num_slots, mine);
      if (blockIdx.x == 0 && i == 0 && threadIdx.x == 0) *a.dev_status = status;
      if (status != MAMBA2_OK) return;
    } else if (*a.dev_status != MAMBA2_OK) {
      return;
    }
    if (i >= num) return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float up, down;
    sigmoids(gv[j], up, down);
    h[j] = fmaf(fmaf(1.0f - lo[j], up, lo[j]), h[j], (1.0f - lo[j]) * down * xv[j]);
  }
  T* y = static_cast<T*>(a.y) + i * a.ld_y;
  if constexpr (kVec) {
    if (!any) return;
    *reinterpret_cast<float4*>(st + channel(0)) = make_float4(h[0], h[1], h[2], h[3]);
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(y + channel(0)) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
      const __nv_bfloat162 p = __floats2bfloat162_rn(h[0], h[1]), q = __floats2bfloat162_rn(h[2], h[3]);
      *reinterpret_cast<uint2*>(y + channel(0)) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (channel(j) < a.dim) {
        st[channel(j)] = h[j];
        y[channel(j)] = Act<T>::from_f(h[j]);
      }
  }
}

bool rows16(const void* p, int64_t ld, size_t e) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (size_t)ld * e % 16 == 0;
}

// CTAs of a launch: so many to an SM, no more than tiles; empty runs need one.
int ctas(int64_t items, int per_sm) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(items, per_sm * (int64_t)device_sm_count()));
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encode_fn() {
  static Encode fn = []() -> Encode {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return fn;
}
// [rows][dim] with a row stride of ld elements: boxes of 128 bytes x kTok rows, zeros past the edges
template <typename T>
bool make_map(CUtensorMap* tm, const void* base, int64_t rows, int64_t dim, int64_t ld) {
  const Encode enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)dim, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * sizeof(T)};
  const cuuint32_t box[2] = {(cuuint32_t)kTileCh<T>, (cuuint32_t)kTok}, estr[2] = {1, 1};
  return enc(tm, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t tiles_at_once() { return (int64_t)kCtas * device_sm_count(); }
// Runs whose chunks are taken in turns: as many as fill the GPU (64 runs of 65 536 x 2 048 took 2 % longer with twice and
// 7 % with four times as many).
int runs_in_turn(int64_t groups) { return (int)((tiles_at_once() + groups - 1) / groups); }
// log2 of the chunks between two published states: as few as keep a state's readers a wave of tiles behind it (the
// fewer, the fewer maps to read and fold). runs: those in turn, on average.
int state_shift(int64_t runs, int64_t groups) {
  int shift = kLeastShift;
  while (shift < kMostShift && (runs * groups << shift) < tiles_at_once()) ++shift;
  return shift;
}

// The plan that both passes share: tiles, and the chain (cleared on the stream) when a run has several.
struct Tiles {
  int groups, items;
  Chain chain;
  int turn;  // runs that take turns; 0: none do
  cudaError_t status;
};
Tiles plan(const SeqTable& t, mamba2_dtype act, int32_t dim, void* ws, cudaStream_t st) {
  Tiles p;
  p.chain = {};
  p.turn = 0;
  p.status = cudaSuccess;
  const int width = act == MAMBA2_BF16 ? kTileCh<__nv_bfloat16> : kTileCh<float>;
  p.groups = (dim + width - 1) / width;
  const int64_t chunks = t.tile[t.n], items = chunks * p.groups;
  if (items > 0x3fffffff) {
    p.status = cudaErrorInvalidValue;
    return p;
  }
  p.items = (int)items;
  int longest = 0;
  for (int i = 0; i < t.n; ++i) longest = std::max(longest, t.tile[i + 1] - t.tile[i]);
  if (longest > 1) {
    if (t.n > 1) p.turn = runs_in_turn(p.groups);
    const int shift = state_shift(p.turn == 0 ? 1 : std::min<int64_t>(p.turn, chunks / longest), p.groups);
    p.chain = chain_at(ws, chunks, (int64_t)p.groups * width, shift);
    p.status = cudaMemsetAsync(ws, 0xff, chain_bytes(chunks, t.n, (int64_t)p.groups * width, shift), st);
  }
  return p;
}

template <typename T, bool kVec>
cudaError_t run_fwd(const RecArgs& a, const Tiles& p, cudaStream_t st) {
  constexpr int smem = kFwdStages<kVec> * kFwdStage<kVec>;
  CUtensorMap mx, mg;
  std::memset(&mx, 0, sizeof mx);
  std::memset(&mg, 0, sizeof mg);
  const int rows = a.tab.cu[a.tab.n];
  if (kVec && rows > 0 && !(make_map<T>(&mx, a.x, rows, a.dim, a.ld_x) && make_map<T>(&mg, a.gate, rows, a.dim, a.ld_gate)))
    return cudaErrorInvalidValue;
  auto run = [&](auto kernel, auto most) {
    Runs<decltype(most)::value> runs;
    fill_runs(runs, a.tab, p.turn);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<ctas(p.items, kCtas), kThreads, smem, st>>>(a, runs, mx, mg, p.chain, p.items, p.groups);
    return cudaGetLastError();
  };
  if (a.tab.n <= kFewRuns) return run(rec_fwd_kernel<T, kVec, kFewRuns>, std::integral_constant<int, kFewRuns>());
  return run(rec_fwd_kernel<T, kVec, MAMBA2_MAX_SEQS>, std::integral_constant<int, MAMBA2_MAX_SEQS>());
}
template <typename T, bool kVec>
cudaError_t run_bwd(const RecBwdArgs& a, const Tiles& p, float* part, cudaStream_t st) {
  constexpr int smem = kBwdStages * kBwdStage<kVec>;
  CUtensorMap mx, mg, md;
  std::memset(&mx, 0, sizeof mx);
  std::memset(&mg, 0, sizeof mg);
  std::memset(&md, 0, sizeof md);
  const int rows = a.tab.cu[a.tab.n];
  if (kVec && rows > 0 &&
      !(make_map<T>(&mx, a.x, rows, a.dim, a.ld_x) && make_map<T>(&mg, a.gate, rows, a.dim, a.ld_gate) &&
        make_map<T>(&md, a.dy, rows, a.dim, a.ld_dy)))
    return cudaErrorInvalidValue;
  auto run = [&](auto kernel, auto most) {
    Runs<decltype(most)::value> runs;
    fill_runs(runs, a.tab, p.turn);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<ctas(p.items, kCtas), kThreads, smem, st>>>(a, runs, mx, mg, md, p.chain, part, p.items, p.groups);
    return cudaGetLastError();
  };
  if (a.tab.n <= kFewRuns) return run(rec_bwd_kernel<T, kVec, kFewRuns>, std::integral_constant<int, kFewRuns>());
  return run(rec_bwd_kernel<T, kVec, MAMBA2_MAX_SEQS>, std::integral_constant<int, MAMBA2_MAX_SEQS>());
}

}  // namespace

size_t recurrence_workspace(int64_t chunks, bool chained, int32_t runs, int32_t dim, bool backward) {
  const size_t part = backward ? ((size_t)chunks * dim * 4 + 255) / 256 * 256 : 0;
  // (either type's groups together are at most 63 channels wider than dim)
  return part + (chained ? (chain_bytes(chunks, runs, (int64_t)dim + 63, kLeastShift) + 255) / 256 * 256 : 0);
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
    return vec ? run_fwd<__nv_bfloat16, true>(a, p, st)
               : run_fwd<__nv_bfloat16, false>(a, p, st);
  return vec ? run_fwd<float, true>(a, p, st)
             : run_fwd<float, false>(a, p, st);
}

cudaError_t launch_recurrence_backward(const RecBwdArgs& a, mamba2_dtype act, void* ws, cudaStream_t st) {
  const int64_t chunks = a.tab.tile[a.tab.n];
  float* part = a.dlower ? static_cast<float*>(ws) : nullptr;
  const Tiles p = plan(a.tab, act, a.dim, static_cast<char*>(ws) + recurrence_workspace(chunks, false, 0, a.dim, true), st);
  if (p.status != cudaSuccess) return p.status;
  const size_t es = act == MAMBA2_BF16 ? 2 : 4;
  const bool vec = rows16(a.x, a.ld_x, es) && rows16(a.gate, a.ld_gate, es) && rows16(a.dy, a.ld_dy, es) &&
                   rows16(a.dx, a.ld_dx, es) && rows16(a.dgate, a.ld_dgate, es);
  cudaError_t e;
  if (act == MAMBA2_BF16)
    e = vec ? run_bwd<__nv_bfloat16, true>(a, p, part, st)
            : run_bwd<__nv_bfloat16, false>(a, p, part, st);
  else
    e = vec ? run_bwd<float, true>(a, p, part, st)
            : run_bwd<float, false>(a, p, part, st);
  if (e == cudaSuccess && a.dlower) e = launch_column_sum(a.dlower, part, (int)chunks, a.dim, st);
  return e;
}

cudaError_t launch_recurrence_step(const RecStepArgs& a, mamba2_dtype act, cudaStream_t st) {
  if (a.dev_slots && a.n > kCheckHere) {
    const cudaError_t e = launch_check_device_batch(a.dev_slots, a.dev_n, a.n, a.num_slots, a.dev_status, st);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((a.dim + 4 * kStepThreads - 1) / (4 * kStepThreads), a.n);
  const size_t e = act == MAMBA2_BF16 ? 2 : 4;
  auto fours = [&](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & (4 * e - 1)) == 0 && ld % 4 == 0; };
  const bool vec = a.dim % 4 == 0 && fours(a.x, a.ld_x) && fours(a.gate, a.ld_gate) && fours(a.y, a.ld_y);
  if (act == MAMBA2_BF16) {
    if (vec) rec_step_kernel<__nv_bfloat16, true><<<grid, kStepThreads, 0, st>>>(a);
    else rec_step_kernel<__nv_bfloat16, false><<<grid, kStepThreads, 0, st>>>(a);
  } else {
    if (vec) rec_step_kernel<float, true><<<grid, kStepThreads, 0, st>>>(a);
    else rec_step_kernel<float, false><<<grid, kStepThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace mamba2
