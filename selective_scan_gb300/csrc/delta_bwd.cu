// Gated delta rule, backward (delta.h), bf16, d_state and headdim of at most 128; delta_chunk.cu has the notation.
//
// With dO the gradient of y, dS1 that of the state behind a chunk, everything that depends on both directions of time
// goes through dS. For a chunk, rows of tokens:
//   dU = left (K dS1^T) + P^T dO,  dV = Inv^T (beta dU),  dS0 = exp(G_C) dS1 + (upq dO)^T Q - (up dV)^T K
// Three kernels: the records of every chunk and head; dS through a run's chunks from its last to its first, a warp to 16
// of its rows as in the forward pass, which leaves dV and every chunk's dS1; then the other gradients, every chunk by
// itself. For those, with r the corrections (u = beta r) and D_ij = exp(G_i - G_j),
//   Pr = dO r^T,  Er = dV r^T,  F_ij = beta_j Pr_ij D_ij scale kappa_q,i kappa_j (j <= i),  E_ij = beta_j Er_ij D_ij kappa_i kappa_j (j < i)
//   dq = upq dO S0 + F K,   dk = - up dV S0 - E K + F^T Q - E^T K + beta left r dS1   (lengths taken as constant)
//   dbeta_j = left_j (r dS1)_j . k_j + sum_i P_ij Pr_ij - sum_i L_ij Er_ij
// and g_t reaches what a state before it gives to a row at or behind it:
//   dg_t = exp(G_C) <dS1, S0> + sum_{i>=t} a_i + sum_{j<t} b_j + sum_{i>=t>j} W_ij,
//   W_ij = beta_j (P_ij Pr_ij - L_ij Er_ij),  a_i = upq_i dO_i S0 q_i - up_i dV_i S0 k_i,  b_j = beta_j left_j (r dS1)_j . k_j,
// summed without differences of its terms: what a token forgets is an exact zero in each, so dg is 0 where nothing is left
// of the state. For t in the chunk's 16 rows T, the double sum is that of W's column sums over row blocks I > T up to
// column t, of its rows from t to T's last left of T's columns, and of the same rows within T's own block.
//
// What is rounded: dS, dU, dV and the triangles enter products that end in dS or dV as two bf16 numbers each (2^-16 of
// them), and so do S0, R and Inv where they end in r: r is what the state has not predicted of v, a small difference of
// large numbers once the state has learnt them, and dbeta and a part of dk are proportional to it. r itself, and what
// else ends in dq, dk, dg and dbeta, which are bf16, enters as one (2^-9). dV between the kernels is its output in bf16, a
// chunk's dS1 a bf16 operand; their sums are fp32.
//
// 8 192 tokens, 8 runs, 16 heads of 128 x 128: the records 32 us, dS 123, the other gradients 206, of which r from
// operands in two parts 23 and dg 4 (0.32 GB in and out of the call in all: 0.9 TB/s).
#include <algorithm>
#include <type_traits>

#include "../../include/delta.h"
#include "common.cuh"
#include "delta_tiles.h"
#include "host.h"

namespace mamba2 {

__device__ unsigned int g_delta_back_timeouts = 0;

namespace {

#include "delta_mma.cuh"

using bf16 = __nv_bfloat16;

// A state as an operand: 64 of its rows to a tile (those behind the last strip of 16 are not written).
template <int DK>
constexpr int kStateTile = 64 * DK * 2;
__host__ __device__ constexpr int state_tiles(int dv) { return (dv + 63) / 64; }

// ------------------------------------------------------------------ dS through the chunks

// As the forward chain: products that wait for one another, in two warps a scheduler.

template <int DK, int NW>
struct Back : Stages<DK, true, NW, 2> {
  // Inv and P, of one chunk: the next one's come while dS is updated (two of them would leave an SM one CTA)
  static constexpr int kTriangles = Stages<DK, true, NW, 2>::kEnd, kOffBar = kTriangles + 4 * kTri, kSmem = kOffBar + 32;
};

template <int DK, int NW>
__global__ void __launch_bounds__(32 * NW, 2) delta_back_kernel(const __grid_constant__ DeltaBwdArgs a, const __grid_constant__ DeltaMaps maps, const unsigned char* records, unsigned char* ds) {
  using L = Back<DK, NW>;
  constexpr int KS = DK / 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = sm32(smem);
  if (not_aligned(base, &g_delta_back_timeouts)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int run = a.order[blockIdx.z], h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int dv0 = blockIdx.x * 16 * NW, dv = dv0 + 16 * warp;
  const int first = a.tab.cu[run], len = a.tab.cu[run + 1] - first, n = (len + kC - 1) / kC;
  auto bar = [&](int ch) { return base + L::kOffBar + 8u * (uint32_t)(ch & 1); };
  const uint32_t tri_bar = base + L::kOffBar + 16, rec = base + L::kTriangles;
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBar + 24);
  if (threadIdx.x == 0) {
    bar_init(bar(0), 32);
    bar_init(bar(1), 32);
    bar_init(tri_bar, 1);
    *gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  float s[2 * KS][4];  // dS: rows dv + g and + 8, columns 8 n + 2 t and + 1
  const int64_t at0 = (int64_t)(dv + g) * a.dk + 2 * t, mine = ((int64_t)run * a.heads + h) * a.dv * a.dk;
  auto each = [&](auto f) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
      if (dv + 8 * half < a.dv)
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i)
          if (8 * i < a.dk) f(s[i] + 2 * half, at0 + (int64_t)(8 * half) * a.dk + 8 * i);
  };
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
  if (a.dstate_end)
    each([&](float* v, int64_t at) {
      const float2 f = *reinterpret_cast<const float2*>(a.dstate_end + mine + at);
      v[0] = f.x;
      v[1] = f.y;
    });
  auto fetch = [&](int ch) {  // (warp 0)
    load_stage<DK, true, NW, 2>(ch, base, bar(ch), a, maps, a.dy, a.ld_dy,
                             records + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * record_bytes(true),
                             first + (int64_t)ch * kC, min(kC, len - ch * kC), grp, h, dv0, lane);
  };
  auto fetch_triangles = [&](int ch) {  // (a thread)
    const unsigned char* from = records + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * record_bytes(true);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tri_bar), "r"((uint32_t)(4 * kTri)) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(rec), "l"(from), "r"((uint32_t)(4 * kTri)), "r"(tri_bar) : "memory");
  };
  if (n > 0 && warp == 0) {
    fetch(n - 1);
    if (lane == 0) fetch_triangles(n - 1);
  }
  for (int ch = n - 1; ch >= 0; --ch) {
    if (ch < n - 1) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (dv was written where another chunk's dO comes)
      __syncthreads();  // every warp is done with the other stage
    }
    if (ch > 0 && warp == 0) fetch(ch - 1);
    bar_wait(bar(ch), (uint32_t)(((n - 1 - ch) >> 1) & 1), gave_up);
    __syncwarp();
    const uint32_t at = base + L::k(ch), qt = base + L::q(ch), dt = base + L::v(ch) + warp * L::kStrip;
    const float* f = reinterpret_cast<const float*>(smem + L::rec(ch));
    {  // dS1, for the gradients that take it as an operand (rounded as such), as they hold it in shared memory
      unsigned char* o = ds + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * state_tiles(a.dv) * kStateTile<DK> +
                         (dv >> 6) * kStateTile<DK>;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i)
          *reinterpret_cast<uint32_t*>(o + wide_at((dv & 63) + g + 8 * half, i) + 4 * t) = pair(s[i][2 * half], s[i][2 * half + 1]);
    }
    // dU^T = left (dS1^T)^T K^T + dO^T P
    float x[8][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t sh[4], sl[4], b[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(s[2 * ks + (j >> 1)][2 * (j & 1)], s[2 * ks + (j >> 1)][2 * (j & 1) + 1], sh[j], sl[j]);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        load4(b[nb], at + wide_rows(16 * nb, 2 * ks, lane));
        mma_if(ks == 0, x[2 * nb], sh, b[nb][0], b[nb][1]);
        mma_if(ks == 0, x[2 * nb + 1], sh, b[nb][2], b[nb][3]);
      }
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        mma(x[2 * nb], sl, b[nb][0], b[nb][1]);
        mma(x[2 * nb + 1], sl, b[nb][2], b[nb][3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 w = *reinterpret_cast<const float2*>(f + kLeft + 8 * i + 2 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] *= j & 1 ? w.y : w.x;
    }
    bar_wait(tri_bar, (uint32_t)((n - 1 - ch) & 1), gave_up);
    __syncwarp();
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      uint32_t v[4];
      load4t(v, dt + narrow_cols(16 * ib, lane));
      const uint32_t d[4] = {v[0], v[2], v[1], v[3]};
#pragma unroll
      for (int jb = 0; jb <= ib; ++jb) {
        uint32_t b[4];
        load4t(b, rec + kOffP + block_at(ib, jb) + narrow_cols(0, lane));
        mma(x[2 * jb], d, b[0], b[1]);
        mma(x[2 * jb + 1], d, b[2], b[3]);
      }
#pragma unroll
      for (int jb = 0; jb <= ib; ++jb) {
        uint32_t b[4];
        load4t(b, rec + kOffPLo + block_at(ib, jb) + narrow_cols(0, lane));
        mma(x[2 * jb], d, b[0], b[1]);
        mma(x[2 * jb + 1], d, b[2], b[3]);
      }
    }
    // dV^T = (beta dU)^T Inv
    float y[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = 0.0f;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      uint32_t uh[4], ul[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 2 * ib + (j >> 1);
        const float2 w = *reinterpret_cast<const float2*>(f + kBeta + 8 * i + 2 * t);
        split(x[i][2 * (j & 1)] * w.x, x[i][2 * (j & 1) + 1] * w.y, uh[j], ul[j]);
      }
#pragma unroll
      for (int jb = 0; jb <= ib; ++jb) {
        uint32_t bh[4], bl[4];
        load4t(bh, rec + block_at(ib, jb) + narrow_cols(0, lane));
        load4t(bl, rec + kOffInvLo + block_at(ib, jb) + narrow_cols(0, lane));
        mma(y[2 * jb], uh, bh[0], bh[1]);
        mma(y[2 * jb + 1], uh, bh[2], bh[3]);
        mma(y[2 * jb], ul, bh[0], bh[1]);
        mma(y[2 * jb + 1], ul, bh[2], bh[3]);
        mma(y[2 * jb], uh, bl[0], bl[1]);
        mma(y[2 * jb + 1], uh, bl[2], bl[3]);
      }
    }
    if (ch > 0) {
      __syncthreads();  // every warp is done with the triangles
      if (threadIdx.x == 0) fetch_triangles(ch - 1);
    }
    // dS0 = gamma dS1 + (upq dO)^T Q - (up dV)^T K
    const float gamma = f[kGamma];
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] *= gamma;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t v[4], oh[4], ol[4], vh[4], vl[4];
      load4t(v, dt + narrow_cols(16 * jb, lane));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 2 * jb + (j >> 1);
        const float2 wq = *reinterpret_cast<const float2*>(f + kUpQ + 8 * i + 2 * t);
        const float2 w = *reinterpret_cast<const float2*>(f + kUp + 8 * i + 2 * t);
        const uint32_t o = v[(j >> 1) + 2 * (j & 1)];
        split(__uint_as_float(o << 16) * wq.x, __uint_as_float(o & 0xffff0000u) * wq.y, oh[j], ol[j]);
        split(-w.x * y[i][2 * (j & 1)], -w.y * y[i][2 * (j & 1) + 1], vh[j], vl[j]);
      }
#pragma unroll
      for (int nb = 0; nb < KS; ++nb) {
        uint32_t b[4];
        load4t(b, qt + wide_cols(16 * jb, 2 * nb, lane));
        mma(s[2 * nb], oh, b[0], b[1]);
        mma(s[2 * nb + 1], oh, b[2], b[3]);
        mma(s[2 * nb], ol, b[0], b[1]);
        mma(s[2 * nb + 1], ol, b[2], b[3]);
        load4t(b, at + wide_cols(16 * jb, 2 * nb, lane));
        mma(s[2 * nb], vh, b[0], b[1]);
        mma(s[2 * nb + 1], vh, b[2], b[3]);
        mma(s[2 * nb], vl, b[0], b[1]);
        mma(s[2 * nb + 1], vl, b[2], b[3]);
      }
    }
    __syncwarp();  // every lane has read dO
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
      store4t(dt + narrow_cols(16 * jb, lane), pair(y[2 * jb][0], y[2 * jb][1]), pair(y[2 * jb + 1][0], y[2 * jb + 1][1]),
              pair(y[2 * jb][2], y[2 * jb][3]), pair(y[2 * jb + 1][2], y[2 * jb + 1][3]));
    __syncwarp();
    const int m = min(kC, len - ch * kC), col = dv + 8 * (lane & 1);
    bf16* out = static_cast<bf16*>(a.dv_out) + (first + (int64_t)ch * kC) * a.ld_dv + (int64_t)h * a.dv + col;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int tok = 16 * it + (lane >> 1);
      if (tok < m && col < a.dv)
        *reinterpret_cast<uint4*>(out + tok * a.ld_dv) =
            *reinterpret_cast<const uint4*>(smem + (dt - base) + narrow_at(tok, lane & 1));
    }
  }
  if (a.dstate) each([&](float* v, int64_t at) { *reinterpret_cast<float2*>(a.dstate + mine + at) = make_float2(v[0], v[1]); });
  if (lane == 0 && *gave_up) atomicAdd(&g_delta_back_timeouts, 1u);
}

// ------------------------------------------------------------------ the other gradients

// An item is a chunk and one group of keys, its heads one after another, so that what they add to a query or key is
// summed in registers in their order; a head in steps of 64 of its v channels, whose tiles are copied while the step
// before is worked on. A CTA an SM takes every so-manieth item (two an SM of half the width, one step's tiles at a time,
// took 254 us where this took 199 then). Bound by latency and shared memory: a product's operands are read again by every
// warp that has a part of it. A warp: 16 rows of the chunk, half of the columns; of
// the 64 x 64 products the first half has Pr and the other Er.
constexpr int kGradWarps = 8, kGradThreads = 32 * kGradWarps;

template <int DK>
struct Grad {
  static constexpr int kTileK = kC * DK * 2, kState = kStateTile<DK>, kTile = kC * 64 * 2;
  static constexpr int kK = 0, kQ = kTileK, kS0 = 4 * kTileK;  // K and Q twice: of the chunk at hand and the next
  // of each step, twice: dS, V (then R), dO, dV (then F and E, the last step of a head)
  static constexpr int kStep = kS0 + kState, kDS = 0, kV = kState, kDO = kV + kTile, kDV = kDO + kTile, kStepBytes = kDV + kTile;
  static constexpr int kF = kDO, kE = kDV;
  // kWide: S0 in fp32, until it is an operand; then what S0 and R leave of themselves as bf16 numbers
  static constexpr int kR = kStep + 2 * kStepBytes, kWide = kR + kTile, kS0Lo = kWide, kRLo = kWide + kState;
  // of each head, twice: Inv and the factors; Inv's second part once
  static constexpr int kHead = kWide + 64 * DK * 4, kFac = kTri, kHeadBytes = kTri + 9 * kC * 4, kInvLo = kHead + 2 * kHeadBytes;
  // floats at kVec: W's part of dg from a token's own row block [2 halves], sums of W's columns [2][4 row blocks] (without
  // beta), its diagonal, a and the write's rows
  // [2 halves], the inner product [8 warps]
  static constexpr int kVec = kInvLo + kTri;
  static constexpr int kRow = 0, kCol = 2 * kC, kDiag = 10 * kC, kA = 11 * kC, kWrite = 13 * kC, kDot = 15 * kC;
  static constexpr int kBar = kVec + (15 * kC + 16) * 4, kSmem = kBar + 32;  // barriers: the steps' two, S0's; the flag
  static_assert(kRLo + kTile <= kHead && kSmem <= 232448, "shared memory plan exceeds 227 KB");
};
struct GradMaps {
  CUtensorMap k, q, v, dy, dv;  // 64 rows of 64 columns of a head
};

__device__ __forceinline__ float sum_quad(float v) {  // over the lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float sum_behind(float v, int lane) {  // of this row and those behind it (of 8)
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += u;
  }
  return v;
}
__device__ __forceinline__ float sum_rows(float v) {  // over the lanes of a column
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

template <int DK>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaBwdArgs a, const __grid_constant__ GradMaps maps,
                                                                     const unsigned char* records, const unsigned char* ds) {
  using L = Grad<DK>;
  constexpr int KS = DK / 16, NK = DK / 16;  // steps over columns; column tiles of 8 of a half
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = sm32(smem);
  if (not_aligned(base, &g_delta_back_timeouts)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // (a scheduler's two warps have rows that add up to the same work in the triangles)
  const int part = warp >> 2, rb = part ? 3 - (warp & 3) : warp & 3, r0 = 16 * rb;
  const bool second = part == 1;  // of the 64 x 64 products: Er
  const int per = a.heads / a.groups, halves = state_tiles(a.dv), steps = per * halves;
  const unsigned items = (unsigned)a.tab.tile[a.tab.n] * (unsigned)a.groups, groups = (unsigned)a.groups;
  float* vec = reinterpret_cast<float*>(smem + L::kVec);
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kBar + 24);
  auto bar = [&](int i) { return base + L::kBar + 8u * (uint32_t)i; };  // 0, 1: a step's tiles; 2: its S0

  if (threadIdx.x == 0) {
    bar_init(bar(0), kGradThreads);
    bar_init(bar(1), kGradThreads);
    bar_init(bar(2), 1);
    *gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  auto bulk = [](uint32_t to, const void* from, int bytes, uint32_t b) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(to), "l"(from), "r"(bytes), "r"(b) : "memory");
  };
  // Of an item (a chunk and a group) and its i-th step the tiles, by every thread: whole chunks by tensor maps, a run's
  // last rows one by one (zeros behind them). n: steps of this CTA before it, m: items.
  auto fetch = [&](const Chunk& c, int chunk, int grp, int i, int n, int m) {
    const int h = grp * per + i / halves, half = i % halves;
    const uint32_t b = bar(n & 1), to = base + L::kStep + (uint32_t)(n & 1) * L::kStepBytes, kq = base + (uint32_t)(m & 1) * (2 * L::kTileK);
    if (threadIdx.x == 0) {
      const int64_t item = (int64_t)chunk * a.heads + h;
      const bool whole = c.len == kC;
      uint32_t bytes = L::kState + (whole ? 3 * L::kTile : 0);
      if (half == 0) bytes += L::kHeadBytes;
      if (i == 0 && whole) bytes += 2 * L::kTileK;
      asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
      bulk(to + L::kDS, ds + (item * halves + half) * L::kState, L::kState, b);
      if (whole) {
        if (i == 0) {
#pragma unroll
          for (int x = 0; x < DK / 64; ++x) {
            tma_3d(kq + L::kK + x * kC * 128, &maps.k, 64 * x, grp, c.row, b);
            tma_3d(kq + L::kQ + x * kC * 128, &maps.q, 64 * x, grp, c.row, b);
          }
        }
        tma_3d(to + L::kV, &maps.v, 64 * half, h, c.row, b);
        tma_3d(to + L::kDO, &maps.dy, 64 * half, h, c.row, b);
        tma_3d(to + L::kDV, &maps.dv, 64 * half, h, c.row, b);
      }
      if (half == 0) {
        const unsigned char* rec = records + item * record_bytes(true);
        const uint32_t head = base + L::kHead + (uint32_t)((m * per + i / halves) & 1) * L::kHeadBytes;
        bulk(head, rec, kTri, b);
        bulk(head + L::kFac, rec + off_factors(true), 9 * kC * 4, b);
      }
    }
    if (c.len < kC) {
      auto rows = [&](uint32_t at, const void* from, int64_t ld, int64_t col, int width, int units) {
        const bf16* p = static_cast<const bf16*>(from) + col;
        for (int e = threadIdx.x; e < kC * units; e += kGradThreads) {
          const int r = e / units, u = e % units;
          const bool in = r < c.len && 8 * u < width;
          copy16(at + wide_at(r, u), p + (int64_t)(c.row + (in ? r : 0)) * ld + (in ? 8 * u : 0), in);
        }
      };
      if (i == 0) {
        rows(kq + L::kK, a.k, a.ld_k, (int64_t)grp * a.dk, a.dk, DK / 8);
        rows(kq + L::kQ, a.q, a.ld_q, (int64_t)grp * a.dk, a.dk, DK / 8);
      }
      const int64_t col = (int64_t)h * a.dv + 64 * half;
      const int width = a.dv - 64 * half;
      rows(to + L::kV, a.v, a.ld_v, col, width, 8);
      rows(to + L::kDO, a.dy, a.ld_dy, col, width, 8);
      rows(to + L::kDV, a.dv_out, a.ld_dv, col, width, 8);
      bar_arrive_copies(b);  // (the barrier counts every thread)
    } else {
      bar_arrive(b);
    }
  };

  // And its S0, in fp32, with the second part of Inv: into the places that the step before has emptied (a thread).
  auto fetch_state = [&](int chunk, int grp, int i) {
    const int half = i % halves, rows = min(64, a.dv - 64 * half);
    const int64_t item = (int64_t)chunk * a.heads + grp * per + i / halves;
    const uint32_t bytes = (uint32_t)(rows * a.dk * 4 + (half == 0 ? kTri : 0));
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar(2)), "r"(bytes) : "memory");
    bulk(base + L::kWide, a.ckpt + (item * a.dv + 64 * half) * a.dk, rows * a.dk * 4, bar(2));
    if (half == 0) bulk(base + L::kInvLo, records + item * record_bytes(true) + kOffInvLo, kTri, bar(2));
  };

  float dq[NK][4], dk[NK][4];
  uint32_t kq0 = 0;  // where the item's K and Q are
  // the pair of a key or query that this thread's sum (column tile i of its half, row g + 8 e) is of
  auto pair_at = [&](uint32_t tile, int i, int e) -> uint32_t* {
    return reinterpret_cast<uint32_t*>(smem + kq0 + tile + wide_at(r0 + g + 8 * e, part * NK + i) + 4 * t);
  };
  float x[4][2][4], at_row[2], write_row[2], dot = 0.0f;  // Pr or Er; rows' parts of a and of the write; <dS1, S0>

  unsigned item = blockIdx.x;  // (no more CTAs than items)
  Chunk c = chunk_of(a.tab, (int)(item / groups));
  fetch(c, (int)(item / groups), (int)(item % groups), 0, 0, 0);
  if (threadIdx.x == 0) fetch_state((int)(item / groups), (int)(item % groups), 0);
  int n = 0;
  for (int m = 0; item < items; ++m, item += gridDim.x) {
  const int chunk = (int)(item / groups), grp = (int)(item % groups);
  const unsigned after = item + gridDim.x;
  const Chunk next = after < items ? chunk_of(a.tab, (int)(after / groups)) : c;
  kq0 = (uint32_t)(m & 1) * (2 * L::kTileK);
  const uint32_t kq = base + kq0;
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dq[i][j] = dk[i][j] = 0.0f;
  for (int i = 0; i < steps; ++i, ++n) {
    const int half = i % halves, hh = i / halves, h = grp * per + hh;
    const uint32_t st = L::kStep + (uint32_t)(n & 1) * L::kStepBytes;
    const unsigned char* head = smem + L::kHead + ((m * per + hh) & 1) * L::kHeadBytes;
    const uint32_t inv = sm32(head);
    const float* f = reinterpret_cast<const float*>(head + L::kFac);
    const int rows = min(64, a.dv - 64 * half);
    bar_wait(bar(n & 1), (uint32_t)((n >> 1) & 1), gave_up);
    bar_wait(bar(2), (uint32_t)(n & 1), gave_up);
    if (half == 0) {
      dot = at_row[0] = at_row[1] = write_row[0] = write_row[1] = 0.0f;
#pragma unroll
      for (int o = 0; o < 4; ++o)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[o][n][j] = 0.0f;
    }
    uint4 s0_lo[DK / 32];
#pragma unroll
    for (int z = 0; z < DK / 32; ++z) {  // S0 as an operand in two parts, and its product with dS1
      const int e = threadIdx.x + z * kGradThreads, r = e / (DK / 8), u = e % (DK / 8);
      uint4 w = make_uint4(0, 0, 0, 0);
      s0_lo[z] = w;
      if (r >= rows) *reinterpret_cast<uint4*>(smem + st + L::kDS + wide_at(r, u)) = w;  // (rows that the state has not)
      if (r < rows && 8 * u < a.dk) {
        float v[8], d[8];
        const float* from = reinterpret_cast<const float*>(smem + L::kWide) + r * a.dk + 8 * u;
        Vec16<float>::load(from, v);
        Vec16<float>::load(from + 4, v + 4);
        Vec16<bf16>::unpack(*reinterpret_cast<const uint4*>(smem + st + L::kDS + wide_at(r, u)), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(v[j], d[j], dot);
        split(v[0], v[1], w.x, s0_lo[z].x);
        split(v[2], v[3], w.y, s0_lo[z].y);
        split(v[4], v[5], w.z, s0_lo[z].z);
        split(v[6], v[7], w.w, s0_lo[z].w);
      }
      *reinterpret_cast<uint4*>(smem + L::kS0 + wide_at(r, u)) = w;
    }
    __syncthreads();  // S0 has been read
#pragma unroll
    for (int z = 0; z < DK / 32; ++z) {
      const int e = threadIdx.x + z * kGradThreads;
      *reinterpret_cast<uint4*>(smem + L::kS0Lo + wide_at(e / (DK / 8), e % (DK / 8))) = s0_lo[z];
    }
    __syncthreads();
    if (i + 1 < steps) fetch(c, chunk, grp, i + 1, n + 1, m);
    else if (after < items) fetch(next, (int)(after / groups), (int)(after % groups), 0, n + 1, m + 1);
    // R = V - up K S0^T, in V's place and kRLo: 32 channels a half
    {
      float y[4][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t k[4], b[4];
        load4(k, kq + L::kK + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          load4(b, base + L::kS0 + wide_rows(32 * part + 16 * n, 2 * ks, lane));
          mma_if(ks == 0, y[2 * n], k, b[0], b[1]);
          mma_if(ks == 0, y[2 * n + 1], k, b[2], b[3]);
          load4(b, base + L::kS0Lo + wide_rows(32 * part + 16 * n, 2 * ks, lane));
          mma(y[2 * n], k, b[0], b[1]);
          mma(y[2 * n + 1], k, b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float up = f[kUp + r0 + g + 8 * e];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t at = wide_at(r0 + g + 8 * e, 4 * part + n) + 4 * t;
          uint32_t* p = reinterpret_cast<uint32_t*>(smem + st + L::kV + at);
          split(fmaf(-up, y[n][2 * e], __uint_as_float(*p << 16)), fmaf(-up, y[n][2 * e + 1], __uint_as_float(*p & 0xffff0000u)), *p,
                *reinterpret_cast<uint32_t*>(smem + L::kRLo + at));
        }
      }
    }
    __syncthreads();
    {  // r = Inv R
      float y[4][4];
#pragma unroll
      for (int jb = 0; jb < 4; ++jb)
        if (jb <= rb) {
          uint32_t w[4], wl[4], b[4];
          load4(w, inv + block_at(rb, jb) + narrow_cols(0, lane));
          load4(wl, base + L::kInvLo + block_at(rb, jb) + narrow_cols(0, lane));
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            load4t(b, base + st + L::kV + wide_cols(16 * jb, 4 * part + 2 * n, lane));
            mma_if(jb == 0, y[2 * n], w, b[0], b[1]);
            mma_if(jb == 0, y[2 * n + 1], w, b[2], b[3]);
            mma(y[2 * n], wl, b[0], b[1]);
            mma(y[2 * n + 1], wl, b[2], b[3]);
            load4t(b, base + L::kRLo + wide_cols(16 * jb, 4 * part + 2 * n, lane));
            mma(y[2 * n], w, b[0], b[1]);
            mma(y[2 * n + 1], w, b[2], b[3]);
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          *reinterpret_cast<uint32_t*>(smem + L::kR + wide_at(r0 + g + 8 * e, 4 * part + n) + 4 * t) = pair(y[n][2 * e], y[n][2 * e + 1]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the second parts were written where the next S0 comes)
    __syncthreads();
    if (threadIdx.x == 0) {
      if (i + 1 < steps) fetch_state(chunk, grp, i + 1);
      else if (after < items) fetch_state((int)(after / groups), (int)(after % groups), 0);
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {  // Pr or Er
      uint32_t w[4], b[4];
      load4(w, base + st + (second ? L::kDV : L::kDO) + wide_cols(r0, 2 * ks, lane));
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (p <= rb) {
          load4(b, base + L::kR + wide_rows(16 * p, 2 * ks, lane));
          mma(x[p][0], w, b[0], b[1]);
          mma(x[p][1], w, b[2], b[3]);
        }
    }
    // what goes through the states, one product after another (all three at once take more registers than there are)
    auto through = [&](uint32_t left, uint32_t right, float (&y)[NK][4]) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t w[4], b[4];
        load4(w, left + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int nb = 0; nb < NK / 2; ++nb) {
          load4t(b, right + wide_cols(16 * ks, part * NK + 2 * nb, lane));
          mma_if(ks == 0, y[2 * nb], w, b[0], b[1]);
          mma_if(ks == 0, y[2 * nb + 1], w, b[2], b[3]);
        }
      }
    };
    // adds w y to a gradient; gives y . (query or key) of the row
    auto add = [&](const float (&y)[NK][4], int e, float w, uint32_t with, float (&to)[NK][4]) {
      float dots[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t p = *pair_at(with, i, e);
        dots[0] = fmaf(y[i][2 * e], __uint_as_float(p << 16), dots[0]);
        dots[1] = fmaf(y[i][2 * e + 1], __uint_as_float(p & 0xffff0000u), dots[1]);
        to[i][2 * e] = fmaf(w, y[i][2 * e], to[i][2 * e]);
        to[i][2 * e + 1] = fmaf(w, y[i][2 * e + 1], to[i][2 * e + 1]);
      }
      return dots[0] + dots[1];
    };
    {
      float y[NK][4];
      through(base + st + L::kDO, base + L::kS0, y);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float w = f[kUpQ + r0 + g + 8 * e];
        at_row[e] = fmaf(w, add(y, e, w, L::kQ, dq), at_row[e]);
      }
      through(base + st + L::kDV, base + L::kS0, y);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float w = -f[kUp + r0 + g + 8 * e];
        at_row[e] = fmaf(w, add(y, e, w, L::kK, dk), at_row[e]);
      }
      through(base + L::kR, base + st + L::kDS, y);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // (the write's product without beta, which dbeta is without)
        const float w = f[kLeft + r0 + g + 8 * e];
        write_row[e] = fmaf(w, add(y, e, w * f[kBeta + r0 + g + 8 * e], L::kK, dk), write_row[e]);
      }
    }
    if (half == halves - 1) {
      // Q K^T (or K K^T), by blocks of 16 columns (of every head again: 32 registers held took 197 us for 177, spills)
      float qk[4][2][4];
#pragma unroll
      for (int o = 0; o < 4; ++o)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) qk[o][n][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t v[4], b[4];
        load4(v, kq + (second ? L::kK : L::kQ) + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int o = 0; o < 4; ++o)
          if (o <= rb) {
            load4(b, kq + L::kK + wide_rows(16 * o, 2 * ks, lane));
            mma(qk[o][0], v, b[0], b[1]);
            mma(qk[o][1], v, b[2], b[3]);
          }
      }
      __syncthreads();  // dO and dV have been read
      // F or -E, and W's sums
      float row[2] = {0.0f, 0.0f}, own[2][2][2] = {};  // rows left of their own block; that block [n][e][j]
      float mine[2], mine_hi[2], mine_lo[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = r0 + g + 8 * e;
        mine[e] = second ? f[kKn + at] : f[kQn + at] * a.scale;
        mine_hi[e] = f[kGHi + at];
        mine_lo[e] = f[kGLo + at];
      }
#pragma unroll
      for (int o = 0; o < 4; ++o)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int to0 = 16 * o + 8 * n + 2 * t;
          float col[2] = {0.0f, 0.0f};
          if (o <= rb) {
            auto pairs = [&](int from) { return *reinterpret_cast<const float2*>(f + from + to0); };
            const float2 hi = pairs(kGHi), lo = pairs(kGLo), kn = pairs(kKn), beta = pairs(kBeta);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = r0 + g + 8 * e;
              float out[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int to = to0 + j;
                const float b = j ? beta.y : beta.x;
                const float apart = (mine_hi[e] - (j ? hi.y : hi.x)) + (mine_lo[e] - (j ? lo.y : lo.x));
                const float d = to <= at ? ex2(apart) * ((j ? kn.y : kn.x) * mine[e]) : 0.0f;
                const float p = x[o][n][2 * e + j] * d, w = p * qk[o][n][2 * e + j];
                const bool diagonal = to == at;
                out[j] = second ? (diagonal ? 0.0f : -p * b) : p * b;
                if (!second && diagonal) vec[L::kDiag + at] = w;
                const float below = diagonal ? 0.0f : w;
                if (o == rb) own[n][e][j] = b * below;
                else row[e] = fmaf(b, below, row[e]);
                col[j] += below;
              }
              *reinterpret_cast<uint32_t*>(smem + st + (second ? L::kE : L::kF) + wide_at(at, 2 * o + n) + 4 * t) = pair(out[0], out[1]);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float total = sum_rows(col[j]);
            if (g == 0) vec[L::kCol + ((second ? 4 : 0) + rb) * kC + to0 + j] = total;
          }
        }
      // rows from each on, and of its own block's columns those before it (rows 0-7 have none of columns 8-15)
      row[1] = sum_behind(row[1], lane);
      row[0] = sum_behind(row[0], lane) + __shfl_sync(0xffffffffu, row[1], t);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float left = sum_behind(own[0][1][j], lane), right = sum_behind(own[1][1][j], lane);
        const float top = sum_behind(own[0][0][j], lane) + __shfl_sync(0xffffffffu, left, t);
        row[0] += 2 * t + j < g ? top : 0.0f;
        row[1] += left + (2 * t + j < g ? right : 0.0f);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = sum_quad(row[e]), av = sum_quad(at_row[e]), wr = sum_quad(write_row[e]);
        if (t == 0) {
          vec[L::kRow + part * kC + r0 + g + 8 * e] = s;
          vec[L::kA + part * kC + r0 + g + 8 * e] = av;
          vec[L::kWrite + part * kC + r0 + g + 8 * e] = wr;
        }
      }
      float d = dot;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) vec[L::kDot + warp] = d;
      __syncthreads();
      // within the chunk
      for (int jb = 0; jb <= rb; ++jb) {
        uint32_t w[4], e[4], b[4];
        load4(w, base + st + L::kF + wide_cols(r0, 2 * jb, lane));
        load4(e, base + st + L::kE + wide_cols(r0, 2 * jb, lane));
#pragma unroll
        for (int nb = 0; nb < NK / 2; ++nb) {
          load4t(b, kq + L::kK + wide_cols(16 * jb, part * NK + 2 * nb, lane));
          mma(dq[2 * nb], w, b[0], b[1]);
          mma(dq[2 * nb + 1], w, b[2], b[3]);
          mma(dk[2 * nb], e, b[0], b[1]);
          mma(dk[2 * nb + 1], e, b[2], b[3]);
        }
      }
      for (int ib = rb; ib < 4; ++ib) {
        uint32_t w[4], e[4], b[4];
        load4t(w, base + st + L::kF + wide_rows(16 * ib, 2 * rb, lane));
        load4t(e, base + st + L::kE + wide_rows(16 * ib, 2 * rb, lane));
#pragma unroll
        for (int nb = 0; nb < NK / 2; ++nb) {
          load4t(b, kq + L::kQ + wide_cols(16 * ib, part * NK + 2 * nb, lane));
          mma(dk[2 * nb], w, b[0], b[1]);
          mma(dk[2 * nb + 1], w, b[2], b[3]);
          load4t(b, kq + L::kK + wide_cols(16 * ib, part * NK + 2 * nb, lane));
          mma(dk[2 * nb], e, b[0], b[1]);
          mma(dk[2 * nb + 1], e, b[2], b[3]);
        }
      }
      if (warp == 0 && (a.dg || a.dbeta)) {  // tokens 2 lane and + 1
        float inner = 0.0f, out[2], db[2], av[2], write[2], col[3][2];  // col: of row blocks 1 to 3, left of them
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) inner += vec[L::kDot + w];
        inner *= f[kGamma];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = 2 * lane + j;
          float sums[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[i] = vec[L::kCol + i * kC + at] - vec[L::kCol + (4 + i) * kC + at];
          const float wr = vec[L::kWrite + at] + vec[L::kWrite + kC + at], beta = f[kBeta + at];
          av[j] = vec[L::kA + at] + vec[L::kA + kC + at];
          out[j] = inner + (vec[L::kRow + at] - vec[L::kRow + kC + at]);
          db[j] = wr + vec[L::kDiag + at] + ((sums[0] + sums[1]) + (sums[2] + sums[3]));
          write[j] = beta * wr;
#pragma unroll
          for (int i = 0; i < 3; ++i) col[i][j] = lane < 8 * (i + 1) ? beta * sums[i + 1] : 0.0f;
        }
        auto before = [&](const float (&v)[2], bool take) {  // adds the tokens before each of this lane's
          float sum = v[0] + v[1];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
          }
          sum = __shfl_up_sync(0xffffffffu, sum, 1);
          if (lane == 0) sum = 0.0f;
          if (take) {
            out[0] += sum;
            out[1] += sum + v[0];
          }
        };
        before(write, true);
#pragma unroll
        for (int i = 0; i < 3; ++i) before(col[i], lane < 8 * (i + 1));
        float behind = av[0] + av[1];  // of this lane's tokens on
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float u = __shfl_down_sync(0xffffffffu, behind, o);
          if (lane + o < 32) behind += u;
        }
        behind = __shfl_down_sync(0xffffffffu, behind, 1);
        if (lane == 31) behind = 0.0f;
        out[0] += behind + av[1] + av[0];
        out[1] += behind + av[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = 2 * lane + j;
          if (at >= c.len) break;
          const int64_t to = (int64_t)(c.row + at) * a.heads + h;
          if (a.dg) static_cast<bf16*>(a.dg)[to] = __float2bfloat16_rn(out[j]);
          if (a.dbeta) static_cast<bf16*>(a.dbeta)[to] = __float2bfloat16_rn(db[j]);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (R was written where a later step's v comes)
    __syncthreads();  // this step's tiles have been read
  }
  // (any head's lengths; the copies under way go to the other)
  const float* f = reinterpret_cast<const float*>(smem + L::kHead + ((m * per + per - 1) & 1) * L::kHeadBytes + L::kFac);
  // a length's own gradient: d - kappa^2 (x . d) x
  if (a.l2_eps >= 0.0f) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float dots[2] = {0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        const uint32_t q = *pair_at(L::kQ, n, e), k = *pair_at(L::kK, n, e);
        dots[0] = fmaf(dq[n][2 * e], __uint_as_float(q << 16), fmaf(dq[n][2 * e + 1], __uint_as_float(q & 0xffff0000u), dots[0]));
        dots[1] = fmaf(dk[n][2 * e], __uint_as_float(k << 16), fmaf(dk[n][2 * e + 1], __uint_as_float(k & 0xffff0000u), dots[1]));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float d = sum_quad(dots[j]);
        if (t == 0) vec[(2 * j + part) * kC + r0 + g + 8 * e] = d;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int at = r0 + g + 8 * e;
    float wq = 0.0f, wk = 0.0f;
    if (a.l2_eps >= 0.0f) {
      wq = f[kQn + at] * f[kQn + at] * (vec[at] + vec[kC + at]);
      wk = f[kKn + at] * f[kKn + at] * (vec[2 * kC + at] + vec[3 * kC + at]);
    }
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      uint32_t *q = pair_at(L::kQ, n, e), *k = pair_at(L::kK, n, e);
      *q = pair(fmaf(-wq, __uint_as_float(*q << 16), dq[n][2 * e]), fmaf(-wq, __uint_as_float(*q & 0xffff0000u), dq[n][2 * e + 1]));
      *k = pair(fmaf(-wk, __uint_as_float(*k << 16), dk[n][2 * e]), fmaf(-wk, __uint_as_float(*k & 0xffff0000u), dk[n][2 * e + 1]));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kC * DK / 8; e += kGradThreads) {
    const int r = e / (DK / 8), u = e % (DK / 8);
    if (r >= c.len || 8 * u >= a.dk) continue;
    const int64_t col = (int64_t)grp * a.dk + 8 * u;
    *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dq) + (int64_t)(c.row + r) * a.ld_dq + col) =
        *reinterpret_cast<const uint4*>(smem + kq0 + L::kQ + wide_at(r, u));
    *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dk_out) + (int64_t)(c.row + r) * a.ld_dk + col) =
        *reinterpret_cast<const uint4*>(smem + kq0 + L::kK + wide_at(r, u));
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the gradients were written where later keys come)
  __syncthreads();
  c = next;
  }
  if (threadIdx.x == 0 && *gave_up) atomicAdd(&g_delta_back_timeouts, 1u);
}

template <int DK, int NW>
cudaError_t run_back(const DeltaBwdArgs& a, const DeltaMaps& maps, const unsigned char* records, unsigned char* ds, cudaStream_t st) {
  using L = Back<DK, NW>;
  auto kernel = delta_back_kernel<DK, NW>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.dv + 16 * NW - 1) / (16 * NW), a.heads, a.tab.n);
  kernel<<<grid, 32 * NW, L::kSmem, st>>>(a, maps, records, ds);
  return cudaGetLastError();
}

template <int DK>
cudaError_t run_grad(const DeltaBwdArgs& a, const DeltaMaps& both, const unsigned char* records, const unsigned char* ds, cudaStream_t st) {
  using L = Grad<DK>;
  const int chunks = a.tab.tile[a.tab.n];
  if (chunks == 0) return cudaSuccess;
  const int64_t rows = a.tab.cu[a.tab.n];
  GradMaps maps;
  maps.k = both.k;
  maps.q = both.q;
  if (!delta_map(&maps.v, a.v, rows, a.heads, a.dv, a.ld_v, 64) || !delta_map(&maps.dy, a.dy, rows, a.heads, a.dv, a.ld_dy, 64) ||
      !delta_map(&maps.dv, a.dv_out, rows, a.heads, a.dv, a.ld_dv, 64))
    return cudaErrorInvalidValue;
  auto kernel = delta_grad_kernel<DK>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)chunks * a.groups;
  if (items + device_sm_count() > 0xffffffffll) return cudaErrorInvalidValue;  // (queries that no memory holds)
  kernel<<<(unsigned)std::min<int64_t>(items, device_sm_count()), kGradThreads, L::kSmem, st>>>(a, maps, records, ds);
  return cudaGetLastError();
}

template <int DK>
cudaError_t run_backward(const DeltaBwdArgs& a, const DeltaMaps& maps, const unsigned char* records, unsigned char* ds, cudaStream_t st) {
  // Four warps share a chunk's tiles where that leaves most SMs a CTA; eight never were faster (us of 8, 4 and 2 warps,
  // 8 192 tokens, 16 heads of 128 x 128: 8 runs 169, 122, 127; 16 runs 110, 109, 116; 32 runs 119, 105, 126; of 4 runs
  // 159 and 156 of 4 and 2 warps, of 2 runs 312 and 304).
  const int64_t blocks = (int64_t)a.tab.n * a.heads * ((a.dv + 15) / 16);  // of 16 rows
  const cudaError_t e = blocks >= 4 * device_sm_count() ? run_back<DK, 4>(a, maps, records, ds, st)
                                                        : run_back<DK, 2>(a, maps, records, ds, st);
  return e == cudaSuccess ? run_grad<DK>(a, maps, records, ds, st) : e;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

unsigned int read_delta_back_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_back_timeouts, sizeof v) != cudaSuccess) return 0xffffffffu;
  return v;
}

size_t delta_backward_workspace(int64_t chunks, int heads, int dv, int dk) {
  const size_t states = (size_t)chunks * heads * state_tiles(dv) * (dk <= 64 ? kStateTile<64> : kStateTile<128>);
  return round256(delta_records(chunks, heads, true)) + round256(states);
}

cudaError_t launch_delta_backward(const DeltaBwdArgs& a, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  unsigned char* ds = records + round256(delta_records(a.tab.tile[a.tab.n], a.heads, true));
  DeltaMaps maps;
  if (a.tab.cu[a.tab.n] > 0 && !delta_maps(&maps, a, a.dy, a.ld_dy)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_delta_records(a, maps, ws, st);
  if (e != cudaSuccess) return e;
  return a.dk <= 64 ? run_backward<64>(a, maps, records, ds, st) : run_backward<128>(a, maps, records, ds, st);
}

}  // namespace mamba2
