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
// a running sum over t of rows and columns of the same W, so that what cancels cancels exactly.
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

// ------------------------------------------------------------------ dS through the chunks

template <int DK, int NW>
struct Back : Stages<DK, true, NW, 2> {
  static constexpr int kOffBar = Stages<DK, true, NW, 2>::kEnd, kSmem = kOffBar + 32;
};

template <int DK, int NW>
__global__ void __launch_bounds__(32 * NW) delta_back_kernel(const __grid_constant__ DeltaBwdArgs a, const __grid_constant__ DeltaMaps maps, const unsigned char* records, bf16* ds) {
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
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBar + 16);
  if (threadIdx.x == 0) {
    bar_init(bar(0), 32);
    bar_init(bar(1), 32);
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
  if (n > 0 && warp == 0) fetch(n - 1);
  for (int ch = n - 1; ch >= 0; --ch) {
    if (ch < n - 1) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (dv was written where another chunk's dO comes)
      __syncthreads();  // every warp is done with the other stage
    }
    if (ch > 0 && warp == 0) fetch(ch - 1);
    bar_wait(bar(ch), (uint32_t)(((n - 1 - ch) >> 1) & 1), gave_up);
    __syncwarp();
    const uint32_t at = base + L::k(ch), qt = base + L::q(ch), rec = base + L::rec(ch), dt = base + L::v(ch) + warp * L::kStrip;
    const float* f = reinterpret_cast<const float*>(smem + (rec - base) + off_factors(true));
    {  // dS1, for the gradients that take it as an operand (rounded as such)
      bf16* o = ds + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * a.dv * a.dk;
      each([&](float* v, int64_t to) { *reinterpret_cast<uint32_t*>(o + to) = pair(v[0], v[1]); });
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

// A CTA takes a chunk and one group of keys, its heads one after another, so that what they add to a query or key is
// summed in registers in their order. Warp w: rows 16 (w % 4) of the chunk, columns of half w / 4.
constexpr int kGradThreads = 256;

template <int DK, int DV>
struct Grad {
  static constexpr int kState = DV * DK * 2, kTileK = kC * DK * 2, kTileV = kC * DV * 2, kSq = kC * kC * 2;
  static constexpr int kS0 = 0, kDS = kState, kV = 2 * kState, kDO = kV + kTileV, kDV = kDO + kTileV, kR = kDV + kTileV;
  static constexpr int kK = kR + kTileV, kQ = kK + kTileK, kF = kQ + kTileK, kE = kF + kSq, kInv = kE + kSq;
  static constexpr int kFac = kInv + kTri, kVec = kFac + 9 * kC * 4;
  // floats at kVec: sums of W's rows [2 halves], columns [2][4 row blocks], its diagonal, a and the write's rows [2 halves]
  static constexpr int kRow = 0, kCol = 2 * kC, kDiag = 10 * kC, kA = 11 * kC, kWrite = 13 * kC, kDot = 15 * kC;
  static constexpr int kSmem = kVec + (15 * kC + 8) * 4;
  static_assert(kSmem <= 232448, "shared memory plan exceeds 227 KB");
};

__device__ __forceinline__ float sum_quad(float v) {  // over the lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float sum_rows(float v) {  // over the lanes of a column
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaBwdArgs a, const unsigned char* records, const bf16* ds) {
  using L = Grad<DK, DV>;
  constexpr int KS = DK / 16, VS = DV / 16, NK = DK / 16, NV = DV / 16;  // steps over columns; column tiles of a half
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = sm32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rb = warp & 3, half = warp >> 2, r0 = 16 * rb;
  const int grp = blockIdx.y, per = a.heads / a.groups;
  const Chunk c = chunk_of(a.tab, blockIdx.x);
  float* vec = reinterpret_cast<float*>(smem + L::kVec);
  const float* f = reinterpret_cast<const float*>(smem + L::kFac);

  auto tile = [&](uint32_t to, const void* from, int64_t ld, int64_t col, int width, auto cols) {  // 64 rows, zeros past the matrix
    constexpr int C = decltype(cols)::value, units = C / 8;
    const bf16* p = static_cast<const bf16*>(from) + col;
    for (int e = threadIdx.x; e < kC * units; e += kGradThreads) {
      const int r = e / units, u = e % units;
      const bool in = r < c.len && 8 * u < width;
      copy16(base + to + wide_at(r, u), p + (int64_t)(c.row + (in ? r : 0)) * ld + (in ? 8 * u : 0), in);
    }
  };
  tile(L::kK, a.k, a.ld_k, (int64_t)grp * a.dk, a.dk, std::integral_constant<int, DK>{});
  tile(L::kQ, a.q, a.ld_q, (int64_t)grp * a.dk, a.dk, std::integral_constant<int, DK>{});

  float dq[NK][4], dk[NK][4], qk[8][4];  // qk: Q K^T in the first half's warps, K K^T in the second's
#pragma unroll
  for (int i = 0; i < NK; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dq[i][j] = dk[i][j] = 0.0f;
  // the pair of a [64][C] tile that this thread's sum (column tile i of its half, row g + 8 e) is of
  auto pair_at = [&](uint32_t tile_off, int i, int e, auto cols) -> uint32_t* {
    constexpr int C = decltype(cols)::value;
    return reinterpret_cast<uint32_t*>(smem + tile_off + wide_at(r0 + g + 8 * e, half * (C / 16) + i) + 4 * t);
  };
  constexpr std::integral_constant<int, DK> wide_k{};
  constexpr std::integral_constant<int, DV> wide_v{};

  for (int hh = 0; hh < per; ++hh) {
    const int h = grp * per + hh;
    if (hh > 0) __syncthreads();  // the last head's tiles have been read
    tile(L::kV, a.v, a.ld_v, (int64_t)h * a.dv, a.dv, wide_v);
    tile(L::kDO, a.dy, a.ld_dy, (int64_t)h * a.dv, a.dv, wide_v);
    tile(L::kDV, a.dv_out, a.ld_dv, (int64_t)h * a.dv, a.dv, wide_v);
    const int64_t item = (int64_t)blockIdx.x * a.heads + h;
    const unsigned char* rec = records + item * record_bytes(true);
    for (int e = threadIdx.x; e < kTri / 16; e += kGradThreads) copy16(base + L::kInv + 16 * e, rec + 16 * e, true);
    for (int e = threadIdx.x; e < 9 * kC / 4; e += kGradThreads) copy16(base + L::kFac + 16 * e, rec + off_factors(true) + 16 * e, true);
    copies_end();
    {  // S0 as bf16, dS1, and their inner product
      const float* s0 = a.ckpt + item * a.dv * a.dk;
      const bf16* s1 = ds + item * a.dv * a.dk;
      float dot = 0.0f;
      for (int e = threadIdx.x; e < DV * DK / 8; e += kGradThreads) {
        const int r = e / (DK / 8), u = e % (DK / 8);
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (r < a.dv && 8 * u < a.dk) {
          float v[8], d[8];
          Vec16<float>::load_stream(s0 + (int64_t)r * a.dk + 8 * u, v);
          Vec16<float>::load_stream(s0 + (int64_t)r * a.dk + 8 * u + 4, v + 4);
          w1 = __ldcs(reinterpret_cast<const uint4*>(s1 + (int64_t)r * a.dk + 8 * u));
          Vec16<bf16>::unpack(w1, d);
#pragma unroll
          for (int j = 0; j < 8; ++j) dot = fmaf(v[j], d[j], dot);
          w0 = Vec16<bf16>::pack(v);
        }
        *reinterpret_cast<uint4*>(smem + L::kS0 + wide_at<DV>(r, u)) = w0;
        *reinterpret_cast<uint4*>(smem + L::kDS + wide_at<DV>(r, u)) = w1;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) vec[L::kDot + warp] = dot;
    }
    copies_done();
    __syncthreads();
    if (hh == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) qk[i][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t x[4], b[4];
        load4(x, base + (half ? L::kK : L::kQ) + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          if (nb <= rb) {
            load4(b, base + L::kK + wide_rows(16 * nb, 2 * ks, lane));
            mma(qk[2 * nb], x, b[0], b[1]);
            mma(qk[2 * nb + 1], x, b[2], b[3]);
          }
      }
    }
    // R = V - up K S0^T, in V's place
    {
      float x[NV][4];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t k[4], b[4];
        load4(k, base + L::kK + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int nb = 0; nb < NV / 2; ++nb) {
          load4(b, base + L::kS0 + wide_rows<DV>(half * (DV / 2) + 16 * nb, 2 * ks, lane));
          mma(x[2 * nb], k, b[0], b[1]);
          mma(x[2 * nb + 1], k, b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float up = f[kUp + r0 + g + 8 * e];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t* p = pair_at(L::kV, i, e, wide_v);
          *p = pair(fmaf(-up, x[i][2 * e], __uint_as_float(*p << 16)), fmaf(-up, x[i][2 * e + 1], __uint_as_float(*p & 0xffff0000u)));
        }
      }
    }
    __syncthreads();
    {  // r = Inv R
      float x[NV][4];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
      for (int jb = 0; jb <= rb; ++jb) {
        uint32_t w[4], b[4];
        load4(w, base + L::kInv + block_at(rb, jb) + narrow_cols(0, lane));
#pragma unroll
        for (int nb = 0; nb < NV / 2; ++nb) {
          load4t(b, base + L::kV + wide_cols(16 * jb, half * (DV / 16) + 2 * nb, lane));
          mma(x[2 * nb], w, b[0], b[1]);
          mma(x[2 * nb + 1], w, b[2], b[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < NV; ++i) *pair_at(L::kR, i, e, wide_v) = pair(x[i][2 * e], x[i][2 * e + 1]);
    }
    __syncthreads();
    {  // Pr (first half) or Er, F or -E, and W's sums
      float x[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < VS; ++ks) {
        uint32_t d[4], b[4];
        load4(d, base + (half ? L::kDV : L::kDO) + wide_cols(r0, 2 * ks, lane));
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          if (nb <= rb) {
            load4(b, base + L::kR + wide_rows(16 * nb, 2 * ks, lane));
            mma(x[2 * nb], d, b[0], b[1]);
            mma(x[2 * nb + 1], d, b[2], b[3]);
          }
      }
      float row[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float col[2] = {0.0f, 0.0f};
        if (i / 2 <= rb) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = r0 + g + 8 * e;
            const float mine = half ? f[kKn + at] : f[kQn + at] * a.scale;
            float out[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int to = 8 * i + 2 * t + j;
              const bool in = half ? to < at : to <= at;
              const float d = in ? ex2((f[kGHi + at] - f[kGHi + to]) + (f[kGLo + at] - f[kGLo + to])) * f[kKn + to] * mine : 0.0f;
              const float p = x[i][2 * e + j] * d, w = p * qk[i][2 * e + j];
              out[j] = half ? -p * f[kBeta + to] : p * f[kBeta + to];
              if (to < at) {
                row[e] = fmaf(f[kBeta + to], w, row[e]);
                col[j] += w;
              } else if (to == at && !half) {
                vec[L::kDiag + at] = w;
              }
            }
            *reinterpret_cast<uint32_t*>(smem + (half ? L::kE : L::kF) + wide_at(at, i) + 4 * t) = pair(out[0], out[1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float total = sum_rows(col[j]);
          if (g == 0) vec[L::kCol + (4 * half + rb) * kC + 8 * i + 2 * t + j] = total;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row[e] = sum_quad(row[e]);
        if (t == 0) vec[L::kRow + half * kC + r0 + g + 8 * e] = row[e];
      }
    }
    {  // what goes through the states
      float x[NK][4], at[2] = {0.0f, 0.0f};
      auto product = [&](uint32_t left, uint32_t right) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < VS; ++ks) {
          uint32_t d[4], b[4];
          load4(d, base + left + wide_cols(r0, 2 * ks, lane));
#pragma unroll
          for (int nb = 0; nb < NK / 2; ++nb) {
            load4t(b, base + right + wide_cols<DV>(16 * ks, half * (DK / 16) + 2 * nb, lane));
            mma(x[2 * nb], d, b[0], b[1]);
            mma(x[2 * nb + 1], d, b[2], b[3]);
          }
        }
      };
      // adds w x to a gradient, and gives w x . (query or key) of the row
      auto add = [&](float (&to)[NK][4], int e, float w, uint32_t with) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const uint32_t p = *pair_at(with, i, e, wide_k);
          dot = fmaf(x[i][2 * e], __uint_as_float(p << 16), dot);
          dot = fmaf(x[i][2 * e + 1], __uint_as_float(p & 0xffff0000u), dot);
          to[i][2 * e] = fmaf(w, x[i][2 * e], to[i][2 * e]);
          to[i][2 * e + 1] = fmaf(w, x[i][2 * e + 1], to[i][2 * e + 1]);
        }
        return dot * w;
      };
      product(L::kDO, L::kS0);
#pragma unroll
      for (int e = 0; e < 2; ++e) at[e] += add(dq, e, f[kUpQ + r0 + g + 8 * e], L::kQ);
      product(L::kDV, L::kS0);
#pragma unroll
      for (int e = 0; e < 2; ++e) at[e] += add(dk, e, -f[kUp + r0 + g + 8 * e], L::kK);
      product(L::kR, L::kDS);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = r0 + g + 8 * e;
        float dot = 0.0f;  // without beta, which dbeta is without
        const float left = f[kLeft + i], w = left * f[kBeta + i];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          const uint32_t p = *pair_at(L::kK, n, e, wide_k);
          dot = fmaf(x[n][2 * e], __uint_as_float(p << 16), dot);
          dot = fmaf(x[n][2 * e + 1], __uint_as_float(p & 0xffff0000u), dot);
          dk[n][2 * e] = fmaf(w, x[n][2 * e], dk[n][2 * e]);
          dk[n][2 * e + 1] = fmaf(w, x[n][2 * e + 1], dk[n][2 * e + 1]);
        }
        dot = sum_quad(dot * left);
        const float av = sum_quad(at[e]);
        if (t == 0) {
          vec[L::kWrite + half * kC + i] = dot;
          vec[L::kA + half * kC + i] = av;
        }
      }
    }
    __syncthreads();
    // within the chunk
    for (int jb = 0; jb <= rb; ++jb) {
      uint32_t w[4], e[4], b[4];
      load4(w, base + L::kF + wide_cols(r0, 2 * jb, lane));
      load4(e, base + L::kE + wide_cols(r0, 2 * jb, lane));
#pragma unroll
      for (int nb = 0; nb < NK / 2; ++nb) {
        load4t(b, base + L::kK + wide_cols(16 * jb, half * (DK / 16) + 2 * nb, lane));
        mma(dq[2 * nb], w, b[0], b[1]);
        mma(dq[2 * nb + 1], w, b[2], b[3]);
        mma(dk[2 * nb], e, b[0], b[1]);
        mma(dk[2 * nb + 1], e, b[2], b[3]);
      }
    }
    for (int ib = rb; ib < 4; ++ib) {
      uint32_t w[4], e[4], b[4];
      load4t(w, base + L::kF + wide_rows(16 * ib, 2 * rb, lane));
      load4t(e, base + L::kE + wide_rows(16 * ib, 2 * rb, lane));
#pragma unroll
      for (int nb = 0; nb < NK / 2; ++nb) {
        load4t(b, base + L::kQ + wide_cols(16 * ib, half * (DK / 16) + 2 * nb, lane));
        mma(dk[2 * nb], w, b[0], b[1]);
        mma(dk[2 * nb + 1], w, b[2], b[3]);
        load4t(b, base + L::kK + wide_cols(16 * ib, half * (DK / 16) + 2 * nb, lane));
        mma(dk[2 * nb], e, b[0], b[1]);
        mma(dk[2 * nb + 1], e, b[2], b[3]);
      }
    }
    if (warp == 0 && (a.dg || a.dbeta)) {  // tokens 2 lane and + 1
      float dot = 0.0f, step[2], all = 0.0f, db[2];
#pragma unroll
      for (int w = 0; w < kGradThreads / 32; ++w) dot += vec[L::kDot + w];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        float col = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) col += vec[L::kCol + r * kC + i] - vec[L::kCol + (4 + r) * kC + i];
        const float av = vec[L::kA + i] + vec[L::kA + kC + i], wr = vec[L::kWrite + i] + vec[L::kWrite + kC + i];
        db[j] = wr + vec[L::kDiag + i] + col;
        step[j] = f[kBeta + i] * (wr + col) - av - (vec[L::kRow + i] - vec[L::kRow + kC + i]);
        all += av;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      float before = step[0] + step[1];  // of the lanes before this one, exclusive
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      before -= step[0] + step[1];
      const float start = fmaf(f[kGamma], dot, all);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * lane + j;
        if (i >= c.len) break;
        const int64_t to = (int64_t)(c.row + i) * a.heads + h;
        if (a.dg) static_cast<bf16*>(a.dg)[to] = __float2bfloat16_rn(start + before + (j ? step[0] : 0.0f));
        if (a.dbeta) static_cast<bf16*>(a.dbeta)[to] = __float2bfloat16_rn(db[j]);
      }
    }
  }
  __syncthreads();
  // a length's own gradient: d - kappa^2 (x . d) x
  if (a.l2_eps >= 0.0f) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float dots[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t q = *pair_at(L::kQ, i, e, wide_k), k = *pair_at(L::kK, i, e, wide_k);
        dots[0] = fmaf(dq[i][2 * e], __uint_as_float(q << 16), fmaf(dq[i][2 * e + 1], __uint_as_float(q & 0xffff0000u), dots[0]));
        dots[1] = fmaf(dk[i][2 * e], __uint_as_float(k << 16), fmaf(dk[i][2 * e + 1], __uint_as_float(k & 0xffff0000u), dots[1]));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float d = sum_quad(dots[j]);
        if (t == 0) vec[(2 * j + half) * kC + r0 + g + 8 * e] = d;
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
    for (int i = 0; i < NK; ++i) {
      uint32_t *q = pair_at(L::kQ, i, e, wide_k), *k = pair_at(L::kK, i, e, wide_k);
      *q = pair(fmaf(-wq, __uint_as_float(*q << 16), dq[i][2 * e]), fmaf(-wq, __uint_as_float(*q & 0xffff0000u), dq[i][2 * e + 1]));
      *k = pair(fmaf(-wk, __uint_as_float(*k << 16), dk[i][2 * e]), fmaf(-wk, __uint_as_float(*k & 0xffff0000u), dk[i][2 * e + 1]));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kC * DK / 8; e += kGradThreads) {
    const int r = e / (DK / 8), u = e % (DK / 8);
    if (r >= c.len || 8 * u >= a.dk) continue;
    const int64_t col = (int64_t)grp * a.dk + 8 * u;
    *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dq) + (int64_t)(c.row + r) * a.ld_dq + col) =
        *reinterpret_cast<const uint4*>(smem + L::kQ + wide_at(r, u));
    *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dk_out) + (int64_t)(c.row + r) * a.ld_dk + col) =
        *reinterpret_cast<const uint4*>(smem + L::kK + wide_at(r, u));
  }
}

template <int DK, int NW>
cudaError_t run_back(const DeltaBwdArgs& a, const DeltaMaps& maps, const unsigned char* records, bf16* ds, cudaStream_t st) {
  using L = Back<DK, NW>;
  auto kernel = delta_back_kernel<DK, NW>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.dv + 16 * NW - 1) / (16 * NW), a.heads, a.tab.n);
  kernel<<<grid, 32 * NW, L::kSmem, st>>>(a, maps, records, ds);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t run_grad(const DeltaBwdArgs& a, const unsigned char* records, const bf16* ds, cudaStream_t st) {
  using L = Grad<DK, DV>;
  const int chunks = a.tab.tile[a.tab.n];
  if (chunks == 0) return cudaSuccess;
  auto kernel = delta_grad_kernel<DK, DV>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(chunks, a.groups), kGradThreads, L::kSmem, st>>>(a, records, ds);
  return cudaGetLastError();
}

template <int DK>
cudaError_t run_backward(const DeltaBwdArgs& a, const unsigned char* records, bf16* ds, cudaStream_t st) {
  DeltaMaps maps;
  if (a.tab.cu[a.tab.n] > 0 && !delta_maps(&maps, a, a.dy, a.ld_dy)) return cudaErrorInvalidValue;
  const int64_t chains = (int64_t)a.tab.n * a.heads, sms = device_sm_count();
  cudaError_t e;
  if (a.dv > 64 && chains >= sms) e = run_back<DK, 8>(a, maps, records, ds, st);
  else if (a.dv > 32 && 2 * chains >= sms) e = run_back<DK, 4>(a, maps, records, ds, st);
  else e = run_back<DK, 2>(a, maps, records, ds, st);
  if (e != cudaSuccess) return e;
  return a.dv <= 64 ? run_grad<DK, 64>(a, records, ds, st) : run_grad<DK, 128>(a, records, ds, st);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

unsigned int read_delta_back_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_back_timeouts, sizeof v) != cudaSuccess) return 0xffffffffu;
  return v;
}

size_t delta_backward_workspace(int64_t chunks, int heads, int dv, int dk) {
  return round256(delta_records(chunks, heads, true)) + round256((size_t)chunks * heads * dv * dk * 2);
}

cudaError_t launch_delta_backward(const DeltaBwdArgs& a, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  bf16* ds = reinterpret_cast<bf16*>(records + round256(delta_records(a.tab.tile[a.tab.n], a.heads, true)));
  const cudaError_t e = launch_delta_records(a, ws, st);
  if (e != cudaSuccess) return e;
  return a.dk <= 64 ? run_backward<64>(a, records, ds, st) : run_backward<128>(a, records, ds, st);
}

}  // namespace mamba2
