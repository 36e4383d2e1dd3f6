// Gated delta rule over packed runs in chunks of 64 tokens (delta.h), bf16, d_state and headdim of at most 128.
//
// In a chunk, with G the sums of g from its start, kappa the keys' reciprocal lengths (1 without l2_eps), S0 the state
// before it and
//   L_ij = kappa_i kappa_j (k_i . k_j) exp(G_i - G_j)   (j < i),
// the corrections r (u = beta r) satisfy (I + L diag(beta)) r = R, R_i = v_i - exp(G_i) kappa_i S0 k_i, so
//   r = Inv R,   y_i = scale (exp(G_i) S0 q_i + sum_{j<=i} P_ij u_j),   S = exp(G_C) S0 + sum_j exp(G_C - G_j) kappa_j u_j k_j^T.
//
// Two kernels. The first takes every chunk and head by itself: Inv, P and the factors of its tokens, into a record. The
// second carries the state through a run's chunks. A warp owns 16 rows of the state (v channels) in registers, as the
// sums of its products are laid out, and every product of the chain has the state, R or u as its left operand:
//   X^T = S0 K^T,  r^T = R^T Inv^T,  Y^T = S0 Q^T + u^T P^T,  S += u^T K
// which is again the sums' own layout. So nothing that the chain makes leaves the warp, and warps meet once a chunk, for
// the tiles that they share. A chain's products are small (16 x 64 x 128) and wait for one another, which is why they run
// on warp products: 21 cycles from one to the next, where a tensor-memory round trip takes several hundred.
#include <algorithm>
#include <type_traits>

#include "../../include/delta.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {
namespace {

#include "delta_mma.cuh"

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ chunks by themselves

constexpr int kPrepThreads = 128;
constexpr int kLdA = kC + 4;  // floats between the rows of an fp32 triangle in shared memory

struct PrepSmem {
  static constexpr int kTiles = 2 * kC * 128 * 2;      // K and Q; then Inv in fp32
  static constexpr int kA = kTiles;                    // L diag(beta), fp32
  static constexpr int kVec = kA + kC * kLdA * 4;      // per token: G (two parts), beta, lengths
  static constexpr int kBytes = kVec + 6 * kC * 4;
};

// G_i (in units of log 2) as a sum of two floats.
__device__ __forceinline__ void scan_decays(float g, float& hi, float& lo, int lane) {
  hi = g;
  lo = 0.0f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const DF u = {__shfl_up_sync(0xffffffffu, hi, o), __shfl_up_sync(0xffffffffu, lo, o)};
    if (lane >= o) {
      const DF s = df_add(DF{hi, lo}, u);
      hi = s.hi;
      lo = s.lo;
    }
  }
}

template <int DK, bool kBackward>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(const __grid_constant__ DeltaArgs a, unsigned char* records) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, grp = h / (a.heads / a.groups);
  const Chunk c = chunk_of(a.tab, blockIdx.x);
  float* vec = reinterpret_cast<float*>(smem + PrepSmem::kVec);
  float *ghi = vec, *glo = vec + kC, *beta = vec + 2 * kC, *kn = vec + 3 * kC, *qn = vec + 4 * kC;
  const uint32_t sk = sm32(smem), sq = sk + kC * DK * 2;
  {
    const bf16* k = static_cast<const bf16*>(a.k) + (int64_t)grp * a.dk;
    const bf16* q = static_cast<const bf16*>(a.q) + (int64_t)grp * a.dk;
    constexpr int units = DK / 8;
    for (int e = threadIdx.x; e < kC * units; e += kPrepThreads) {
      const int r = e / units, u = e % units;
      const bool in = r < c.len && 8 * u < a.dk;
      const int64_t row = c.row + (in ? r : 0), col = in ? 8 * u : 0;
      copy16(sk + wide_at<DK>(r, u), k + row * a.ld_k + col, in);
      copy16(sq + wide_at<DK>(r, u), q + row * a.ld_q + col, in);
    }
    copies_end();
  }
  if (warp == 0) {
    float hi[2], lo[2], last[2] = {0.0f, 0.0f};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * half + lane;
      const int64_t at = (int64_t)(c.row + i) * a.heads + h;
      float gv = i < c.len && a.g ? a.g[at] : 0.0f;
      if (gv < -10000.0f) gv = -10000.0f;  // (a NaN stays one)
      scan_decays(gv * kLog2e, hi[half], lo[half], lane);
      const DF s = df_add(DF{hi[half], lo[half]}, DF{last[0], last[1]});
      ghi[i] = s.hi;
      glo[i] = s.lo;
      last[0] = __shfl_sync(0xffffffffu, s.hi, 31);
      last[1] = __shfl_sync(0xffffffffu, s.lo, 31);
      beta[i] = i < c.len ? (a.beta ? a.beta[at] : 1.0f) : 0.0f;
    }
  }
  copies_done();
  __syncthreads();
  {  // reciprocal lengths: a thread a row
    const int r = threadIdx.x & (kC - 1);
    const bool is_q = threadIdx.x >= kC;
    float n = 1.0f;
    if (a.l2_eps >= 0.0f) {
      float s = 0.0f;
      for (int u = 0; u < DK / 8; ++u) {
        float v[8];
        Vec16<bf16>::unpack(*reinterpret_cast<const uint4*>(smem + (is_q ? kC * DK * 2 : 0) + wide_at<DK>(r, u)), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
      }
      n = rsqrtf(s + a.l2_eps);
    }
    if (r >= c.len) n = 0.0f;
    (is_q ? qn : kn)[r] = n;
  }
  // K K^T and Q K^T below and on the diagonal blocks: a warp 16 rows
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[n][j] = qk[n][j] = 0.0f;
  const int r0 = 16 * warp;
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t ak[4], aq[4], b[4];
    load4(ak, sk + wide_cols<DK>(r0, 2 * ks, lane));
    load4(aq, sq + wide_cols<DK>(r0, 2 * ks, lane));
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      if (nb <= warp) {
        load4(b, sk + wide_rows<DK>(16 * nb, 2 * ks, lane));
        mma(kk[2 * nb], ak, b[0], b[1]);
        mma(kk[2 * nb + 1], ak, b[2], b[3]);
        mma(qk[2 * nb], aq, b[0], b[1]);
        mma(qk[2 * nb + 1], aq, b[2], b[3]);
      }
  }
  __syncthreads();  // lengths are there; K and Q have been read
  float* A = reinterpret_cast<float*>(smem + PrepSmem::kA);
  float* inv = reinterpret_cast<float*>(smem);
  unsigned char* rec = records + ((int64_t)blockIdx.x * a.heads + h) * record_bytes(kBackward);
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (n / 2 > warp) continue;
    const int j0 = 8 * n + 2 * t;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = r0 + g + 8 * half;
      float l[2], p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + e;
        const float d = j <= i ? ex2((ghi[i] - ghi[j]) + (glo[i] - glo[j])) * kn[j] : 0.0f;
        l[e] = j < i ? kk[n][2 * half + e] * d * kn[i] * beta[j] : 0.0f;
        p[e] = j <= i ? qk[n][2 * half + e] * d * (qn[i] * a.scale) : 0.0f;
      }
      *reinterpret_cast<float2*>(A + i * kLdA + j0) = make_float2(l[0], l[1]);
      uint32_t hi, lo;
      split(p[0], p[1], hi, lo);
      const uint32_t at = block_at(warp, n >> 1) + narrow_at(g + 8 * half, n & 1) + 4 * t;
      *reinterpret_cast<uint32_t*>(rec + kOffP + at) = hi;
      if (kBackward) *reinterpret_cast<uint32_t*>(rec + kOffPLo + at) = lo;
    }
  }
  {  // the tokens' factors
    float* f = reinterpret_cast<float*>(rec + off_factors(kBackward));
    const float chi = ghi[kC - 1], clo = glo[kC - 1];
    for (int i = threadIdx.x; i < kC; i += kPrepThreads) {
      const float up = ex2(ghi[i] + glo[i]), left = ex2((chi - ghi[i]) + (clo - glo[i]));
      f[kUp + i] = up * kn[i];
      f[kLeft + i] = left * kn[i];
      f[kUpQ + i] = up * (qn[i] * a.scale);
      f[kBeta + i] = beta[i];
      if (kBackward) {
        f[kGHi + i] = ghi[i];
        f[kGLo + i] = glo[i];
        f[kKn + i] = kn[i];
        f[kQn + i] = qn[i];
      }
    }
    if (threadIdx.x == 0) f[kGamma] = ex2(chi + clo);
  }
  __syncwarp();
  // Inv: the diagonal blocks by substitution, a column a lane (a warp's own rows of A are what it wrote)
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int l = 0; l < i; ++l) s = fmaf(-A[(r0 + i) * kLdA + r0 + l], x[l], s);
      x[i] = s;
      inv[(r0 + i) * kLdA + r0 + lane] = s;
    }
  }
  __syncthreads();
  // the blocks below them, transposed, a block column a warp: Inv_ij^T = -(sum_l Inv_lj^T A_il^T) Inv_ii^T, l from j to
  // i - 1, each factor in two bf16 parts (three products)
  {
    auto right = [&](const float* m, int i, int l, uint32_t (&bh)[2][2], uint32_t (&bl)[2][2]) {  // m_il^T
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(m + (16 * i + 8 * n + g) * kLdA + 16 * l + 8 * k + 2 * t);
          split(v.x, v.y, bh[n][k], bl[n][k]);
        }
    };
    auto left = [&](const float (&d)[2][4], uint32_t (&ah)[4], uint32_t (&al)[4]) {
      split(d[0][0], d[0][1], ah[0], al[0]);
      split(d[0][2], d[0][3], ah[1], al[1]);
      split(d[1][0], d[1][1], ah[2], al[2]);
      split(d[1][2], d[1][3], ah[3], al[3]);
    };
    auto times = [&](float (&d)[2][4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[2][2],
                     const uint32_t (&bl)[2][2]) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mma(d[n], al, bh[n][0], bh[n][1]);
        mma(d[n], ah, bl[n][0], bl[n][1]);
        mma(d[n], ah, bh[n][0], bh[n][1]);
      }
    };
    const int j = warp;
    uint32_t ih[3][4], il[3][4], bh[2][2], bl[2][2];  // Inv_lj^T of l = j, j + 1, j + 2
    {
      float d[2][4];  // Inv_jj^T: (row g: column g of Inv_jj, its rows 2t, 2t + 1)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = inv[(16 * j + 8 * n + 2 * t + (e & 1)) * kLdA + 16 * j + g + 8 * (e >> 1)];
      left(d, ih[0], il[0]);
    }
#pragma unroll
    for (int s = 1; s < 4; ++s) {
      const int i = j + s;
      if (i > 3) break;
      float m[2][4] = {}, d[2][4] = {};
#pragma unroll
      for (int l = 0; l < s; ++l) {
        right(A, i, j + l, bh, bl);
        times(m, ih[l], il[l], bh, bl);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[n][e] = -m[n][e];
      uint32_t mh[4], ml[4];
      left(m, mh, ml);
      right(inv, i, i, bh, bl);
      times(d, mh, ml, bh, bl);
      if (s < 3) left(d, ih[s], il[s]);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) inv[(16 * i + 8 * n + 2 * t + (e & 1)) * kLdA + 16 * j + g + 8 * (e >> 1)] = d[n][e];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 10 * 32; e += kPrepThreads) {  // a 16-byte unit of each part
    const int blk = e >> 5, r = (e >> 1) & 15, u = e & 1;
    const int i = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, j = blk - i * (i + 1) / 2;
    const float* from = inv + (16 * i + r) * kLdA + 16 * j + 8 * u;
    const float4 x = *reinterpret_cast<const float4*>(from), y = *reinterpret_cast<const float4*>(from + 4);
    uint4 hi, lo;
    split(x.x, x.y, hi.x, lo.x);
    split(x.z, x.w, hi.y, lo.y);
    split(y.x, y.y, hi.z, lo.z);
    split(y.z, y.w, hi.w, lo.w);
    *reinterpret_cast<uint4*>(rec + blk * 512 + narrow_at(r, u)) = hi;
    *reinterpret_cast<uint4*>(rec + kOffInvLo + blk * 512 + narrow_at(r, u)) = lo;
  }
}

// ------------------------------------------------------------------ the state through the chunks

template <int DK, int NW>
struct Chain {
  static constexpr int kTile = kC * DK * 2;
  static constexpr int kQ = kTile, kRec = 2 * kTile, kV = kRec + record_bytes(false);
  static constexpr int kStage = kV + NW * kC * 32;
  static constexpr int kSmem = 2 * kStage;
};

template <int DK, int NW>
__global__ void __launch_bounds__(32 * NW) delta_chain_kernel(const __grid_constant__ DeltaArgs a, const unsigned char* records) {
  using L = Chain<DK, NW>;
  constexpr int kThreads = 32 * NW, KS = DK / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = sm32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int run = blockIdx.z, h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int dv0 = blockIdx.x * 16 * NW, dv = dv0 + 16 * warp;  // this CTA's, this warp's first row
  const int first = a.tab.cu[run], len = a.tab.cu[run + 1] - first, n = (len + kC - 1) / kC;
  const bool fresh = seq_fresh(a.tab, run);
  if (len == 0 && !fresh) return;
  // the state: rows dv + g and + 8, columns 8 n + 2 t and + 1
  float s[2 * KS][4];
  float* st = a.state + ((int64_t)seq_slot(a.tab, run) * a.heads + h) * a.dv * a.dk;
  const int64_t at0 = (int64_t)(dv + g) * a.dk + 2 * t;
  auto each = [&](auto f) {  // f(the registers' first, offset in [dv, dk]) of what there is
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
  if (!fresh)
    each([&](float* v, int64_t at) {
      const float2 f = *reinterpret_cast<const float2*>(st + at);
      v[0] = f.x;
      v[1] = f.y;
    });
  auto fetch = [&](int ch) {
    const uint32_t to = base + (uint32_t)(ch & 1) * L::kStage;
    const int64_t row0 = first + (int64_t)ch * kC;
    const int m = min(kC, len - ch * kC);
    constexpr int units = DK / 8;
    const bf16* k = static_cast<const bf16*>(a.k) + (int64_t)grp * a.dk;
    const bf16* q = static_cast<const bf16*>(a.q) + (int64_t)grp * a.dk;
    for (int e = threadIdx.x; e < kC * units; e += kThreads) {
      const int r = e / units, u = e % units;
      const bool in = r < m && 8 * u < a.dk;
      const int64_t row = row0 + (in ? r : 0);
      const int col = in ? 8 * u : 0;
      copy16(to + wide_at<DK>(r, u), k + row * a.ld_k + col, in);
      copy16(to + L::kQ + wide_at<DK>(r, u), q + row * a.ld_q + col, in);
    }
    const unsigned char* rec = records + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * record_bytes(false);
    for (int e = threadIdx.x; e < record_bytes(false) / 16; e += kThreads) copy16(to + L::kRec + 16 * e, rec + 16 * e, true);
    const bf16* v = static_cast<const bf16*>(a.v) + (int64_t)h * a.dv + dv0;
    for (int e = threadIdx.x; e < kC * 2 * NW; e += kThreads) {
      const int r = e / (2 * NW), u = e % (2 * NW);
      const bool in = r < m && dv0 + 8 * u < a.dv;
      copy16(to + L::kV + (u >> 1) * (kC * 32) + narrow_at(r, u & 1), v + (row0 + (in ? r : 0)) * a.ld_v + (in ? 8 * u : 0), in);
    }
    copies_end();
  };
  if (n > 0) fetch(0);
  for (int ch = 0; ch < n; ++ch) {
    copies_done();
    __syncthreads();  // this chunk's tiles are there, and every warp is done with the other stage
    if (ch + 1 < n) fetch(ch + 1);
    const uint32_t at = base + (uint32_t)(ch & 1) * L::kStage, rec = at + L::kRec, vt = at + L::kV + warp * (kC * 32);
    const float* f = reinterpret_cast<const float*>(smem + (rec - base) + off_factors(false));
    if (a.ckpt) {
      float* o = a.ckpt + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * a.dv * a.dk;
      each([&](float* v, int64_t to) { *reinterpret_cast<float2*>(o + to) = make_float2(v[0], v[1]); });
    }
    // X^T = S0 K^T (the state in two parts) and S0 Q^T (in one: it ends in a bf16 output)
    float x[8][4], y[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = y[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t sh[4], sl[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(s[2 * ks + (j >> 1)][2 * (j & 1)], s[2 * ks + (j >> 1)][2 * (j & 1) + 1], sh[j], sl[j]);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        load4(b, at + wide_rows<DK>(16 * nb, 2 * ks, lane));
        mma(x[2 * nb], sh, b[0], b[1]);
        mma(x[2 * nb + 1], sh, b[2], b[3]);
        mma(x[2 * nb], sl, b[0], b[1]);
        mma(x[2 * nb + 1], sl, b[2], b[3]);
        load4(b, at + L::kQ + wide_rows<DK>(16 * nb, 2 * ks, lane));
        mma(y[2 * nb], sh, b[0], b[1]);
        mma(y[2 * nb + 1], sh, b[2], b[3]);
      }
    }
    // R = V - up X, as left operands of 16 tokens each
    uint32_t ah[4][4], al[4][4];
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t v[4];
      load4t(v, vt + narrow_cols(16 * jb, lane));
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // tokens 16 jb + 8 (j / 2) + 2 t and + 1, rows + 8 (j % 2)
        const int i = 2 * jb + (j >> 1);
        const float2 up = *reinterpret_cast<const float2*>(f + kUp + 8 * i + 2 * t);
        const uint32_t w = v[(j >> 1) + 2 * (j & 1)];
        split(fmaf(-up.x, x[i][2 * (j & 1)], __uint_as_float(w << 16)),
              fmaf(-up.y, x[i][2 * (j & 1) + 1], __uint_as_float(w & 0xffff0000u)), ah[jb][j], al[jb][j]);
      }
    }
    // r^T = R^T Inv^T
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        uint32_t bh[4], bl[4];
        load4(bh, rec + block_at(ib, jb) + narrow_rows(0, lane));
        load4(bl, rec + kOffInvLo + block_at(ib, jb) + narrow_rows(0, lane));
        mma(x[2 * ib], ah[jb], bh[0], bh[1]);
        mma(x[2 * ib + 1], ah[jb], bh[2], bh[3]);
        mma(x[2 * ib], al[jb], bh[0], bh[1]);
        mma(x[2 * ib + 1], al[jb], bh[2], bh[3]);
        mma(x[2 * ib], ah[jb], bl[0], bl[1]);
        mma(x[2 * ib + 1], ah[jb], bl[2], bl[3]);
      }
    // u = beta r; the scores' product takes it as it is, the state's with what is left of it at the chunk's end
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 b = *reinterpret_cast<const float2*>(f + kBeta + 8 * i + 2 * t);
      const float2 up = *reinterpret_cast<const float2*>(f + kUpQ + 8 * i + 2 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] *= j & 1 ? b.y : b.x;
        y[i][j] *= j & 1 ? up.y : up.x;
      }
    }
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t uh[4], ul[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(x[2 * jb + (j >> 1)][2 * (j & 1)], x[2 * jb + (j >> 1)][2 * (j & 1) + 1], uh[j], ul[j]);
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        uint32_t b[4];
        load4(b, rec + kOffP + block_at(ib, jb) + narrow_rows(0, lane));
        mma(y[2 * ib], uh, b[0], b[1]);
        mma(y[2 * ib + 1], uh, b[2], b[3]);
        mma(y[2 * ib], ul, b[0], b[1]);
        mma(y[2 * ib + 1], ul, b[2], b[3]);
      }
    }
    // S = gamma S + (left u)^T K
    const float gamma = f[kGamma];
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] *= gamma;
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t uh[4], ul[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 2 * jb + (j >> 1);
        const float2 w = *reinterpret_cast<const float2*>(f + kLeft + 8 * i + 2 * t);
        split(x[i][2 * (j & 1)] * w.x, x[i][2 * (j & 1) + 1] * w.y, uh[j], ul[j]);
      }
#pragma unroll
      for (int nb = 0; nb < KS; ++nb) {
        uint32_t b[4];
        load4t(b, at + wide_cols<DK>(16 * jb, 2 * nb, lane));
        mma(s[2 * nb], uh, b[0], b[1]);
        mma(s[2 * nb + 1], uh, b[2], b[3]);
        mma(s[2 * nb], ul, b[0], b[1]);
        mma(s[2 * nb + 1], ul, b[2], b[3]);
      }
    }
    // y takes the place of the warp's v and goes out a token's 32 bytes at a time
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
      store4t(vt + narrow_cols(16 * jb, lane), pair(y[2 * jb][0], y[2 * jb][1]), pair(y[2 * jb + 1][0], y[2 * jb + 1][1]),
              pair(y[2 * jb][2], y[2 * jb][3]), pair(y[2 * jb + 1][2], y[2 * jb + 1][3]));
    __syncwarp();
    const int m = min(kC, len - ch * kC), col = dv + 8 * (lane & 1);
    bf16* out = static_cast<bf16*>(a.y) + (first + (int64_t)ch * kC) * a.ld_y + (int64_t)h * a.dv + col;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int tok = 16 * it + (lane >> 1);
      if (tok < m && col < a.dv)
        *reinterpret_cast<uint4*>(out + tok * a.ld_y) =
            *reinterpret_cast<const uint4*>(smem + (vt - base) + narrow_at(tok, lane & 1));
    }
  }
  each([&](float* v, int64_t at) { *reinterpret_cast<float2*>(st + at) = make_float2(v[0], v[1]); });
}

template <int DK, int NW>
cudaError_t run_chain(const DeltaArgs& a, const unsigned char* records, cudaStream_t st) {
  using L = Chain<DK, NW>;
  auto kernel = delta_chain_kernel<DK, NW>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.dv + 16 * NW - 1) / (16 * NW), a.heads, a.tab.n);
  kernel<<<grid, 32 * NW, L::kSmem, st>>>(a, records);
  return cudaGetLastError();
}

template <int DK, bool kBackward>
cudaError_t run_prep(const DeltaArgs& a, unsigned char* records, cudaStream_t st) {
  const int chunks = a.tab.tile[a.tab.n];
  if (chunks == 0) return cudaSuccess;
  auto kernel = delta_prep_kernel<DK, kBackward>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(chunks, a.heads), kPrepThreads, PrepSmem::kBytes, st>>>(a, records);
  return cudaGetLastError();
}

template <int DK>
cudaError_t run_forward(const DeltaArgs& a, unsigned char* records, cudaStream_t st) {
  const cudaError_t e = run_prep<DK, false>(a, records, st);
  if (e != cudaSuccess) return e;
  const int64_t chains = (int64_t)a.tab.n * a.heads, sms = device_sm_count();
  if (a.dv > 64 && chains >= sms) return run_chain<DK, 8>(a, records, st);
  if (a.dv > 32 && 2 * chains >= sms) return run_chain<DK, 4>(a, records, st);
  return run_chain<DK, 2>(a, records, st);
}

}  // namespace

bool delta_chunked_supported(mamba2_dtype act, int dv, int dk) { return act == MAMBA2_BF16 && dk <= 128 && dv <= 128; }

size_t delta_records(int64_t chunks, int heads, bool backward) { return (size_t)chunks * heads * record_bytes(backward); }

cudaError_t launch_delta_records(const DeltaArgs& a, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  return a.dk <= 64 ? run_prep<64, true>(a, records, st) : run_prep<128, true>(a, records, st);
}

cudaError_t launch_delta_chunked(const DeltaArgs& a, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  return a.dk <= 64 ? run_forward<64>(a, records, st) : run_forward<128>(a, records, st);
}

}  // namespace mamba2
