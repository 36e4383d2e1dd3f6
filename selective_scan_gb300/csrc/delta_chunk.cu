// Gated delta rule over packed runs in chunks of 64 tokens (delta.h), bf16, d_state and headdim of at most 128.
//
// In a chunk, with G the sums of g from its start, kappa the keys' reciprocal lengths (1 without l2_eps), S0 the state
// before it and
//   L_ij = kappa_i kappa_j (k_i . k_j) exp(G_i - G_j)   (j < i),
// the corrections r (u = beta r) satisfy (I + L diag(beta)) r = R, R_i = v_i - exp(G_i) kappa_i S0 k_i, so
//   r = Inv R,   y_i = scale (exp(G_i) S0 q_i + sum_{j<=i} P_ij u_j),   S = exp(G_C) S0 + sum_j exp(G_C - G_j) kappa_j u_j k_j^T.
//
// Two kernels, one after the other. The first takes every chunk and head by itself: Inv, P and the factors of its tokens, into a record. The
// second carries the state through a run's chunks. A warp owns 16 rows of the state (v channels) in registers, as the
// sums of its products are laid out, and every product of the chain has the state, R or u as its left operand:
//   X^T = S0 K^T,  r^T = R^T Inv^T,  Y^T = S0 Q^T + u^T P^T,  S += u^T K
// which is again the sums' own layout. So nothing that the chain makes leaves the warp, and warps meet once a chunk, for
// the tiles that they share. A chain's products are small (16 x 64 x 128) and wait for one another, which is why they run
// on warp products: 21 cycles from one to the next, where a tensor-memory round trip takes several hundred. (A form in
// tensor memory, where several chains of an SM would fill in for each other, has not been measured.)
//
// What is rounded: the state, R, r and u enter products that end in the state as two bf16 numbers each (2^-16 of them),
// Inv likewise; S0 Q^T and P, which end in a bf16 output, as one. So y is 2.2e-3 off in the 2-norm where its own rounding
// is 1.7e-3 (P; S0 adds 1e-4 to 3e-4 of it), and an end state 2e-6, all of it from u: in three parts that is 1.1e-6, and
// 24 prompts of 16 384 tokens take 212 us for 195, one run of 32 768 1 249 for 1 170.
#include <algorithm>
#include <type_traits>

#include "../../include/delta.h"
#include "common.cuh"
#include "delta_tiles.h"
#include "host.h"

namespace mamba2 {

__device__ unsigned int g_delta_timeouts = 0;

namespace {

#include "delta_mma.cuh"

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ chunks by themselves

// A warp has 16 of the chunk's 64 rows. Bound by latency and issue (42 % of the issue slots, 23 % of the tensor pipe):
// a CTA's phases wait for one another, and four CTAs an SM fill in for each other. 16 384 chunks and heads of 128
// channels, two heads a group, take 176 us (0.54 GB of records and inputs: 3.1 TB/s), 4 240 take 52 us.
constexpr int kPrepThreads = 128;
constexpr int kLdA = kC + 4;  // floats between the rows of an fp32 triangle in shared memory

template <bool kBackward>
struct PrepSmem {
  // K and Q; then A = L diag(beta) and Inv in fp32, and in A's place Inv in two bf16 parts
  static constexpr int kInv = kC * kLdA * 4, kTiles = 2 * kInv;
  static_assert(kTiles >= 2 * kC * 128 * 2, "K and Q");
  static constexpr int kScores = kTiles;  // the rest of the record: P and the factors
  static constexpr int kToken = kScores + record_bytes(kBackward) - kOffP, kQn = kToken + kC * 16, kBar = kQn + kC * 4;
  static constexpr int kBytes = kBar + 16;  // the tiles' barrier and the flag
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
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prep_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps, unsigned char* records, int several) {
  using L = PrepSmem<kBackward>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sk = sm32(smem), sq = sk + kC * DK * 2, bar = sk + L::kBar;
  if (not_aligned(sk, &g_delta_timeouts)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h0 = blockIdx.y * several, grp = h0 / (a.heads / a.groups);  // the first of this CTA's heads
  // The last 16 rows have four times the first's work, so which warp has which goes round: the warps of a scheduler
  // then have all kinds.
  const int rb = (warp + (int)(blockIdx.x + blockIdx.y)) & 3, r0 = 16 * rb;
  const Chunk c = chunk_of(a.tab, blockIdx.x);
  float4* token = reinterpret_cast<float4*>(smem + L::kToken);  // G in two parts, kappa, beta
  float* qn = reinterpret_cast<float*>(smem + L::kQn);
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kBar + 8);
  if (c.len == kC) {
    if (threadIdx.x == 0) {
      bar_init(bar, 1);
      *gave_up = 0u;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(2u * kC * DK * 2) : "memory");
#pragma unroll
      for (int b = 0; b < DK / 64; ++b) {
        tma_3d(sk + b * kC * 128, &maps.k, 64 * b, grp, c.row, bar);
        tma_3d(sq + b * kC * 128, &maps.q, 64 * b, grp, c.row, bar);
      }
    }
  } else {  // the rows behind the run's last, which may be another run's, are zeros
    const bf16* k = static_cast<const bf16*>(a.k) + (int64_t)grp * a.dk;
    const bf16* q = static_cast<const bf16*>(a.q) + (int64_t)grp * a.dk;
    constexpr int units = DK / 8;
#pragma unroll 4
    for (int e = threadIdx.x; e < kC * units; e += kPrepThreads) {
      const int r = e / units, u = e % units;
      const bool in = r < c.len && 8 * u < a.dk;
      const int64_t row = c.row + (in ? r : 0);
      const int col = in ? 8 * u : 0;
      copy16(sk + wide_at(r, u), k + row * a.ld_k + col, in);
      copy16(sq + wide_at(r, u), q + row * a.ld_q + col, in);
    }
    copies_end();
  }
  // The decays of a head: asked for early, and summed by the warp with the least of the products.
  float gv[2] = {}, bv[2] = {};
  auto ask = [&](int h) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * half + lane;
      const int64_t at = (int64_t)(c.row + i) * a.heads + h;
      gv[half] = i < c.len && a.g ? a.g[at] : 0.0f;
      bv[half] = i < c.len ? (a.beta ? a.beta[at] : 1.0f) : 0.0f;
    }
  };
  auto sum_decays = [&]() {
    float hi[2], lo[2], last[2] = {0.0f, 0.0f};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (gv[half] < -10000.0f) gv[half] = -10000.0f;  // (a NaN stays one)
      scan_decays(gv[half] * kLog2e, hi[half], lo[half], lane);
      const DF s = df_add(DF{hi[half], lo[half]}, DF{last[0], last[1]});
      const int i = 32 * half + lane;
      token[i].x = s.hi;
      token[i].y = s.lo;
      token[i].w = bv[half];
      last[0] = __shfl_sync(0xffffffffu, s.hi, 31);
      last[1] = __shfl_sync(0xffffffffu, s.lo, 31);
    }
  };
  if (rb == 0) ask(h0);
  copies_done();
  __syncthreads();
  if (rb == 0) sum_decays();
  if (c.len == kC) {
    bar_wait(bar, 0, gave_up);
    __syncwarp();
  }
  // K K^T and Q K^T below and on the diagonal blocks, a warp 16 rows; and of Q Q^T what has the queries' lengths
  float kk[8][4], qk[8][4], qq[2][4] = {};
  const bool l2 = a.l2_eps >= 0.0f;
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[n][j] = qk[n][j] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t ak[4], aq[4], b[4];
    load4(ak, sk + wide_cols(r0, 2 * ks, lane));
    load4(aq, sq + wide_cols(r0, 2 * ks, lane));
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      if (nb <= rb) {
        load4(b, sk + wide_rows(16 * nb, 2 * ks, lane));
        mma(kk[2 * nb], ak, b[0], b[1]);
        mma(kk[2 * nb + 1], ak, b[2], b[3]);
        mma(qk[2 * nb], aq, b[0], b[1]);
        mma(qk[2 * nb + 1], aq, b[2], b[3]);
      }
    if (l2) {
      load4(b, sq + wide_rows(r0, 2 * ks, lane));
      mma(qq[0], aq, b[0], b[1]);
      mma(qq[1], aq, b[2], b[3]);
    }
  }
  if (t == g >> 1) {  // reciprocal lengths, from the diagonals
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float k2 = 0.0f;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
        if (nb == rb) k2 = g & 1 ? kk[2 * nb + half][2 * half + 1] : kk[2 * nb + half][2 * half];
      const float q2 = g & 1 ? qq[half][2 * half + 1] : qq[half][2 * half];
      const int r = r0 + g + 8 * half;
      token[r].z = r >= c.len ? 0.0f : l2 ? rsqrtf(k2 + a.l2_eps) : 1.0f;
      qn[r] = r >= c.len ? 0.0f : l2 ? rsqrtf(q2 + a.l2_eps) : 1.0f;
    }
  }
  __syncthreads();  // lengths are there; K and Q have been read
  float* A = reinterpret_cast<float*>(smem);
  float* inv = reinterpret_cast<float*>(smem + L::kInv);
  unsigned char* scores = smem + L::kScores;
  for (int hh = 0; hh < several; ++hh) {
  if (hh > 0) {
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();  // the last record has been copied
    if (rb == 0) sum_decays();
    __syncthreads();
  }
  if (rb == 0 && hh + 1 < several) ask(h0 + hh + 1);
  const float4 row[2] = {token[r0 + g], token[r0 + g + 8]};
  const float rq[2] = {qn[r0 + g] * a.scale, qn[r0 + g + 8] * a.scale};
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (n / 2 > rb) continue;
    const int j0 = 8 * n + 2 * t;
    const float4 col[2] = {token[j0], token[j0 + 1]};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = r0 + g + 8 * half;
      float l[2], p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + e;
        const float d = j <= i ? ex2((row[half].x - col[e].x) + (row[half].y - col[e].y)) * col[e].z : 0.0f;
        l[e] = j < i ? kk[n][2 * half + e] * d * row[half].z * col[e].w : 0.0f;
        p[e] = qk[n][2 * half + e] * d * rq[half];
        if (j > i) p[e] = 0.0f;
      }
      *reinterpret_cast<float2*>(A + i * kLdA + j0) = make_float2(l[0], l[1]);
      const uint32_t at = block_at(rb, n >> 1) + narrow_at(g + 8 * half, n & 1) + 4 * t;
      if constexpr (kBackward) {
        uint32_t hi, lo;
        split(p[0], p[1], hi, lo);
        *reinterpret_cast<uint32_t*>(scores + at) = hi;
        *reinterpret_cast<uint32_t*>(scores + kTri + at) = lo;
      } else {
        *reinterpret_cast<uint32_t*>(scores + at) = pair(p[0], p[1]);
      }
    }
  }
  if (threadIdx.x < kC) {  // the tokens' factors
    float* f = reinterpret_cast<float*>(scores + off_factors(kBackward) - kOffP);
    const int i = threadIdx.x;
    const float4 v = token[i], end = token[kC - 1];
    const float up = ex2(v.x + v.y), left = ex2((end.x - v.x) + (end.y - v.y));
    f[kUp + i] = up * v.z;
    f[kLeft + i] = left * v.z;
    f[kUpQ + i] = up * (qn[i] * a.scale);
    f[kBeta + i] = v.w;
    f[kGamma + i] = ex2(end.x + end.y);
    if (kBackward) {
      f[kGHi + i] = v.x;
      f[kGLo + i] = v.y;
      f[kKn + i] = v.z;
      f[kQn + i] = qn[i];
    }
  }
  __syncwarp();
  // Inv: the diagonal blocks by substitution, a column a lane (a warp's own rows of A are what it wrote)
  if (lane < 16) {
    float x[16];
    const float* rows = A + r0 * kLdA + r0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 v = *reinterpret_cast<const float4*>(rows + i * kLdA + l);
        s = fmaf(-v.x, x[l], s);
        if (l + 1 < i) s = fmaf(-v.y, x[l + 1], s);
        if (l + 2 < i) s = fmaf(-v.z, x[l + 2], s);
        if (l + 3 < i) s = fmaf(-v.w, x[l + 3], s);
      }
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
      for (int n = 0; n < 2; ++n) mma(d[n], al, bh[n][0], bh[n][1]);
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(d[n], ah, bl[n][0], bl[n][1]);
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(d[n], ah, bh[n][0], bh[n][1]);
    };
    const int j = 3 - rb;  // (the first column has the most blocks: for the warp that had the fewest rows)
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
#pragma unroll
  for (int e = threadIdx.x; e < 10 * 32; e += kPrepThreads) {  // a 16-byte unit of each part, where A was
    const int blk = e >> 5, r = (e >> 1) & 15, u = e & 1;
    const int i = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, j = blk - i * (i + 1) / 2;
    const float* from = inv + (16 * i + r) * kLdA + 16 * j + 8 * u;
    const float4 x = *reinterpret_cast<const float4*>(from), y = *reinterpret_cast<const float4*>(from + 4);
    uint4 hi, lo;
    split(x.x, x.y, hi.x, lo.x);
    split(x.z, x.w, hi.y, lo.y);
    split(y.x, y.y, hi.z, lo.z);
    split(y.z, y.w, hi.w, lo.w);
    *reinterpret_cast<uint4*>(smem + blk * 512 + narrow_at(r, u)) = hi;
    *reinterpret_cast<uint4*>(smem + kOffInvLo + blk * 512 + narrow_at(r, u)) = lo;
  }
  // the record goes out in two copies
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned char* rec = records + ((int64_t)blockIdx.x * a.heads + h0 + hh) * record_bytes(kBackward);
    auto out = [](unsigned char* to, uint32_t from, int bytes) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
    };
    out(rec, sk, kOffP);
    out(rec + kOffP, sk + L::kScores, record_bytes(kBackward) - kOffP);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  }
  if (threadIdx.x == 0) {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (c.len == kC && *gave_up) atomicAdd(&g_delta_timeouts, 1u);
  }
}

// ------------------------------------------------------------------ the state through the chunks

// Four warps share a chunk's tiles, two CTAs an SM (of 128 channels: 113 KB, 243 registers). Bound by the tensor pipe,
// busy 68 % of the time, and by two warps a scheduler that wait for their own products in between: 24 prompts of 16 384
// tokens in all, 16 heads of 128 x 128, take 142 us (0.25 GB in and out: 1.8 TB/s). Eight warps to a chunk's tiles took
// 157 us, three CTAs an SM (168 registers, the keys alone held twice) 153 us, so it is instructions that they share, not
// latency that more warps would fill.
template <int DK, int NW>
struct Chain : Stages<DK, false, NW, 2> {
  static constexpr int kOffBar = Stages<DK, false, NW, 2>::kEnd, kSmem = kOffBar + 32;
};

template <int DK, int NW>
__global__ void __launch_bounds__(32 * NW, 2) delta_chain_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps, const unsigned char* records) {
  using L = Chain<DK, NW>;
  constexpr int KS = DK / 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = sm32(smem);
  if (not_aligned(base, &g_delta_timeouts)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int run = a.order[blockIdx.z], h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int dv0 = blockIdx.x * 16 * NW, dv = dv0 + 16 * warp;  // this CTA's, this warp's first row
  const int first = a.tab.cu[run], len = a.tab.cu[run + 1] - first, n = (len + kC - 1) / kC;
  const bool fresh = seq_fresh(a.tab, run);
  if (len == 0 && !fresh) return;
  auto bar = [&](int ch) { return base + L::kOffBar + 8u * (uint32_t)(ch & 1); };
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBar + 16);
  if (threadIdx.x == 0) {
    bar_init(bar(0), 32);
    bar_init(bar(1), 32);
    *gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
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
  auto fetch = [&](int ch) {  // (warp 0)
    load_stage<DK, false, NW, 2>(ch, base, bar(ch), a, maps, a.v, a.ld_v,
                              records + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * record_bytes(false),
                              first + (int64_t)ch * kC, min(kC, len - ch * kC), grp, h, dv0, lane);
  };
  if (n > 0 && warp == 0) fetch(0);
  auto kept = [&](int ch) { return a.ckpt + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * a.dv * a.dk; };
  if (a.ckpt && n > 0) each([&](float* v, int64_t at) { *reinterpret_cast<float2*>(kept(0) + at) = make_float2(v[0], v[1]); });
  for (int ch = 0; ch < n; ++ch) {
    if (ch > 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (y was written where the next chunk's v comes)
      __syncthreads();  // every warp is done with the other stage
    }
    if (ch + 1 < n && warp == 0) fetch(ch + 1);
    bar_wait(bar(ch), (uint32_t)((ch >> 1) & 1), gave_up);
    __syncwarp();
    const uint32_t at = base + L::k(ch), qt = base + L::q(ch), rec = base + L::rec(ch), vt = base + L::v(ch) + warp * L::kStrip;
    const float* f = reinterpret_cast<const float*>(smem + (rec - base) + off_factors(false));
    // X^T = S0 K^T (the state in two parts) and S0 Q^T (in one: it ends in a bf16 output)
    float x[8][4], y[8][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t sh[4], sl[4], b[4][4], c[4];
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
        load4(c, qt + wide_rows(16 * nb, 2 * ks, lane));
        mma_if(ks == 0, y[2 * nb], sh, c[0], c[1]);
        mma_if(ks == 0, y[2 * nb + 1], sh, c[2], c[3]);
        mma(x[2 * nb], sl, b[nb][0], b[nb][1]);
        mma(x[2 * nb + 1], sl, b[nb][2], b[nb][3]);
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
    for (int jb = 0; jb < 4; ++jb)
    {
      uint32_t b[4][4];
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        load4(b[ib], rec + block_at(ib, jb) + narrow_rows(0, lane));
        mma_if(jb == 0, x[2 * ib], ah[jb], b[ib][0], b[ib][1]);
        mma_if(jb == 0, x[2 * ib + 1], ah[jb], b[ib][2], b[ib][3]);
      }
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        mma(x[2 * ib], al[jb], b[ib][0], b[ib][1]);
        mma(x[2 * ib + 1], al[jb], b[ib][2], b[ib][3]);
      }
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        load4(b[ib], rec + kOffInvLo + block_at(ib, jb) + narrow_rows(0, lane));
        mma(x[2 * ib], ah[jb], b[ib][0], b[ib][1]);
        mma(x[2 * ib + 1], ah[jb], b[ib][2], b[ib][3]);
      }
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
      uint32_t b[4][4];
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        load4(b[ib], rec + kOffP + block_at(ib, jb) + narrow_rows(0, lane));
        mma(y[2 * ib], uh, b[ib][0], b[ib][1]);
        mma(y[2 * ib + 1], uh, b[ib][2], b[ib][3]);
      }
#pragma unroll
      for (int ib = jb; ib < 4; ++ib) {
        mma(y[2 * ib], ul, b[ib][0], b[ib][1]);
        mma(y[2 * ib + 1], ul, b[ib][2], b[ib][3]);
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
      for (int n0 = 0; n0 < KS; n0 += 4) {
        uint32_t b[4][4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          load4t(b[nb], at + wide_cols(16 * jb, 2 * (n0 + nb), lane));
          mma(s[2 * (n0 + nb)], uh, b[nb][0], b[nb][1]);
          mma(s[2 * (n0 + nb) + 1], uh, b[nb][2], b[nb][3]);
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          mma(s[2 * (n0 + nb)], ul, b[nb][0], b[nb][1]);
          mma(s[2 * (n0 + nb) + 1], ul, b[nb][2], b[nb][3]);
        }
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
    // The next chunk's checkpoint by way of y's place, 32 columns at a time: from the registers a store would touch eight
    // lines for 256 bytes (8 192 tokens, 16 heads, 8 runs 125 us, with lines whole 122; 16 runs 106 and 101).
    if (a.ckpt && ch + 1 < n) {
      unsigned char* turn = smem + (vt - base);
      auto unit = [](int row, int u) { return row * 128 + ((u ^ (2 * (row & 3))) << 4); };
#pragma unroll
      for (int r = 0; r < DK / 32; ++r) {
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float2*>(turn + unit(g + 8 * half, 2 * i + (t >> 1)) + 8 * (t & 1)) =
                make_float2(s[4 * r + i][2 * half], s[4 * r + i][2 * half + 1]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int row = 4 * it + (lane >> 3), c = 32 * r + 4 * (lane & 7);
          if (dv + row < a.dv && c < a.dk)
            *reinterpret_cast<float4*>(kept(ch + 1) + (int64_t)(dv + row) * a.dk + c) =
                *reinterpret_cast<const float4*>(turn + unit(row, lane & 7));
        }
      }
    }
  }
  each([&](float* v, int64_t at) { *reinterpret_cast<float2*>(st + at) = make_float2(v[0], v[1]); });
  if (lane == 0 && *gave_up) atomicAdd(&g_delta_timeouts, 1u);
}

// ------------------------------------------------------------------ the same with two warps to 16 rows
//
// Where there are few chains, a chunk's time is that of its products one after another. Here two warps share 16 rows of
// the state: each holds one half of its columns, so each has half of the products with K and Q; they add up their parts
// of X and Y, each takes half of the tokens through Inv and P, and they exchange the u that come out. The first and last
// 16 tokens are warp 0's, those between warp 1's: both have five of the ten blocks of a triangle. One more warp copies.
// Bound by latency: one run of 32 768 tokens, 32 heads of 128 x 128, takes 990 us, 3 800 cycles a chunk (one warp to 16
// rows: 5 200), of which the tensor pipe works 47 %.
constexpr int kAhead = 3;  // chunks whose tiles are held (with two, 970 of a chunk's 4 300 cycles were waiting for them)

template <int DK, int NP>
struct Pairs : Stages<DK, false, NP, kAhead> {
  static constexpr int kMail = 12 * 512;  // of a warp: 48 registers of every lane
  static constexpr int kOffMail = Stages<DK, false, NP, kAhead>::kEnd, kOffBar = kOffMail + 2 * NP * kMail;
  static constexpr int kOffFlag = kOffBar + 8 * 2 * kAhead, kSmem = kOffFlag + 16;
  enum Bar : int { kFull = 0, kEmpty = kAhead };  // + chunk % kAhead
  static_assert(kSmem <= 232448, "shared memory plan exceeds 227 KB");
};

__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory"); }

template <int DK, int NP>
__global__ void __launch_bounds__(64 * NP + 32, 1) delta_pairs_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps, const unsigned char* records) {
  using L = Pairs<DK, NP>;
  constexpr int KS = DK / 32;  // k-steps of a half
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = sm32(smem);
  if (not_aligned(base, &g_delta_timeouts)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int pr = warp >> 1, half = warp & 1;
  const int run = a.order[blockIdx.z], h = blockIdx.y, grp = h / (a.heads / a.groups);
  const int dv0 = blockIdx.x * 16 * NP, dv = dv0 + 16 * pr;
  const int first = a.tab.cu[run], len = a.tab.cu[run + 1] - first, n = (len + kC - 1) / kC;
  const bool fresh = seq_fresh(a.tab, run);
  if (len == 0 && !fresh) return;
  auto bar = [&](int id) { return base + L::kOffBar + 8u * (uint32_t)id; };
  volatile uint32_t* gave_up = reinterpret_cast<volatile uint32_t*>(smem + L::kOffFlag);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kAhead; ++i) {
      bar_init(bar(L::kFull + i), 32);
      bar_init(bar(L::kEmpty + i), 2 * NP);
    }
    *gave_up = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (warp == 2 * NP) {
    for (int ch = 0; ch < n; ++ch) {
      if (ch >= kAhead) bar_wait(bar(L::kEmpty + ch % kAhead), (uint32_t)((ch / kAhead - 1) & 1), gave_up);
      load_stage<DK, false, NP, kAhead>(ch, base, bar(L::kFull + ch % kAhead), a, maps, a.v, a.ld_v,
                                records + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * record_bytes(false),
                                first + (int64_t)ch * kC, min(kC, len - ch * kC), grp, h, dv0, lane);
    }
    copies_end();
    copies_done();
    return;
  }
  const int own[2] = {half, 3 - half};  // this warp's blocks of 16 tokens
  float s[2 * KS][4];
  float* st = a.state + ((int64_t)seq_slot(a.tab, run) * a.heads + h) * a.dv * a.dk;
  const int col0 = half * (DK / 2);
  const int64_t at0 = (int64_t)(dv + g) * a.dk + col0 + 2 * t;
  auto each = [&](auto f) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (dv + 8 * r < a.dv)
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i)
          if (col0 + 8 * i < a.dk) f(s[i] + 2 * r, at0 + (int64_t)(8 * r) * a.dk + 8 * i);
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
  unsigned char* mail = smem + L::kOffMail + warp * L::kMail;          // what the other warp reads
  const unsigned char* post = smem + L::kOffMail + (warp ^ 1) * L::kMail;  // what it has written
  auto put = [&](int i, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    *reinterpret_cast<uint4*>(mail + i * 512 + lane * 16) = make_uint4(w0, w1, w2, w3);
  };
  auto get = [&](const unsigned char* from, int i) { return *reinterpret_cast<const uint4*>(from + i * 512 + lane * 16); };
  for (int ch = 0; ch < n; ++ch) {
    bar_wait(bar(L::kFull + ch % kAhead), (uint32_t)((ch / kAhead) & 1), gave_up);
    __syncwarp();
    const uint32_t at = base + L::k(ch), qt = base + L::q(ch), rec = base + L::rec(ch), vt = base + L::v(ch) + pr * L::kStrip;
    const float* f = reinterpret_cast<const float*>(smem + (rec - base) + off_factors(false));
    if (a.ckpt) {
      float* o = a.ckpt + ((int64_t)(a.tab.tile[run] + ch) * a.heads + h) * a.dv * a.dk;
      each([&](float* v, int64_t to) { *reinterpret_cast<float2*>(o + to) = make_float2(v[0], v[1]); });
    }
    float x[8][4];
    uint32_t sh[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t sl[4], b[4][4];
      const int unit = half * (DK / 16) + 2 * ks;
#pragma unroll
      for (int j = 0; j < 4; ++j) split(s[2 * ks + (j >> 1)][2 * (j & 1)], s[2 * ks + (j >> 1)][2 * (j & 1) + 1], sh[ks][j], sl[j]);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        load4(b[nb], at + wide_rows(16 * nb, unit, lane));
        mma_if(ks == 0, x[2 * nb], sh[ks], b[nb][0], b[nb][1]);
        mma_if(ks == 0, x[2 * nb + 1], sh[ks], b[nb][2], b[nb][3]);
      }
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        mma(x[2 * nb], sl, b[nb][0], b[nb][1]);
        mma(x[2 * nb + 1], sl, b[nb][2], b[nb][3]);
      }
    }
    pair_sync(pr);  // the other has read its mail of the last chunk
#pragma unroll
    for (int i = 0; i < 8; ++i) put(i, __float_as_uint(x[i][0]), __float_as_uint(x[i][1]), __float_as_uint(x[i][2]), __float_as_uint(x[i][3]));
    // (this half's part of Y, which nothing of the chain waits for, while the mail is on its way)
    float yo[2][2][4];  // Y of this warp's tokens
    {
      float y[8][4];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t c[4];
          load4(c, qt + wide_rows(16 * nb, half * (DK / 16) + 2 * ks, lane));
          mma_if(ks == 0, y[2 * nb], sh[ks], c[0], c[1]);
          mma_if(ks == 0, y[2 * nb + 1], sh[ks], c[2], c[3]);
        }
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // (block 3 o of the tokens is warp 0's, block 1 + o warp 1's)
            yo[o][i][j] = half ? y[2 * (1 + o) + i][j] : y[6 * o + i][j];
            w[j] = __float_as_uint(half ? y[6 * o + i][j] : y[2 * (1 + o) + i][j]);
          }
          put(8 + 2 * o + i, w[0], w[1], w[2], w[3]);
        }
    }
    pair_sync(pr);
    auto plus = [&](float (&d)[4], const uint4& w) {
      d[0] += __uint_as_float(w.x);
      d[1] += __uint_as_float(w.y);
      d[2] += __uint_as_float(w.z);
      d[3] += __uint_as_float(w.w);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) plus(x[i], get(post, i));
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 2; ++i) plus(yo[o][i], get(post, 8 + 2 * o + i));
    // R = V - up X, as left operands of 16 tokens each
    uint32_t ah[4][4], al[4][4];
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t v[4];
      load4t(v, vt + narrow_cols(16 * jb, lane));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 2 * jb + (j >> 1);
        const float2 up = *reinterpret_cast<const float2*>(f + kUp + 8 * i + 2 * t);
        const uint32_t w = v[(j >> 1) + 2 * (j & 1)];
        split(fmaf(-up.x, x[i][2 * (j & 1)], __uint_as_float(w << 16)),
              fmaf(-up.y, x[i][2 * (j & 1) + 1], __uint_as_float(w & 0xffff0000u)), ah[jb][j], al[jb][j]);
      }
    }
    pair_sync(pr);  // both have read the mail
    // r of this warp's tokens, and from it u: for the scores as it is, for the state with what is left at the chunk's end
    float r[2][2][4], rl[2][2][4];  // (two sums, for a shorter chain)
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t b[2][4], c[2][4];
#pragma unroll
      for (int o = 0; o < 2; ++o)
        if (jb <= own[o]) {
          load4(b[o], rec + block_at(own[o], jb) + narrow_rows(0, lane));
          load4(c[o], rec + kOffInvLo + block_at(own[o], jb) + narrow_rows(0, lane));
          mma_if(jb == 0, r[o][0], ah[jb], b[o][0], b[o][1]);
          mma_if(jb == 0, r[o][1], ah[jb], b[o][2], b[o][3]);
          mma_if(jb == 0, rl[o][0], al[jb], b[o][0], b[o][1]);
          mma_if(jb == 0, rl[o][1], al[jb], b[o][2], b[o][3]);
          mma(rl[o][0], ah[jb], c[o][0], c[o][1]);
          mma(rl[o][1], ah[jb], c[o][2], c[o][3]);
        }
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      uint32_t uh[4], ul[4], wh[4], wl[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 16 * own[o] + 8 * i + 2 * t;
        const float2 b = *reinterpret_cast<const float2*>(f + kBeta + tok);
        const float2 left = *reinterpret_cast<const float2*>(f + kLeft + tok);
        const float2 up = *reinterpret_cast<const float2*>(f + kUpQ + tok);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float u0 = (r[o][i][2 * e] + rl[o][i][2 * e]) * b.x, u1 = (r[o][i][2 * e + 1] + rl[o][i][2 * e + 1]) * b.y;
          split(u0, u1, uh[2 * i + e], ul[2 * i + e]);
          split(u0 * left.x, u1 * left.y, wh[2 * i + e], wl[2 * i + e]);
          yo[o][i][2 * e] *= up.x;
          yo[o][i][2 * e + 1] *= up.y;
        }
      }
      put(4 * o, uh[0], uh[1], uh[2], uh[3]);
      put(4 * o + 1, ul[0], ul[1], ul[2], ul[3]);
      put(4 * o + 2, wh[0], wh[1], wh[2], wh[3]);
      put(4 * o + 3, wl[0], wl[1], wl[2], wl[3]);
    }
    const float gamma = f[kGamma];
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] *= gamma;
    pair_sync(pr);
    auto mail_of = [&](int jb) {  // block jb's u: whose it is; it is that one's block jb / 2
      return ((jb == 0 || jb == 3) == (half == 0)) ? static_cast<const unsigned char*>(mail) : post;
    };
    // S = gamma S + (left u)^T K, which the next chunk waits for
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t b[KS][4];
      const uint4 h4 = get(mail_of(jb), 4 * (jb >> 1) + 2), l4 = get(mail_of(jb), 4 * (jb >> 1) + 3);
      const uint32_t wh[4] = {h4.x, h4.y, h4.z, h4.w}, wl[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
      for (int nb = 0; nb < KS; ++nb) {
        load4t(b[nb], at + wide_cols(16 * jb, half * (DK / 16) + 2 * nb, lane));
        mma(s[2 * nb], wh, b[nb][0], b[nb][1]);
        mma(s[2 * nb + 1], wh, b[nb][2], b[nb][3]);
      }
#pragma unroll
      for (int nb = 0; nb < KS; ++nb) {
        mma(s[2 * nb], wl, b[nb][0], b[nb][1]);
        mma(s[2 * nb + 1], wl, b[nb][2], b[nb][3]);
      }
    }
    // Y = scale exp(G) S0 q + u^T P^T
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      const uint4 h4 = get(mail_of(jb), 4 * (jb >> 1)), l4 = get(mail_of(jb), 4 * (jb >> 1) + 1);
      const uint32_t uh[4] = {h4.x, h4.y, h4.z, h4.w}, ul[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (jb <= own[e]) {
          uint32_t c[4];
          load4(c, rec + kOffP + block_at(own[e], jb) + narrow_rows(0, lane));
          mma(yo[e][0], uh, c[0], c[1]);
          mma(yo[e][1], uh, c[2], c[3]);
          mma(yo[e][0], ul, c[0], c[1]);
          mma(yo[e][1], ul, c[2], c[3]);
        }
    }
    // y takes the place of its tokens' v (both warps have read it)
    const int m = min(kC, len - ch * kC), col = dv + 8 * (lane & 1);
    bf16* out = static_cast<bf16*>(a.y) + (first + (int64_t)ch * kC) * a.ld_y + (int64_t)h * a.dv + col;
#pragma unroll
    for (int o = 0; o < 2; ++o)
      store4t(vt + narrow_cols(16 * own[o], lane), pair(yo[o][0][0], yo[o][0][1]), pair(yo[o][1][0], yo[o][1][1]),
              pair(yo[o][0][2], yo[o][0][3]), pair(yo[o][1][2], yo[o][1][3]));
    __syncwarp();
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int tok = 16 * own[o] + (lane >> 1);
      if (tok < m && col < a.dv)
        *reinterpret_cast<uint4*>(out + tok * a.ld_y) = *reinterpret_cast<const uint4*>(smem + (vt - base) + narrow_at(tok, lane & 1));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (y was written where a later chunk's v comes)
    __syncwarp();
    if (lane == 0) bar_arrive(bar(L::kEmpty + ch % kAhead));
  }
  if (lane == 0 && *gave_up) atomicAdd(&g_delta_timeouts, 1u);
  each([&](float* v, int64_t at) { *reinterpret_cast<float2*>(st + at) = make_float2(v[0], v[1]); });
}

template <int DK, int NP>
cudaError_t run_pairs(const DeltaArgs& a, const DeltaMaps& maps, const unsigned char* records, cudaStream_t st) {
  using L = Pairs<DK, NP>;
  auto kernel = delta_pairs_kernel<DK, NP>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.dv + 16 * NP - 1) / (16 * NP), a.heads, a.tab.n);
  kernel<<<grid, 64 * NP + 32, L::kSmem, st>>>(a, maps, records);
  return cudaGetLastError();
}

template <int DK, int NW>
cudaError_t run_chain(const DeltaArgs& a, const DeltaMaps& maps, const unsigned char* records, cudaStream_t st) {
  using L = Chain<DK, NW>;
  auto kernel = delta_chain_kernel<DK, NW>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.dv + 16 * NW - 1) / (16 * NW), a.heads, a.tab.n);
  kernel<<<grid, 32 * NW, L::kSmem, st>>>(a, maps, records);
  return cudaGetLastError();
}

template <int DK, bool kBackward>
cudaError_t run_prep(const DeltaArgs& a, const DeltaMaps& maps, unsigned char* records, cudaStream_t st) {
  const int chunks = a.tab.tile[a.tab.n];
  if (chunks == 0) return cudaSuccess;
  auto kernel = delta_prep_kernel<DK, kBackward>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem<kBackward>::kBytes);
  if (e != cudaSuccess) return e;
  // Heads of a group that a CTA takes one after another, from one product of keys and queries: as many, up to eight, as
  // leave three quarters of the SMs' places a CTA (us of 1, 2, 4 and 8 heads, chunks of 128 channels and 16 heads: 512
  // chunks of one group 108, 89, 84, 83; 128 of two groups 31, 27, 26, 37; 64 of eight groups 18.4 and 16.6 of 1 and 2
  // heads, 32 of them 10.5 and 11.6).
  int several = 1;
  for (int d = 2; d <= 8; ++d)
    if (a.heads / a.groups % d == 0 && (int64_t)chunks * (a.heads / d) >= 3 * device_sm_count()) several = d;
  kernel<<<dim3(chunks, a.heads / several), kPrepThreads, PrepSmem<kBackward>::kBytes, st>>>(a, maps, records, several);
  return cudaGetLastError();
}

template <int DK>
cudaError_t run_forward(const DeltaArgs& a, unsigned char* records, cudaStream_t st) {
  DeltaMaps maps;
  if (a.tab.cu[a.tab.n] > 0 && !delta_maps(&maps, a, a.v, a.ld_v)) return cudaErrorInvalidValue;
  const cudaError_t e = run_prep<DK, false>(a, maps, records, st);
  if (e != cudaSuccess) return e;
  // Two warps to 16 rows while the SMs have room for them, so that a chunk takes less time; beyond that one warp, which
  // does no product twice and needs no exchange. Microseconds of (two warps, one block of 16 rows a CTA | two blocks |
  // one warp, four blocks), 8 192 tokens, 16 heads of 128 x 128: 128 blocks in all 230 | 250 | 348, 256 blocks
  // 232 | 182 | 253, 384 blocks 235 | 146 | 156, 512 blocks 221 | 137 | 129, 1 024 blocks 214 | 123 | 97.
  const int64_t blocks = (int64_t)a.tab.n * a.heads * ((a.dv + 15) / 16), sms = device_sm_count();
  if (blocks <= sms) return run_pairs<DK, 1>(a, maps, records, st);
  if (blocks <= 3 * sms) return run_pairs<DK, 2>(a, maps, records, st);
  return run_chain<DK, 4>(a, maps, records, st);
}

}  // namespace

unsigned int read_delta_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_timeouts, sizeof v) != cudaSuccess) return 0xffffffffu;
  return v;
}

bool delta_chunked_supported(mamba2_dtype act, int dv, int dk) { return act == MAMBA2_BF16 && dk <= 128 && dv <= 128; }

size_t delta_records(int64_t chunks, int heads, bool backward) { return (size_t)chunks * heads * record_bytes(backward); }

cudaError_t launch_delta_records(const DeltaArgs& a, const DeltaMaps& maps, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  return a.dk <= 64 ? run_prep<64, true>(a, maps, records, st) : run_prep<128, true>(a, maps, records, st);
}

cudaError_t launch_delta_chunked(const DeltaArgs& a, void* ws, cudaStream_t st) {
  unsigned char* records = static_cast<unsigned char*>(ws);
  return a.dk <= 64 ? run_forward<64>(a, records, st) : run_forward<128>(a, records, st);
}

}  // namespace mamba2
