// Matrix product with bias, activation and residual in its epilogue (block.h), from bf16
// or e4m3 operands, and its backward pass: tcgen05 products, fp32 accumulators in tensor
// memory, operands by TMA.
//
// Many rows: pairs of CTAs (cta_group::2), persistent, 256 x 256 output tiles, N fastest.
// Each CTA of a pair loads its half of A (128 rows) and of B (128 columns) per k-block of
// 128 bytes, so a pair moves 64 KB from L2 per 256 x 256 x 64 (bf16) products, two thirds
// of what two CTAs with 128 x 256 tiles of their own would. Roles in each CTA:
//   warp 0      TMA loads, completing on the leader's barrier of the stage
//   warp 1      (leader) tcgen05.mma into one of two 256-column accumulators; commits
//               free the stage and publish the accumulator in both CTAs
//   warps 2-9   epilogue of this CTA's 128 rows while the next tile's products run:
//               tensor memory -> registers -> shared memory (32 x 32 blocks, so that a
//               warp's loads and stores of global memory follow the rows) -> scales,
//               bias, activation, residual -> global
// Few rows: the weight takes the instruction's 128 rows and the tokens its N, and a
// cluster splits the K axis, see few_rows_kernel.
//
// Measured (GB300, bf16, six calls in a graph on an idle GPU; in brackets without a pause, where
// the power limit holds the clock down): 16 384 x 2 048 x 4 096 with bias, SiLU and residual
// 171 us [197] (1 610 TFLOP/s, 84 % of the measured cuBLAS rate in bursts), without any of them
// 158 [179], with `pre` too 182 [207], GELU 188 [208]; the products alone, the epilogue's work
// left out, took 139 (1 980), so what remains is the last tile's epilogue (6 us), the fill and
// what the epilogue takes from the products beside it. e4m3 16 001 x 4 096 x 4 096 with residual
// 174 us [201] (3 090 TFLOP/s). Both backward products of 8 192 x 2 048 x 4 096 152 us [179]
// (1 810 TFLOP/s). 5 x 2 048 x 8 192 9.5 us with weights from HBM (3.5 TB/s; 7.5 us with three
// weights in turn, which L2 holds in good part), in e4m3 7.5 us (2.2 TB/s).
//
// Every mbarrier wait is bounded; a timeout stops the CTA's roles, drains what was
// issued, frees tensor memory and counts the CTA in g_linear_timeouts.
#include <cuda.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "../../include/block.h"
#include "common.cuh"
#include "host.h"

namespace mamba2 {

__device__ unsigned int g_linear_timeouts = 0;

namespace {

#include "tc.cuh"

// The flushing forms of the exponential and the reciprocal: what they flush is below 2^-126 (and the others scale
// around that at several instructions each).
__device__ __forceinline__ float exp2_ftz(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
__device__ __forceinline__ float recip_ftz(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_ftz(float v) { return recip_ftz(1.0f + exp2_ftz(v * -kLog2e)); }

// The normal distribution's tail 1 - Phi(|v|), and bell = exp(-v^2 / 2). The tail is t P(t) bell with t = 1 / (1 + 0.3 |v|)
// (the form that Hastings gave erfc), P of degree 7 fitted to the ratio of the two, for |v| up to 13.5, by least relative
// error: 1.3e-7 of the tail, however small it is, where a fit of the same form to erfc's absolute error loses digits from
// -2 on. No branch. bell is rounded as v^2 / 2 is: the tail's relative error is at most (64 + 2 v^2) 2^-24. Below 2^-126
// (|v| above 13.2) both are 0.
__device__ __forceinline__ void normal_tail(float v, float& tail, float& bell) {
  const float x = fabsf(v), t = recip_ftz(fmaf(0.3f, x, 1.0f));
  bell = exp2_ftz(x * x * (-0.5f * kLog2e));
  float p = fmaf(t, 0.03593175858f, -0.15827606618f);
  p = fmaf(t, p, 0.20820668340f);
  p = fmaf(t, p, -0.05539390445f);
  p = fmaf(t, p, 0.12946923077f);
  p = fmaf(t, p, 0.09963748604f);
  p = fmaf(t, p, 0.12079836428f);
  p = fmaf(t, p, 0.11962639540f);
  tail = t * p * bell;
}
__device__ __forceinline__ float gelu(float v) {
  float tail, bell;
  normal_tail(v, tail, bell);
  return v * (v < 0.0f ? tail : 1.0f - tail);
}
// max(v, 0); a NaN stays one.
__device__ __forceinline__ float relu(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}
// (one branch for all of them)
template <int n>
__device__ __forceinline__ void activate_all(float (&v)[n], int act) {
  if (act == MAMBA2_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] *= sigmoid_ftz(v[i]);
  } else if (act == MAMBA2_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = gelu(v[i]);
  } else if (act == MAMBA2_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = relu(v[i]);
  }
}
__device__ __forceinline__ float slope(float v, int act) {
  switch (act) {
    case MAMBA2_ACT_RELU: return v > 0.0f ? 1.0f : v <= 0.0f ? 0.0f : v;  // (a NaN's is NaN)
    case MAMBA2_ACT_SILU: {
      const float p = sigmoid_ftz(v);
      return p * fmaf(v, 1.0f - p, 1.0f);
    }
    case MAMBA2_ACT_GELU: {
      float tail, bell;
      normal_tail(v, tail, bell);
      return fmaf(v * 0.39894228040143268f, bell, v < 0.0f ? tail : 1.0f - tail);
    }
  }
  return 1.0f;
}

// One product D[M][N] = sum_k A(m, k) B(n, k) and what its epilogue does:
// D * scale_m[m] * scale_n[n] + bias[n] -> pre; activation; + residual -> out.
struct Product {
  int M, N, K;
  void* out;
  int64_t ld_out;
  const void* residual;
  int64_t ld_res;
  __nv_bfloat16* pre;  // row stride N
  const float* scale_m;
  const float* scale_n;
  const float* bias;
  int act;
  int vec;  // four columns at once: every matrix of the epilogue has rows aligned for them
};

// Four columns of one output row.
template <typename TO> struct Quad;
template <> struct Quad<__nv_bfloat16> {
  using Raw = uint2;
  __device__ __forceinline__ static void unpack(Raw r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x << 16);
    v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16);
    v[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  __device__ __forceinline__ static Raw pack(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <> struct Quad<float> {
  using Raw = float4;
  __device__ __forceinline__ static void unpack(Raw r, float (&v)[4]) {
    v[0] = r.x;
    v[1] = r.y;
    v[2] = r.z;
    v[3] = r.w;
  }
  __device__ __forceinline__ static Raw pack(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};

// Per-column constants of four columns from col on (those past N are not used).
struct Columns {
  float scale[4], bias[4];
};
__device__ __forceinline__ Columns load_columns(const Product& g, int col) {
  Columns c;
  if (col + 4 <= g.N) {  // (col is a multiple of four, and both vectors are 16-byte aligned)
    const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f), none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 sc = g.scale_n ? __ldg(reinterpret_cast<const float4*>(g.scale_n + col)) : one;
    const float4 bi = g.bias ? __ldg(reinterpret_cast<const float4*>(g.bias + col)) : none;
    return {{sc.x, sc.y, sc.z, sc.w}, {bi.x, bi.y, bi.z, bi.w}};
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = col + j < g.N;
    c.scale[j] = g.scale_n && in ? g.scale_n[col + j] : 1.0f;
    c.bias[j] = g.bias && in ? g.bias[col + j] : 0.0f;
  }
  return c;
}

template <typename TO>
__device__ __forceinline__ typename Quad<TO>::Raw load_residual(const Product& g, int64_t row, int col) {
  typename Quad<TO>::Raw r = {};
  if (!g.residual || row >= g.M || col >= g.N) return r;
  const TO* p = static_cast<const TO*>(g.residual) + row * g.ld_res + col;
  if (g.vec && col + 4 <= g.N) return *reinterpret_cast<const typename Quad<TO>::Raw*>(p);
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = col + j < g.N ? Act<TO>::to_f(p[j]) : 0.0f;
  return Quad<TO>::pack(v);
}

template <typename TO>
__device__ __forceinline__ void finish(const Product& g, int64_t row, int col, float (&v)[4], const Columns& c,
                                       typename Quad<TO>::Raw res) {
  if (row >= g.M || col >= g.N) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j], c.scale[j], c.bias[j]);
  const bool whole = g.vec && col + 4 <= g.N;
  if (g.pre) {
    __nv_bfloat16* p = g.pre + row * g.N + col;
    if (whole) {
      *reinterpret_cast<uint2*>(p) = Quad<__nv_bfloat16>::pack(v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < g.N) p[j] = __float2bfloat16_rn(v[j]);
    }
  }
  activate_all(v, g.act);
  if (g.residual) {
    float r[4];
    Quad<TO>::unpack(res, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += r[j];
  }
  TO* o = static_cast<TO*>(g.out) + row * g.ld_out + col;
  if (whole) {
    *reinterpret_cast<typename Quad<TO>::Raw*>(o) = Quad<TO>::pack(v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < g.N) o[j] = Act<TO>::from_f(v[j]);
  }
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// Descriptor of a staged operand: rows of 128 bytes, 128-byte swizzle. K along the row, or
// (mn) M or N along the row, the k-block's kRows rows deep, 64 columns to a block of kRows rows.
template <bool mn, int kRows>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return mn ? sdesc(addr, kRows * 128, 1024) : sdesc(addr, 16, 1024);
}
// One tcgen05.mma takes 32 bytes of K: a step along the row, or 16 rows of 128 bytes.
template <bool mn>
__device__ __forceinline__ uint64_t k_step(int k) {
  return mn ? (uint64_t)((k * 2048) >> 4) : (uint64_t)(2 * k);
}
__host__ __device__ constexpr uint32_t idesc(bool f8, int M, int N, bool a_mn, bool b_mn) {
  const uint32_t type = f8 ? 0u : 1u;  // kind::f8f6f4: e4m3 = 0; kind::f16: bf16 = 1
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

constexpr uint32_t kRowBytes = 128;  // a k-block: 64 bf16 or 128 e4m3

// ------------------------------------------------------------------ many rows

constexpr int kBM = 256, kBN = 256, kStages = 5;
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kHalf = 128 * kRowBytes;  // one CTA's half of A or B: 16 KB
constexpr uint32_t kStage = 2 * kHalf;
constexpr uint32_t kOffEpi = kStages * kStage;
constexpr int kEpiLd = 36;  // floats between the rows of a warp's 32 x 32 block: 16-byte accesses without conflicts
constexpr uint32_t kEpiBytes = 32 * kEpiLd * 4;
constexpr uint32_t kOffBar = kOffEpi + kEpiWarps * kEpiBytes;
enum Bar : int { kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = 2 * kStages + 2,
                 kDone = 2 * kStages + 4, kNumBars = 2 * kStages + 5 };
constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory plan exceeds 227 KB");

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <bool F8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (F8)
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
  else
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {  // arrives at this offset in both CTAs
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"((uint16_t)3) : "memory");
}

// How an operand is laid out, and the box that its tensor map loads: K along the row (128 rows of 128 bytes); or K
// down the rows, 64 rows of 128 bytes, of two neighbouring blocks of 64 columns at once where the matrix is
// whole blocks wide, else of one (one copy to a stage instead of two: 87 us against 96 for dw of 8 192 x 2 048 x
// 4 096).
enum Layout : int { kAlong = 0, kDown = 1, kDownPaired = 2 };

// The operand's k-block kb, 128 of its rows (or columns) from r0 on, into dst.
template <bool F8, int layout>
__device__ __forceinline__ void load_half(uint32_t dst, const CUtensorMap* tm, int kb, int r0, uint32_t bar) {
  constexpr int depth = F8 ? 128 : 64;
  if constexpr (layout == kDownPaired) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(kb * depth), "r"(r0 / 64), "r"(bar) : "memory");
  } else if constexpr (layout == kDown) {
    tma_load_pair(dst, tm, r0, kb * depth, bar);
    tma_load_pair(dst + kHalf / 2, tm, r0 + 64, kb * depth, bar);
  } else {
    tma_load_pair(dst, tm, kb * depth, r0, bar);
  }
}

// Both products of the backward pass in one launch (dw first: its tiles, over all rows, are the longer ones),
// so that they fill the last wave together: pair p takes every npairs-th tile of dw, and the tiles
// [start[p], start[p + 1]) of dx.
constexpr int kMaxPairs = 80;
struct Split {
  int start[kMaxPairs + 1];
};
template <bool kGrad>
struct Job {
  Product g[kGrad ? 2 : 1];
  CUtensorMap a[kGrad ? 2 : 1], b[kGrad ? 2 : 1];
  int layout_a[2], layout_b[2];
  Split split;
};
template <>
struct Job<false> {
  Product g[1];
  CUtensorMap a[1], b[1];
};

// kGrad: product 0 is dw (rows of both operands are K), product 1 dx (rows of the second are); else the only
// product has K along the rows of both.
template <bool F8, bool kGrad, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
pair_kernel(const __grid_constant__ Job<kGrad> job) {
  static_assert(!F8 || !kGrad, "8-bit operands have K along the row");
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = su32(smem_raw);
  unsigned char* smem = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
  const uint32_t sbase = su32(smem);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc + 4);
  auto bar = [&](int id) { return sbase + kOffBar + 8u * (uint32_t)id; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  constexpr int depth = F8 ? 128 : 64;
  const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;
  // this pair's tiles: the first product's pair, + npairs, ..., then the second's range
  const int tiles0 = (job.g[0].M + kBM - 1) / kBM * ((job.g[0].N + kBN - 1) / kBN);
  const int mine0 = pair < tiles0 ? (tiles0 - 1 - pair) / npairs + 1 : 0;
  int mine = mine0;
  if constexpr (kGrad) mine += job.split.start[pair + 1] - job.split.start[pair];
  struct Tile {
    int which, m0, n0;
  };
  auto tile = [&](int t) -> Tile {  // N fastest
    int which = 0, i = pair + t * npairs;
    if constexpr (kGrad)
      if (t >= mine0) {
        which = 1;
        i = job.split.start[pair] + t - mine0;
      }
    const int across = (job.g[which].N + kBN - 1) / kBN;
    return {which, i / across * kBM, i % across * kBN};
  };
  auto kblocks = [&](int which) { return (job.g[which].K + depth - 1) / depth; };

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(su32(s_tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kFull + s), 1);   // (leader) its own expect_tx; both CTAs' bytes
      mbar_init(bar(kEmpty + s), 1);  // the products' commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kAccFull + b), 1);
      mbar_init(bar(kAccEmpty + b), 2 * kEpiWarps);  // (leader) both CTAs' epilogue warps
    }
    mbar_init(bar(kDone), 1);
    *s_abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready before either signals the other's
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 0) {
    // =================== TMA producer (one thread, and nothing in its loop that can go before it: at a k-block
    // every 280 ns it is what the rest waits for if it takes long)
    if (lane == 0) {
      const uint32_t full0 = at_rank(bar(kFull), 0);
      uint32_t s = 0, turn = 0;
      int issued = 0;
      bool ok = true;
      auto run = [&](const Tile& w, auto la, auto lb) {
        const int m0 = w.m0 + (int)rank * 128, n0 = w.n0 + (int)rank * 128, nkb = kblocks(w.which);
        const CUtensorMap* ma = &job.a[w.which];
        const CUtensorMap* mb = &job.b[w.which];
        for (int kb = 0; kb < nkb; ++kb) {
          // (the first turn's wait is for the phase before the first: over already)
          if (!wait_bar(bar(kEmpty) + 8 * s, turn ^ 1u, s_abort)) {
            ok = false;
            return;
          }
          const uint32_t dst = sbase + s * kStage, full = full0 + 8 * s;
          if (leader) mbar_expect_tx(bar(kFull) + 8 * s, 2 * kStage);
          load_half<F8, decltype(la)::value>(dst, ma, kb, m0, full);
          load_half<F8, decltype(lb)::value>(dst + kHalf, mb, kb, n0, full);
          ++issued;
          if (++s == kStages) {
            s = 0;
            turn ^= 1u;
          }
        }
      };
      using Along = std::integral_constant<int, kAlong>;
      using Down = std::integral_constant<int, kDown>;
      using Paired = std::integral_constant<int, kDownPaired>;
      for (int t = 0; t < mine && ok; ++t) {
        const Tile w = tile(t);
        if constexpr (!kGrad) {
          run(w, Along{}, Along{});
        } else {
          auto with_b = [&](auto la) {
            if (job.layout_b[w.which] == kDownPaired) run(w, la, Paired{});
            else run(w, la, Down{});
          };
          if (job.layout_a[w.which] == kDownPaired) with_b(Paired{});
          else if (job.layout_a[w.which] == kDown) with_b(Down{});
          else with_b(Along{});
        }
      }
      // on an abort, let the loads in flight land before the pair exits
      if (leader && *s_abort)
        for (int i = max(0, issued - kStages); i < issued; ++i)
          drain_bar(bar(kFull + i % kStages), (uint32_t)((i / kStages) & 1));
    }
    __syncwarp();
  } else if (warp == 1) {
    // =================== MMA issuer
    if (leader && lane == 0) {
      uint32_t s = 0, turn = 0;
      bool ok = true;
      for (int t = 0; t < mine && ok; ++t) {
        const int buf = t & 1;
        if (t >= 2 && !wait_bar(bar(kAccEmpty + buf), (uint32_t)(((t >> 1) - 1) & 1), s_abort)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * kBN);
        const int which = tile(t).which, nkb = kblocks(which);
        auto run = [&](auto down) {  // (is K down A's rows)
          constexpr bool a_mn = decltype(down)::value;
          constexpr uint32_t id = idesc(F8, kBM, kBN, a_mn, kGrad);
          for (int kb = 0; kb < nkb; ++kb) {
            if (!wait_bar(bar(kFull) + 8 * s, turn, s_abort)) {
              ok = false;
              return;
            }
            tc_fence_after();
            const uint32_t a0 = sbase + s * kStage;
            const uint64_t ad = operand<a_mn, depth>(a0), bd = operand<kGrad, depth>(a0 + kHalf);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_pair<F8>(d, ad + k_step<a_mn>(k), bd + k_step<kGrad>(k), id, (kb > 0 || k > 0) ? 1u : 0u);
            commit_pair(bar(kEmpty) + 8 * s);
            if (++s == kStages) {
              s = 0;
              turn ^= 1u;
            }
          }
        };
        if (kGrad && which == 0) run(std::bool_constant<kGrad>{});
        else run(std::false_type{});
        if (!ok) break;
        commit_pair(bar(kAccFull + buf));
      }
      // everything issued completes before the pair frees tensor memory
      commit_pair(bar(kDone));
      drain_bar(bar(kDone), 0u);
    }
    __syncwarp();
  } else {
    // =================== epilogue: lanes 32 (warp % 4) .. + 31, one half of the columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    float* blk = reinterpret_cast<float*>(smem + kOffEpi + (uint32_t)(warp - 2) * kEpiBytes);
    // what a chunk of 32 columns needs from global memory is fetched a chunk ahead, across tiles: waited for in
    // its place, it took the epilogue to 15 us a tile (with SiLU and a residual), where 32 k-blocks take 9.
    // The residual is 32 words: four columns of eight rows, or at an edge and where rows are not aligned for that
    // a column of 32 rows (8 192 x 1 024 x 4 095 81 us, 91 when only the first was fetched ahead).
    using Raw = typename Quad<TO>::Raw;
    struct Chunk {
      uint32_t res[32];
      Columns cols;
    };
    constexpr int kRaw = sizeof(Raw) / 4;
    auto whole = [&](const Product& g, int64_t row0, int col0) {  // the same for the whole warp
      return g.vec && col0 + 32 <= g.N && row0 + 32 <= g.M;
    };
    auto fetch = [&](const Tile& w, int c, Chunk& k) {
      const Product& g = job.g[w.which];
      const int col0 = w.n0 + half * 128 + c, col = col0 + 4 * (lane & 7);
      const int64_t row0 = (int64_t)w.m0 + (int)rank * 128 + q * 32;
      if (kGrad) return;  // (gradients are the products as they are)
      k.cols = load_columns(g, col);
      if (!g.residual) return;
      const TO* res = static_cast<const TO*>(g.residual);
      if (whole(g, row0, col0)) {
        const TO* p = res + (row0 + (lane >> 3)) * g.ld_res + col;
#pragma unroll
        for (int i = 0; i < 8; ++i, p += 4 * g.ld_res) {
          const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
          for (int j = 0; j < kRaw; ++j) k.res[kRaw * i + j] = reinterpret_cast<const uint32_t*>(&r)[j];
        }
      } else if (col0 + lane < g.N) {
        const TO* p = res + row0 * g.ld_res + col0 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += g.ld_res)
          if (row0 + i < g.M) {
            if constexpr (sizeof(TO) == 2) k.res[i] = *reinterpret_cast<const uint16_t*>(p);
            else k.res[i] = *reinterpret_cast<const uint32_t*>(p);
          }
      }
    };
    Chunk now;
    Tile at = tile(0);
    if (mine > 0) fetch(at, 0, now);
    for (int t = 0; t < mine; ++t) {
      const int buf = t & 1;
      const Product& g = job.g[at.which];
      const int64_t row0 = (int64_t)at.m0 + (int)rank * 128 + q * 32;
      const int n0 = at.n0 + half * 128;
      const Tile after = tile(min(t + 1, mine - 1));
      const float sm = !kGrad && g.scale_m && row0 + lane < g.M ? g.scale_m[row0 + lane] : 1.0f;
      if (!warp_wait(bar(kAccFull + buf), (uint32_t)((t >> 1) & 1), s_abort)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        const int col = n0 + c + 4 * (lane & 7);
        Chunk next;
        if (c < 96) fetch(at, c + 32, next);
        else fetch(after, 0, next);
        if (n0 + c < g.N && row0 < g.M) {  // the same for the whole warp
          uint32_t r[32];
          tmem_ld32(tmem + lane_off + (uint32_t)(buf * kBN + half * 128 + c), r);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(blk + lane * kEpiLd + 4 * j) =
                make_float4(__uint_as_float(r[4 * j]) * sm, __uint_as_float(r[4 * j + 1]) * sm,
                            __uint_as_float(r[4 * j + 2]) * sm, __uint_as_float(r[4 * j + 3]) * sm);
          __syncwarp();
          const float* mine = blk + (lane >> 3) * kEpiLd + 4 * (lane & 7);
          const int64_t row = row0 + (lane >> 3);
          if (whole(g, row0, n0 + c)) {
            // the whole block: a step at a time over 32 values, so that the branches are the block's
            float v[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = *reinterpret_cast<const float4*>(mine + 4 * i * kEpiLd);
              v[i][0] = kGrad ? f.x : fmaf(f.x, now.cols.scale[0], now.cols.bias[0]);
              v[i][1] = kGrad ? f.y : fmaf(f.y, now.cols.scale[1], now.cols.bias[1]);
              v[i][2] = kGrad ? f.z : fmaf(f.z, now.cols.scale[2], now.cols.bias[2]);
              v[i][3] = kGrad ? f.w : fmaf(f.w, now.cols.scale[3], now.cols.bias[3]);
            }
            if (!kGrad && g.pre) {
              __nv_bfloat16* p = g.pre + row * g.N + col;
#pragma unroll
              for (int i = 0; i < 8; ++i, p += 4 * (int64_t)g.N) *reinterpret_cast<uint2*>(p) = Quad<__nv_bfloat16>::pack(v[i]);
            }
            if (!kGrad) activate_all(reinterpret_cast<float(&)[32]>(v), g.act);
            if (!kGrad && g.residual) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float r4[4];
                Raw r;
#pragma unroll
                for (int j = 0; j < kRaw; ++j) reinterpret_cast<uint32_t*>(&r)[j] = now.res[kRaw * i + j];
                Quad<TO>::unpack(r, r4);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] += r4[j];
              }
            }
            TO* o = static_cast<TO*>(g.out) + row * g.ld_out + col;
#pragma unroll
            for (int i = 0; i < 8; ++i, o += 4 * g.ld_out)
              *reinterpret_cast<typename Quad<TO>::Raw*>(o) = Quad<TO>::pack(v[i]);
          } else {
            // an edge of the matrix, or rows of any alignment: a row an instruction, a column a lane
            const int one = n0 + c + lane;
            const int rows = (int)min((int64_t)32, g.M - row0);
            if (one < g.N) {
              const float sc = !kGrad && g.scale_n ? g.scale_n[one] : 1.0f;
              const float bi = !kGrad && g.bias ? g.bias[one] : 0.0f;
              TO* o = static_cast<TO*>(g.out) + row0 * g.ld_out + one;
              __nv_bfloat16* pre = !kGrad && g.pre ? g.pre + row0 * g.N + one : nullptr;
              const float* from = blk + lane;
              constexpr int kSome = 16;
              auto some = [&](auto first) {  // kSome rows, or as many of them as there are
                constexpr int i0 = decltype(first)::value;
                float v[kSome];
#pragma unroll
                for (int i = 0; i < kSome; ++i) v[i] = kGrad ? from[(i0 + i) * kEpiLd] : fmaf(from[(i0 + i) * kEpiLd], sc, bi);
                if (pre) {
#pragma unroll
                  for (int i = 0; i < kSome; ++i, pre += g.N)
                    if (i0 + i < rows) *pre = __float2bfloat16_rn(v[i]);
                }
                if (!kGrad) activate_all(v, g.act);
                if (!kGrad && g.residual) {
#pragma unroll
                  for (int i = 0; i < kSome; ++i)
                    v[i] += __uint_as_float(sizeof(TO) == 2 ? now.res[i0 + i] << 16 : now.res[i0 + i]);
                }
#pragma unroll
                for (int i = 0; i < kSome; ++i, o += g.ld_out)
                  if (i0 + i < rows) *o = Act<TO>::from_f(v[i]);
              };
              some(std::integral_constant<int, 0>{});
              if (rows > kSome) some(std::integral_constant<int, kSome>{});
            }
          }
          __syncwarp();
        }
        now = next;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                     :: "r"(at_rank(bar(kAccEmpty + buf), 0)) : "memory");
      at = after;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) atomicAdd(&g_linear_timeouts, 1u);
  cluster_sync();  // neither CTA's shared memory goes before the other is done with it
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem));
}

// ------------------------------------------------------------------ few rows

// The product transposed: a tile is 128 rows of w by kN tokens, so a weight of few tokens is read at the
// rate of memory without 256 rows of output to fill. A cluster of CTAs shares a tile, each over its part of
// the K axis; they leave their fp32 parts in shared memory, and each then adds up every S-th token's parts in
// the order of the ranks (over distributed shared memory) and finishes those rows of the output.
template <int kN>
struct Few {
  static constexpr uint32_t kTileW = 128 * kRowBytes, kTileX = kN * kRowBytes, kStage = kTileW + kTileX;
  // two CTAs to an SM
  static constexpr int kStages = (int)(110u * 1024u / kStage) > 6 ? 6 : (int)(110u * 1024u / kStage);
  static constexpr uint32_t kOffBar = kStages * kStage;
  enum Bar : int { kFull = 0, kEmpty = kStages, kDone = 2 * kStages, kNumBars = 2 * kStages + 1 };
  static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
  static constexpr uint32_t kCols = kN < 32 ? 32 : kN;
  static_assert(kN * 128 * 4 <= (int)kOffBar, "the parts take the place of the stages");
};
constexpr int kFewThreads = 256;

template <bool F8>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (F8)
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
  else
    mma_ss(d, a, b, id, acc);
}

template <bool F8, int kN, typename TO>
__global__ void __launch_bounds__(kFewThreads, 2)
few_rows_kernel(const __grid_constant__ Product g, const __grid_constant__ CUtensorMap tmw,
                const __grid_constant__ CUtensorMap tmx) {
  using L = Few<kN>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = su32(smem_raw);
  unsigned char* smem = smem_raw + (((raw_base + 1023u) & ~1023u) - raw_base);
  const uint32_t sbase = su32(smem);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile uint32_t* s_abort = reinterpret_cast<volatile uint32_t*>(smem + L::kOffMisc + 4);
  auto bar = [&](int id) { return sbase + L::kOffBar + 8u * (uint32_t)id; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int depth = F8 ? 128 : 64;
  const int kblocks = (g.K + depth - 1) / depth, S = (int)gridDim.x, rank = (int)blockIdx.x;
  const int kb0 = (int)((int64_t)kblocks * rank / S), n_kb = (int)((int64_t)kblocks * (rank + 1) / S) - kb0;
  const int n0 = (int)blockIdx.y * 128, m0 = (int)blockIdx.z * kN;
  auto load = [&](int i) {  // the i-th k-block of this CTA's
    const int s = i % L::kStages;
    const uint32_t dst = sbase + (uint32_t)s * L::kStage;
    mbar_expect_tx(bar(L::kFull + s), L::kStage);
    tma_load_2d(dst, &tmw, (kb0 + i) * depth, n0, bar(L::kFull + s));
    tma_load_2d(dst + L::kTileW, &tmx, (kb0 + i) * depth, m0, bar(L::kFull + s));
  };

  if (warp == 0) {
    // the first turn of the stages is under way before anything else is set up
    if (lane == 0) {
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(bar(L::kFull + s), 1);
        mbar_init(bar(L::kEmpty + s), 1);
      }
      mbar_init(bar(L::kDone), 1);
      *s_abort = 0u;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("griddepcontrol.wait;" ::: "memory");  // launched as a programmatic dependent
      for (int i = 0; i < min(n_kb, L::kStages); ++i) load(i);
    }
    __syncwarp();
  } else if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(su32(s_tmem)), "n"(L::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 0) {
    if (lane == 0) {
      int issued = min(n_kb, L::kStages);
      for (int i = L::kStages; i < n_kb; ++i) {
        if (!wait_bar(bar(L::kEmpty + i % L::kStages), (uint32_t)((i / L::kStages - 1) & 1), s_abort)) break;
        load(i);
        issued = i + 1;
      }
      if (*s_abort)
        for (int i = max(0, issued - L::kStages); i < issued; ++i)
          drain_bar(bar(L::kFull + i % L::kStages), (uint32_t)((i / L::kStages) & 1));
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id = idesc(F8, 128, kN, false, false);
      for (int i = 0; i < n_kb; ++i) {
        const int s = i % L::kStages;
        if (!wait_bar(bar(L::kFull + s), (uint32_t)((i / L::kStages) & 1), s_abort)) break;
        tc_fence_after();
        const uint32_t a0 = sbase + (uint32_t)s * L::kStage;
        const uint64_t ad = operand<false, depth>(a0), bd = operand<false, depth>(a0 + L::kTileW);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_one<F8>(tmem, ad + k_step<false>(k), bd + k_step<false>(k), id, (i > 0 || k > 0) ? 1u : 0u);
        mma_commit(bar(L::kEmpty + s));
      }
      mma_commit(bar(L::kDone));
    }
  }
  __syncwarp();
  // ---- every product done, every stage read: the parts take the stages' place, [token][128 features]
  float* part = reinterpret_cast<float*>(smem);
  const bool done = warp_wait(bar(L::kDone), 0u, s_abort);
  if (!done) drain_bar(bar(L::kDone), 0u);
  tc_fence_after();
  __syncthreads();
  if (done && warp >= 4) {
    const int q = warp & 3;
#pragma unroll
    for (int c = 0; c < kN; c += 16) {
      float v[16];
      tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = v[j];
    }
  }
  tc_fence_before();
  cluster_sync();
  {
    const int col = n0 + 4 * lane;
    const Columns cc = load_columns(g, col);
    const int tokens = min(kN, g.M - m0);
    for (int t = rank + S * warp; t < tokens; t += S * (kFewThreads / 32)) {
      const int64_t row = m0 + t;
      const typename Quad<TO>::Raw res = load_residual<TO>(g, row, col);
      const float sm = g.scale_m ? g.scale_m[row] : 1.0f;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t at = su32(part + t * 128 + 4 * lane);
      for (int r = 0; r < S; ++r) {
        float u[4];
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]) : "r"(at_rank(at, (uint32_t)r)) : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += u[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= sm;
      finish<TO>(g, row, col, v, cc, res);
    }
  }
  if (threadIdx.x == 0 && *s_abort) atomicAdd(&g_linear_timeouts, 1u);
  __syncthreads();
  cluster_sync();  // nobody reads this CTA's parts any more
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(L::kCols));
}

// ------------------------------------------------------------------ tensor maps

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

// [rows][cols] with a row stride of ld elements: boxes of 128 bytes x box_rows, 128-byte swizzle, zeros past the edges
bool make_map(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f8) {
  std::memset(tm, 0, sizeof *tm);
  const Encode enc = encode_fn();
  if (!enc) return false;
  const int e = f8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * e};
  const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / e), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same matrix as an operand with K down its rows: blocks of 64 columns are the third dimension where the matrix
// is whole blocks wide (so that no box reaches past a row).
bool make_map_down(CUtensorMap* tm, int* layout, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  if (cols % 64 != 0) {
    *layout = kDown;
    return make_map(tm, base, rows, cols, ld, 64, false);
  }
  *layout = kDownPaired;
  std::memset(tm, 0, sizeof *tm);
  const Encode enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, kRowBytes};
  const cuuint32_t box[3] = {64, 64, 2}, estr[3] = {1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t pair_tiles(const Product& g) { return (int64_t)((g.M + kBM - 1) / kBM) * ((g.N + kBN - 1) / kBN); }

template <bool F8, bool kGrad, typename TO>
cudaError_t start_pairs(const Job<kGrad>& job, int pairs, cudaStream_t st) {
  auto kernel = pair_kernel<F8, kGrad, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<2 * pairs, kThreads, kSmem, st>>>(job);
  return cudaGetLastError();
}
int pair_count(int64_t tiles) {
  return (int)std::max<int64_t>(1, std::min<int64_t>({tiles, (int64_t)device_sm_count() / 2, (int64_t)kMaxPairs}));
}

template <bool F8, typename TO>
cudaError_t launch_pairs(const Product& g, const void* x, int64_t ldx, const void* w, cudaStream_t st) {
  Job<false> job = {};
  job.g[0] = g;
  if (!make_map(&job.a[0], x, g.M, g.K, ldx, 128, F8) || !make_map(&job.b[0], w, g.N, g.K, g.K, 128, F8))
    return cudaErrorInvalidValue;
  const int64_t tiles = pair_tiles(g);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  return start_pairs<F8, false, TO>(job, pair_count(tiles), st);
}

// The most rows that the few-rows kernel takes: as long as the pairs' tiles would leave half of the SMs idle (K and N
// of 2 048 and 4 096: 512 rows, 32 tiles, 15.7 us against 17.1 by pairs; 768 rows, 48 tiles, 22.0 against 17.6).
int few_rows_most(const Product& g) {
  const int64_t tiles = pair_tiles(g);
  return g.M <= 128 || 4 * tiles < device_sm_count() ? g.M : 0;
}

template <bool F8, int kN, typename TO>
cudaError_t launch_few(const Product& g, const void* x, int64_t ldx, const void* w, cudaStream_t st) {
  using L = Few<kN>;
  CUtensorMap tmw, tmx;
  if (!make_map(&tmw, w, g.N, g.K, g.K, 128, F8) || !make_map(&tmx, x, g.M, g.K, ldx, kN, F8)) return cudaErrorInvalidValue;
  auto kernel = few_rows_kernel<F8, kN, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles_w = (g.N + 127) / 128, tiles_x = (g.M + kN - 1) / kN;
  const int kblocks = (g.K + (F8 ? 127 : 63)) / (F8 ? 128 : 64);
  // as many parts of K as fill two CTAs an SM, each of two k-blocks at least (weights from HBM, 5 x 2 048 x 8 192: 4 parts
  // 9.5 us, 2 10.1, 1 13.0; 5 x 4 096 x 4 096: 8 and 4 parts 9.9 to 10.3, 2 13.1, 1 20.6)
  const int S = std::max(1, std::min({8, kblocks / 2, (int)(2 * (int64_t)device_sm_count() / ((int64_t)tiles_w * tiles_x))}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, (unsigned)tiles_w, (unsigned)tiles_x);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, g, tmw, tmx);
}

// out = x . w^T by the kernel that suits the number of rows.
template <bool F8, typename TO>
cudaError_t launch_forward(const Product& g, const void* x, int64_t ldx, const void* w, cudaStream_t st) {
  if ((g.N + 127) / 128 <= 65535) {
    if (g.M <= 16) return launch_few<F8, 16, TO>(g, x, ldx, w, st);
    if (g.M <= 32) return launch_few<F8, 32, TO>(g, x, ldx, w, st);
    if (g.M <= 64) return launch_few<F8, 64, TO>(g, x, ldx, w, st);
    if (g.M <= few_rows_most(g)) return launch_few<F8, 128, TO>(g, x, ldx, w, st);
  }
  return launch_pairs<F8, TO>(g, x, ldx, w, st);
}

// ------------------------------------------------------------------ backward: dp and the bias

// dp = dy * activation'(pre) rounded to bf16, and the column sums of each kPartRows rows, unrounded. A CTA takes
// 256 columns of them, a warp every eighth row, a lane 8 columns: adjacent ones where rows are 16-byte aligned,
// else every 32nd. Bound by HBM: dy and pre in, dp out
// (with the bias's sums 36 us for 8 192 x 4 096 and GELU).
// The rounding: the tensor cores take bf16 operands, as dy is, so dp carries one rounding more than its formula; dx and dw
// are off by 2.35e-3 of their 2-norm instead of the 1.66e-3 of their own rounding alone. The bias's sums, which no product
// takes, have none.
constexpr int kPartRows = 64;
constexpr int kPartCols = 256;

template <bool kVec, int act>
__global__ void __launch_bounds__(256) dp_kernel(const LinearBwdArgs a) {
  __shared__ float sums[8][kPartCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * kPartCols;
  const int64_t m0 = (int64_t)blockIdx.x * kPartRows;
  auto col = [&](int j) { return c0 + (kVec ? 8 * lane + j : lane + 32 * j); };
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.0f;
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy);
  const __nv_bfloat16* pre = static_cast<const __nv_bfloat16*>(a.pre);
  if (!kVec || col(0) < a.ld_dp) {
#pragma unroll 2
    for (int i = 0; i < kPartRows / 8; ++i) {
      const int64_t m = m0 + 8 * i + warp;
      if (m >= a.rows) break;
      float v[8], p[8];
      const int64_t at = m * a.out_f;
      if constexpr (kVec) {
        if (col(0) < a.out_f) {
          Vec16<__nv_bfloat16>::load_stream(dy + at + col(0), v);
          if (act) Vec16<__nv_bfloat16>::load_stream(pre + at + col(0), p);
        } else {  // the padding
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = p[j] = 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = col(j) < a.out_f ? __bfloat162float(dy[at + col(j)]) : 0.0f;
          p[j] = act && col(j) < a.out_f ? __bfloat162float(pre[at + col(j)]) : 0.0f;
        }
      }
      if (act) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= slope(p[j], act);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += v[j];
      if (a.dp) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.dp) + m * a.ld_dp;
        if constexpr (kVec) {
          Vec16<__nv_bfloat16>::store(o + col(0), v);  // (the products read it next, from L2 as far as it holds)
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col(j) < a.ld_dp) o[col(j)] = __float2bfloat16_rn(v[j]);
        }
      }
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[warp][col(j) - c0] = s[j];
  __syncthreads();
  const int c = c0 + (int)threadIdx.x;
  if (c < a.out_f) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
    a.partial[(int64_t)blockIdx.x * a.out_f + c] = t;
  }
}

bool quad_ok(const void* p, int64_t ld, size_t elem) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & (4 * elem - 1)) == 0 && ld % 4 == 0);
}

}  // namespace

unsigned int read_linear_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_linear_timeouts, sizeof v) != cudaSuccess) return 0xffffffffu;
  return v;
}

cudaError_t launch_linear(const LinearArgs& a, mamba2_dtype in, mamba2_dtype out, int act, cudaStream_t st) {
  const size_t oe = out == MAMBA2_F32 ? 4 : 2;
  Product g = {a.rows, a.out_f, a.in_f, a.out, a.ld_out, a.residual, a.ld_res, static_cast<__nv_bfloat16*>(a.pre),
               a.x_scale, a.w_scale, a.bias, act, 0};
  g.vec = quad_ok(a.out, a.ld_out, oe) && quad_ok(a.residual, a.ld_res, oe) && quad_ok(a.pre, a.out_f, 2);
  if (in == MAMBA2_BF16) {
    if (out == MAMBA2_BF16) return launch_forward<false, __nv_bfloat16>(g, a.x, a.ld_x, a.w, st);
    return launch_forward<false, float>(g, a.x, a.ld_x, a.w, st);
  }
  if (out == MAMBA2_BF16) return launch_forward<true, __nv_bfloat16>(g, a.x, a.ld_x, a.w, st);
  return launch_forward<true, float>(g, a.x, a.ld_x, a.w, st);
}

int linear_bias_parts(int32_t rows) { return (rows + kPartRows - 1) / kPartRows; }

cudaError_t launch_linear_backward(const LinearBwdArgs& args, int act, cudaStream_t st) {
  LinearBwdArgs a = args;
  if (a.rows == 0) {
    cudaError_t e = a.dw ? cudaMemsetAsync(a.dw, 0, (size_t)a.out_f * a.in_f * 2, st) : cudaSuccess;
    if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, (size_t)a.out_f * 4, st);
    return e;
  }
  const int parts = linear_bias_parts(a.rows);
  const void* dp = a.dp;
  if (act == MAMBA2_ACT_NONE && a.out_f % 8 == 0) {  // dy itself, whose rows TMA can take
    dp = a.dy;
    a.ld_dp = a.out_f;
    a.dp = nullptr;
  }
  if (!a.dx && !a.dw) a.dp = nullptr;
  if (a.dp || a.dbias) {
    const dim3 grid((unsigned)parts, (unsigned)((a.ld_dp + kPartCols - 1) / kPartCols));
    if (grid.y > 65535) return cudaErrorInvalidValue;
    auto run = [&](auto of) {
      constexpr int kAct = decltype(of)::value;
      if (a.out_f % 8 == 0) dp_kernel<true, kAct><<<grid, 256, 0, st>>>(a);
      else dp_kernel<false, kAct><<<grid, 256, 0, st>>>(a);
    };
    switch (act) {
      case MAMBA2_ACT_RELU: run(std::integral_constant<int, MAMBA2_ACT_RELU>{}); break;
      case MAMBA2_ACT_SILU: run(std::integral_constant<int, MAMBA2_ACT_SILU>{}); break;
      case MAMBA2_ACT_GELU: run(std::integral_constant<int, MAMBA2_ACT_GELU>{}); break;
      default: run(std::integral_constant<int, MAMBA2_ACT_NONE>{});
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dbias) e = launch_column_sum(a.dbias, a.partial, parts, a.out_f, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.dx && !a.dw) return cudaSuccess;
  Job<true> job = {};
  for (int i = 0; i < 2; ++i) {
    Product& g = job.g[i];
    g.N = a.in_f;
    g.ld_out = a.in_f;
    g.vec = 1;  // in_f is a multiple of 8
  }
  if (a.dw) {  // dw[n][k] = sum_m dp[m][n] x[m][k]
    job.g[0].M = a.out_f;
    job.g[0].K = a.rows;
    job.g[0].out = a.dw;
    // (dp's own rows are padded with zeros to whole blocks)
    if (!make_map_down(&job.a[0], &job.layout_a[0], dp, a.rows, a.dp ? a.ld_dp : a.out_f, a.ld_dp) ||
        !make_map_down(&job.b[0], &job.layout_b[0], a.x, a.rows, a.in_f, a.ld_x))
      return cudaErrorInvalidValue;
  }
  if (a.dx) {  // dx[m][k] = sum_n dp[m][n] w[n][k]
    job.g[1].M = a.rows;
    job.g[1].K = a.out_f;
    job.g[1].out = a.dx;
    job.layout_a[1] = kAlong;
    if (!make_map(&job.a[1], dp, a.rows, a.out_f, a.ld_dp, 128, false) ||
        !make_map_down(&job.b[1], &job.layout_b[1], a.w, a.out_f, a.in_f, a.in_f))
      return cudaErrorInvalidValue;
  }
  const int64_t t0 = pair_tiles(job.g[0]), t1 = pair_tiles(job.g[1]);
  if (t0 + t1 > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = pair_count(t0 + t1);
  // dx's tiles go to the pairs with the least of dw, under the lowest load that takes them all
  const int64_t c0 = (job.g[0].K + 63) / 64 + 1, c1 = (job.g[1].K + 63) / 64 + 1;  // (one for the epilogue's share)
  auto room = [&](int p, int64_t cap) {
    const int64_t has = (p < t0 ? (t0 - 1 - p) / pairs + 1 : 0) * c0;
    return cap > has ? (cap - has) / c1 : 0;
  };
  int64_t lo = 0, hi = (t0 / pairs + 1) * c0 + (t1 / pairs + 1) * c1;
  while (lo < hi) {
    const int64_t cap = (lo + hi) / 2;
    int64_t n = 0;
    for (int p = 0; p < pairs; ++p) n += room(p, cap);
    if (n >= t1) hi = cap;
    else lo = cap + 1;
  }
  int64_t given = 0;
  for (int p = 0; p <= pairs; ++p) {
    job.split.start[p] = (int)given;
    if (p < pairs) given = std::min(t1, given + room(p, hi));
  }
  return start_pairs<false, true, __nv_bfloat16>(job, pairs, st);
}

}  // namespace mamba2
