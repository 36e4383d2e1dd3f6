// What the chunked kernels of the gated delta rule share: warp matrix products (bf16, fp32 sums), their fragments in
// shared memory, and the records that the chunks' first pass leaves to the others (internal to libmamba2). Included
// inside an anonymous namespace of each translation unit that uses it.
//
// Fragments of a warp's m16n8k16 product, g = lane / 4, t = lane % 4: the sum's registers hold (row g, columns 2t, 2t+1)
// and (row g + 8, the same); two neighbouring sums are, packed to bf16 pairs, the left operand of the next product.
#pragma once

constexpr int kC = MAMBA2_DELTA_CHUNK;  // tokens of a chunk
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t sm32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ float ex2(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}

__device__ __forceinline__ uint32_t pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two values as a bf16 pair and the pair of what it leaves of them: together off by at most 2^-16 of each.
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pair(a, b);
  lo = pair(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// (not volatile: a product that takes the sum of the one before it waits 21 cycles, one of another sum 8)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_if(bool first, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (first) mma_new(d, a, b0, b1);  // (known when compiled)
  else mma(d, a, b0, b1);
}
__device__ __forceinline__ void load4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void store4t(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
               :: "r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---- tiles in shared memory; 16-byte units are placed so that eight rows of a unit fall on different banks, as the
// tensor maps' swizzles place them (tiles begin at multiples of 1024 bytes)
// [rows][columns] bf16 in blocks of 64 columns: byte offset of 16-byte unit c of row r
template <int kRows = kC>
__device__ __forceinline__ uint32_t wide_at(int r, int c) {
  return (uint32_t)((c >> 3) * kRows * 128 + r * 128 + (((c ^ r) & 7) << 4));
}
// [rows][16] bf16
__device__ __forceinline__ uint32_t narrow_at(int r, int c) { return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }

// Addresses of the 16 x 16 block at row r0 and unit c0 (lane's own row for ldmatrix.x4): the four matrices are
// rows 0-7 | rows 0-7, columns 8-15 | rows 8-15 | rows 8-15, columns 8-15: as loaded, the right operand of two products
// whose columns are the block's rows.
template <int kRows = kC>
__device__ __forceinline__ uint32_t wide_rows(int r0, int c0, int lane) {
  return wide_at<kRows>(r0 + (lane & 7) + ((lane & 16) >> 1), c0 + ((lane >> 3) & 1));
}
__device__ __forceinline__ uint32_t narrow_rows(int r0, int lane) {
  return narrow_at(r0 + (lane & 7) + ((lane & 16) >> 1), (lane >> 3) & 1);
}
// The same block with rows 8-15 second: transposed as loaded, the right operand of two products whose columns are the
// block's columns.
template <int kRows = kC>
__device__ __forceinline__ uint32_t wide_cols(int r0, int c0, int lane) {
  return wide_at<kRows>(r0 + (lane & 15), c0 + (lane >> 4));
}
__device__ __forceinline__ uint32_t narrow_cols(int r0, int lane) { return narrow_at(r0 + (lane & 15), lane >> 4); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// ---- barriers on which copies in shared memory are waited for. A wait gives up after about a second, raises the CTA's
// flag, and from then on no wait of the CTA waits: its warps run to their ends (what they write is then wrong, and
// counted), so that none is left at a barrier of its pair.
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An arrival once this thread's copies so far have landed.
__device__ __forceinline__ void bar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_over(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred P;\nmbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\nselp.u32 %0, 1, 0, P;\n}\n"
               : "=r"(done) : "r"(bar), "r"(parity), "r"(1000u) : "memory");
  return done != 0;
}
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up) {
  for (uint32_t i = 0; i < 1u << 20; ++i) {
    if (bar_over(bar, parity) || *gave_up) return;
  }
  *gave_up = 1u;
}

// The swizzled tiles need a base at a multiple of 1024 bytes; a CTA that has none does nothing, and is counted.
__device__ __forceinline__ bool not_aligned(uint32_t base, unsigned int* count) {
  if ((base & 1023u) == 0) return false;
  if (threadIdx.x == 0) atomicAdd(count, 1u);
  return true;
}

// ---- records: for each chunk and head, what depends on keys, queries, decays and betas alone
// Lower triangles of 64 x 64, as 16 x 16 blocks of bf16 (narrow tiles), block (i, j) at i (i + 1) / 2 + j.
constexpr int kTri = 10 * 512;
__device__ __forceinline__ constexpr int block_at(int i, int j) { return (i * (i + 1) / 2 + j) * 512; }
// Inv = (I + L diag(beta))^-1 in two bf16 parts, then the scores P (in two, for the backward pass), then the factors.
constexpr int kOffInvLo = kTri, kOffP = 2 * kTri, kOffPLo = 3 * kTri;
// Per token: exp(G) kappa, exp(G_C - G) kappa, scale exp(G) kappa_q, beta; exp(G_C); and for the backward pass G in two
// parts (in units of log 2), kappa and kappa_q.
enum Factor : int { kUp = 0, kLeft = kC, kUpQ = 2 * kC, kBeta = 3 * kC, kGamma = 4 * kC, kGHi = 5 * kC, kGLo = 6 * kC,
                    kKn = 7 * kC, kQn = 8 * kC };
__host__ __device__ constexpr int off_factors(bool backward) { return (backward ? 4 : 3) * kTri; }
// What the chains copy with a chunk's tiles: all of it, or (backward) the factors alone.
__host__ __device__ constexpr int copied_from(bool backward) { return backward ? off_factors(true) : 0; }
__host__ __device__ constexpr int copied_bytes(bool backward) { return (backward ? 0 : off_factors(false)) + 5 * kC * 4; }
__host__ __device__ constexpr int record_bytes(bool backward) { return off_factors(backward) + (backward ? 9 : 5) * kC * 4; }

// Which run, and which of its chunks, the batch's chunk is.
struct Chunk {
  int run, at, row, len;  // at: in the run; row: its first; len: its tokens
};
template <typename Table>
__device__ __forceinline__ Chunk chunk_of(const Table& t, int chunk) {
  Chunk c;
  c.run = find_tile_seq(t, chunk);
  c.at = chunk - t.tile[c.run];
  c.row = t.cu[c.run] + c.at * kC;
  c.len = min(kC, t.cu[c.run + 1] - c.row);
  return c;
}

// ---- a chunk's tiles: keys and queries of a group, the record of a head, and 16 columns of values (or gradients of y)
// for each of kStrips strips of the state's rows
// (kDepth of each, for the chunk at hand and the next)
template <int DK, bool kBackward, int kStrips, int kDepth>
struct Stages {
  static constexpr int kTile = kC * DK * 2, kStrip = kC * 32, kRecBytes = copied_bytes(kBackward);
  static constexpr int kV = kDepth * 2 * kTile, kRec = kV + kDepth * kStrips * kStrip, kEnd = kRec + kDepth * kRecBytes;
  static constexpr int kCopied = 2 * kTile + kRecBytes + kStrips * kStrip;
  __device__ static __forceinline__ uint32_t k(int ch) { return (uint32_t)(ch % kDepth) * (2 * kTile); }
  __device__ static __forceinline__ uint32_t q(int ch) { return k(ch) + kTile; }
  __device__ static __forceinline__ uint32_t v(int ch) { return kV + (uint32_t)(ch % kDepth) * (kStrips * kStrip); }
  __device__ static __forceinline__ uint32_t rec(int ch) { return kRec + (uint32_t)(ch % kDepth) * kRecBytes; }
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// By a whole warp; `bar` counts its 32 lanes. Whole chunks by tensor maps; the rows behind a run's last chunk, which may
// be another run's, are zeros, so that one comes row by row. v: the head's columns from v0 on, of a.dv in all.
template <int DK, bool kBackward, int kStrips, int kDepth>
__device__ __forceinline__ void load_stage(int ch, uint32_t base, uint32_t bar, const DeltaArgs& a, const DeltaMaps& maps, const void* vp,
                                           int64_t ld_v, const unsigned char* rec, int64_t row0, int m, int grp, int h, int v0,
                                           int lane) {
  using L = Stages<DK, kBackward, kStrips, kDepth>;
  const uint32_t tk = base + L::k(ch), tq = base + L::q(ch), tv = base + L::v(ch), tr = base + L::rec(ch);
  if (m == kC) {
    if (lane == 0) {
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((uint32_t)L::kCopied) : "memory");
#pragma unroll
      for (int b = 0; b < DK / 64; ++b) tma_3d(tk + b * kC * 128, &maps.k, 64 * b, grp, (int)row0, bar);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                   ::"r"(tr), "l"(rec + copied_from(kBackward)), "r"((uint32_t)L::kRecBytes), "r"(bar) : "memory");
#pragma unroll
      for (int b = 0; b < DK / 64; ++b) tma_3d(tq + b * kC * 128, &maps.q, 64 * b, grp, (int)row0, bar);
#pragma unroll
      for (int s = 0; s < kStrips; ++s) tma_3d(tv + s * kC * 32, &maps.v, v0 + 16 * s, h, (int)row0, bar);
    } else {
      bar_arrive(bar);
    }
    return;
  }
  constexpr int units = DK / 8;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + (int64_t)grp * a.dk;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)grp * a.dk;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(vp) + (int64_t)h * a.dv + v0;
#pragma unroll 4
  for (int e = lane; e < kC * units; e += 32) {
    const int r = e / units, u = e % units;
    const bool in = r < m && 8 * u < a.dk;
    const int64_t row = row0 + (in ? r : 0);
    const int col = in ? 8 * u : 0;
    copy16(tk + wide_at(r, u), k + row * a.ld_k + col, in);
    copy16(tq + wide_at(r, u), q + row * a.ld_q + col, in);
  }
#pragma unroll 4
  for (int e = lane; e < L::kRecBytes / 16; e += 32) copy16(tr + 16 * e, rec + copied_from(kBackward) + 16 * e, true);
#pragma unroll 4
  for (int e = lane; e < kC * 2 * kStrips; e += 32) {
    const int r = e / (2 * kStrips), u = e % (2 * kStrips);
    const bool in = r < m && v0 + 8 * u < a.dv;
    copy16(tv + (u >> 1) * (kC * 32) + narrow_at(r, u & 1), v + (row0 + (in ? r : 0)) * ld_v + (in ? 8 * u : 0), in);
  }
  bar_arrive_copies(bar);
}
