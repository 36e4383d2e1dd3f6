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

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// ---- tiles in shared memory; 16-byte units are placed so that eight rows of a unit fall on different banks
// [rows][kCols] bf16: byte offset of 16-byte unit c of row r
template <int kCols>
__device__ __forceinline__ uint32_t wide_at(int r, int c) {
  return (uint32_t)(r * kCols * 2 + ((c ^ (r & 7)) << 4));
}
// [rows][16] bf16
__device__ __forceinline__ uint32_t narrow_at(int r, int c) { return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }

// Addresses of the 16 x 16 block at row r0 and unit c0 (lane's own row for ldmatrix.x4): the four matrices are
// rows 0-7 | rows 0-7, columns 8-15 | rows 8-15 | rows 8-15, columns 8-15: as loaded, the right operand of two products
// whose columns are the block's rows.
template <int kCols>
__device__ __forceinline__ uint32_t wide_rows(int r0, int c0, int lane) {
  return wide_at<kCols>(r0 + (lane & 7) + ((lane & 16) >> 1), c0 + ((lane >> 3) & 1));
}
__device__ __forceinline__ uint32_t narrow_rows(int r0, int lane) {
  return narrow_at(r0 + (lane & 7) + ((lane & 16) >> 1), (lane >> 3) & 1);
}
// The same block with rows 8-15 second: transposed as loaded, the right operand of two products whose columns are the
// block's columns.
template <int kCols>
__device__ __forceinline__ uint32_t wide_cols(int r0, int c0, int lane) {
  return wide_at<kCols>(r0 + (lane & 15), c0 + (lane >> 4));
}
__device__ __forceinline__ uint32_t narrow_cols(int r0, int lane) { return narrow_at(r0 + (lane & 15), lane >> 4); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

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
