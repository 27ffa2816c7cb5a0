// Shared pieces of the gated delta rule's chunked kernels: the operand tiles
// ("images"), products of fp16 pairs on the tensor cores, and the scales that
// keep fp32 values inside fp16's range.
//
// Why fp16 pairs. The states, the carried gradients and the sums behind dg and
// dbeta are fp32 results, so every operand that is itself a result (T, P, u,
// the states) enters a product as hi + lo, two fp16 values of 11 bits each:
// 22 bits, against 16 of a bf16 pair, at the same tensor-core rate. q, k, v and
// do of bfloat16 calls have 8 bits and are exact as one fp16 value after a
// scale by a power of two, so a product with them takes two mma (a b_hi +
// a b_lo) and a product of two pairs three (the lo lo term is 2^-22 of it).
// fp16 has 5 exponent bits: every tile carries a power-of-two scale that puts
// its largest magnitude just below 2^14 (pow2_scale). A value keeps the 22 bits
// down to 2^-17 of that, fewer below, and is lost at 2^-39, which costs nothing in
// a sum that holds the larger ones. So a scale comes from the values themselves: a
// bound that is loose by more than 2^10 or so costs bits of all of them.
//
// Images. A tile lives in global memory exactly as in shared memory: rows of
// 128 bytes (64 fp16 values; wider tiles are several such panels one after the
// other) whose eight 16-byte pieces are permuted by the row (piece ^ (row &
// 7)), so that ldmatrix reads eight rows from eight different bank groups and a
// whole tile moves by one bulk copy. A lower triangular 64 x 64 tile keeps only its ten lower 16 x 16
// blocks (tri), each with rows of 32 bytes whose two pieces are swapped in
// every other four rows. The hi part comes first, then the lo part.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gdr_launch.h"
#include "wkv7_common.cuh"

namespace gdr {

using wkv7::mbar_arrive_expect_tx;
using wkv7::mbar_init;
using wkv7::mbar_wait_bounded;
using wkv7::smem_addr;

// ------------------------------------------------------------ elements ---

template <typename T> struct In;
template <> struct In<__nv_bfloat16> {
  static constexpr int kParts = 1;  // fp16 parts that hold a value exactly (after scaling)
};
template <> struct In<float> {
  static constexpr int kParts = 2;
};

__device__ __forceinline__ void load8(float (&x)[8], const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint4 u;
  uint32_t* w = &u.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
// The squares of vectors that are normalised are formed of the vector times kSmall,
// the epsilon's part with them: in fp32's range up to a length of 2^115.
constexpr float kSmall = 0x1p-52f, kSmallEps = 1e-6f * 0x1p-104f;
// ---------------------------------------------------------- fp16 pairs ---

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// (a, b) as a packed hi and, for kP = 2, a packed lo.
template <int kP>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(a, b);
  if constexpr (kP == 2) {
    const float2 f = unpack_f16(hi);
    lo = pack_f16(a - f.x, b - f.y);
  }
}

// The power of two s with largest * s in [2^13, 2^14), its exponent held to
// +-120 so that s and 1/s are normal floats (0 gives 2^120; infinity and NaN
// give 2^-115, and the values themselves carry them into the products).
__device__ __forceinline__ float pow2_scale(float largest) {
  int e = (int)((__float_as_uint(largest) >> 23) & 255u) - 127;
  e = 13 - e;
  e = e > 120 ? 120 : (e < -120 ? -120 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Largest of a warp's non-negative floats (NaN counts as larger than all).
__device__ __forceinline__ float warp_max_abs(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
__device__ __forceinline__ float abs_max(float m, float x) {  // keeps NaN
  return __uint_as_float(max(__float_as_uint(m), __float_as_uint(x) & 0x7FFFFFFFu));
}

// ------------------------------------------------------------- images ----

// Offset (in halves) of (row, col) in an image of `rows` rows.
__device__ __forceinline__ int img(int rows, int row, int col) {
  return (col >> 6) * rows * 64 + row * 64 + ((((col >> 3) & 7) ^ (row & 7)) << 3) + (col & 7);
}

// Lower triangular images: the block (i, j), j <= i < 4, and a place in it. The
// blocks of a column follow one another.
constexpr int kTriPart = 10 * 256;
__host__ __device__ constexpr int tri_block(int i, int j) { return (j * (7 - j) / 2 + i) * 256; }
__device__ __forceinline__ int tri_at(int row, int col) { return row * 16 + (((col >> 3) ^ ((row >> 2) & 1)) << 3) + (col & 7); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void stsm4(__half* p, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(smem_addr(p)), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stsm4t(void* p, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(smem_addr(p)), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a b: adds to the zero register, which takes no instruction to clear d.
__device__ __forceinline__ void mma16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Fragments of m16n8k16 for one 16-deep block, from an image of `rows` rows
// (lo part `part` halves after the hi part). With g = lane / 4, t = lane % 4
// the accumulator holds C[g][2t, 2t+1] and C[g+8][2t, 2t+1].
//   a_mk: A[m][k] stored [m][k];  a_km: A stored [k][m]
//   b_nk: B (16 columns) stored [n][k];  b_kn: B stored [k][n]
template <int kP>
struct Frag {
  uint32_t h[4];
  uint32_t l[kP == 2 ? 4 : 1];
};
template <int kP>
__device__ __forceinline__ void a_mk(Frag<kP>& f, const __half* s, int rows, int part, int m0, int k0, int lane) {
  const __half* p = s + img(rows, m0 + (lane & 15), k0 + (lane >> 4) * 8);
  ldsm4(f.h, p);
  if constexpr (kP == 2) ldsm4(f.l, p + part);
}
template <int kP>
__device__ __forceinline__ void a_km(Frag<kP>& f, const __half* s, int rows, int part, int m0, int k0, int lane) {
  const __half* p = s + img(rows, k0 + (lane & 7) + (lane >> 4) * 8, m0 + ((lane >> 3) & 1) * 8);
  ldsm4t(f.h, p);
  if constexpr (kP == 2) ldsm4t(f.l, p + part);
}
template <int kP>
__device__ __forceinline__ void b_nk(Frag<kP>& f, const __half* s, int rows, int part, int n0, int k0, int lane) {
  const __half* p = s + img(rows, n0 + (lane & 7) + (lane >> 4) * 8, k0 + ((lane >> 3) & 1) * 8);
  ldsm4(f.h, p);
  if constexpr (kP == 2) ldsm4(f.l, p + part);
}
template <int kP>
__device__ __forceinline__ void b_kn(Frag<kP>& f, const __half* s, int rows, int part, int n0, int k0, int lane) {
  const __half* p = s + img(rows, k0 + (lane & 15), n0 + (lane >> 4) * 8);
  ldsm4t(f.h, p);
  if constexpr (kP == 2) ldsm4t(f.l, p + part);
}
// A fragments from a lower triangular pair image: its block (i, j), or that
// block transposed (A[m][k] = X[16 i + k][16 j + m]).
__device__ __forceinline__ void a_tri(Frag<2>& f, const __half* s, int i, int j, int lane) {
  const __half* p = s + tri_block(i, j) + tri_at(lane & 15, (lane >> 4) * 8);
  ldsm4(f.h, p);
  ldsm4(f.l, p + kTriPart);
}
__device__ __forceinline__ void a_tri_t(Frag<2>& f, const __half* s, int i, int j, int lane) {
  const __half* p = s + tri_block(i, j) + tri_at((lane & 7) + (lane >> 4) * 8, ((lane >> 3) & 1) * 8);
  ldsm4t(f.h, p);
  ldsm4t(f.l, p + kTriPart);
}
__device__ __forceinline__ void put2_tri(__half* s, int row, int col, float x0, float x1) {
  uint32_t hi, lo;
  split2<2>(x0, x1, hi, lo);
  const int at = tri_block(row >> 4, col >> 4) + tri_at(row & 15, col & 15);
  *reinterpret_cast<uint32_t*>(s + at) = hi;
  *reinterpret_cast<uint32_t*>(s + at + kTriPart) = lo;
}

// Two n8 tiles += a b, the small terms first.
template <bool kFirst = false>
__device__ __forceinline__ void mma_pair(float (&d0)[4], float (&d1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  if constexpr (kFirst) {
    mma16_first(d0, a, b[0], b[1]);
    mma16_first(d1, a, b[2], b[3]);
  } else {
    mma16(d0, a, b[0], b[1]);
    mma16(d1, a, b[2], b[3]);
  }
}
template <int kA, int kB>
__device__ __forceinline__ void mma_parts(float (&d0)[4], float (&d1)[4], const Frag<kA>& a, const Frag<kB>& b) {
  if constexpr (kA == 2) mma_pair(d0, d1, a.l, b.h);
  if constexpr (kB == 2) mma_pair(d0, d1, a.h, b.l);
  mma_pair(d0, d1, a.h, b.h);
}

template <int kA, int kB>
__device__ __forceinline__ void mma_parts_first(float (&d0)[4], float (&d1)[4], const Frag<kA>& a, const Frag<kB>& b) {
  if constexpr (kA == 2) mma_pair<true>(d0, d1, a.l, b.h);
  if constexpr (kB == 2) mma_pair<kA != 2>(d0, d1, a.h, b.l);
  mma_pair<kA != 2 && kB != 2>(d0, d1, a.h, b.h);
}

// N pairs of n8 tiles += a b[n] (or, kFirst, = a b[n]): part by part over all of
// them, so that two mma on one accumulator stand 2 N apart (a dependent mma waits
// 38 cycles, an independent one 8 to 16).
template <int N, bool kFirst = false, int kA, int kB, int kTilesOf>
__device__ __forceinline__ void mma_row(float (&d)[kTilesOf][4], const Frag<kA>& a, const Frag<kB> (&b)[N]) {
  if constexpr (kA == 2)
#pragma unroll
    for (int n = 0; n < N; ++n) mma_pair<kFirst>(d[2 * n], d[2 * n + 1], a.l, b[n].h);
  if constexpr (kB == 2)
#pragma unroll
    for (int n = 0; n < N; ++n) mma_pair<kFirst && kA != 2>(d[2 * n], d[2 * n + 1], a.h, b[n].l);
#pragma unroll
  for (int n = 0; n < N; ++n) mma_pair<kFirst && kA != 2 && kB != 2>(d[2 * n], d[2 * n + 1], a.h, b[n].h);
}

// Two accumulator tiles (16 rows, columns k0 .. k0+7 and k0+8 .. k0+15) times s
// as the A fragment of a product over those columns.
template <int kP>
__device__ __forceinline__ void to_a(Frag<kP>& f, const float (&x)[4], const float (&y)[4], float s) {
  uint32_t l[4];
  split2<kP>(x[0] * s, x[1] * s, f.h[0], l[0]);
  split2<kP>(x[2] * s, x[3] * s, f.h[1], l[1]);
  split2<kP>(y[0] * s, y[1] * s, f.h[2], l[2]);
  split2<kP>(y[2] * s, y[3] * s, f.h[3], l[3]);
  if constexpr (kP == 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) f.l[i] = l[i];
}
// ---------------------------------------------------------- bulk copies ---

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A thread that started copies, after it gave up: no copy is left in flight, either
// phase of each barrier is waited for, for a millisecond at most.
__device__ __forceinline__ void drain(uint64_t* bar) {
  mbar_wait_bounded(nullptr, bar, 0, 1000000);
  mbar_wait_bounded(nullptr, bar, 1, 1000000);
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int N>
__device__ __forceinline__ float warp_max(const float (&x)[N][4]) {
  // four chains of max; a NaN is passed over here and carries itself into the products
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fabsf(x[n][e]));
  return warp_max_abs(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
}
template <int N>
__device__ __forceinline__ void zero(float (&x)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
}

// --------------------------------------------------- sequences and chunks ---

struct SeqRange {
  int b;       // batch row the sequence lies in
  int t0, t1;  // its tokens there
  long long slot;  // its first chunk slot
};
// Packed starts are clamped into [0, T] and to non-negative lengths, so that
// no value in them can take an access out of a buffer.
__device__ __forceinline__ SeqRange seq_range(const Shape& a, int s) {
  SeqRange r;
  if (a.starts) {
    const int x0 = min(max(a.starts[s], 0), a.T), x1 = min(max(a.starts[s + 1], 0), a.T);
    r.b = 0, r.t0 = x0, r.t1 = max(x0, x1), r.slot = x0 / kC + s;
  } else {
    r.b = s, r.t0 = 0, r.t1 = a.T, r.slot = (long long)s * ((a.T + kC - 1) / kC);
  }
  return r;
}
// Of a packed call: the tokens that sequences cover, of the first's start to the
// last's end; those before and behind lie in none.
__device__ __forceinline__ int2 covered(const Shape& a) {
  return make_int2(seq_range(a, 0).t0, seq_range(a, a.nseq - 1).t1);
}
struct ChunkAt {
  int b, t0, len;
  bool last;  // the sequence's last chunk
};
__device__ __forceinline__ bool chunk_at(const Shape& a, int slot, ChunkAt& c) {
  if (a.starts) {
    int lo = 0, hi = a.nseq - 1;  // the last sequence whose first slot is <= slot
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (min(max(a.starts[mid], 0), a.T) / kC + mid <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
    const SeqRange r = seq_range(a, lo);
    const int at = slot - (int)r.slot;
    if (at < 0 || r.t0 + at * kC >= r.t1) return false;
    c.b = 0, c.t0 = r.t0 + at * kC, c.len = min(kC, r.t1 - c.t0), c.last = c.t0 + kC >= r.t1;
    return true;
  }
  const int nc = (a.T + kC - 1) / kC;
  c.b = slot / nc;
  c.t0 = (slot - c.b * nc) * kC;
  c.len = min(kC, a.T - c.t0);
  c.last = c.t0 + kC >= a.T;
  return true;
}

}  // namespace gdr
