// Shared pieces of the chunked linear attention kernels: operands as sums of
// bfloat16 parts, their tiles in shared memory, products of them, decays, and
// where chunks lie.
//
// Why bfloat16 parts. A bfloat16 value is exact in one part; an fp32 value in
// three (8 bits each, 24 in all). Parts have fp32's exponents, so no operand needs
// a scale, whatever its range: nothing is lost of a value beside much larger ones.
// A product of operands with a and b parts is the sum of the products of the parts
// i + j < 3 (the rest is below 2^-24 of it), accumulated in fp32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "linattn_launch.h"
#include "wkv7_common.cuh"

namespace linattn {

using wkv7::smem_addr;
typedef __nv_bfloat16 bf16_t;

template <typename T> struct In;
template <> struct In<bf16_t> {
  static constexpr int kParts = 1;
};
template <> struct In<float> {
  static constexpr int kParts = 3;
};

__device__ __forceinline__ void load8(float (&x)[8], const bf16_t* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
// Two floats at once: a - b (exact where b is a's rounding), a b.
__device__ __forceinline__ float2 minus2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n sub.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 times2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// (a, b) as kP packed parts, each the rounding of what the ones before leave. (An infinity
// leaves NaN; the products that meet it are non-finite anyway.)
template <int kP>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&p)[kP]) {
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    p[i] = pack2(a, b);
    if (i + 1 < kP) {
      const float2 f = unpack2(p[i]), r = minus2(make_float2(a, b), f);
      a = r.x, b = r.y;
    }
  }
}

// --------------------------------------------------------------- tiles ----

// A tile of `rows` rows in shared memory: panels of 64 columns, rows of 128 bytes
// whose eight 16-byte pieces are permuted by the row, so that ldmatrix reads eight
// rows from eight bank groups.
__device__ __forceinline__ int at(int rows, int row, int col) {
  return (col >> 6) * rows * 64 + row * 64 + ((((col >> 3) & 7) ^ (row & 7)) << 3) + (col & 7);
}
// Eight values as kP parts, `part` elements from part to part.
template <int kP>
__device__ __forceinline__ void put8(bf16_t* p, int part, const float (&x)[8]) {
  uint32_t u[4][kP];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<kP>(x[2 * i], x[2 * i + 1], u[i]);
#pragma unroll
  for (int j = 0; j < kP; ++j) *reinterpret_cast<uint4*>(p + j * part) = make_uint4(u[0][j], u[1][j], u[2][j], u[3][j]);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const bf16_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const bf16_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of m16n8k16 for one 16-deep block, from a tile of `rows` rows. With g = lane / 4,
// t = lane % 4 the accumulator holds C[g][2t, 2t+1] and C[g+8][2t, 2t+1].
//   a_mk: A[m][k] stored [m][k];  a_km: A stored [k][m]
//   b_nk: B (16 columns) stored [n][k];  b_kn: B stored [k][n]
template <int kP>
struct Frag {
  uint32_t p[kP][4];
};
template <int kP>
__device__ __forceinline__ void a_mk(Frag<kP>& f, const bf16_t* s, int rows, int part, int m0, int k0, int lane) {
  const bf16_t* p = s + at(rows, m0 + (lane & 15), k0 + (lane >> 4) * 8);
#pragma unroll
  for (int i = 0; i < kP; ++i) ldsm4(f.p[i], p + i * part);
}
template <int kP>
__device__ __forceinline__ void a_km(Frag<kP>& f, const bf16_t* s, int rows, int part, int m0, int k0, int lane) {
  const bf16_t* p = s + at(rows, k0 + (lane & 7) + (lane >> 4) * 8, m0 + ((lane >> 3) & 1) * 8);
#pragma unroll
  for (int i = 0; i < kP; ++i) ldsm4t(f.p[i], p + i * part);
}
template <int kP>
__device__ __forceinline__ void b_nk(Frag<kP>& f, const bf16_t* s, int rows, int part, int n0, int k0, int lane) {
  const bf16_t* p = s + at(rows, n0 + (lane & 7) + (lane >> 4) * 8, k0 + ((lane >> 3) & 1) * 8);
#pragma unroll
  for (int i = 0; i < kP; ++i) ldsm4(f.p[i], p + i * part);
}
template <int kP>
__device__ __forceinline__ void b_kn(Frag<kP>& f, const bf16_t* s, int rows, int part, int n0, int k0, int lane) {
  const bf16_t* p = s + at(rows, k0 + (lane & 15), n0 + (lane >> 4) * 8);
#pragma unroll
  for (int i = 0; i < kP; ++i) ldsm4t(f.p[i], p + i * part);
}
// Two n8 tiles += a b, the small terms first.
template <int kA, int kB>
__device__ __forceinline__ void mma_parts(float (&d0)[4], float (&d1)[4], const Frag<kA>& a, const Frag<kB>& b) {
#pragma unroll
  for (int sum = 2; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < kA; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (i + j == sum) {
          mma16(d0, a.p[i], b.p[j][0], b.p[j][1]);
          mma16(d1, a.p[i], b.p[j][2], b.p[j][3]);
        }
}
// The same added to the tiles in fp32: the tensor cores cut what they add to an accumulator (2^-23 of it, always
// towards 0), which over the tens of steps of these sums came to 1e-6.
template <int kA, int kB>
__device__ __forceinline__ void mma_added(float (&d0)[4], float (&d1)[4], const Frag<kA>& a, const Frag<kB>& b) {
  float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
  mma_parts(x, y, a, b);
#pragma unroll
  for (int e = 0; e < 4; ++e) d0[e] += x[e], d1[e] += y[e];
}
// Two accumulator tiles (columns k0 .. k0+7 and k0+8 .. k0+15 of 16 rows) as the A
// fragment of a product over those columns.
template <int kP>
__device__ __forceinline__ void to_a(Frag<kP>& f, const float (&x)[4], const float (&y)[4]) {
  uint32_t u[kP];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e < 2)
      split2<kP>(x[2 * e], x[2 * e + 1], u);
    else
      split2<kP>(y[2 * e - 4], y[2 * e - 3], u);
#pragma unroll
    for (int i = 0; i < kP; ++i) f.p[i][e] = u[i];
  }
}
template <int N>
__device__ __forceinline__ void zero(float (&x)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
}
// Rows 0 .. kRows-1 (zeros from `len` on) and columns 0 .. ceil(cols / 64) 64 - 1 (zeros from `cols`
// on) of a tile, times w[row] where w is given; src is row 0, `stride` elements from row to row.
template <int kP, int kRows, typename T>
__device__ __forceinline__ void fill_tile(bf16_t* dst, const T* src, long long stride, int len, int cols, const float* w,
                                          int tid, int threads) {
  constexpr int kBatch = 8;  // loads on their way together
  const int shift = cols > 64 ? 4 : 3, total = kRows << shift, part = total * 8;
  for (int i0 = tid; i0 < total; i0 += kBatch * threads) {
    float x[kBatch][8];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * threads, row = i >> shift, col = (i - (row << shift)) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[b][e] = 0.f;
      if (row < len && col < cols) load8(x[b], src + row * stride + col);  // (len <= kRows)
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * threads, row = i >> shift, col = (i - (row << shift)) * 8;
      if (i >= total) break;
      if (w) {
        const float f = w[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[b][e] *= f;
      }
      put8<kP>(dst + at(kRows, row, col), part, x[b]);
    }
  }
}

// ---------------------------------------------------------------- decays ---

// The running sums of a chunk's log decays as unrounded sums of two floats (their differences
// stand in exponents: after a reset, -1e6, a rounded sum would lose those of the tokens behind it). A log
// decay below -1e6 counts as that: both empty the state.
constexpr float kReset = -1e6f;
__device__ __forceinline__ float2 two_sum(float2 a, float2 b) {
  const float s = a.x + b.x, bb = s - a.x;
  const float e = (a.x - (s - bb)) + (b.x - bb) + a.y + b.y;
  const float h = s + e;
  return make_float2(h, e - (h - s));
}
__device__ __forceinline__ float minus(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }
// The difference as two floats, and e to it: an exponent of tens loses up to 2^-20 when it is rounded to one float, and e^x as much
// of itself. (The second float is at most half a unit of the first.)
__device__ __forceinline__ float2 minus_both(float2 a, float2 b) { return two_sum(a, make_float2(-b.x, -b.y)); }
__device__ __forceinline__ float exp_both(float2 x) { return expf(x.x) * (1.f + x.y); }
// The running sums of 32 kPer tokens by a warp, kPer a lane: of r, log decays.
template <int kPer>
__device__ __forceinline__ void running_sums(float2 (&G)[kPer], const float (&r)[kPer], int lane) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    G[i] = make_float2(r[i] < kReset ? kReset : r[i], 0.f);  // (a NaN stays)
    if (i) G[i] = two_sum(G[i - 1], G[i]);
  }
  float2 s = G[kPer - 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float2 y = make_float2(__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o));
    if (lane >= o) s = two_sum(s, y);
  }
  float2 e = make_float2(__shfl_up_sync(0xffffffffu, s.x, 1), __shfl_up_sync(0xffffffffu, s.y, 1));
  if (lane == 0) e = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPer; ++i) G[i] = two_sum(e, G[i]);
}
// A lane's log decays, `stride` floats from token to token; 0 from token `len` on.
template <int kPer>
__device__ __forceinline__ void load_decays(float (&r)[kPer], const float* g, long long stride, int len, int lane) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) r[i] = kPer * lane + i < len ? g[(kPer * lane + i) * stride] : 0.f;
}
template <int kPer>
__device__ __forceinline__ void running_sums(float2* G, const float* g, long long stride, int len, int lane) {
  float r[kPer];
  float2 x[kPer];
  load_decays(r, g, stride, len, lane);
  running_sums(x, r, lane);
#pragma unroll
  for (int i = 0; i < kPer; ++i) G[kPer * lane + i] = x[i];
}

// --------------------------------------------------- sequences and chunks ---

struct SeqRange {
  int b;           // batch row the sequence lies in
  int t0, t1;      // its tokens there
  long long slot;  // its first slot
};
// Packed starts are clamped into [0, T] and to non-negative lengths, so that
// no value in them can take an access out of a buffer.
__device__ __forceinline__ SeqRange seq_range(const Shape& a, int s, int tokens) {
  SeqRange r;
  if (a.starts) {
    const int x0 = min(max(a.starts[s], 0), a.T), x1 = min(max(a.starts[s + 1], 0), a.T);
    r.b = 0, r.t0 = x0, r.t1 = max(x0, x1), r.slot = x0 / tokens + s;
  } else {
    r.b = s, r.t0 = 0, r.t1 = a.T, r.slot = (long long)s * ((a.T + tokens - 1) / tokens);
  }
  return r;
}
struct ChunkAt {
  int b, t0, len;  // batch row, first token, tokens
  int seq, first;  // its sequence, and that one's first token
};
// The stretch of `tokens` tokens (a chunk, or a segment of chunks) that has the slot; false: none.
__device__ __forceinline__ bool chunk_at(const Shape& a, int slot, int tokens, ChunkAt& c) {
  int n;
  if (a.starts) {
    int lo = 0, hi = a.nseq - 1;  // the last sequence whose first slot is <= slot
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (min(max(a.starts[mid], 0), a.T) / tokens + mid <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
    c.seq = lo;
  } else {
    c.seq = slot / ((a.T + tokens - 1) / tokens);
  }
  const SeqRange r = seq_range(a, c.seq, tokens);
  n = slot - (int)r.slot;
  if (n < 0 || r.t0 + (long long)n * tokens >= r.t1) return false;
  c.b = r.b, c.first = r.t0, c.t0 = r.t0 + n * tokens, c.len = min(tokens, r.t1 - c.t0);
  return true;
}
// The slot of the chunk that begins at token t0 of a sequence.
__device__ __forceinline__ long long chunk_slot(const Shape& a, const ChunkAt& c, int t0) {
  const int n = (t0 - c.first) / a.C;
  return (a.starts ? (long long)c.first / a.C + c.seq : (long long)c.seq * ((a.T + a.C - 1) / a.C)) + n;
}

}  // namespace linattn
