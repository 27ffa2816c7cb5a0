// The fifth-generation tensor cores (tcgen05) as linear attention's kernels use them: chunks of 128
// tokens, which are the 128 rows (lanes of tensor memory) of a product's accumulator.
//
// A tile (linattn_common.cuh) is an operand as it lies: rows of 128 bytes with permuted pieces are
// the 128-byte swizzle, read along the row (K-major) or across it (MN-major), so that one copy of q,
// k, v and do in shared memory serves every product they stand in.
#pragma once

#include "linattn_common.cuh"
#include "linattn_maps.h"
#include "wkv7_tmem.cuh"

namespace linattn {

using wkv7::fence_proxy_async_smem;
using wkv7::mbar_init;
using wkv7::mbar_wait_bounded;
using wkv7::tmem_fence_after_sync;
using wkv7::tmem_fence_before_sync;

constexpr int kCT = kCBf16;
constexpr int kRowPanel = kCT * 128;  // bytes of a panel of 128 rows

// Descriptor of an operand in shared memory: start, leading and stride byte offsets, version 1, 128-byte
// swizzle. `lead`: MN-major, from one 64-wide panel to the next.
__device__ __forceinline__ uint64_t desc(const void* tile, uint32_t lead = 16) {
  const uint32_t lo = (smem_addr(tile) >> 4) | (lead >> 4) << 16, hi = (1024u >> 4) | 1u << 14 | 2u << 29;
  return (uint64_t)hi << 32 | lo;
}
// bfloat16 operands, fp32 accumulator, m x n.
__host__ __device__ constexpr uint32_t product_of(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// d += a b, or = where !add; a in shared memory, or (tc_mma_t) in tensor memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
               "l"(a), "l"(b), "r"(what), "r"((uint32_t)add)
               : "memory");
}
__device__ __forceinline__ void tc_mma_t(uint32_t d, uint32_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(what), "r"((uint32_t)add)
               : "memory");
}
// The barrier gets an arrival when this thread's products so far are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// True in one lane of a whole warp (an election, so that the compiler sees that descriptors are uniform).
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Products. `step` and `panel` are 16-byte units from one 16-deep block to the next.
// K-major operand of `rows` rows: block ks of its columns.
template <int kRows>
__device__ __forceinline__ constexpr uint32_t along(int ks) {
  return ((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4;
}
// MN-major: block ks of its rows.
__device__ __forceinline__ constexpr uint32_t across(int ks) { return ks * 2048 >> 4; }

// 32 columns of a thread's lane, complete.
__device__ __forceinline__ void tc_load32(float (&v)[32], uint32_t taddr) { wkv7::tmem_ld<32>(taddr, v); }
__device__ __forceinline__ void tc_loaded32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                 "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_load16(float (&v)[16], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
                 "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc_loaded16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
template <int N>
__device__ __forceinline__ void tc_read(float (&v)[N], uint32_t taddr) {
  if constexpr (N == 16) {
    tc_load16(v, taddr);
    tc_loaded16(v);
  } else {
    tc_load32(v, taddr);
    tc_loaded32(v);
  }
}
// 16 or 32 columns of 16 rows (those of a 64-row accumulator) as mma.sync's accumulator tiles.
__device__ __forceinline__ void tc_load_tiles(float (&x)[2][4], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0][0]), "=f"(x[0][1]), "=f"(x[0][2]), "=f"(x[0][3]), "=f"(x[1][0]), "=f"(x[1][1]), "=f"(x[1][2]), "=f"(x[1][3])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0][0]), "+f"(x[0][1]), "+f"(x[0][2]), "+f"(x[0][3]), "+f"(x[1][0]), "+f"(x[1][1]), "+f"(x[1][2]), "+f"(x[1][3])
               :
               : "memory");
}
__device__ __forceinline__ void tc_load_tiles(float (&x)[4][4], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=f"(x[0][0]), "=f"(x[0][1]), "=f"(x[0][2]), "=f"(x[0][3]), "=f"(x[1][0]), "=f"(x[1][1]), "=f"(x[1][2]), "=f"(x[1][3]),
                 "=f"(x[2][0]), "=f"(x[2][1]), "=f"(x[2][2]), "=f"(x[2][3]), "=f"(x[3][0]), "=f"(x[3][1]), "=f"(x[3][2]), "=f"(x[3][3])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0][0]), "+f"(x[0][1]), "+f"(x[0][2]), "+f"(x[0][3]), "+f"(x[1][0]), "+f"(x[1][1]), "+f"(x[1][2]), "+f"(x[1][3]),
                 "+f"(x[2][0]), "+f"(x[2][1]), "+f"(x[2][2]), "+f"(x[2][3]), "+f"(x[3][0]), "+f"(x[3][1]), "+f"(x[3][2]), "+f"(x[3][3])
               :
               : "memory");
}
__device__ __forceinline__ void stsm4(bf16_t* p, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(smem_addr(p)), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// Registers of a thread of the calling four warps, of those the block was launched with.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Barrier `id` of some of a block's warps: `n` threads in all meet there, or announce themselves and go on.
__device__ __forceinline__ void meet(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void announce(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// A wait that a warp gives up on once: from then on it goes through its steps without waiting (all accesses
// are in bounds whatever the data) and starts no copy, so that barriers and tensor memory are left in order.
struct Patience {
  unsigned* status;
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_bounded(status, bar, parity & 1);
  }
};

// Where a wait was given up, before the block ends: no product and (by the thread that started them) no copy is left in
// flight, a millisecond or two at most for each. (Which of a barrier's phases the copy in flight completes is not known then.)
constexpr uint64_t kLastWaitNs = 1000000;
__device__ __forceinline__ void finish_products(uint64_t* bar) {  // by the issuing warp; bar's first use
  if (elected()) tc_commit(bar);
  __syncwarp();
  mbar_wait_bounded(nullptr, bar, 0, kLastWaitNs);
}
__device__ __forceinline__ void finish_copies(uint64_t* bar) {
  for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait_bounded(nullptr, bar, parity, kLastWaitNs);
}
#ifdef WKV7_DEBUG
__device__ __forceinline__ bool skipped(const Args& a, int what, int n) { return a.skip_what == what && a.skip_n == n; }
#define LINATTN_SKIPPED(what, n) skipped(a, what, n)
#else
#define LINATTN_SKIPPED(what, n) false
#endif

// ---------------------------------------------------------------- copies ---

// kCols columns of a tile from token t on; the bytes that will arrive.
template <int kCols>
__device__ __forceinline__ void load_tile(bf16_t* dst, const CUtensorMap* map, uint64_t* bar, int col, int head, int t, int b) {
#pragma unroll
  for (int c = 0; c < kCols; c += 64) wkv7::tma_load_4d(dst + c * kCT, map, bar, col + c, head, t, b);
}
// The rows of a packed chunk from `len` on, which belong to another sequence (whose values may be anything).
template <int kCols>
__device__ __forceinline__ void clear_rows(bf16_t* tile, int len, int tid, int threads) {
  for (int i = tid; i < (kCT - len) * (kCols / 8); i += threads)
    *reinterpret_cast<uint4*>(tile + at(kCT, len + i / (kCols / 8), i % (kCols / 8) * 8)) = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)), "l"(src),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------------- decays ---

// A chunk's factors, by one warp:
//   head: scale e^G and tail: e^{Gc - G}. Of the state's part of a row, and of a token in the next state (forward),
//     or the other way round (backward)
//   to, from: e^{G - m} and e^{m - G} with m the middle of the range of G in a token's block of 32. Where that range is
//     at most kNear, products of them are the decays of the diagonal's blocks, and with e^{G_i - m} those of the others
//     (at most 1 times e^30 where no log decay is above 0). Exponentials of every element instead cost 30 us of 86 in a
//     chain at 4 x 4096 x 32 x 64, and 40 of 176 in the gradients
constexpr float kNear = 60.f;
struct alignas(16) Decays {
  float2 G[kCT];
  float head[kCT], tail[kCT], to[kCT], from[kCT];
  float middle[4];  // m
  float whole;      // e^{Gc}
  int up;           // a log decay is above 0 (or NaN)
  int near;         // bit b: block b's range is at most kNear
};
// kFull: for fp32 results, exponents in two floats (those of 32 tokens span tens: rounded to one, each factor is off by up to 1e-6; 2 % of
// the time in fp32, 4 % of a bfloat16 chain's, whose results do not show it).
template <bool kFull>
__device__ __forceinline__ float exp_of(float2 x) {
  return kFull ? exp_both(x) : expf(x.x + x.y);
}
template <bool kFull>
__device__ __forceinline__ float2 apart(float2 a, float2 b) {
  return kFull ? minus_both(a, b) : make_float2(minus(a, b), 0.f);
}
template <bool kFull>
__device__ __forceinline__ void make_decays(Decays& d, const float (&r)[4], float scale, int lane) {
  float2 G[4];
  running_sums(G, r, lane);
  const float2 last = make_float2(__shfl_sync(0xffffffffu, G[3].x, 31), __shfl_sync(0xffffffffu, G[3].y, 31));
  float hi = fmaxf(fmaxf(G[0].x, G[1].x), fmaxf(G[2].x, G[3].x)), lo = fminf(fminf(G[0].x, G[1].x), fminf(G[2].x, G[3].x));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o)), lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  const float m = 0.5f * (hi + lo);
  const bool sound = G[0].x == G[0].x && G[1].x == G[1].x && G[2].x == G[2].x && G[3].x == G[3].x;
  const unsigned near = __ballot_sync(0xffffffffu, hi - lo <= kNear && sound);
  const bool up = __any_sync(0xffffffffu, !(r[0] <= 0.f && r[1] <= 0.f && r[2] <= 0.f && r[3] <= 0.f));
  float4 head, tail, to, from;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = apart<kFull>(G[i], make_float2(m, 0.f));
    (&head.x)[i] = scale * exp_of<kFull>(G[i]), (&tail.x)[i] = exp_of<kFull>(apart<kFull>(last, G[i]));
    (&to.x)[i] = exp_of<kFull>(x), (&from.x)[i] = exp_of<kFull>(make_float2(-x.x, -x.y));
  }
  reinterpret_cast<float4*>(d.G)[2 * lane] = make_float4(G[0].x, G[0].y, G[1].x, G[1].y);
  reinterpret_cast<float4*>(d.G)[2 * lane + 1] = make_float4(G[2].x, G[2].y, G[3].x, G[3].y);
  reinterpret_cast<float4*>(d.head)[lane] = head, reinterpret_cast<float4*>(d.tail)[lane] = tail;
  reinterpret_cast<float4*>(d.to)[lane] = to, reinterpret_cast<float4*>(d.from)[lane] = from;
  if ((lane & 7) == 0) d.middle[lane >> 3] = m;
  if (lane == 0) {
    d.whole = exp_of<kFull>(last), d.up = up;
    d.near = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) d.near |= ((near >> 8 * b & 255u) == 255u) << b;
  }
}

// 32 columns (block `blk`) of a row's products times scale e^{G_i - G_j}, 0 outside the mask. kFull: for fp32 results (the fast
// exponential is off by 1.2 |x| + 2 units in the last place).
template <bool kUpper, bool kFull>
__device__ __forceinline__ void decayed(float (&x)[32], const Decays& d, int row, int blk, float scale) {
  const bool diagonal = blk == row >> 5;
  const int at = row - 32 * blk;  // the diagonal's column
  if (!(d.near >> blk & 1) || (!diagonal && d.up)) {
    const float2 Gr = d.G[row];
    const float4* G = reinterpret_cast<const float4*>(d.G + 32 * blk);  // two tokens
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float4 g = G[j / 2];
      const float d0 = minus(Gr, make_float2(g.x, g.y)), d1 = minus(Gr, make_float2(g.z, g.w));
      // (selects, no branches: a masked place takes the exponent 0)
      const bool k0 = kUpper ? j >= at : j <= at, k1 = kUpper ? j + 1 >= at : j + 1 <= at;
      const float x0 = k0 ? (kUpper ? -d0 : d0) : 0.f, x1 = k1 ? (kUpper ? -d1 : d1) : 0.f;
      const float e0 = scale * (kFull ? expf(x0) : __expf(x0)), e1 = scale * (kFull ? expf(x1) : __expf(x1));
      x[j] = k0 ? x[j] * e0 : 0.f, x[j + 1] = k1 ? x[j + 1] * e1 : 0.f;
    }
    return;
  }
  const float2 y = apart<kFull>(d.G[row], make_float2(d.middle[blk], 0.f));
  const float r = scale * (diagonal ? (kUpper ? d.from : d.to)[row]
                           : kFull  ? exp_both(kUpper ? make_float2(-y.x, -y.y) : y)
                                    : __expf(kUpper ? -y.x : y.x));
  const float4* c = reinterpret_cast<const float4*>((kUpper ? d.to : d.from) + 32 * blk);
  const float2 rr = make_float2(r, r);
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 f = c[j / 4];
    const float2 a = times2(make_float2(x[j], x[j + 1]), times2(make_float2(f.x, f.y), rr));
    const float2 b = times2(make_float2(x[j + 2], x[j + 3]), times2(make_float2(f.z, f.w), rr));
    x[j] = a.x, x[j + 1] = a.y, x[j + 2] = b.x, x[j + 3] = b.y;
  }
  if (diagonal) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (kUpper ? j < at : j > at) x[j] = 0.f;
  }
}
// 32 columns of a left operand in kP parts into tensor memory, 16 columns a part (eight at a time, for fewer
// registers), or zeros.
__device__ __forceinline__ void tc_store8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
template <int kP>
__device__ __forceinline__ void store_parts(uint32_t taddr, const float (&x)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[kP][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t p[kP];
      split2<kP>(x[16 * h + 2 * j], x[16 * h + 2 * j + 1], p);
#pragma unroll
      for (int i = 0; i < kP; ++i) v[i][j] = p[i];
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) tc_store8(taddr + 16 * i + 8 * h, v[i]);
  }
}
template <int kP>
__device__ __forceinline__ void store_zeros(uint32_t taddr) {
  const uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 2 * kP; ++i) tc_store8(taddr + 8 * i, v);
}
// The same in three parts of which two take the 32 columns' own place, where a product left them, and the third is handed
// back: 16 columns, for tc_store16.
__device__ __forceinline__ void store_two(uint32_t taddr, const float (&x)[32], uint32_t (&third)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t p[3];
      split2<3>(x[16 * h + 2 * j], x[16 * h + 2 * j + 1], p);
      v[0][j] = p[0], v[1][j] = p[1], third[8 * h + j] = p[2];
    }
    tc_store8(taddr + 8 * h, v[0]), tc_store8(taddr + 16 + 8 * h, v[1]);
  }
}
__device__ __forceinline__ void tc_store16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
               "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}
// Where part `part` of the columns 16 ks .. of that operand lies; `third`: of the block of 32 columns, from the first part's place on.
__device__ __forceinline__ uint32_t two_and_third(int ks, int part, int third) {
  return (part < 2 ? (ks >> 1) * 32 + part * 16 : third) + (ks & 1) * 8;
}
// Where part `part` of the columns 16 ks .. of that operand lies.
template <int kP>
__device__ __forceinline__ constexpr uint32_t part_at(int ks, int part) {
  return (ks >> 1) * 16 * kP + part * 16 + (ks & 1) * 8;
}
// The products of the parts of operands with kA and kB of them: f(part of a, part of b, whether it is the first),
// the small ones first. A loop: most kernels run it a few times only, and code that runs cold costs more than the loop.
struct Terms {
  int count = 0;
  uint32_t a = 0, b = 0;  // two bits each
  __host__ __device__ constexpr Terms(int parts_a, int parts_b) {
    for (int sum = parts_a + parts_b - 2 < 2 ? parts_a + parts_b - 2 : 2; sum >= 0; --sum)
      for (int i = 0; i < parts_a; ++i)
        if (sum - i >= 0 && sum - i < parts_b) a |= (uint32_t)i << 2 * count, b |= (uint32_t)(sum - i) << 2 * count, ++count;
  }
};
template <int kA, int kB, typename F>
__device__ __forceinline__ void terms(F f) {
  constexpr Terms t(kA, kB);
#pragma unroll 1
  for (int n = 0; n < t.count; ++n) f((int)(t.a >> 2 * n & 3u), (int)(t.b >> 2 * n & 3u), n == 0);
}

}  // namespace linattn
