// The fifth-generation tensor cores (tcgen05) as the gated delta rule's chains
// use them: products with 64 rows, the left operand (what a warp computed) and the
// accumulator in tensor memory, the right one an image in shared memory. (With the
// left operand in shared memory too, an mma of 64 x 64 x 16 took the 37 cycles in
// which 4 KB come out of it, and everybody else's accesses waited.)
//
// An image (gdr_common.cuh) is an operand as it lies: its rows of 128 bytes with
// permuted pieces are the 128-byte swizzle, read along the row (K-major: tc_rows)
// or across it (MN-major: tc_columns); the 32-byte rows of the triangular images'
// blocks are the 32-byte swizzle.
//
// With 64 rows an accumulator's row i lies in lane 32 (i / 16) + i % 16: warp w
// of four reads rows 16 w .., and by 16 x 256 bits it gets them as mma.sync's
// accumulator tiles, so that the code around the products is the same for both.
#pragma once

#include "gdr_common.cuh"
#include "wkv7_tmem.cuh"

namespace gdr {

using wkv7::tmem_fence_after_sync;
using wkv7::tmem_fence_before_sync;

// Descriptor of a right operand: start, leading and stride byte offsets, version 1,
// layout (2: 128-byte swizzle, 6: 32-byte). Made once a product; the parts and
// steps in it lie at offsets that are constants (addresses stay below 2^18, so
// adding to the low word is enough).
struct Right {
  uint32_t lo, hi;
  __device__ __forceinline__ Right(const void* image, uint32_t lbo, uint32_t sbo, uint32_t layout)
      : lo((smem_addr(image) >> 4) | (lbo >> 4) << 16), hi((sbo >> 4) | 1u << 14 | layout << 29) {}
  __device__ __forceinline__ uint64_t at(int bytes) const {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
    return d;
  }
};
constexpr int kPanel = kC * 128;  // bytes of a panel: 64 rows
// A triangular image spread out to whole columns: its block (i, j) is block 4 j + i.
constexpr int kSpreadPart = 16 * 256;

// fp16 operands, fp32 accumulator, 64 x n.
__host__ __device__ constexpr uint32_t product_of(int n, bool b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(64 >> 4) << 24);
}
// The left operand lies in tensor memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(what), "r"((uint32_t)add)
      : "memory");
}
// The barrier gets an arrival when this thread's products so far are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// The terms of a product in parts: the small ones first, lo lo left out.
template <int kA, int kB, typename F>
__device__ __forceinline__ void tc_terms(F term) {
  if constexpr (kA == 2) term(1, 0, true);
  if constexpr (kB == 2) term(0, 1, kA != 2);
  term(0, 0, kA != 2 && kB != 2);
}
// d = a b^T: b's rows (64) are the columns of d, its KP columns the sum's.
template <int kA, int kB, int KP>
__device__ __forceinline__ void tc_rows(uint32_t d, uint32_t a, const __half* b) {
  const Right r(b, 16, 1024, 2);
  tc_terms<kA, kB>([&](int pa, int pb, bool first) {
#pragma unroll
    for (int ks = 0; ks < KP / 16; ++ks)
      tc_mma(d, a + 8 * (pa * (KP / 16) + ks), r.at(pb * kC * KP * 2 + (ks >> 2) * kPanel + 32 * (ks & 3)), product_of(64, false),
             !first || ks > 0);
  });
}
// d = a b: b's KP columns are those of d, its rows (64) the sum's.
template <int kA, int kB, int KP>
__device__ __forceinline__ void tc_columns(uint32_t d, uint32_t a, const __half* b) {
  const Right r(b, kPanel, 1024, 2);
  tc_terms<kA, kB>([&](int pa, int pb, bool first) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc_mma(d, a + 8 * (4 * pa + ks), r.at(pb * kC * KP * 2 + 2048 * ks), product_of(KP, true), !first || ks > 0);
  });
}
// d = a X^T with X a triangular image: columns of X 16 j .. meet the rows from 16 j on.
template <int kA, int kB>
__device__ __forceinline__ void tc_tri_rows(uint32_t d, uint32_t a, const __half* tri) {
  const Right r(tri, 16, 256, 6);
  tc_terms<kA, kB>([&](int pa, int pb, bool first) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tc_mma(d + 16 * j, a + 8 * (4 * pa + j), r.at(2 * (pb * kTriPart + tri_block(j, j))), product_of(64 - 16 * j, false),
             !first || j > 0);
  });
}
// d = a X with X spread out: rows of X 16 i .. meet the columns up to them.
template <int kA, int kB>
__device__ __forceinline__ void tc_tri_columns(uint32_t d, uint32_t a, const __half* tri) {
  const Right r(tri, 2048, 256, 6);
  tc_terms<kA, kB>([&](int pa, int pb, bool first) {
#pragma unroll
    for (int i = 3; i >= 0; --i)
      tc_mma(d, a + 8 * (4 * pa + i), r.at(2 * pb * kSpreadPart + 512 * i), product_of(16 * i + 16, true), !first || i < 3);
  });
}

// Columns of a warp's 16 rows as accumulator tiles, and the wait for the loads so
// far (x depends on it, so that no use moves before).
__device__ __forceinline__ void tc_load(float (&x)[8][4], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
               "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=f"(x[0][0]), "=f"(x[0][1]), "=f"(x[0][2]), "=f"(x[0][3]), "=f"(x[1][0]), "=f"(x[1][1]),
                 "=f"(x[1][2]), "=f"(x[1][3]), "=f"(x[2][0]), "=f"(x[2][1]), "=f"(x[2][2]), "=f"(x[2][3]),
                 "=f"(x[3][0]), "=f"(x[3][1]), "=f"(x[3][2]), "=f"(x[3][3]), "=f"(x[4][0]), "=f"(x[4][1]),
                 "=f"(x[4][2]), "=f"(x[4][3]), "=f"(x[5][0]), "=f"(x[5][1]), "=f"(x[5][2]), "=f"(x[5][3]),
                 "=f"(x[6][0]), "=f"(x[6][1]), "=f"(x[6][2]), "=f"(x[6][3]), "=f"(x[7][0]), "=f"(x[7][1]),
                 "=f"(x[7][2]), "=f"(x[7][3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc_loaded(float (&x)[8][4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0][0]), "+f"(x[0][1]), "+f"(x[0][2]), "+f"(x[0][3]), "+f"(x[1][0]), "+f"(x[1][1]),
                 "+f"(x[1][2]), "+f"(x[1][3]), "+f"(x[2][0]), "+f"(x[2][1]), "+f"(x[2][2]), "+f"(x[2][3]),
                 "+f"(x[3][0]), "+f"(x[3][1]), "+f"(x[3][2]), "+f"(x[3][3]), "+f"(x[4][0]), "+f"(x[4][1]),
                 "+f"(x[4][2]), "+f"(x[4][3]), "+f"(x[5][0]), "+f"(x[5][1]), "+f"(x[5][2]), "+f"(x[5][3]),
                 "+f"(x[6][0]), "+f"(x[6][1]), "+f"(x[6][2]), "+f"(x[6][3]), "+f"(x[7][0]), "+f"(x[7][1]),
                 "+f"(x[7][2]), "+f"(x[7][3])
               :
               : "memory");
}
__device__ __forceinline__ void tc_load(float (&x)[4][4], uint32_t taddr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
               "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=f"(x[0][0]), "=f"(x[0][1]), "=f"(x[0][2]), "=f"(x[0][3]), "=f"(x[1][0]), "=f"(x[1][1]),
                 "=f"(x[1][2]), "=f"(x[1][3]), "=f"(x[2][0]), "=f"(x[2][1]), "=f"(x[2][2]), "=f"(x[2][3]),
                 "=f"(x[3][0]), "=f"(x[3][1]), "=f"(x[3][2]), "=f"(x[3][3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tc_loaded(float (&x)[4][4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0][0]), "+f"(x[0][1]), "+f"(x[0][2]), "+f"(x[0][3]), "+f"(x[1][0]), "+f"(x[1][1]),
                 "+f"(x[1][2]), "+f"(x[1][3]), "+f"(x[2][0]), "+f"(x[2][1]), "+f"(x[2][2]), "+f"(x[2][3]),
                 "+f"(x[3][0]), "+f"(x[3][1]), "+f"(x[3][2]), "+f"(x[3][3])
               :
               : "memory");
}

// True in one lane of a whole warp. (Under a branch on the thread's number the
// compiler cannot tell that descriptors are uniform, and an mma took 60 cycles to issue.)
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Two floats at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 pair_of(const float (&x)[4], int h) { return make_float2(x[2 * h], x[2 * h + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[4], int h, float2 y) { x[2 * h] = y.x, x[2 * h + 1] = y.y; }

// 16-deep blocks of a left operand (one part), as A fragments, into tensor memory;
// complete after tc_stored.
__device__ __forceinline__ void tc_store(uint32_t taddr, const uint32_t (&f)[4][4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
               "r"(f[0][0]), "r"(f[0][1]), "r"(f[0][2]), "r"(f[0][3]), "r"(f[1][0]), "r"(f[1][1]), "r"(f[1][2]),
               "r"(f[1][3]), "r"(f[2][0]), "r"(f[2][1]), "r"(f[2][2]), "r"(f[2][3]), "r"(f[3][0]), "r"(f[3][1]),
               "r"(f[3][2]), "r"(f[3][3])
               : "memory");
}
__device__ __forceinline__ void tc_store(uint32_t taddr, const uint32_t (&f)[2][4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(f[0][0]), "r"(f[0][1]), "r"(f[0][2]), "r"(f[0][3]), "r"(f[1][0]), "r"(f[1][1]), "r"(f[1][2]),
               "r"(f[1][3])
               : "memory");
}
__device__ __forceinline__ void tc_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Accumulator tiles times s as N such blocks, hi and lo `part` columns behind.
template <int kP, int N>
struct Operand {
  uint32_t h[N][4], l[kP == 2 ? N : 1][4];
  __device__ __forceinline__ void split(const float (&x)[2 * N][4], float s) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = mul2(pair_of(x[2 * j + (e >> 1)], e & 1), make_float2(s, s));
        h[j][e] = pack_f16(y.x, y.y);
        if constexpr (kP == 2) {
          const float2 z = fma2(unpack_f16(h[j][e]), make_float2(-1.f, -1.f), y);
          l[j][e] = pack_f16(z.x, z.y);
        }
      }
  }
  __device__ __forceinline__ void store(uint32_t taddr, int part) const {
    tc_store(taddr, h);
    if constexpr (kP == 2) tc_store(taddr + part, l);
  }
  // rows of 16 of an image, from column k0 on
  __device__ __forceinline__ void put(__half* image, int part, int k0, int lane) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      __half* p = image + img(16, lane & 15, k0 + 16 * j + (lane >> 4) * 8);
      stsm4(p, h[j]);
      if constexpr (kP == 2) stsm4(p + part, l[j]);
    }
  }
};

constexpr int kWarps = 4, kChains = 2 * kWarps;  // of 16 rows each: two chain warps, half of the columns each

// Registers of a thread of the calling four warps, of those the block was launched with.
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// The two warps of 16 rows, each with half of the columns, meet at barrier `id`;
// the larger of their values.
__device__ __forceinline__ void both_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float both_max(float m, float* slot, int half, int id, int lane) {
  if (lane == 0) slot[half] = m;
  both_sync(id);
  return fmaxf(m, slot[half ^ 1]);
}

// A wait that a warp gives up on once: from then on it goes through its steps
// without waiting (all accesses are in bounds whatever the data), so that the
// block's barriers and its tensor memory are left in order.
struct Patience {
  unsigned* status;
  bool ok = true;
  __device__ __forceinline__ void operator()(const Asked& b) {
    if (ok) ok = b.wait(status);
  }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_bounded(status, bar, parity & 1);
  }
};

enum { kQ = 2, kT, kP };  // barriers of full places: two of k, q, t, p
// The filling thread at its end: the last of n copies into each place (k by turns)
// has landed, also where the warps that would wait for it gave up before. A
// millisecond at most each.
__device__ __forceinline__ void drain_last(uint64_t* full, int n) {
#pragma unroll 1
  for (int b = 0; b < 5; ++b) {
    const int copies = b < 2 ? (n + 1 - b) / 2 : n;
    mbar_wait_bounded(nullptr, full + b, (copies - 1) & 1, 1000000);
  }
}

}  // namespace gdr
