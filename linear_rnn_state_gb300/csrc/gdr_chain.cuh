// What the forward and the backward chain of the gated delta rule share, beside
// the tensor cores' part (gdr_tc.cuh): barriers, the rows of v, o, do and dv, the
// state.
//
// Two warps have 16 rows of the state (value columns), half of the keys and half of
// the tokens each. With the rows as the m of every product (S k^T, r T^T, u P^T,
// w^T k are 16 x 64 or 16 x keys) the result of one is, scaled and packed to fp16
// pairs, the left operand of the next, the two exchange nothing but a maximum, and
// every scale is the exact maximum of the 16 rows. Between two products all is in
// registers, laid out as mma.sync's accumulator tiles.
//
// The chain's warps make only what the next state waits for; helper warps beside
// them make the rest, o in the forward and the products with do in the backward,
// and move the rows and images to and from memory. They meet at a barrier for
// each thing full and one for it free again.
//
// History of a step at 64 keys, bfloat16, forward: tiles of 16 tokens by 16
// columns a warp with intermediates in shared memory, 411 us for 64 steps (42 % of
// it shared-memory reads, 25 % three barriers); 16 rows a warp by mma.sync, in
// registers, 254; helper warps, 194; barriers asked early, 178; tcgen05 with left
// operands in shared memory, 183 to 210; in tensor memory, 189; products issued by
// warps of their own, 138; two warps for the 16 rows, 127.
#pragma once

#include "gdr_common.cuh"

namespace gdr {

// A barrier asked early (a try_wait takes some 85 cycles to answer) and waited
// for only where the answer was no.
struct Asked {
  uint64_t* bar;
  uint32_t parity;
  bool there;
  __device__ __forceinline__ Asked(uint64_t* b, uint32_t p) : bar(b), parity(p & 1), there(wkv7::mbar_try_wait(b, p & 1)) {}
  __device__ __forceinline__ bool wait(unsigned* status) const { return there || mbar_wait_bounded(status, bar, parity); }
};
// What a warp did before is done for whoever waits on the barrier: its last read
// of a place, or its writes of one.
__device__ __forceinline__ void signal(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Accumulator tiles handed from one warp to another as they are.
template <int N>
__device__ __forceinline__ void tiles_get(float (&x)[N][4], const float4* buf, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float4 v = buf[n * 32 + lane];
    x[n][0] = v.x, x[n][1] = v.y, x[n][2] = v.z, x[n][3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void tiles_put(float4* buf, const float (&x)[N][4], float s, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) buf[n * 32 + lane] = make_float4(x[n][0] * s, x[n][1] * s, x[n][2] * s, x[n][3] * s);
}
// ------------------------------------------- 64 tokens x 16 value columns ---
//
// A warp's part of v or do, by asynchronous copies into its own buffer, and its
// part of o or dv out of it. In registers they are the transpose, x[nt] the
// accumulator tile of rows (columns of v) by tokens 8 nt .. 8 nt + 7: for
// bfloat16 ldmatrix and stmatrix transpose on the way, fp32 goes by words, its
// rows 80 bytes apart so that the four tokens of an access differ by 8 banks.

template <typename T>
constexpr int kRowsBytes = sizeof(T) == 2 ? kC * 32 : kC * 80;

__device__ __forceinline__ void copy_async16(void* dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // 0: sixteen bytes of zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// rows points at token 0 of the chunk; len of its tokens and cols of the 16 columns
// exist. All for tokens 8 n0 .. 8 (n0 + N) - 1 (n0 even).
template <int N, typename T>
__device__ __forceinline__ void rows_in(unsigned char* buf, const T* rows, long long stride_t, int len, int cols, int n0, int lane) {
  constexpr int kPer = 16 / sizeof(T), kPieces = 16 / kPer;  // values and pieces of 16 bytes
#pragma unroll
  for (int i = 0; i < N * 8 * kPieces / 32; ++i) {
    const int id = i * 32 + lane, row = 8 * n0 + id / kPieces, c = id % kPieces;
    const bool there = row < len && c * kPer < cols;
    unsigned char* dst = sizeof(T) == 2 ? buf + 2 * tri_at(row, c * 8) : buf + row * 80 + c * 16;
    copy_async16(dst, there ? rows + row * stride_t + c * kPer : rows, there);
  }
}
template <int N>
__device__ __forceinline__ void rows_get(float (&x)[N][4], const unsigned char* buf, int n0, int lane, const __nv_bfloat16*) {
#pragma unroll
  for (int q = 0; q < N / 2; ++q) {
    uint32_t r[4];
    ldsm4t(r, reinterpret_cast<const __half*>(buf) + tri_at(8 * n0 + 16 * q + (lane & 15), (lane >> 4) * 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* y = &x[2 * q + (i & 1)][i & 2];
      y[0] = __uint_as_float(r[i] << 16), y[1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void rows_get(float (&x)[N][4], const unsigned char* buf, int n0, int lane, const float*) {
  const float* s = reinterpret_cast<const float*>(buf);
#pragma unroll
  for (int nt = 0; nt < N; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[nt][e] = s[(8 * (n0 + nt) + 2 * (lane & 3) + (e & 1)) * 20 + (lane >> 2) + 8 * (e >> 1)];
}
template <int N>
__device__ __forceinline__ void rows_put(const float (&x)[N][4], unsigned char* buf, int n0, int lane, const __nv_bfloat16*) {
#pragma unroll
  for (int q = 0; q < N / 2; ++q) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* y = &x[2 * q + (i & 1)][i & 2];
      const __nv_bfloat162 v = __floats2bfloat162_rn(y[0], y[1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    stsm4t(reinterpret_cast<__half*>(buf) + tri_at(8 * n0 + 16 * q + (lane & 15), (lane >> 4) * 8), r);
  }
}
template <int N>
__device__ __forceinline__ void rows_put(const float (&x)[N][4], unsigned char* buf, int n0, int lane, const float*) {
  float* s = reinterpret_cast<float*>(buf);
#pragma unroll
  for (int nt = 0; nt < N; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[(8 * (n0 + nt) + 2 * (lane & 3) + (e & 1)) * 20 + (lane >> 2) + 8 * (e >> 1)] = x[nt][e];
}
// x to memory by way of buf.
template <int N, typename T>
__device__ __forceinline__ void rows_out(const float (&x)[N][4], unsigned char* buf, T* rows, long long stride_t, int len, int cols,
                                         int n0, int lane) {
  constexpr int kPer = 16 / sizeof(T), kPieces = 16 / kPer;
  rows_put(x, buf, n0, lane, rows);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < N * 8 * kPieces / 32; ++i) {
    const int id = i * 32 + lane, row = 8 * n0 + id / kPieces, c = id % kPieces;
    const unsigned char* src = sizeof(T) == 2 ? buf + 2 * tri_at(row, c * 8) : buf + row * 80 + c * 16;
    if (row < len && c * kPer < cols) *reinterpret_cast<uint4*>(rows + row * stride_t + c * kPer) = *reinterpret_cast<const uint4*>(src);
  }
  __syncwarp();
}
// Asks for rows into L2 (N a multiple of 4).
template <int N, typename T>
__device__ __forceinline__ void rows_ask(const T* rows, long long stride_t, int len, int n0, int lane) {
#pragma unroll
  for (int i = 0; i < N * 8; i += 32) {
    const int row = 8 * n0 + i + lane;
    if (row < len) prefetch_l2(rows + row * stride_t);
  }
}

// The state of a warp: rows g4 (+ 8), keys key0 + 8 nt + 2 t4 (+ 1).
template <int N>
__device__ __forceinline__ void load_state(float (&S)[N][4], const float* src, int rows, int key0, int K, int lane) {
#pragma unroll
  for (int nt = 0; nt < N; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (lane >> 2) + 8 * h, key = key0 + 8 * nt + 2 * (lane & 3);
      float2 x = make_float2(0.f, 0.f);
      if (src && row < rows && key < K) x = *reinterpret_cast<const float2*>(src + (size_t)row * K + key);
      S[nt][2 * h] = x.x, S[nt][2 * h + 1] = x.y;
    }
}
template <int N>
__device__ __forceinline__ void store_state(const float (&S)[N][4], float* dst, int rows, int key0, int K, int lane) {
#pragma unroll
  for (int nt = 0; nt < N; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = (lane >> 2) + 8 * h, key = key0 + 8 * nt + 2 * (lane & 3);
      if (row < rows && key < K) *reinterpret_cast<float2*>(dst + (size_t)row * K + key) = make_float2(S[nt][2 * h], S[nt][2 * h + 1]);
    }
}

__device__ __forceinline__ void copy_arrive(uint64_t* bar) {  // once this lane's copies so far have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace gdr
