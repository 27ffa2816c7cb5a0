// Norms around a block, forward and backward: each row is read once, kept in
// registers as fp32, reduced and written.
//
//   add:    h = residual + scale x,  r = 1 / sqrt(mean(h^2) + eps),  n = h r w
//   gated:  r = 1 / sqrt(mean(o^2) + eps),  y = o r w z sigmoid(z)
// Backward, with u = h r (or o r) and t = dn w (or dy z sigmoid(z) w), the
// gradients of the upstream side:
//   dh = (dh) + r (t - u mean(t u)),   dw = sum over rows of dn u (dy z sig u)
//   add:    dresidual = dh, dx = scale dh, dscale = sum over rows of dh x
//   gated:  dz = dy u w sig (1 + z (1 - sig))
// h is formed again from x and residual, so n and its gradient see it before
// its rounding to the residual's type.
//
// A row belongs to a group of kGroup threads with kVec pieces of eight values
// each; a block of 256 threads holds 256 / kGroup rows. All are bound by memory:
// the pieces are 16-byte loads where rows allow them, and 2048 threads an SM keep
// some 64 KB in flight. The sums over rows: a block walks rows a grid apart, keeps its columns' sums in
// registers and writes them as one partial row; a last kernel adds the
// partial rows in order (no atomics, the same bits every time).
//
// Measured: add, 16384 x 2048, x bfloat16 and residual fp32, 60 us forward (6.7
// TB/s, a copy's rate) and 107 backward (5.6 TB/s, the two sums kept beside the
// rows); gated, 16384 x 32 rows of 64, bfloat16, 40 us forward (5.0 TB/s) and 58
// backward (5.8 TB/s): a row of 64 leaves a thread eight values between its loads
// and its store, two rows a thread gave 38 us and took the add norm to 62. The
// sums' kernel adds 5 us. One row: 2.1 us on the device, the rest is the call.
#include <cuda_bf16.h>

#include "blocknorm_launch.h"
#include "gdr_launch.h"

namespace blocknorm {
namespace {

// Threads of a block whose rows have groups of kGroup.
template <int kGroup>
constexpr int kThreads = kGroup > 256 ? kGroup : 256;
constexpr int kSumThreads = 256;

__device__ __forceinline__ void unpack(float (&x)[8], uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// Eight values of a row of D from column c on, kStep apart; places past the row
// are 0. kStep 1: D is a multiple of eight and the rows are 16-byte aligned.
// Elsewhere they are a group of threads apart, so that the threads of a group
// access neighbours (2047 columns, bfloat16 and fp32 residual: 117 -> 42 us forward
// of 16 M values, 191 -> 105 backward, against eight neighbours a thread).
template <int kStep>
__device__ __forceinline__ void load8(float (&x)[8], const __nv_bfloat16* row, int c, int D) {
  if (kStep == 1) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (c < D) u = *reinterpret_cast<const uint4*>(row + c);
    unpack(x, u);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e * kStep < D ? one(row + c + e * kStep) : 0.f;
  }
}
template <int kStep>
__device__ __forceinline__ void load8(float (&x)[8], const float* row, int c, int D) {
  if (kStep == 1) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c < D) a = *reinterpret_cast<const float4*>(row + c), b = *reinterpret_cast<const float4*>(row + c + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e * kStep < D ? one(row + c + e * kStep) : 0.f;
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int kStep>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int D, const float (&x)[8]) {
  if (kStep == 1) {
    if (c < D)
      *reinterpret_cast<uint4*>(row + c) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e * kStep < D) put(row + c + e * kStep, x[e]);
  }
}
template <int kStep>
__device__ __forceinline__ void store8(float* row, int c, int D, const float (&x)[8]) {
  if (kStep == 1) {
    if (c < D) {
      *reinterpret_cast<float4*>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e * kStep < D) put(row + c + e * kStep, x[e]);
  }
}

// Where thread tg of a group begins in piece v.
template <int kStep, int kGroup>
__device__ __forceinline__ int column(int v, int tg) {
  return kStep == 1 ? (v * kGroup + tg) * 8 : v * kGroup * 8 + tg;
}

// Sum over a row's group of threads; every thread of the block calls it.
template <int kGroup>
__device__ __forceinline__ float group_sum(float x, float* red) {
#pragma unroll
  for (int o = 1; o < (kGroup < 32 ? kGroup : 32); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (kGroup > 32) {
    constexpr int kWarps = kGroup / 32;
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // the sums of the row before have been read
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    __syncthreads();
    x = 0.f;
    const int w0 = warp / kWarps * kWarps;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += red[w0 + w];
  }
  return x;
}

// Of a value of type T. For bfloat16 the fast exponential and quotient, whose errors
// (2^-24 times 2 + |z|, and 0 for z < -87.3) stay far below a rounding to 8 bits.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 4)
    return 1.f / (1.f + expf(-z));
  else
    return __fdividef(1.f, 1.f + __expf(-z));
}

// Where row `row` of an input starts: `t` elements from token to token, H rows a
// token (dense where t is H * D, which takes no division).
__device__ __forceinline__ long long row_at(const Args& p, long long row, long long t) {
  if (t == (long long)p.H * p.D) return row * p.D;
  const unsigned r = (unsigned)row, tok = r / (unsigned)p.H;
  return (long long)tok * t + (long long)(r - tok * p.H) * p.D;
}

// kGate: the gated norm (a = o, b = z); otherwise the add norm (a = x, b = residual).
template <typename TA, typename TB, bool kGate, int kGroup, int kVec, bool kWhole>
__global__ void __launch_bounds__(kThreads<kGroup>) forward_kernel(const Args p) {
  __shared__ float red[kThreads<kGroup> / 32];
  constexpr int kRows = kThreads<kGroup> / kGroup, kStep = kWhole ? 1 : kGroup;
  const int tg = threadIdx.x % kGroup;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kGroup;
  const bool in = row < p.rows;
  const int D = p.D;
  const TA* ra = static_cast<const TA*>(p.a) + (in ? row_at(p, row, p.a_t) : 0);
  const TB* rb = p.b ? static_cast<const TB*>(p.b) + (in ? row_at(p, row, p.b_t) : 0) : nullptr;
  float h[kVec][8], z[kGate ? kVec : 1][8], s2 = 0.f;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int c = in ? column<kStep, kGroup>(v, tg) : D;
    if constexpr (kGate) {
      load8<kStep>(h[v], ra, c, D);
      load8<kStep>(z[v], rb, c, D);
    } else {
      load8<kStep>(h[v], rb, c, D);
      if (p.a) {
        float x[8], s[8];
        load8<kStep>(x, ra, c, D);
        if (p.scale) {
          load8<kStep>(s, p.scale, c, D);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] = fmaf(s[e], x[e], h[v][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] += x[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s2 = fmaf(h[v][e], h[v][e], s2);
  }
  s2 = group_sum<kGroup>(s2, red);
  const float r = 1.f / sqrtf(s2 / (float)D + p.eps);
  if (!in) return;
  if (tg == 0 && p.rstd) p.rstd[row] = r;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const int c = column<kStep, kGroup>(v, tg);
    float w[8], y[8];
    load8<kStep>(w, p.w, c, D);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = h[v][e] * r * w[e];
      if constexpr (kGate) y[e] *= z[v][e] * sigmoid<TA>(z[v][e]);
    }
    store8<kStep>(static_cast<TA*>(p.out) + row * D, c, D, y);
    if constexpr (!kGate)
      if (p.h) store8<kStep>(static_cast<TB*>(p.h) + row * D, c, D, h[v]);
  }
}

template <typename TA, typename TB, bool kGate, int kGroup, int kVec, bool kWhole>
__global__ void __launch_bounds__(kThreads<kGroup>) backward_kernel(const Args p) {
  __shared__ float red[kThreads<kGroup> / 32];
  constexpr int kRows = kThreads<kGroup> / kGroup, kSums = kGate ? 1 : 2, kStep = kWhole ? 1 : kGroup;
  __shared__ float join[kRows > 1 ? kSums * kThreads<kGroup> * 8 : 1];
  const int tg = threadIdx.x % kGroup, sub = threadIdx.x / kGroup, D = p.D;
  gdr::grid_go();
  float dw[kVec][8], ds[kGate ? 1 : kVec][8];
#pragma unroll
  for (int v = 0; v < kVec; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[v][e] = 0.f;
      if constexpr (!kGate) ds[v][e] = 0.f;
    }
  for (long long base = (long long)blockIdx.x * kRows; base < p.rows; base += (long long)gridDim.x * kRows) {
    const long long row = base + sub;
    const bool in = row < p.rows;
    const TA* ra = static_cast<const TA*>(p.a) + (in ? row_at(p, row, p.a_t) : 0);
    const TB* rb = p.b ? static_cast<const TB*>(p.b) + (in ? row_at(p, row, p.b_t) : 0) : nullptr;
    const TA* rg = static_cast<const TA*>(p.dout) + (in ? row : 0) * D;
    const float r = in ? p.rstd[row] : 0.f;
    float u[kVec][8], t[kVec][8], x[kVec][8], c1 = 0.f;  // x: of the add norm; dz's factor of the gated
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = in ? column<kStep, kGroup>(v, tg) : D;
      float w[8], g[8];
      load8<kStep>(w, p.w, c, D);
      load8<kStep>(g, rg, c, D);
      if constexpr (kGate) {
        float z[8];
        load8<kStep>(u[v], ra, c, D);
        load8<kStep>(z, rb, c, D);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sigmoid<TA>(z[e]), gate = z[e] * s;
          u[v][e] *= r;
          t[v][e] = g[e] * gate * w[e];
          x[v][e] = g[e] * u[v][e] * w[e] * (s * fmaf(z[e], 1.f - s, 1.f));
          dw[v][e] = fmaf(g[e] * gate, u[v][e], dw[v][e]);
        }
      } else {
        load8<kStep>(u[v], rb, c, D);
        if (p.a) {
          load8<kStep>(x[v], ra, c, D);
          if (p.scale) {
            float s[8];
            load8<kStep>(s, p.scale, c, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[v][e] = fmaf(s[e], x[v][e], u[v][e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[v][e] += x[v][e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[v][e] *= r;
          t[v][e] = g[e] * w[e];
          dw[v][e] = fmaf(g[e], u[v][e], dw[v][e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) c1 = fmaf(t[v][e], u[v][e], c1);
    }
    c1 = group_sum<kGroup>(c1, red) / (float)D;
    if (in) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int c = column<kStep, kGroup>(v, tg);
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = r * fmaf(-u[v][e], c1, t[v][e]);
        if constexpr (kGate) {
          store8<kStep>(static_cast<TA*>(p.da) + row * D, c, D, d);
          store8<kStep>(static_cast<TB*>(p.db) + row * D, c, D, x[v]);
        } else {
          if (p.dh) {
            float up[8];
            load8<kStep>(up, static_cast<const TB*>(p.dh) + row * D, c, D);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] += up[e];
          }
          store8<kStep>(static_cast<TB*>(p.db) + row * D, c, D, d);
          if (p.a) {
            if (p.scale) {
              float s[8];
              load8<kStep>(s, p.scale, c, D);
#pragma unroll
              for (int e = 0; e < 8; ++e) ds[v][e] = fmaf(d[e], x[v][e], ds[v][e]), d[e] *= s[e];
            }
            if (p.da) store8<kStep>(static_cast<TA*>(p.da) + row * D, c, D, d);
          }
        }
      }
    }
  }
  // the block's rows of sums as one: [block][sum][D]
  float* part = p.part + (size_t)blockIdx.x * kSums * D;
  if constexpr (kRows > 1) {
    static_assert(kRows == 1 || kVec == 1, "a group smaller than the block has one piece a thread");
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = sub * kGroup * 8 + column<kStep, kGroup>(0, tg) + e * kStep;
      join[at] = dw[0][e];
      if constexpr (!kGate) join[kThreads<kGroup> * 8 + at] = ds[0][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kSums * kGroup * 8; i += kThreads<kGroup>) {
      const int sum = i / (kGroup * 8), c = i % (kGroup * 8);
      float s = 0.f;
      for (int q = 0; q < kRows; ++q) s += join[(sum * kThreads<kGroup> + q * kGroup) * 8 + c];
      if (c < D) part[sum * D + c] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = column<kStep, kGroup>(v, tg);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e * kStep < D) {
          part[c + e * kStep] = dw[v][e];
          if constexpr (!kGate) part[D + c + e * kStep] = ds[v][e];
        }
    }
  }
}

// The partial rows' sums, column by column: 32 columns a block, eight threads each.
__global__ void __launch_bounds__(kSumThreads) sums_kernel(const float* part, int parts, int sums, int D, float* dw, float* ds) {
  __shared__ float red[8][33];
  gdr::grid_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x, n = sums * D;
  float s = 0.f;
  if (c < n)
    for (int q = y; q < parts; q += 8) s += part[(size_t)q * n + c];
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && c < n) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += red[q][x];
    if (c < D)
      dw[c] = s;
    else if (ds)
      ds[c - D] = s;
  }
}

template <typename TA, typename TB, bool kGate, int kGroup, int kVec, bool kWhole>
cudaError_t forward(const Args& p, cudaStream_t s) {
  constexpr int rows = kThreads<kGroup> / kGroup;
  forward_kernel<TA, TB, kGate, kGroup, kVec, kWhole><<<(unsigned)((p.rows + rows - 1) / rows), kThreads<kGroup>, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename TA, typename TB, bool kGate, int kGroup, int kVec, bool kWhole>
cudaError_t backward(const Args& p, cudaStream_t s) {
  const int parts = part_rows(p.rows, p.D);
  backward_kernel<TA, TB, kGate, kGroup, kVec, kWhole><<<parts, kThreads<kGroup>, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int sums = kGate ? 1 : 2;
  return gdr::launch_after(true, sums_kernel, (unsigned)((sums * p.D + 31) / 32), (unsigned)kSumThreads, 0, s, (const float*)p.part, parts, sums, p.D,
                           p.dw, p.dscale);
}
template <typename TA, typename TB, bool kGate, int kGroup, int kVec, bool kWhole>
cudaError_t launch(const Args& p, bool bw, cudaStream_t s) {
  return bw ? backward<TA, TB, kGate, kGroup, kVec, kWhole>(p, s) : forward<TA, TB, kGate, kGroup, kVec, kWhole>(p, s);
}
// A group of threads is the least power of two with eight values each; rows
// wider than 2048 take more pieces a thread, but past 4096 the backward's sums would
// leave a block an SM: there a thread has one (8192, 16 M values of bfloat16 and
// fp32 residual: 165 -> 117 us; to 4096 it loses, 105 -> 109, and so does the
// forward, 44 -> 50).
template <typename TA, typename TB, bool kGate, bool kWhole>
cudaError_t pick(const Args& p, bool bw, cudaStream_t s) {
  const int need = (p.D + 7) / 8;
  if (need <= 8) return launch<TA, TB, kGate, 8, 1, kWhole>(p, bw, s);
  if (need <= 16) return launch<TA, TB, kGate, 16, 1, kWhole>(p, bw, s);
  if (need <= 32) return launch<TA, TB, kGate, 32, 1, kWhole>(p, bw, s);
  if (need <= 64) return launch<TA, TB, kGate, 64, 1, kWhole>(p, bw, s);
  if (need <= 128) return launch<TA, TB, kGate, 128, 1, kWhole>(p, bw, s);
  if (need <= 256) return launch<TA, TB, kGate, 256, 1, kWhole>(p, bw, s);
  if (need <= 512) return launch<TA, TB, kGate, 256, 2, kWhole>(p, bw, s);
  return bw ? backward<TA, TB, kGate, 1024, 1, kWhole>(p, s) : forward<TA, TB, kGate, 256, 4, kWhole>(p, s);
}
template <typename TA, typename TB, bool kGate>
cudaError_t whole(const Args& p, bool bw, cudaStream_t s) {
  const bool w = p.D % 8 == 0 && p.a_t % 8 == 0 && p.b_t % 8 == 0;
  return w ? pick<TA, TB, kGate, true>(p, bw, s) : pick<TA, TB, kGate, false>(p, bw, s);
}

}  // namespace

int part_rows(long long rows, int D) {
  int g = 8;
  while (g < 256 && g * 8 < D) g *= 2;
  const long long blocks = (rows + 256 / g - 1) / (256 / g);
  return (int)(blocks < kParts ? (blocks < 1 ? 1 : blocks) : kParts);
}

cudaError_t launch_add(const Args& p, bool a_bf16, bool b_bf16, bool bw, cudaStream_t s) {
  if (!a_bf16) return whole<float, float, false>(p, bw, s);
  return b_bf16 ? whole<__nv_bfloat16, __nv_bfloat16, false>(p, bw, s) : whole<__nv_bfloat16, float, false>(p, bw, s);
}
cudaError_t launch_gated(const Args& p, bool bf16, bool bw, cudaStream_t s) {
  return bf16 ? whole<__nv_bfloat16, __nv_bfloat16, true>(p, bw, s) : whole<float, float, true>(p, bw, s);
}

}  // namespace blocknorm
