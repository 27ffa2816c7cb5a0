// Norms of queries and keys, a head at a time, with the position rotation, forward and backward: each row
// is read once, kept in registers as fp32, reduced, turned and written.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,  y = R n   (R turns pairs by position * freq)
//   backward: d = R^T dy, u = x r, t = d w:  dx = r (t - u mean(t u)),  dw = sum over rows of d u
//
// Bound by memory. A row belongs to a group of kGroup lanes with eight values each (16-byte
// loads); a block takes a stretch of rows, heads of a token beside one another, and a thread has
// kIter of them on their way at once. The cosines and sines of the tokens of a stretch are
// formed once, by all threads, in shared memory, and serve all heads of a token.
//
// Angles. freq / (2 pi) as a 64-bit fraction of a turn, times the position modulo 2^64, is the angle as a
// fraction of a turn, off by no more than position * 2^-63; its upper 32 bits go to fp32 as a signed
// part of half a turn (2^-25 of it). In fp32, position * freq would be off by 0.06 at 2^20.
//
// Pairs (j, half + j) lie in two lanes: with half a multiple of eight a lane's partner has the other
// eight values and they are exchanged by shuffles, else through shared memory.
#include <cuda_bf16.h>

#include "gdr_launch.h"
#include "qkrope_launch.h"

namespace qkrope {
namespace {

constexpr int kThreads = 256, kSumThreads = 256;
enum How { kInterleaved, kHalves, kOddHalves };
typedef __nv_bfloat16 bf16_t;

template <typename T> struct Raw;  // eight values as they come
template <> struct Raw<bf16_t> { uint4 u; };
template <> struct Raw<float> { float4 a, b; };

__device__ __forceinline__ void fetch(Raw<bf16_t>& r, const bf16_t* p) { r.u = __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void fetch(Raw<float>& r, const float* p) {
  r.a = __ldg(reinterpret_cast<const float4*>(p)), r.b = __ldg(reinterpret_cast<const float4*>(p + 4));
}
__device__ __forceinline__ void clear(Raw<bf16_t>& r) { r.u = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void clear(Raw<float>& r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void values(float (&x)[8], const Raw<bf16_t>& r) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void values(float (&x)[8], const Raw<float>& r) {
  x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w, x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void put(bf16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void put(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <int kGroup>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// freq / (2 pi) modulo 1 as a 64-bit fraction: freq = m 2^e, m of 53 bits, times 2^66 / (2 pi), by integers.
__device__ __forceinline__ unsigned long long turns_of(double freq) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(freq);
  const int ex = (int)(bits >> 52) & 2047;
  const unsigned long long m = (bits & ((1ull << 52) - 1)) | (ex ? 1ull << 52 : 0ull);
  const unsigned long long c = 0xA2F9836E4E441529ull, cl = 0xFC2757D1F534DDC0ull;  // 2 / pi = c 2^-64 + cl 2^-128
  // m 2^11 (64 bits) * (2 / pi) / 4, as a fraction times 2^128 in (hi, lo), is turns * 2^-(e' ) for e' = ex - 1086
  const unsigned long long M = m << 11;
  unsigned long long hi = __umul64hi(M, c), lo = M * c;
  const unsigned long long add = __umul64hi(M, cl);
  lo += add;
  hi += lo < add;
  // M = freq 2^(1075 + 11 - ex): freq * 2/pi = (hi 2^64 + lo) 2^-64 * 2^(ex - 1086); turns = that / 4. The fraction
  // of 64 bits is turns 2^64 = (hi 2^64 + lo) 2^(ex - 1088), modulo 2^64.
  const int s = ex - 1088;
  unsigned long long t;
  if (s >= 64)
    t = 0;  // freq of 2^130 and more: whole turns as far as 117 bits tell
  else if (s >= 0)
    t = lo << s;
  else if (s > -64)
    t = (lo >> -s) | (hi << (64 + s));
  else if (s > -128)
    t = hi >> (-s - 64);
  else
    t = 0;
  return bits >> 63 ? 0ull - t : t;
}
__device__ __forceinline__ float2 cos_sin(unsigned long long turns, int position) {
  const unsigned long long a = turns * (unsigned long long)(long long)position;
  float s, c;
  sincospif((float)(int)(a >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// The stretch [r0, r1) of rows: the table of its tokens, [token][half].
__device__ __forceinline__ void fill_table(float2* table, const Args& p, long long r0, long long r1, int H) {
  const unsigned t0 = (unsigned)r0 / (unsigned)H;
  const int n = (int)((unsigned)(r1 - 1) / (unsigned)H - t0 + 1) * p.half;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int t = i / p.half, j = i - t * p.half;
    const unsigned tok = t0 + t;
    table[i] = cos_sin(turns_of(p.freq[j]), p.positions ? p.positions[tok] : (int)(tok % p.T));
  }
}

// x's pairs turned (kBack: back) in the group's row. c: where the lane's eight values begin; cs: the token's table.
template <int kHow, int kGroup, bool kBack>
__device__ __forceinline__ void rotate(float (&x)[8], const float2* cs, int c, int half, int lane, float* row) {
  if constexpr (kHow == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int j = (c + e) >> 1;
      if (j < half) {
        const float2 f = cs[j];
        const float s = kBack ? -f.y : f.y, a = x[e], b = x[e + 1];
        x[e] = fmaf(a, f.x, -b * s), x[e + 1] = fmaf(a, s, b * f.x);
      }
    }
  } else if constexpr (kHow == kHalves) {
    const bool first = c < half, in = c < 2 * half;
    const int src = (lane & ~(kGroup - 1)) + (in ? (first ? c + half : c - half) >> 3 : lane & (kGroup - 1));
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, x[e], src);
    if (in) {
      const float2* f = cs + (first ? c : c - half);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 g = *reinterpret_cast<const float4*>(f + e);
        const float s0 = first != kBack ? -g.y : g.y, s1 = first != kBack ? -g.w : g.w;
        x[e] = fmaf(x[e], g.x, o[e] * s0), x[e + 1] = fmaf(x[e + 1], g.z, o[e + 1] * s1);
      }
    }
  } else {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) row[c + e] = x[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e;
      if (i < 2 * half) {
        const bool first = i < half;
        const float2 f = cs[first ? i : i - half];
        x[e] = fmaf(x[e], f.x, row[first ? i + half : i - half] * (first != kBack ? -f.y : f.y));
      }
    }
  }
}

template <typename T>
struct Row {
  const T *x, *dy;
  T* out;
  bool key;
};
template <typename T>
__device__ __forceinline__ Row<T> row_at(const Args& p, long long row, int H) {
  const long long tok = (unsigned)row / (unsigned)H;  // (fewer than 2^31 rows)
  const int h = (int)(row - tok * H);
  Row<T> r;
  r.key = h >= p.Hq;
  if (r.key) {
    const long long at = (tok * p.Hk + h - p.Hq) * p.D;
    r.x = static_cast<const T*>(p.k) + tok * p.k_t + (long long)(h - p.Hq) * p.D;
    r.dy = static_cast<const T*>(p.dko) + at, r.out = static_cast<T*>(p.ko) + at;
  } else {
    const long long at = (tok * p.Hq + h) * p.D;
    r.x = static_cast<const T*>(p.q) + tok * p.q_t + (long long)h * p.D;
    r.dy = static_cast<const T*>(p.dqo) + at, r.out = static_cast<T*>(p.qo) + at;
  }
  return r;
}

// What a block keeps in shared memory: for odd halves its groups' rows, then the table.
template <int kHow>
constexpr int kRowBytes = kHow == kOddHalves ? kThreads * 8 * 4 : 0;

template <typename T, int kHow, int kGroup, int kIter>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Args p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kGroups = kThreads / kGroup;
  float2* table = reinterpret_cast<float2*>(smem + kRowBytes<kHow>);
  const int lane = threadIdx.x & 31, group = threadIdx.x / kGroup, c = threadIdx.x % kGroup * 8, H = p.Hq + p.Hk;
  float* line = reinterpret_cast<float*>(smem) + group * kGroup * 8;
  const long long r0 = (long long)blockIdx.x * kGroups * kIter, r1 = min(r0 + kGroups * kIter, p.rows);
  Raw<T> raw[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long row = r0 + i * kGroups + group;
    clear(raw[i]);
    if (row < r1 && c < p.D) fetch(raw[i], row_at<T>(p, row, H).x + c);
  }
  fill_table(table, p, r0, r1, H);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long row = r0 + i * kGroups + group;
    const bool in = row < r1;
    const Row<T> at = row_at<T>(p, in ? row : r0, H);
    const float2* cs = table + ((unsigned)(in ? row : r0) / (unsigned)H - (unsigned)r0 / (unsigned)H) * p.half;
    float x[8], w[8];
    values(x, raw[i]);
    if (c < p.D) {
      Raw<float> rw;
      fetch(rw, (at.key ? p.wk : p.wq) + c);
      values(w, rw);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0.f;
    }
    float s2 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s2 = fmaf(x[e], x[e], s2);
    const float r = 1.f / sqrtf(group_sum<kGroup>(s2) / (float)p.D + p.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
    rotate<kHow, kGroup, false>(x, cs, c, p.half, lane, line);
    if (in && c < p.D) put(at.out + c, x);
  }
}

template <typename T, int kHow, int kGroup>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kGroups = kThreads / kGroup, kIter = 2;
  __shared__ float join[kThreads * 8];
  float2* table = reinterpret_cast<float2*>(smem + kRowBytes<kHow>);
  const int lane = threadIdx.x & 31, group = threadIdx.x / kGroup, c = threadIdx.x % kGroup * 8, H = p.Hq + p.Hk;
  float* line = reinterpret_cast<float*>(smem) + group * kGroup * 8;
  float dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  for (long long r0 = (long long)blockIdx.x * kGroups * kIter; r0 < p.rows; r0 += (long long)gridDim.x * kGroups * kIter) {
    const long long r1 = min(r0 + kGroups * kIter, p.rows);
    Raw<T> raw[kIter], rawd[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const long long row = r0 + i * kGroups + group;
      clear(raw[i]), clear(rawd[i]);
      if (row < r1 && c < p.D) {
        const Row<T> at = row_at<T>(p, row, H);
        fetch(raw[i], at.x + c), fetch(rawd[i], at.dy + c);
      }
    }
    __syncthreads();  // the stretch before is done with the table
    fill_table(table, p, r0, r1, H);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const long long row = r0 + i * kGroups + group;
      const bool in = row < r1;
      const Row<T> at = row_at<T>(p, in ? row : r0, H);
      const float2* cs = table + ((unsigned)(in ? row : r0) / (unsigned)H - (unsigned)r0 / (unsigned)H) * p.half;
      float x[8], d[8], t[8], w[8];
      values(x, raw[i]), values(d, rawd[i]);
      if (c < p.D) {
        Raw<float> rw;
        fetch(rw, (at.key ? p.wk : p.wq) + c);
        values(w, rw);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 0.f;
      }
      rotate<kHow, kGroup, true>(d, cs, c, p.half, lane, line);
      float s2 = 0.f, c1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = d[e] * w[e], s2 = fmaf(x[e], x[e], s2), c1 = fmaf(t[e], x[e], c1);
      const float r = 1.f / sqrtf(group_sum<kGroup>(s2) / (float)p.D + p.eps);
      const float m = group_sum<kGroup>(c1) * r / (float)p.D;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = x[e] * r, g = d[e] * u;
        if (at.key)
          dwk[e] += in ? g : 0.f;
        else
          dwq[e] += in ? g : 0.f;
        t[e] = r * fmaf(-u, m, t[e]);
      }
      if (in && c < p.D) put(at.out + c, t);
    }
  }
  // the block's sums as one row: [block][q, k][D]
  float* part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) join[threadIdx.x * 8 + e] = s ? dwk[e] : dwq[e];
    __syncthreads();
    for (int i = threadIdx.x; i < p.D; i += kThreads) {
      float x = 0.f;
      for (int g = 0; g < kGroups; ++g) x += join[g * kGroup * 8 + i];
      part[s * p.D + i] = x;
    }
  }
}

// The partial rows' sums, column by column: 32 columns a block, eight threads each.
__global__ void __launch_bounds__(kSumThreads) sums_kernel(const Args p, int parts) {
  __shared__ float red[8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x, n = 2 * p.D;
  float s = 0.f;
  if (c < n)
    for (int q = y; q < parts; q += 8) s += p.part[(size_t)q * n + c];
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && c < n) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += red[q][x];
    if (c < p.D)
      p.dwq[c] = s;
    else
      p.dwk[c - p.D] = s;
  }
}

int group_of(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }
// Bytes of the table of a stretch of `rows` rows: the tokens it can touch.
size_t table_bytes(const Args& p, int rows) {
  const int H = p.Hq + p.Hk;
  return (size_t)((rows + 2 * H - 2) / H) * p.half * 8;
}

template <typename T, int kHow, int kGroup, int kIter>
cudaError_t forward(const Args& p, cudaStream_t s) {
  constexpr int rows = kThreads / kGroup * kIter;
  forward_kernel<T, kHow, kGroup, kIter><<<(unsigned)((p.rows + rows - 1) / rows), kThreads, kRowBytes<kHow> + table_bytes(p, rows), s>>>(p);
  return cudaGetLastError();
}
template <typename T, int kHow, int kGroup>
cudaError_t run(const Args& p, bool backward, cudaStream_t s) {
  if (!backward) return p.rows <= 152 * 2 * (kThreads / kGroup) ? forward<T, kHow, kGroup, 1>(p, s) : forward<T, kHow, kGroup, 2>(p, s);
  const int parts = part_rows(p.rows, p.D);
  backward_kernel<T, kHow, kGroup><<<parts, kThreads, kRowBytes<kHow> + table_bytes(p, kThreads / kGroup * 2), s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  sums_kernel<<<(unsigned)((2 * p.D + 31) / 32), kSumThreads, 0, s>>>(p, parts);
  return cudaGetLastError();
}
template <typename T, int kHow>
cudaError_t pick(const Args& p, bool backward, cudaStream_t s) {
  switch (group_of(p.D)) {
    case 4: return run<T, kHow, 4>(p, backward, s);
    case 8: return run<T, kHow, 8>(p, backward, s);
    case 16: return run<T, kHow, 16>(p, backward, s);
    default: return run<T, kHow, 32>(p, backward, s);
  }
}
template <typename T>
cudaError_t how(const Args& p, bool backward, cudaStream_t s) {
  if (p.interleaved) return pick<T, kInterleaved>(p, backward, s);
  return p.half % 8 ? pick<T, kOddHalves>(p, backward, s) : pick<T, kHalves>(p, backward, s);
}

}  // namespace

int part_rows(long long rows, int D) {
  const long long each = kThreads / group_of(D) * 2, blocks = (rows + each - 1) / each;
  return (int)(blocks < kParts ? (blocks < 1 ? 1 : blocks) : kParts);
}
cudaError_t launch(const Args& p, bool bf16, bool backward, cudaStream_t s) {
  return bf16 ? how<bf16_t>(p, backward, s) : how<float>(p, backward, s);
}

}  // namespace qkrope
