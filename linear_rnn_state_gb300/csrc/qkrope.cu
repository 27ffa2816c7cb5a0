// Norms of queries and keys, a head at a time, with the position rotation, forward and backward: each row
// is read once, kept in registers as fp32, reduced, turned and written.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,  y = R n   (R turns pairs by position * freq)
//   backward: d = R^T dy, u = x r, t = d w:  dx = r (t - u mean(t u)),  dw = sum over rows of d u
//
// Bound by memory. A row belongs to a group of kGroup lanes with eight values each (16-byte
// loads), and up to kIter heads of q or of k of a token to a group, all on their way at once. The cosines and sines
// of a block's tokens are formed once, by all threads, in shared memory; a lane takes those of its values, and its
// weights, once for its heads. Measured: 16384 x 64 x 64 bfloat16 47 us forward (5.7 TB/s) and 92 + 3 backward (4.4), bound
// by instructions and latency at 12 to 24 warps an SM; 32768 x 24 x 64 fp32 66 us (6.1) and 111 + 3 (5.4).
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

constexpr int kThreads = 256, kSumThreads = 1024;
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
__device__ __forceinline__ void values(float2 (&x)[4], const Raw<bf16_t>& r) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void values(float2 (&x)[4], const Raw<float>& r) {
  x[0] = make_float2(r.a.x, r.a.y), x[1] = make_float2(r.a.z, r.a.w), x[2] = make_float2(r.b.x, r.b.y), x[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void put(bf16_t* p, const float2 (&x)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0].x, x[0].y), pack2(x[1].x, x[1].y), pack2(x[2].x, x[2].y), pack2(x[3].x, x[3].y));
}
__device__ __forceinline__ void put(float* p, const float2 (&x)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}
template <int kGroup>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 1 / sqrt(x) by a step of Newton's from the fast one. (0, and what is so small that the fast one overflows, stays as it gives.)
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x), y = fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r);
  return x > 1e-37f && x < 1e37f ? y : r;
}

// Values from 3e18 on, or below 1e-15 without an eps, have squares outside fp32's range: such a row is done once more,
// times a power of two.
__device__ __forceinline__ bool in_range(float mean) { return mean <= 1e37f && mean >= 1e-30f; }
// The mean square of a row so scaled; unit: 1 for rows in range.
template <int kGroup>
__device__ __forceinline__ float scaled_mean(float2 (&v)[4], float& unit, float inv, float eps) {
  float mean = 0.f;
#pragma unroll
  for (int again = 0; again < 2; ++again) {
    unit = !again || in_range(mean) ? 1.f : mean > 1.f ? 0x1p-66f : 0x1p66f;
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e].x *= unit, v[e].y *= unit, s2.x = fmaf(v[e].x, v[e].x, s2.x), s2.y = fmaf(v[e].y, v[e].y, s2.y);
    mean = fmaf(group_sum<kGroup>(s2.x + s2.y), inv, eps * unit * unit);
  }
  return mean;
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

// A lane's cosines and sines of a token, the sines with the signs that its values' partners take in forward (the
// backward turns the other way). kHalves: of its eight values; kInterleaved: of its four pairs.
template <int kHow>
struct Turn {
  float2 c[kHow == kHalves ? 4 : 2], s[kHow == kHalves ? 4 : 2];
  bool first, in;
};
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n"
      " mov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
template <int kHow, bool kBack>
__device__ __forceinline__ void take_turn(Turn<kHow>& t, const float2* cs, int c, int half) {
  if constexpr (kHow == kInterleaved) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = (c >> 1) + 2 * p + e;
        const float2 f = j < half ? cs[j] : make_float2(1.f, 0.f);
        (&t.c[p].x)[e] = f.x, (&t.s[p].x)[e] = kBack ? -f.y : f.y;
      }
  } else if constexpr (kHow == kHalves) {
    t.first = c < half, t.in = c < 2 * half;
    const float sign = t.first != kBack ? -1.f : 1.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float4 g = t.in ? *reinterpret_cast<const float4*>(cs + (t.first ? c : c - half) + 2 * p) : make_float4(1.f, 0.f, 1.f, 0.f);
      t.c[p] = make_float2(g.x, g.z), t.s[p] = make_float2(sign * g.y, sign * g.w);
    }
  }
}
// A row's values turned (kBack: back), four pairs of neighbours a lane. c: where they begin; row: the group's, for odd halves.
template <int kHow, int kGroup, bool kBack>
__device__ __forceinline__ void rotate(float2 (&x)[4], const Turn<kHow>& t, const float2* cs, int c, int half, int lane, float* row) {
  if constexpr (kHow == kInterleaved) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float co = (&t.c[p / 2].x)[p % 2], si = (&t.s[p / 2].x)[p % 2], a = x[p].x, b = x[p].y;
      x[p] = make_float2(fmaf(a, co, -b * si), fmaf(a, si, b * co));
    }
  } else if constexpr (kHow == kHalves) {
    const int own = lane & (kGroup - 1), src = (lane & ~(kGroup - 1)) + (t.in ? own + (t.first ? half : -half) / 8 : own);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 o = make_float2(__shfl_sync(0xffffffffu, x[p].x, src), __shfl_sync(0xffffffffu, x[p].y, src));
      x[p] = fma2(x[p], t.c[p], mul2(o, t.s[p]));
    }
  } else {
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p) *reinterpret_cast<float2*>(row + c + 2 * p) = x[p];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e;
      if (i < 2 * half) {
        const bool first = i < half;
        const float2 f = cs[first ? i : i - half];
        float& v = (&x[e / 2].x)[e % 2];
        v = fmaf(v, f.x, row[first ? i + half : i - half] * (first != kBack ? -f.y : f.y));
      }
    }
  }
}

// A unit: up to kIter heads of q or of k of a token, for a group of lanes.
struct Unit {
  unsigned tok;
  int h, heads, of;  // first head, heads in the unit, all heads
  bool key;
};
template <int kIter>
__device__ __forceinline__ int units_of(const Args& p) {  // of a token
  return (p.Hq + kIter - 1) / kIter + (p.Hk + kIter - 1) / kIter;
}
template <int kIter>
__device__ __forceinline__ Unit unit_at(const Args& p, unsigned u, unsigned units) {
  const int nq = (p.Hq + kIter - 1) / kIter;
  Unit x;
  x.tok = u / units;
  const int r = (int)(u - x.tok * units);
  x.key = r >= nq;
  x.h = (x.key ? r - nq : r) * kIter, x.of = x.key ? p.Hk : p.Hq, x.heads = min(kIter, x.of - x.h);
  return x;
}
// The cosines and sines of the tokens of units [u0, u1): [token][half].
__device__ __forceinline__ void fill_table(float2* table, const Args& p, unsigned t0, unsigned t1) {
  const int n = (int)(t1 - t0 + 1) * p.half;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int t = i / p.half, j = i - t * p.half;
    table[i] = cos_sin(turns_of(p.freq[j]), p.positions ? p.positions[t0 + t] : (int)((t0 + t) % p.T));
  }
}
// Eight weights of a lane.
__device__ __forceinline__ void weights(float2 (&w)[4], const float* p, int c, int D) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = make_float2(0.f, 0.f);
  if (c < D) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + c)), b = __ldg(reinterpret_cast<const float4*>(p + c + 4));
    w[0] = make_float2(a.x, a.y), w[1] = make_float2(a.z, a.w), w[2] = make_float2(b.x, b.y), w[3] = make_float2(b.z, b.w);
  }
}

// What a block keeps in shared memory: for odd halves its groups' rows, then the table.
template <int kHow>
constexpr int kRowBytes = kHow == kOddHalves ? kThreads * 8 * 4 : 0;

template <typename T, int kHow, int kGroup, int kIter>
__global__ void __launch_bounds__(kThreads, kIter == 8 ? 3 : 4) forward_kernel(const Args p, unsigned units) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kGroups = kThreads / kGroup;
  float2* table = reinterpret_cast<float2*>(smem + kRowBytes<kHow>);
  const int lane = threadIdx.x & 31, group = threadIdx.x / kGroup, c = threadIdx.x % kGroup * 8;
  float* line = reinterpret_cast<float*>(smem) + group * kGroup * 8;
  const unsigned u0 = blockIdx.x * kGroups, per = units_of<kIter>(p), u = min(u0 + group, units - 1);
  const bool live = u0 + group < units && c < p.D;
  const Unit x = unit_at<kIter>(p, u, per);
  const T* src = (x.key ? static_cast<const T*>(p.k) + x.tok * p.k_t : static_cast<const T*>(p.q) + x.tok * p.q_t) + x.h * p.D + c;
  T* dst = static_cast<T*>(x.key ? p.ko : p.qo) + ((long long)x.tok * x.of + x.h) * p.D + c;
  Raw<T> raw[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    clear(raw[i]);
    if (live && i < x.heads) fetch(raw[i], src + i * p.D);
  }
  float2 w[4];
  weights(w, x.key ? p.wk : p.wq, c, p.D);
  const unsigned t0 = u0 / per;
  fill_table(table, p, t0, (min(u0 + kGroups, units) - 1) / per);
  __syncthreads();
  const float2* cs = table + (x.tok - t0) * p.half;
  Turn<kHow> turn;
  take_turn<kHow, false>(turn, cs, c, p.half);
  const float inv = 1.f / (float)p.D;
  auto finish = [&](float2 (&v)[4], float mean, int i, bool mine) {
    const float r = inverse_root(mean);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(v[e], make_float2(r, r)), w[e]);
    rotate<kHow, kGroup, false>(v, turn, cs, c, p.half, lane, line);
    if (mine && live && i < x.heads) put(dst + i * p.D, v);
  };
  bool again = false;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    float2 v[4], s2 = make_float2(0.f, 0.f);
    values(v, raw[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) s2 = fma2(v[e], v[e], s2);
    const float mean = fmaf(group_sum<kGroup>(s2.x + s2.y), inv, p.eps);
    again |= live && i < x.heads && !in_range(mean);
    finish(v, mean, i, true);
  }
  if (!__any_sync(0xffffffffu, again)) return;
#pragma unroll 1
  for (int i = 0; i < kIter; ++i) {
    Raw<T> z;
    clear(z);
    if (live && i < x.heads) fetch(z, src + i * p.D);
    float2 v[4];
    values(v, z);
    float unit;
    const float mean = scaled_mean<kGroup>(v, unit, inv, p.eps);
    finish(v, mean, i, unit != 1.f);
  }
}

template <typename T, int kHow, int kGroup, int kIter>
__global__ void __launch_bounds__(kThreads, 2) backward_kernel(const Args p, unsigned units) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kGroups = kThreads / kGroup;
  __shared__ float join[kThreads * 8];
  float2* table = reinterpret_cast<float2*>(smem + kRowBytes<kHow>);
  const int lane = threadIdx.x & 31, group = threadIdx.x / kGroup, c = threadIdx.x % kGroup * 8;
  float* line = reinterpret_cast<float*>(smem) + group * kGroup * 8;
  const unsigned per = units_of<kIter>(p);
  const float inv = 1.f / (float)p.D;
  float2 dwq[4], dwk[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = make_float2(0.f, 0.f);
  for (unsigned u0 = blockIdx.x * kGroups; u0 < units; u0 += gridDim.x * kGroups) {
    const unsigned u = min(u0 + group, units - 1);
    const bool live = u0 + group < units && c < p.D;
    const Unit x = unit_at<kIter>(p, u, per);
    const T* src = (x.key ? static_cast<const T*>(p.k) + x.tok * p.k_t : static_cast<const T*>(p.q) + x.tok * p.q_t) + x.h * p.D + c;
    const long long at = ((long long)x.tok * x.of + x.h) * p.D + c;
    const T* up = static_cast<const T*>(x.key ? p.dko : p.dqo) + at;
    T* dst = static_cast<T*>(x.key ? p.ko : p.qo) + at;
    Raw<T> raw[kIter], rawd[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      clear(raw[i]), clear(rawd[i]);
      if (live && i < x.heads) fetch(raw[i], src + i * p.D), fetch(rawd[i], up + i * p.D);
    }
    float2 w[4];
    weights(w, x.key ? p.wk : p.wq, c, p.D);
    const unsigned t0 = u0 / per;
    __syncthreads();  // the units before are done with the table
    fill_table(table, p, t0, (min(u0 + kGroups, units) - 1) / per);
    __syncthreads();
    const float2* cs = table + (x.tok - t0) * p.half;
    Turn<kHow> turn;
    take_turn<kHow, true>(turn, cs, c, p.half);
    float2 dw[4];
    bool again = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      float2 v[4], d[4], s2 = make_float2(0.f, 0.f), c1 = s2;
      values(v, raw[i]), values(d, rawd[i]);  // (0 where there is no row)
      rotate<kHow, kGroup, true>(d, turn, cs, c, p.half, lane, line);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(v[e], v[e], s2), c1 = fma2(mul2(d[e], w[e]), v[e], c1);
      // (places without a head hold rows of zeros: they add nothing to dw, whatever eps is)
      const float mean = fmaf(group_sum<kGroup>(s2.x + s2.y), inv, p.eps);
      const bool here = u0 + group < units && i < x.heads;
      again |= here && !in_range(mean);
      const float r = here && in_range(mean) ? inverse_root(mean) : 0.f;
      const float m = -(group_sum<kGroup>(c1.x + c1.y) * r * inv);
      const float2 rr = make_float2(r, r), mm = make_float2(m, m);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 z = mul2(v[e], rr);
        dw[e] = fma2(d[e], z, dw[e]);
        d[e] = mul2(fma2(z, mm, mul2(d[e], w[e])), rr);
      }
      if (live && i < x.heads) put(dst + i * p.D, d);
    }
    if (__any_sync(0xffffffffu, again)) {
#pragma unroll 1
      for (int i = 0; i < kIter; ++i) {
        Raw<T> y, z;
        clear(y), clear(z);
        if (live && i < x.heads) fetch(y, src + i * p.D), fetch(z, up + i * p.D);
        float2 v[4], d[4], c1 = make_float2(0.f, 0.f);
        values(v, y), values(d, z);
        rotate<kHow, kGroup, true>(d, turn, cs, c, p.half, lane, line);
        float unit;
        const float mean = scaled_mean<kGroup>(v, unit, inv, p.eps);
        const bool mine = unit != 1.f && u0 + group < units && i < x.heads;
        const float r = mine ? inverse_root(mean) : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) c1 = fma2(mul2(d[e], w[e]), v[e], c1);
        const float m = -(group_sum<kGroup>(c1.x + c1.y) * r * inv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = mul2(v[e], make_float2(r, r)), t = fma2(u, make_float2(m, m), mul2(d[e], w[e]));
          if (mine) dw[e] = fma2(d[e], u, dw[e]);
          d[e] = mul2(mul2(t, make_float2(r, r)), make_float2(unit, unit));
        }
        if (mine && c < p.D) put(dst + i * p.D, d);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (units past the last repeat it, its rows' sums being zeros)
      if (x.key)
        dwk[e].x += dw[e].x, dwk[e].y += dw[e].y;
      else
        dwq[e].x += dw[e].x, dwq[e].y += dw[e].y;
    }
  }
  // the block's sums as one row: [block][q, k][D]
  float* part = p.part + (size_t)blockIdx.x * 2 * p.D;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) reinterpret_cast<float2*>(join)[threadIdx.x * 4 + e] = s ? dwk[e] : dwq[e];
    __syncthreads();
    for (int i = threadIdx.x; i < p.D; i += kThreads) {
      float x = 0.f;
#pragma unroll 8
      for (int g = 0; g < kGroups; ++g) x += join[g * kGroup * 8 + i];
      part[s * p.D + i] = x;
    }
  }
}

// The partial rows' sums, column by column: 32 columns a block, 32 threads each, whose loads are on their way together.
__global__ void __launch_bounds__(kSumThreads) sums_kernel(const Args p, int parts) {
  __shared__ float red[32][33];
  constexpr int kMost = (kParts + 31) / 32;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x, n = 2 * p.D;
  float v[kMost], s = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) v[i] = c < n && y + 32 * i < parts ? p.part[(size_t)(y + 32 * i) * n + c] : 0.f;
#pragma unroll
  for (int i = 0; i < kMost; ++i) s += v[i];
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && c < n) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s += red[q][x];
    if (c < p.D)
      p.dwq[c] = s;
    else
      p.dwk[c - p.D] = s;
  }
}

int group_of(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }
// Heads of a unit, `most` of them where the units that hold fewer are few and there are units enough for the GPU, else
// a half, a quarter or an eighth as many: what a unit costs besides its rows (its place, cosines, sines and weights) is 1.4 heads of
// bfloat16's forward (16384 x 64 x 64: 97, 68, 51 and 48 us with 1, 2, 4 and 8 heads; backward 135, 110 and 87 with 1, 2 and 4)
// and 0.4 of fp32's (32768 x 24 x 64: 74 and 63 us with 1 and 2). More would not fit the registers.
int heads_of(const Args& p, long long tokens, int most) {
  for (int n = most; n > 1; n /= 2) {
    const long long units = (long long)((p.Hq + n - 1) / n) + (p.Hk + n - 1) / n;
    if (units * n <= 5 * (p.Hq + p.Hk) / 4 && tokens * units >= kSms * 4 * (kThreads / group_of(p.D))) return n;
  }
  return 1;
}
unsigned units_in(const Args& p, int heads) {
  const long long tokens = p.rows / (p.Hq + p.Hk);
  return (unsigned)(tokens * ((p.Hq + heads - 1) / heads + (p.Hk + heads - 1) / heads));
}
// Bytes of the table of the tokens that a block's units can touch.
size_t table_bytes(const Args& p, int groups, int heads) {
  const int per = (p.Hq + heads - 1) / heads + (p.Hk + heads - 1) / heads;
  return (size_t)((groups + 2 * per - 2) / per) * p.half * 8;
}

template <typename T, int kHow, int kGroup, int kIter>
cudaError_t run(const Args& p, bool backward, cudaStream_t s) {
  constexpr int kGroups = kThreads / kGroup;
  const unsigned units = units_in(p, kIter);
  const size_t smem = kRowBytes<kHow> + table_bytes(p, kGroups, kIter);
  const unsigned blocks = (units + kGroups - 1) / kGroups;
  if (!backward) {
    forward_kernel<T, kHow, kGroup, kIter><<<blocks, kThreads, smem, s>>>(p, units);
    return cudaGetLastError();
  }
  if constexpr (kIter < 8) {
    const unsigned parts = blocks < (unsigned)kParts ? blocks : kParts;
    backward_kernel<T, kHow, kGroup, kIter><<<parts, kThreads, smem, s>>>(p, units);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    sums_kernel<<<(unsigned)((2 * p.D + 31) / 32), kSumThreads, 0, s>>>(p, (int)parts);
  }
  return cudaGetLastError();
}
template <typename T, int kHow, int kGroup>
cudaError_t heads(const Args& p, bool backward, cudaStream_t s) {
  constexpr bool kBf16 = sizeof(T) == 2;
  const int n = heads_of(p, p.rows / (p.Hq + p.Hk), kBf16 ? backward ? 4 : 8 : 2);
  if constexpr (kBf16) {
    if (n == 8) return run<T, kHow, kGroup, 8>(p, false, s);
    if (n == 4) return run<T, kHow, kGroup, 4>(p, backward, s);
  }
  return n == 2 ? run<T, kHow, kGroup, 2>(p, backward, s) : run<T, kHow, kGroup, 1>(p, backward, s);
}
template <typename T, int kHow>
cudaError_t pick(const Args& p, bool backward, cudaStream_t s) {
  switch (group_of(p.D)) {
    case 4: return heads<T, kHow, 4>(p, backward, s);
    case 8: return heads<T, kHow, 8>(p, backward, s);
    case 16: return heads<T, kHow, 16>(p, backward, s);
    default: return heads<T, kHow, 32>(p, backward, s);
  }
}
template <typename T>
cudaError_t how(const Args& p, bool backward, cudaStream_t s) {
  if (p.interleaved) return pick<T, kInterleaved>(p, backward, s);
  return p.half % 8 ? pick<T, kOddHalves>(p, backward, s) : pick<T, kHalves>(p, backward, s);
}

}  // namespace

int part_rows(long long rows) { return (int)(rows < kParts ? (rows < 1 ? 1 : rows) : kParts); }
cudaError_t launch(const Args& p, bool bf16, bool backward, cudaStream_t s) {
  return bf16 ? how<bf16_t>(p, backward, s) : how<float>(p, backward, s);
}

}  // namespace qkrope
