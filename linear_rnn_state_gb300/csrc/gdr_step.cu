// The gated delta rule a few tokens at a time, states updated in place:
//   u = beta (v - e^g S k),  S <- e^g S + u k^T,  o = scale S q
//
// Bound by the states: each is read once and written once, 64 KB a value head
// at 128 x 128, against a few hundred bytes of q, k, v. A row of S (one value,
// all keys) belongs to a group of lanes with four keys each; rows do not meet,
// so a thread keeps eight rows in registers over all tokens of the call. Both
// products take the state before the update, S' q = e^g S q + u (k.q), so their
// sums are reduced together: sixteen sums over 32 lanes, half of what is left
// handed over at each step, so that each lane ends with one row's (16 shuffles
// and eight to hand the rows' u back, against 80 for each sum on its own).
// Measured: 256 requests x 32 heads of 128 x 128, bfloat16, 158 us, 6.8 TB/s (a
// copy's rate); one request 3.0 us on the device.
#include "gdr_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// kLanes lanes a row: 4 kLanes >= K.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
  constexpr int kRows = kLanes >= 16 ? 8 : 4, kSub = 32 / kLanes, kStep = kLanes / (2 * kRows), kWarpRows = kRows * kSub, kBlockRows = kWarpRows * (kThreads / 32);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / kLanes, cl = lane % kLanes;
  const int tiles = (a.V + kBlockRows - 1) / kBlockRows;
  const int tile = blockIdx.x % tiles, hv = blockIdx.x / tiles % a.Hv, r = blockIdx.x / (tiles * a.Hv);
  const int hk = hv / (a.Hv / a.Hk);
  const int row0 = tile * kBlockRows + warp * kWarpRows + sub;  // + i kSub
  const bool key_in = cl * 4 < a.K;
  const int slot = a.slots ? a.slots[r] : r;
  const bool live = slot >= 0 && slot < a.n_slots;
  float* state = a.state + (((size_t)(live ? slot : 0) * a.Hv + hv) * a.V) * a.K + cl * 4;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kSub;
    S[i] = live && key_in && row < a.V ? __ldcs(reinterpret_cast<const float4*>(state + (size_t)row * a.K)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int t = 0; t < a.T; ++t) {
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
    if (key_in) {
      q = load4(static_cast<const T*>(a.q) + r * a.q_b + t * a.q_t + hk * a.K + cl * 4);
      k = load4(static_cast<const T*>(a.k) + r * a.k_b + t * a.k_t + hk * a.K + cl * 4);
    }
    const size_t tok = (size_t)r * a.T + t;
    const float decay = expf(a.g[tok * a.Hv + hv]), beta = a.beta[tok * a.Hv + hv];
    // each lane ends with the sums of its row `mine`
    const int mine = cl / kStep % kRows, row = row0 + mine * kSub;
    const T* v = static_cast<const T*>(a.v) + r * a.v_b + t * a.v_t + (size_t)hv * a.V;
    const float vr = row < a.V ? load1(v + row) : 0.f;
    const float small = a.l2norm ? kSmall : 1.f;
    q.x *= small, q.y *= small, q.z *= small, q.w *= small;
    k.x *= small, k.y *= small, k.z *= small, k.w *= small;
    float kq = wkv7::group_allreduce<kLanes>(dot4(q, k, 0.f));
    float rq = a.scale, rk = 1.f;
    if (a.l2norm) {
      rq *= 1.f / sqrtf(wkv7::group_allreduce<kLanes>(dot4(q, q, 0.f)) + kSmallEps);
      rk = 1.f / sqrtf(wkv7::group_allreduce<kLanes>(dot4(k, k, 0.f)) + kSmallEps);
    }
    kq *= rk * rq;
    const bool second = cl >= kLanes / 2;  // S q rather than S k
    float x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float sk = dot4(S[i], k, 0.f), sq = dot4(S[i], q, 0.f);
      x[i] = (second ? sq : sk) + __shfl_xor_sync(0xffffffffu, second ? sk : sq, kLanes / 2);
    }
    int bit = kLanes / 4;
#pragma unroll
    for (int n = kRows / 2; n >= 1; n /= 2, bit /= 2) {
      const bool up = cl & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = (up ? x[i + n] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + n], bit);
    }
#pragma unroll
    for (; bit >= 1; bit /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], bit);
    const float other = __shfl_xor_sync(0xffffffffu, x[0], kLanes / 2);
    const float sk = second ? other : x[0], sq = second ? x[0] : other;
    const float u = beta * fmaf(-decay, sk * rk, vr), uk = u * rk;
    if (cl < kLanes / 2 && cl % kStep == 0 && row < a.V)
      store1(static_cast<T*>(a.o) + (tok * a.Hv + hv) * a.V + row, live ? fmaf(u, kq, decay * (sq * rq)) : 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float w = __shfl_sync(0xffffffffu, uk, i * kStep, kLanes);
      S[i].x = fmaf(w, k.x, decay * S[i].x);
      S[i].y = fmaf(w, k.y, decay * S[i].y);
      S[i].z = fmaf(w, k.z, decay * S[i].z);
      S[i].w = fmaf(w, k.w, decay * S[i].w);
    }
  }
  if (live && key_in)
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = row0 + i * kSub;
      if (row < a.V) __stcs(reinterpret_cast<float4*>(state + (size_t)row * a.K), S[i]);
    }
}

template <typename T, int kLanes>
cudaError_t launch(const StepArgs& a, cudaStream_t stream) {
  constexpr int rows = (kLanes >= 16 ? 8 : 4) * (32 / kLanes) * (kThreads / 32);
  step_kernel<T, kLanes><<<(unsigned)((size_t)a.R * a.Hv * ((a.V + rows - 1) / rows)), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t pick(const StepArgs& a, cudaStream_t s) {
  return a.K <= 32 ? launch<T, 8>(a, s) : a.K <= 64 ? launch<T, 16>(a, s) : launch<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? pick<__nv_bfloat16>(a, stream) : pick<float>(a, stream);
}

}  // namespace gdr
