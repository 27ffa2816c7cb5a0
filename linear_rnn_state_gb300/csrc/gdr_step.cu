// The gated delta rule a few tokens at a time, states updated in place:
//   u = beta (v - e^g S k),  S <- e^g S + u k^T,  o = scale S q
//
// Bound by the states: each is read once and written once, 64 KB a value head
// at 128 x 128, against a few hundred bytes of q, k, v. A row of S (one value,
// all keys) belongs to a group of lanes with four keys each; rows do not meet,
// so a thread keeps eight rows in registers over all tokens of the call. Both
// products take the state before the update, S' q = e^g S q + u (k.q), so their
// sums are reduced together.
#include "gdr_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128, kRows = 8;

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
  constexpr int kSub = 32 / kLanes, kWarpRows = kRows * kSub, kBlockRows = kWarpRows * (kThreads / 32);
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
    S[i] = live && key_in && row < a.V ? *reinterpret_cast<const float4*>(state + (size_t)row * a.K) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int t = 0; t < a.T; ++t) {
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
    if (key_in) {
      q = load4(static_cast<const T*>(a.q) + r * a.q_b + t * a.q_t + hk * a.K + cl * 4);
      k = load4(static_cast<const T*>(a.k) + r * a.k_b + t * a.k_t + hk * a.K + cl * 4);
    }
    const size_t tok = (size_t)r * a.T + t;
    const float decay = expf(a.g[tok * a.Hv + hv]), beta = a.beta[tok * a.Hv + hv];
    const T* v = static_cast<const T*>(a.v) + r * a.v_b + t * a.v_t + (size_t)hv * a.V;
    float vs[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) vs[i] = row0 + i * kSub < a.V ? load1(v + row0 + i * kSub) : 0.f;
    float kq = wkv7::group_allreduce<kLanes>(dot4(q, k, 0.f));
    float rq = a.scale, rk = 1.f;
    if (a.l2norm) {
      rq *= 1.f / sqrtf(wkv7::group_allreduce<kLanes>(dot4(q, q, 0.f)) + 1e-6f);
      rk = 1.f / sqrtf(wkv7::group_allreduce<kLanes>(dot4(k, k, 0.f)) + 1e-6f);
    }
    kq *= rk * rq;
    float out = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float sk = wkv7::group_allreduce<kLanes>(dot4(S[i], k, 0.f)), sq = wkv7::group_allreduce<kLanes>(dot4(S[i], q, 0.f));
      const float u = beta * fmaf(-decay, sk * rk, vs[i]), uk = u * rk;
      S[i].x = fmaf(uk, k.x, decay * S[i].x);
      S[i].y = fmaf(uk, k.y, decay * S[i].y);
      S[i].z = fmaf(uk, k.z, decay * S[i].z);
      S[i].w = fmaf(uk, k.w, decay * S[i].w);
      const float o = fmaf(u, kq, decay * (sq * rq));
      if (cl == i) out = o;
    }
    // lane i of a group has row i's o
    const int row = row0 + cl * kSub;
    if (cl < kRows && row < a.V) store1(static_cast<T*>(a.o) + (tok * a.Hv + hv) * a.V + row, live ? out : 0.f);
  }
  if (live && key_in)
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = row0 + i * kSub;
      if (row < a.V) *reinterpret_cast<float4*>(state + (size_t)row * a.K) = S[i];
    }
}

template <typename T, int kLanes>
cudaError_t launch(const StepArgs& a, cudaStream_t stream) {
  constexpr int rows = kRows * (32 / kLanes) * (kThreads / 32);
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
