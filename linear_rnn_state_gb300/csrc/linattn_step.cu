// Linear attention with a decay a few tokens at a time, states updated in place:
//   S <- e^g S + v k^T,  o = scale S q
//
// Bound by the states: each is read once and written once, 64 KB a value head at 128 x 128, against a
// few hundred bytes of q, k, v. A row of S (one value, all keys) belongs to a group of lanes with
// four keys each; rows do not meet, so a thread keeps its rows in registers over all tokens of the
// call. The rows' sums over the lanes are reduced together, half of what is left handed over at each
// step, so that each lane ends with one row's. Measured: 256 requests, 32 heads of 128 x 128, 152 us (1.08 GB, 7.1 TB/s: the
// measured copy rate and 4 %); one request 4.7 us.
#include "linattn_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float4 load4(const bf16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = unpack2(u.x), b = unpack2(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float load1(const bf16_t* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(bf16_t* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

template <int kLanes>
constexpr int kRowsOf = kLanes >= 16 ? 8 : 4;

// kLanes lanes a row: 4 kLanes >= K.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
  constexpr int kRows = kRowsOf<kLanes>, kSub = 32 / kLanes, kBlockRows = kRows * kSub * (kThreads / 32), kStep = kLanes / kRows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / kLanes, cl = lane % kLanes;
  const int tiles = (a.V + kBlockRows - 1) / kBlockRows;
  const int tile = blockIdx.x % tiles, hv = blockIdx.x / tiles % a.Hv, r = blockIdx.x / (tiles * a.Hv);
  const int hk = hv / (a.Hv / a.Hk);
  const int row0 = tile * kBlockRows + warp * kRows * kSub + sub;  // + i kSub
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
    const float decay = expf(a.g[a.fixed ? hv : tok * a.Hv + hv]);
    const T* v = static_cast<const T*>(a.v) + r * a.v_b + t * a.v_t + (size_t)hv * a.V;
    // each lane brings and ends with its row `mine`
    const int mine = cl / kStep, row = row0 + mine * kSub;
    const float vr = row < a.V ? load1(v + row) : 0.f;
    float x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float w = __shfl_sync(0xffffffffu, vr, i * kStep, kLanes);
      S[i].x = fmaf(w, k.x, decay * S[i].x);
      S[i].y = fmaf(w, k.y, decay * S[i].y);
      S[i].z = fmaf(w, k.z, decay * S[i].z);
      S[i].w = fmaf(w, k.w, decay * S[i].w);
      x[i] = fmaf(S[i].x, q.x, fmaf(S[i].y, q.y, fmaf(S[i].z, q.z, S[i].w * q.w)));
    }
    int bit = kLanes / 2;
#pragma unroll
    for (int n = kRows / 2; n >= 1; n /= 2, bit /= 2) {
      const bool up = cl & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = (up ? x[i + n] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + n], bit);
    }
#pragma unroll
    for (; bit >= 1; bit /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], bit);
    if (cl % kStep == 0 && row < a.V) store1(static_cast<T*>(a.o) + (tok * a.Hv + hv) * a.V + row, live ? a.scale * x[0] : 0.f);
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
  constexpr int rows = kRowsOf<kLanes> * (32 / kLanes) * (kThreads / 32);
  step_kernel<T, kLanes><<<(unsigned)((size_t)a.R * a.Hv * ((a.V + rows - 1) / rows)), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t pick(const StepArgs& a, cudaStream_t s) {
  return a.K <= 32 ? launch<T, 8>(a, s) : a.K <= 64 ? launch<T, 16>(a, s) : launch<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t stream) {
  return bf16 ? pick<bf16_t>(a, stream) : pick<float>(a, stream);
}

}  // namespace linattn
