// Linear attention with a decay: the states before every chunk, and backward the gradients of the
// states after every chunk (fp32 with heads above 64; the joining serves segments of the others too).
//
// Within a chunk, with G the running sum of its log decays and Gc the whole sum:
//   forward   S' = e^{Gc} S + sum_j e^{Gc - G_j} v_j k_j^T
//   backward  D  = e^{Gc} D' + sum_i scale e^{G_i} do_i q_i^T
// The sums of all chunks come first, all at once, as products of a chunk's tokens on the tensor cores (the
// scaled values in three bfloat16 parts, 24 bits: states are fp32 results); a second kernel
// runs over the chunks of each sequence, every number of a state on its own, and puts the state
// before each chunk in the place of its sum.
#include "linattn_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128, kC = kCF32, kP = In<float>::kParts;

// A block: a chunk, a value head, 64 values (16 a warp) by all keys.
template <bool kBack, int kTiles>
__global__ void __launch_bounds__(kThreads) sums_kernel(const Args a, float* out) {
  constexpr int kKp = kTiles * 8;
  extern __shared__ __align__(128) unsigned char smem[];
  bf16_t* xs = reinterpret_cast<bf16_t*>(smem);  // [64 tokens][64 values], 3 parts
  bf16_t* bs = xs + kP * kC * 64;                // [64 tokens][keys]
  float2* G = reinterpret_cast<float2*>(bs + kP * kC * kKp);
  float* u = reinterpret_cast<float*>(G + kC);
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = (s.V + 63) >> 6, slice = blockIdx.x % slices, hv = blockIdx.x / slices % s.Hv, slot = blockIdx.x / slices / s.Hv;
  const int hk = hv / (s.Hv / s.Hk), v0 = slice * 64;
  ChunkAt c;
  if (!chunk_at(s, slot, kC, c)) return;
  const size_t tok = (size_t)c.b * s.T + c.t0;
  if (warp == 0) {
    running_sums<kC / 32>(G, s.fixed ? a.g + hv : a.g + tok * s.Hv + hv, s.fixed ? 0 : s.Hv, c.len, lane);
    __syncwarp();
#pragma unroll
    for (int j = lane; j < kC; j += 32) u[j] = kBack ? s.scale * expf(G[j].x + G[j].y) : expf(minus(G[kC - 1], G[j]));
    if (lane == 0 && slice == 0) a.decay[(size_t)slot * s.Hv + hv] = expf(G[kC - 1].x + G[kC - 1].y);
  }
  __syncthreads();
  const float* x = kBack ? static_cast<const float*>(a.d_o) + (tok * s.Hv + hv) * s.V + v0
                     : static_cast<const float*>(a.v) + c.b * s.v_b + c.t0 * s.v_t + (size_t)hv * s.V + v0;
  const float* b = kBack ? static_cast<const float*>(a.q) + c.b * s.q_b + c.t0 * s.q_t + (size_t)hk * s.K
                     : static_cast<const float*>(a.k) + c.b * s.k_b + c.t0 * s.k_t + (size_t)hk * s.K;
  fill_tile<kP, kC>(xs, x, kBack ? (long long)s.Hv * s.V : s.v_t, c.len, min(64, s.V - v0), u, tid, kThreads);
  fill_tile<kP, kC>(bs, b, kBack ? s.q_t : s.k_t, c.len, s.K, nullptr, tid, kThreads);
  __syncthreads();
  float acc[kTiles][4];
  zero(acc);
#pragma unroll
  for (int k0 = 0; k0 < kC; k0 += 16) {
    Frag<kP> fa;
    a_km(fa, xs, kC, kC * 64, 16 * warp, k0, lane);
#pragma unroll
    for (int n = 0; n < kTiles / 2; ++n) {
      Frag<kP> fb;
      b_kn(fb, bs, kC, kC * kKp, 16 * n, k0, lane);
      mma_added(acc[2 * n], acc[2 * n + 1], fa, fb);
    }
  }
  float* dst = out + ((size_t)slot * s.Hv + hv) * s.V * s.K;
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = v0 + 16 * warp + (lane >> 2) + 8 * h, col = 8 * n + 2 * (lane & 3);
      if (row < s.V && col < s.K) *reinterpret_cast<float2*>(dst + (size_t)row * s.K + col) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    }
}

// A thread: four numbers of a state, over the chunks of its sequence, kAhead of them on their way.
constexpr int kAhead = 8;
template <bool kBack>
__global__ void __launch_bounds__(256) join_kernel(const Args a, float* states, int tokens) {
  const Shape& s = a.s;
  const int quads = s.V * s.K / 4, per = (quads + 255) / 256, piece = (blockIdx.x % per) * 256 + threadIdx.x;
  const int hv = blockIdx.x / per % s.Hv, seq = blockIdx.x / per / s.Hv;
  if (piece >= quads) return;
  const SeqRange r = seq_range(s, seq, tokens);
  const int n = (r.t1 - r.t0 + tokens - 1) / tokens;
  const size_t mine = ((size_t)seq * s.Hv + hv) * quads + piece;
  const float* init = kBack ? a.dS_final : a.s_init;
  float4 S = init ? reinterpret_cast<const float4*>(init)[mine] : make_float4(0.f, 0.f, 0.f, 0.f);
  float4* at = reinterpret_cast<float4*>(states) + ((size_t)r.slot * s.Hv + hv) * quads + piece;
  const float* decay = a.decay + (size_t)r.slot * s.Hv + hv;
  const size_t step = (size_t)s.Hv * quads;
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float4 x[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = kBack ? n - 1 - c0 - i : c0 + i;
      if (c0 + i < n) x[i] = at[c * step], d[i] = decay[(size_t)c * s.Hv];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = kBack ? n - 1 - c0 - i : c0 + i;
      if (c0 + i < n) {
        at[c * step] = S;
        S.x = fmaf(d[i], S.x, x[i].x), S.y = fmaf(d[i], S.y, x[i].y), S.z = fmaf(d[i], S.z, x[i].z), S.w = fmaf(d[i], S.w, x[i].w);
      }
    }
  }
  float* last = kBack ? a.dS_init : a.s_final;
  if (last) reinterpret_cast<float4*>(last)[mine] = S;
}

template <bool kBack, int kTiles>
cudaError_t sums(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = (kP * kC * 64 + kP * kC * kTiles * 8) * sizeof(bf16_t) + kC * 12;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(sums_kernel<kBack, kTiles>), smem, done);
  if (e != cudaSuccess) return e;
  sums_kernel<kBack, kTiles><<<(unsigned)((size_t)a.s.slots * a.s.Hv * ((a.s.V + 63) / 64)), kThreads, smem, stream>>>(a, kBack ? a.dstates : a.states);
  return cudaGetLastError();
}

// Tokens in front of the first packed sequence and behind the last.
__global__ void gaps_kernel(const Args a, const Gaps g) {
  const int t0 = seq_range(a.s, 0, a.s.C).t0, t1 = seq_range(a.s, a.s.nseq - 1, a.s.C).t1, none = a.s.T - max(t1 - t0, 0);
  for (int i = 0; i < kGapOutputs; ++i) {
    if (!g.at[i]) continue;
    for (int n = blockIdx.x; n < none; n += gridDim.x) {
      const long long t = n < t0 ? n : n + max(t1 - t0, 0);
      for (long long w = threadIdx.x; w < g.words[i]; w += blockDim.x) g.at[i][t * g.words[i] + w] = 0;
    }
  }
}

// dg of fixed decays: a block the tokens of its part, threads the heads by turns and the tokens beside
// them; then the parts, in order and in 64 bits.
__global__ void __launch_bounds__(256) dg_part_kernel(const Args a, long long tokens) {
  __shared__ double red[256];
  const int Hv = a.s.Hv, lanes = Hv < 256 ? 256 / Hv : 1;
  const long long each = (tokens + kParts - 1) / kParts, t0 = blockIdx.x * each, t1 = min(t0 + each, tokens);
  for (int h0 = 0; h0 < Hv; h0 += 256) {
    const int h = h0 + threadIdx.x % min(Hv, 256), l = threadIdx.x / min(Hv, 256);
    double x = 0;
    if (l < lanes && h < Hv)
      for (long long t = t0 + l; t < t1; t += lanes) x += a.dg[t * Hv + h];
    red[threadIdx.x] = x;
    __syncthreads();
    if (l == 0 && h < Hv) {
      for (int i = 1; i < lanes; ++i) x += red[threadIdx.x + i * min(Hv, 256)];
      a.part[(size_t)blockIdx.x * Hv + h] = x;
    }
    __syncthreads();
  }
}
// A block: a head.
__global__ void __launch_bounds__(kParts) dg_sum_kernel(const Args a) {
  __shared__ double red[kParts / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double x = a.part[(size_t)threadIdx.x * a.s.Hv + blockIdx.x];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_down_sync(0xffffffffu, x, o);
  if (lane == 0) red[warp] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kParts / 32; ++i) x += red[i];
    a.dg_fixed[blockIdx.x] = (float)x;
  }
}

}  // namespace

cudaError_t launch_join(const Args& a, bool backward, int tokens, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((size_t)a.s.nseq * a.s.Hv * ((a.s.V * a.s.K / 4 + 255) / 256));
  if (backward)
    join_kernel<true><<<blocks, 256, 0, stream>>>(a, a.dstates, tokens);
  else
    join_kernel<false><<<blocks, 256, 0, stream>>>(a, a.states, tokens);
  return cudaGetLastError();
}
cudaError_t launch_states(const Args& a, bool backward, cudaStream_t stream) {
  cudaError_t e;
  if (backward)
    e = a.s.K <= 64 ? sums<true, 8>(a, stream) : sums<true, 16>(a, stream);
  else
    e = a.s.K <= 64 ? sums<false, 8>(a, stream) : sums<false, 16>(a, stream);
  return e == cudaSuccess ? launch_join(a, backward, a.s.C, stream) : e;
}
cudaError_t launch_gaps(const Args& a, const Gaps& g, cudaStream_t stream) {
  gaps_kernel<<<(unsigned)(a.s.T < 256 ? a.s.T : 256), 256, 0, stream>>>(a, g);
  return cudaGetLastError();
}
cudaError_t launch_dg_sums(const Args& a, cudaStream_t stream) {
  dg_part_kernel<<<kParts, 256, 0, stream>>>(a, (long long)a.s.B * a.s.T);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  dg_sum_kernel<<<a.s.Hv, kParts, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace linattn
