// Linear attention with a decay: the rows of o, dq, dk and dv of every chunk, all chunks at once.
//
// Each is a masked product of the chunk's own tokens and one with a state. With G the running sum of the
// chunk's log decays, Gc the whole sum, S the state before the chunk and D the gradient of the state after it:
//   o_i  = sum_{j<=i} scale e^{G_i - G_j} (q_i.k_j) v_j   + scale e^{G_i} S q_i
//   dq_i = sum_{j<=i} scale e^{G_i - G_j} (do_i.v_j) k_j  + scale e^{G_i} S^T do_i
//   dv_j = sum_{i>=j} scale e^{G_i - G_j} (k_j.q_i) do_i  + e^{Gc - G_j} D k_j
//   dk_j = sum_{i>=j} scale e^{G_i - G_j} (v_j.do_i) q_i  + e^{Gc - G_j} D^T v_j
// A log decay g_t moves whatever passes it: pairs j < t <= i of the chunk, the state's part that is read
// from t on, what is written before t and read after the chunk, and what passes the whole chunk,
//   dg_t = sum_{j<t<=i} X_ij + sum_{i>=t} q_i.(scale e^{G_i} S^T do_i) + sum_{j<t} k_j.(e^{Gc - G_j} D^T v_j)
//          + e^{Gc} <S, D>,   X_ij = scale e^{G_i - G_j} (q_i.k_j)(do_i.v_j),
// all of them sums: no differences of large ones.
//
// For fp32 heads above 64: three parts of the four tiles of a chunk (393 KB at 128) would not fit the shared memory that
// tcgen05 reads, so products are mma.sync's, of 64 tokens and 64 columns at a time. Bound by latency with eight warps
// an SM: 2 x 4096 x 16 x 128 takes 269 us for o, 266 dv, 475 dq and dg, 361 dk.
#include "linattn_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256, kC = kCF32, kP = In<float>::kParts;
enum Mode { kO, kDv, kDq, kDk };

__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }

struct Tokens {  // a chunk's rows of one head
  const float* p;
  long long stride;
  int cols;
};

// What a block keeps in shared memory; D: the (padded) size of the products' inner dimension.
struct Layout {
  __host__ __device__ static constexpr size_t b(int D) { return (size_t)kP * kC * D * 2; }
  __host__ __device__ static constexpr size_t x(int D) { return 2 * b(D); }
  __host__ __device__ static constexpr size_t s(int D) { return x(D) + (size_t)kP * kC * 64 * 2; }
  __host__ __device__ static constexpr size_t g(int D) { return s(D) + (size_t)kP * 64 * D * 2; }
  __host__ __device__ static constexpr size_t size(int D) { return g(D) + kC * 8 + kC * 4 + 7 * kC * 4; }
};

// rows += a b^T of the warp's 16 rows and the columns that the mask leaves it.
template <bool kUpper>
__device__ __forceinline__ void scores(float (&x)[8][4], const bf16_t* as, const bf16_t* bs, int D, int Dp, int warp, int lane) {
  zero(x);
  for (int k0 = 0; k0 < D; k0 += 16) {
    Frag<kP> fa;
    a_mk(fa, as, kC, kC * Dp, 16 * warp, k0, lane);
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (kUpper ? n >= warp : n <= warp) {
        Frag<kP> fb;
        b_nk(fb, bs, kC, kC * Dp, 16 * n, k0, lane);
        mma_added(x[2 * n], x[2 * n + 1], fa, fb);
      }
  }
}

// A block: a chunk and a value head (o, dv), or a key head with all its value heads (dq, dk). 16 tokens and half of each
// 64 columns of the output a warp; kSlices x 64 columns. (One block's tiles fill shared memory. Both warps of 16 tokens make
// their scores: four warps that made each once took 436 us for 327 for o at 2 x 4096 x 16 x 128.)
template <int kMode, int kSlices>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Args a) {
  constexpr bool kUpper = kMode == kDv || kMode == kDk, kKeys = kMode == kDq || kMode == kDk;  // kKeys: the output is a key's
  using L = Layout;
  extern __shared__ __align__(128) unsigned char smem[];
  const Shape& s = a.s;
  const int D = kKeys ? s.V : s.K, Dx = kKeys ? s.K : s.V, Dp = (D + 63) & ~63;
  bf16_t* as = reinterpret_cast<bf16_t*>(smem);
  bf16_t* bs = reinterpret_cast<bf16_t*>(smem + L::b(Dp));
  bf16_t* xs = reinterpret_cast<bf16_t*>(smem + L::x(Dp));
  bf16_t* ss = reinterpret_cast<bf16_t*>(smem + L::s(Dp));
  float2* G = reinterpret_cast<float2*>(smem + L::g(Dp));
  float* w = reinterpret_cast<float*>(G + kC);
  float* red = w + kC;  // [7][kC]: dg of the warps' rows, the rows' terms by halves, the state's
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5 & 3, half = tid >> 7, gr = lane >> 2, tq = lane & 3;
  const int heads = kKeys ? s.Hk : s.Hv, head = blockIdx.x % heads, slot = blockIdx.x / heads, group = s.Hv / s.Hk;
  ChunkAt c;
  if (!chunk_at(s, slot, kC, c)) return;
  const size_t tok = (size_t)c.b * s.T + c.t0;
  float acc[kSlices][8][4];
#pragma unroll
  for (int i = 0; i < kSlices; ++i) zero(acc[i]);
  const int hk = kKeys ? head : head / group;
  const Tokens q{static_cast<const float*>(a.q) + c.b * s.q_b + c.t0 * s.q_t + (size_t)hk * s.K, s.q_t, s.K};
  const Tokens k{static_cast<const float*>(a.k) + c.b * s.k_b + c.t0 * s.k_t + (size_t)hk * s.K, s.k_t, s.K};
  for (int hv = kKeys ? hk * group : head; hv < (kKeys ? (hk + 1) * group : head + 1); ++hv) {
    const Tokens v{static_cast<const float*>(a.v) + c.b * s.v_b + c.t0 * s.v_t + (size_t)hv * s.V, s.v_t, s.V};
    const Tokens d{static_cast<const float*>(a.d_o) + (tok * s.Hv + hv) * s.V, (long long)s.Hv * s.V, s.V};
    const Tokens&ta = kMode == kO ? q : kMode == kDv ? k : kMode == kDq ? d : v;
    const Tokens&tb = kMode == kO ? k : kMode == kDv ? q : kMode == kDq ? v : d;
    const Tokens&tx = kMode == kO ? v : kMode == kDv ? d : kMode == kDq ? k : q;
    const float* state = (kUpper ? a.dstates : a.states) + ((size_t)slot * s.Hv + hv) * s.V * s.K;
    const bool dg = kKeys && a.dg;
    __syncthreads();  // the head before is done with shared memory
    if (tid < 32) {
      running_sums<2>(G, s.fixed ? a.g + hv : a.g + tok * s.Hv + hv, s.fixed ? 0 : s.Hv, c.len, lane);
      __syncwarp();
#pragma unroll
      for (int j = lane; j < kC; j += 32) w[j] = kUpper ? expf(minus(G[kC - 1], G[j])) : s.scale * expf(G[j].x + G[j].y);
    }
    float qk[8][4];
    if (kMode == kDq && dg) {
      const int Kp = (s.K + 63) & ~63;
      if (Kp <= Dp) {
        fill_tile<kP, kC>(as, q.p, q.stride, c.len, s.K, nullptr, tid, kThreads);
        fill_tile<kP, kC>(bs, k.p, k.stride, c.len, s.K, nullptr, tid, kThreads);
        __syncthreads();
        scores<false>(qk, as, bs, s.K, Kp, warp, lane);
      } else {  // in two halves
        for (int h = 0; h < 2; ++h) {
          fill_tile<kP, kC>(as, q.p + 64 * h, q.stride, c.len, h ? s.K - 64 : 64, nullptr, tid, kThreads);
          fill_tile<kP, kC>(bs, k.p + 64 * h, k.stride, c.len, h ? s.K - 64 : 64, nullptr, tid, kThreads);
          __syncthreads();
          float part[8][4];
          scores<false>(part, as, bs, h ? s.K - 64 : 64, 64, warp, lane);
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) qk[n][e] = h ? qk[n][e] + part[n][e] : part[n][e];
          __syncthreads();
        }
      }
      __syncthreads();
    }
    fill_tile<kP, kC>(as, ta.p, ta.stride, c.len, D, nullptr, tid, kThreads);
    fill_tile<kP, kC>(bs, tb.p, tb.stride, c.len, D, nullptr, tid, kThreads);
    __syncthreads();
    Frag<kP> pf[4];
    {
      float x[8][4];
      scores<kUpper>(x, as, bs, D, Dp, warp, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 16 * warp + gr + 8 * h;
        const float2 Gi = G[i];
        const float sc = s.scale;
        float run = 0.f;  // of the row's X so far
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * n + 2 * tq + e;
            const bool keep = kUpper ? j >= i : j <= i;
            y[e] = keep ? x[n][2 * h + e] * sc * expf(kUpper ? minus(G[j], Gi) : minus(Gi, G[j])) : 0.f;
            x[n][2 * h + e] = y[e];
          }
          if (kMode == kDq && dg) {  // qk: the sums over j' < j of X_ij', where j <= i
            const int j = 8 * n + 2 * tq;
            const float z0 = j < i ? y[0] * qk[n][2 * h] : 0.f, z1 = j + 1 < i ? y[1] * qk[n][2 * h + 1] : 0.f;
            float p = z0 + z1, up = __shfl_up_sync(0xffffffffu, p, 1, 4);
            if (tq >= 1) p += up;
            up = __shfl_up_sync(0xffffffffu, p, 2, 4);
            if (tq >= 2) p += up;
            up = __shfl_up_sync(0xffffffffu, p, 1, 4);
            const float before = run + (tq ? up : 0.f);
            qk[n][2 * h] = j <= i ? before : 0.f;
            qk[n][2 * h + 1] = j + 1 <= i ? before + z0 : 0.f;
            run += __shfl_sync(0xffffffffu, p, 3, 4);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) to_a(pf[n], x[2 * n], x[2 * n + 1]);
    }
    if (kMode == kDq && dg) {  // over the warp's rows
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = qk[n][e] + qk[n][2 + e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (gr == 0 && half == 0) red[warp * kC + 8 * n + 2 * tq + e] = x;
        }
    }
    float dots[2] = {0.f, 0.f}, whole = 0.f;
#pragma unroll
    for (int sl = 0; sl < kSlices; ++sl) {
      const int x0 = 64 * sl, xn = min(64, Dx - x0);
      __syncthreads();
      fill_tile<kP, kC>(xs, tx.p + x0, tx.stride, c.len, xn, nullptr, tid, kThreads);
      // the state's slice: rows of values and 64 keys (kKeys), or 64 rows and all keys
      const int rows = kKeys ? Dp : 64, shift = kKeys || Dp == 64 ? 3 : 4, total = rows << shift;
      constexpr int kBatch = 4;  // loads on their way together
      for (int i0 = tid; i0 < total; i0 += kBatch * kThreads) {
        float f[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b * kThreads, r = i >> shift, col = (i - (r << shift)) * 8;
          const int sr = kKeys ? r : x0 + r, scol = kKeys ? x0 + col : col;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[b][e] = 0.f;
          if (i < total && sr < s.V && scol < s.K) load8(f[b], state + (size_t)sr * s.K + scol);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b * kThreads, r = i >> shift, col = (i - (r << shift)) * 8;
          if (i >= total) break;
          const int sr = kKeys ? r : x0 + r, scol = kKeys ? x0 + col : col;
          if (kMode == kDq && dg && sr < s.V && scol < s.K) {
            float f2[8];
            load8(f2, a.dstates + ((size_t)slot * s.Hv + hv) * s.V * s.K + (size_t)sr * s.K + scol);
#pragma unroll
            for (int e = 0; e < 8; ++e) whole = fmaf(f[b][e], f2[e], whole);
          }
          put8<kP>(ss + at(rows, r, col), 64 * Dp, f[b]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if ((n >> 1) == half && 16 * n < xn) {
          float y0[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
          for (int k0 = 0; k0 < D; k0 += 16) {
            Frag<kP> fa;
            Frag<kP> fb;
            a_mk(fa, as, kC, kC * Dp, 16 * warp, k0, lane);
            if (kKeys)
              b_kn(fb, ss, Dp, 64 * Dp, 16 * n, k0, lane);
            else
              b_nk(fb, ss, 64, 64 * Dp, 16 * n, k0, lane);
            mma_added(y0, y1, fa, fb);
          }
          const float w0 = w[16 * warp + gr], w1 = w[16 * warp + gr + 8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y0[e] *= e < 2 ? w0 : w1, y1[e] *= e < 2 ? w0 : w1;
            acc[sl][2 * n][e] += y0[e], acc[sl][2 * n + 1][e] += y1[e];
          }
          if (dg) {  // q.(the state's part of dq), or k.(that of dk)
            const Tokens& t = kMode == kDq ? q : k;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = 16 * warp + gr + 8 * h, col = x0 + 16 * n + 2 * tq;
              if (row < c.len) {
                const float* p = t.p + row * t.stride + col;
                if (col < Dx) {
                  const float2 z = load2(p);
                  dots[h] = fmaf(z.x, y0[2 * h], fmaf(z.y, y0[2 * h + 1], dots[h]));
                }
                if (col + 8 < Dx) {
                  const float2 z = load2(p + 8);
                  dots[h] = fmaf(z.x, y1[2 * h], fmaf(z.y, y1[2 * h + 1], dots[h]));
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (kUpper ? j >= warp : j <= warp) {
              Frag<kP> fx;
              b_kn(fx, xs, kC, kC * 64, 16 * n, 16 * j, lane);
              mma_added(acc[sl][2 * n], acc[sl][2 * n + 1], pf[j], fx);
            }
        }
    }
    if (dg) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = dots[h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (tq == 0) red[(4 + half) * kC + 16 * warp + gr + 8 * h] = x;
      }
      if (kMode == kDq) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, o);
        if (lane == 0) red[6 * kC + 4 * half + warp] = whole;
      }
      __syncthreads();
      if (tid < 32) {  // two tokens a lane
        float* out = a.dg + tok * s.Hv + hv;
        const float x0 = red[4 * kC + 2 * lane] + red[5 * kC + 2 * lane], x1 = red[4 * kC + 2 * lane + 1] + red[5 * kC + 2 * lane + 1];
        float run = x0 + x1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = kMode == kDq ? __shfl_down_sync(0xffffffffu, run, o) : __shfl_up_sync(0xffffffffu, run, o);
          if (kMode == kDq ? lane + o < 32 : lane >= o) run += y;
        }
        float other = kMode == kDq ? __shfl_down_sync(0xffffffffu, run, 1) : __shfl_up_sync(0xffffffffu, run, 1);
        if (lane == (kMode == kDq ? 31 : 0)) other = 0.f;
        const float y0 = kMode == kDq ? run : other, y1 = kMode == kDq ? other + x1 : other + x0;
        float pass = 0.f;
        if (kMode == kDq) {
#pragma unroll
          for (int i = 0; i < 8; ++i) pass += red[6 * kC + i];
          pass *= expf(G[kC - 1].x + G[kC - 1].y);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * lane + e;
          if (t < c.len) {
            float x = (e ? y1 : y0) + pass;
            if (kMode == kDq)
              x += (red[t] + red[kC + t]) + (red[2 * kC + t] + red[3 * kC + t]);
            else
              x += out[(size_t)t * s.Hv];
            out[(size_t)t * s.Hv] = x;
          }
        }
      }
    }
  }
  float* out = static_cast<float*>(kMode == kO ? a.o : kMode == kDv ? a.dv : kMode == kDq ? a.dq : a.dk);
  out += (tok * heads + head) * Dx;
#pragma unroll
  for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * warp + gr + 8 * h, col = 64 * sl + 8 * n + 2 * tq;
        if ((n >> 2) == half && row < c.len && col < Dx)
          *reinterpret_cast<float2*>(out + (size_t)row * heads * Dx + col) = make_float2(acc[sl][n][2 * h], acc[sl][n][2 * h + 1]);
      }
}

template <int kMode, int kSlices>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr bool kKeys = kMode == kDq || kMode == kDk;
  const int D = kKeys ? a.s.V : a.s.K;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(rows_kernel<kMode, kSlices>), Layout::size(kMaxDim), done);
  if (e != cudaSuccess) return e;
  rows_kernel<kMode, kSlices><<<(unsigned)((size_t)a.s.slots * (kKeys ? a.s.Hk : a.s.Hv)), kThreads, Layout::size((D + 63) & ~63), stream>>>(a);
  return cudaGetLastError();
}
template <int kMode>
cudaError_t pick(const Args& a, cudaStream_t stream) {
  const int Dx = kMode == kDq || kMode == kDk ? a.s.K : a.s.V;
  return Dx <= 64 ? launch<kMode, 1>(a, stream) : launch<kMode, 2>(a, stream);
}

}  // namespace

cudaError_t launch_rows_o(const Args& a, cudaStream_t stream) { return pick<kO>(a, stream); }
cudaError_t launch_rows_grad(const Args& a, cudaStream_t stream) {
  cudaError_t e = pick<kDv>(a, stream);
  if (e == cudaSuccess) e = pick<kDq>(a, stream);
  if (e == cudaSuccess) e = pick<kDk>(a, stream);
  return e;
}

}  // namespace linattn
