// What the gated delta rule's chunks need before the states are known, for
// every chunk of 64 tokens and key head at once.
//
// With G the running sum of g in the chunk and r_ij = e^(G_i - G_j) (j <= i):
//   L_ij = beta_j r_ij k_i.k_j  (j < i),    T = (I + L)^-1
//   P_ij = scale beta_j r_ij q_i.k_j  (j <= i)
// so that with S0 the state before the chunk u = T (v - e^G S0 k) and
// o = scale e^G S0 q + P u. The kernel writes q, k, T and P as the images that
// the chain kernels copy into shared memory, with their scales and the tokens'
// factors (gdr_launch.h, Rows and Scal).
//
// The decay ratios. G is summed in double and kept as two floats, so that no
// difference of it is rounded. g below -200 counts as -200 (e^-200 is 0 in fp32
// either way), which makes -inf a reset of the state instead of inf - inf.
// Where G spans at most 60 in the chunk, r_ij is the product of a row's and a
// column's factor, two multiplications an element; elsewhere it is the
// exponential of the difference, which strong decays cannot overflow.
//
// T in fp32: the four diagonal 16 x 16 blocks by forward substitution, a column
// a thread, then blocks joined two by two, [T1 0; -T2 L21 T1 T2], 16 and then
// 32 wide.
#include "gdr_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kLx = 36;
constexpr int kLd = 68;  // row stride of the fp32 64 x 64 tiles: rows stay 16-byte aligned

template <typename T, int KP>
struct alignas(128) PrepSmem {
  static constexpr int P = In<T>::kParts;
  __half q[P * kC * KP], k[P * kC * KP];
  float L[kC * kLd];            // L, and then T in its place
  float x[32 * kLx];            // L21 T1 in between
  __half out[2 * kTriPart];     // the image of P, then of T
  Rows rows;
  Scal scal;
  float pa[kC], la[kC], cb[kC];  // scale qs fa, ks fa, beta ks fb: P_ij = (q_i.k_j) pa_i cb_j where G is near
  float red[8];
};

// One of q, k: 64 rows into an image, each row scaled by a power of two. A lane
// has eight columns of every kPass-th row; all its loads are issued at once.
template <typename T, int KP>
struct RowLoader {
  static constexpr int P = In<T>::kParts, kLanes = KP / 8, kPass = kThreads / kLanes, kOwn = kC / kPass;
  uint4 raw[kOwn][P];
  __device__ __forceinline__ void load(const T* src, long long stride_t, int len, int K, int tid) {
    const int cl = tid % kLanes;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int row = tid / kLanes + i * kPass;
      const bool in = row < len && cl * 8 < K;
#pragma unroll
      for (int p = 0; p < P; ++p)
        raw[i][p] = in ? reinterpret_cast<const uint4*>(src + (size_t)row * stride_t + cl * 8)[p] : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8], int i) const {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t w[4] = {raw[i][p].x, raw[i][p].y, raw[i][p].z, raw[i][p].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if constexpr (P == 1)
          x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        else
          x[4 * p + e] = __uint_as_float(w[e]);
    }
  }
  // The row's largest magnitude, over its lanes.
  __device__ __forceinline__ float largest(int i) const {
    uint32_t m = 0, lo = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t w[4] = {raw[i][p].x, raw[i][p].y, raw[i][p].z, raw[i][p].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m = max(m, w[e] & 0x7FFFFFFFu);  // magnitudes are ordered as their bits
        if constexpr (P == 1) lo = max(lo, (w[e] << 16) & 0x7FFFFFFFu);
      }
    }
    if constexpr (P == 1) m = max(m & 0xFFFF0000u, lo);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return __uint_as_float(m);
  }
  __device__ __forceinline__ void store(__half* image, float* inv, float* rn, int l2norm, int tid) const {
    const int cl = tid % kLanes;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int row = tid / kLanes + i * kPass;
      const float sc = pow2_scale(largest(i));
      float x[8], r = 1.f;
      values(x, i);
      if (l2norm) {
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s2 = fmaf(x[e], x[e], s2);
        r = 1.f / sqrtf(wkv7::group_allreduce<kLanes>(s2) + 1e-6f);
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2<P>(x[2 * e] * sc, x[2 * e + 1] * sc, hi[e], lo[e]);
      const int at = img(kC, row, cl * 8);
      *reinterpret_cast<uint4*>(image + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (P == 2) *reinterpret_cast<uint4*>(image + kC * KP + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (cl == 0) inv[row] = pow2_inverse(sc) * r, rn[row] = r;
    }
  }
};

// Largest of the block's values; every thread gets it. `red` is reused: a
// barrier stands before and after.
__device__ __forceinline__ float block_max(float x, float* red, int tid) {
  x = warp_max_abs(x);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = x;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = abs_max(m, red[w]);
  return m;
}

// X[i][j] = sign sum_m A[i][m] B[m][j] for the thread's R rows from r and C
// columns from c, m < N; rows of A and B 16-byte aligned.
template <int R, int C, int N>
__device__ __forceinline__ void small_product(float (&x)[R][C], const float* A, int lda, const float* B, int ldb, int r, int c) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) x[i][j] = 0.f;
#pragma unroll 4
  for (int m = 0; m < N; m += 4) {
    float4 a[R];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(A + (r + i) * lda + m);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float b[C];
      if constexpr (C == 4) {
        const float4 v = *reinterpret_cast<const float4*>(B + (m + q) * ldb + c);
        b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(B + (m + q) * ldb + c);
        b[0] = v.x, b[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float s = q == 0 ? a[i].x : q == 1 ? a[i].y : q == 2 ? a[i].z : a[i].w;
#pragma unroll
        for (int j = 0; j < C; ++j) x[i][j] = fmaf(s, b[j], x[i][j]);
      }
    }
  }
}

template <typename T, int KP>
__global__ void __launch_bounds__(kThreads, 4) prep_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  PrepSmem<T, KP>& sm = *reinterpret_cast<PrepSmem<T, KP>*>(raw);
  constexpr int P = In<T>::kParts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / a.s.Hk, hk = blockIdx.x % a.s.Hk;
  if (a.small) grid_go();
  ChunkAt c;
  if (!chunk_at(a.s, slot, c)) return;
  const size_t at_k = (size_t)slot * a.s.Hk + hk;
  const int g4 = lane >> 2, t4 = lane & 3, group = a.s.Hv / a.s.Hk;
  float gin[2] = {0.f, 0.f}, bin[2] = {0.f, 0.f};  // warp 0: g and beta of tokens 2 lane, 2 lane + 1
  auto load_gates = [&](int hv) {
    if (warp == 0)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * lane + e < c.len) {
          const size_t at = ((size_t)c.b * a.s.T + c.t0 + 2 * lane + e) * a.s.Hv + hv;
          gin[e] = a.g[at], bin[e] = a.beta[at];
        }
  };
  load_gates(hk * group);
  {
    const T* q = static_cast<const T*>(a.q) + c.b * a.s.q_b + c.t0 * a.s.q_t + hk * a.s.K;
    const T* k = static_cast<const T*>(a.k) + c.b * a.s.k_b + c.t0 * a.s.k_t + hk * a.s.K;
    RowLoader<T, KP> lq, lk;
    lq.load(q, a.s.q_t, c.len, a.s.K, tid);
    if (P == 1) lk.load(k, a.s.k_t, c.len, a.s.K, tid);  // fp32 rows are too many registers for both at once
    lq.store(sm.q, sm.rows.qs, sm.rows.rq, a.s.l2norm, tid);
    if (P == 2) lk.load(k, a.s.k_t, c.len, a.s.K, tid);
    lk.store(sm.k, sm.rows.ks, sm.rows.rk, a.s.l2norm, tid);
  }
  wkv7::fence_proxy_async_smem();
  __syncthreads();
  constexpr int image = P * kC * KP * 2;
  if (tid == 0) {
    bulk_store(a.b.q_img + at_k * image, sm.q, image);
    bulk_store(a.b.k_img + at_k * image, sm.k, image);
    bulk_commit();
  }

  // q k^T and k k^T, the 16 rows of a warp against the columns up to them
  float qk[8][4], kk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) qk[n][e] = kk[n][e] = 0.f;
#pragma unroll
  for (int kt = 0; kt < KP / 16; ++kt) {
    Frag<P> fq, fk;
    a_mk<P>(fq, sm.q, kC, kC * KP, 16 * warp, 16 * kt, lane);
    a_mk<P>(fk, sm.k, kC, kC * KP, 16 * warp, 16 * kt, lane);
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (n <= warp) {
        Frag<P> fb;
        b_nk<P>(fb, sm.k, kC, kC * KP, 16 * n, 16 * kt, lane);
        mma_parts<P, P>(qk[2 * n], qk[2 * n + 1], fq, fb);
        mma_parts<P, P>(kk[2 * n], kk[2 * n + 1], fk, fb);
      }
  }

#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * warp + g4 + 8 * (e >> 1);
      if (8 * n + 2 * t4 + (e & 1) == i) sm.rows.qk[i] = qk[n][e] * sm.rows.qs[i] * sm.rows.ks[i];
    }
  for (int hg = 0; hg < group; ++hg) {
    const int hv = hk * group + hg;
    const size_t at_v = (size_t)slot * a.s.Hv + hv;
    if (warp == 0) {  // the running sum of g, two tokens a lane
      const double x[2] = {gin[0] < -200.f ? -200.f : gin[0], gin[1] < -200.f ? -200.f : gin[1]};
      double s = x[0] + x[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      const double G[2] = {s - x[1], s}, Gc = __shfl_sync(0xffffffffu, s, 31);
      float top = fmaxf((float)G[0], (float)G[1]), low = fminf((float)G[0], (float)G[1]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
      }
      const float mid = 0.5f * (top + low);
      float bk = 0.f, qm = 0.f, km = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const float b = bin[e], hi = (float)G[e], lo = (float)(G[e] - hi), th = (float)(Gc - G[e]), tl = (float)(Gc - G[e] - th);
        const float mh = (float)(G[e] - mid), ml = (float)(G[e] - mid - mh);
        const float eg = expf(hi) * (1.f + lo), w = expf(th) * (1.f + tl) * b, fa = expf(mh) * (1.f + ml), fb = expf(-mh) * (1.f - ml);
        const float qs = sm.rows.qs[i], ks = sm.rows.ks[i];
        Scal& o = sm.scal;
        o.beta[i] = b, o.gh[i] = hi, o.gl[i] = lo, o.eg[i] = eg, o.fa[i] = fa, o.fb[i] = fb;
        o.ek[i] = eg * ks, o.wk[i] = w * ks, o.eq[i] = a.s.scale * eg * qs;
        sm.pa[i] = a.s.scale * qs * fa, sm.la[i] = ks * fa, sm.cb[i] = b * ks * fb;
        bk = abs_max(bk, b * ks), qm = abs_max(qm, qs), km = abs_max(km, ks);
      }
      bk = warp_max_abs(bk), qm = warp_max_abs(qm), km = warp_max_abs(km);
      // the largest e^(G_i - G_j), j <= i, is 1 unless some g is positive
      const bool grows = __any_sync(0xffffffffu, x[0] > 0 || x[1] > 0);
      if (lane == 31) {
        const float ch = (float)Gc, cl = (float)(Gc - ch), r = grows ? expf(top - low) : 1.f, sr = fabsf(a.s.scale) * r;
        Scal& o = sm.scal;
        o.egc = expf(ch) * (1.f + cl);
        o.near = top - low <= kNear ? 1.f : 0.f;
        o.fb_max = sr * bk, o.eb_max = r * bk, o.f_max = sr * qm, o.e_max = r * km;
      }
    }
    __syncthreads();
    if (hg + 1 < group) load_gates(hv + 1);
    float p[8][4], pm = 0.f;
    if (sm.scal.near != 0.f) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n < 2 * warp + 2) {
          const float2 cb = *reinterpret_cast<const float2*>(sm.cb + 8 * n + 2 * t4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = 16 * warp + g4 + 8 * h, j = 8 * n + 2 * t4;
            const float pa = sm.pa[i], la = sm.la[i];
            float x0 = qk[n][2 * h] * pa * cb.x, x1 = qk[n][2 * h + 1] * pa * cb.y;
            float y0 = kk[n][2 * h] * la * cb.x, y1 = kk[n][2 * h + 1] * la * cb.y;
            if (n >= 2 * warp) {  // the diagonal block
              x0 = j <= i ? x0 : 0.f, x1 = j + 1 <= i ? x1 : 0.f;
              y0 = j < i ? y0 : 0.f, y1 = j + 1 < i ? y1 : 0.f;
            }
            p[n][2 * h] = x0, p[n][2 * h + 1] = x1;
            pm = abs_max(abs_max(pm, x0), x1);
            *reinterpret_cast<float2*>(sm.L + i * kLd + j) = make_float2(y0, y1);
          }
        }
    } else {
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n < 2 * warp + 2)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * warp + g4 + 8 * (e >> 1), j = 8 * n + 2 * t4 + (e & 1);
            float r = 0.f;
            if (j <= i) r = expf((sm.scal.gh[i] - sm.scal.gh[j]) + (sm.scal.gl[i] - sm.scal.gl[j])) * (sm.scal.beta[j] * sm.rows.ks[j]);
            p[n][e] = j <= i ? a.s.scale * (sm.rows.qs[i] * qk[n][e]) * r : 0.f;
            pm = abs_max(pm, p[n][e]);
            sm.L[i * kLd + j] = j < i ? sm.rows.ks[i] * kk[n][e] * r : 0.f;
          }
    }
    pm = block_max(pm, sm.red, tid);
    const float ps = pow2_scale(pm);
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (n < 2 * warp + 2)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          put2_tri(sm.out, 16 * warp + g4 + 8 * h, 8 * n + 2 * t4, p[n][2 * h] * ps, p[n][2 * h + 1] * ps);
    wkv7::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(a.b.p_img + at_v * Layout::tp_img, sm.out, Layout::tp_img);
      bulk_commit();
    }

    // T in the place of L: diagonal blocks, then the blocks left of them
    if (tid < kC) {
      float* D = sm.L + (tid & 48) * (kLd + 1);
      const int j = tid & 15;
      float col[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x0 = i == j ? 1.f : 0.f, x1 = 0.f;
#pragma unroll
        for (int m = 0; m < i; m += 4) {
          const float4 l = *reinterpret_cast<const float4*>(D + i * kLd + m);
          x0 = fmaf(-l.x, col[m], x0);
          if (m + 1 < i) x1 = fmaf(-l.y, col[m + 1], x1);
          if (m + 2 < i) x0 = fmaf(-l.z, col[m + 2], x0);
          if (m + 3 < i) x1 = fmaf(-l.w, col[m + 3], x1);
        }
        col[i] = i < j ? 0.f : x0 + x1;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) D[i * kLd + j] = col[i];
    }
    __syncthreads();
    {
      const int pair = tid >> 6, r = ((tid >> 3) & 7) * 2, cc = (tid & 7) * 2;
      float* T1 = sm.L + 32 * pair * (kLd + 1);
      float *L21 = T1 + 16 * kLd, *X = sm.x + 16 * pair * kLx;
      float x[2][2];
      small_product<2, 2, 16>(x, L21, kLd, T1, kLd, r, cc);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<float2*>(X + (r + i) * kLx + cc) = make_float2(x[i][0], x[i][1]);
      __syncthreads();
      small_product<2, 2, 16>(x, L21 + 16, kLd, X, kLx, r, cc);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<float2*>(L21 + (r + i) * kLd + cc) = make_float2(-x[i][0], -x[i][1]);
    }
    __syncthreads();
    {
      const int r = (tid >> 3) * 2, cc = (tid & 7) * 4;
      float *L21 = sm.L + 32 * kLd, x[2][4];
      // the 16 x 16 block above the diagonal of T1 and of T2 still holds what L's buffer held
      *reinterpret_cast<float4*>(sm.L + 32 * (tid >> 6) * (kLd + 1) + ((tid >> 2) & 15) * kLd + 16 + (tid & 3) * 4) =
          make_float4(0.f, 0.f, 0.f, 0.f);
      __syncthreads();
      small_product<2, 4, 32>(x, L21, kLd, sm.L, kLd, r, cc);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(sm.x + (r + i) * kLx + cc) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
      __syncthreads();
      small_product<2, 4, 32>(x, L21 + 32, kLd, sm.x, kLx, r, cc);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(L21 + (r + i) * kLd + cc) = make_float4(-x[i][0], -x[i][1], -x[i][2], -x[i][3]);
    }
    __syncthreads();
    // two neighbours of a row at a time: ten blocks of 128 pairs
    float2 tv[10];
    float tm = 0.f;
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const int ib = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3, jb = b - ib * (ib + 1) / 2;
      tv[b] = *reinterpret_cast<const float2*>(sm.L + (16 * ib + (tid >> 3)) * kLd + 16 * jb + 2 * (tid & 7));
      tm = abs_max(abs_max(tm, tv[b].x), tv[b].y);
    }
    if (tid == 0) bulk_wait_read();  // P is out
    tm = block_max(tm, sm.red, tid);
    const float ts = pow2_scale(tm);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const int ib = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3, jb = b - ib * (ib + 1) / 2;
      put2_tri(sm.out, 16 * ib + (tid >> 3), 16 * jb + 2 * (tid & 7), tv[b].x * ts, tv[b].y * ts);
    }
    if (tid == 0) {
      sm.scal.inv_p = pow2_inverse(ps), sm.scal.inv_t = pow2_inverse(ts);
    }
    wkv7::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(a.b.t_img + at_v * Layout::tp_img, sm.out, Layout::tp_img);
      bulk_store(a.b.scal + at_v, &sm.scal, sizeof(Scal));
      if (hg == 0) bulk_store(a.b.rows + at_k, &sm.rows, sizeof(Rows));
      bulk_commit();
      bulk_wait_read();  // T and the scalars are out
    }
    if (hg + 1 < group) __syncthreads();
  }
  if (tid == 0) bulk_wait_all();
}

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(PrepSmem<T, KP>);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(prep_kernel<T, KP>), smem, done);
  if (e != cudaSuccess) return e;
  prep_kernel<T, KP><<<(unsigned)((size_t)a.s.slots * a.s.Hk), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep(const Args& a, bool bf16, cudaStream_t stream) {
  const bool wide = padded_k(a.s.K) == 128;
  if (bf16) return wide ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
  return wide ? launch<float, 128>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace gdr
