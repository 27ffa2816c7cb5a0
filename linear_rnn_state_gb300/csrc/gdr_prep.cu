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
// The decay ratios. G is summed and kept as an unrounded sum of two floats, so
// that no difference of it is rounded (doubles took 3600 of a chunk's 31000
// cycles). g below -200 counts as -200 (e^-200 is 0 in fp32
// either way), which makes -inf a reset of the state instead of inf - inf.
// Where G spans at most 60 in the chunk, r_ij is the product of a row's and a
// column's factor, two multiplications an element; elsewhere it is the
// exponential of the difference, which strong decays cannot overflow.
//
// T in fp32: the four diagonal 16 x 16 blocks by forward substitution, a column
// a thread, then blocks joined two by two, [T1 0; -T2 L21 T1 T2], 16 and then
// 32 wide, the products of the joins on the tensor cores in fp16 pairs (as fp32
// multiply-adds they took 7000 of a chunk's 31000 cycles).
//
// A block of four warps has a chunk of a key head: 54 KB in and out (64 keys,
// bfloat16; 87 KB fp32) in some 25000 cycles of small dependent parts, so what
// bounds it is their latency against the blocks that an SM has room for (four; at
// most 128 registers a thread, 47 KB). Measured: 4 x 4096 tokens x 32 heads of 64,
// bfloat16, 148 us, 3.0 TB/s; 8 x 4096 x 12 x 64 fp32 148 us, 3.6 TB/s; 65536 x 40
// x 64 fp32 930 us, 3.8 TB/s. (Five blocks, with q k^T made after T in the
// registers of k k^T and images in the places of what they follow: 157 us.)
#include "gdr_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kLd = 68;  // row stride of the fp32 64 x 64 tiles: rows stay 16-byte aligned

template <typename T, int KP>
struct alignas(128) PrepSmem {
  static constexpr int P = In<T>::kParts;
  __half q[P * kC * KP], k[P * kC * KP];
  float L[kC * kLd];            // L, and then T in its place
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
        for (int e = 0; e < 8; ++e) s2 = fmaf(x[e] * kSmall, x[e] * kSmall, s2);
        s2 = wkv7::group_allreduce<kLanes>(s2) + kSmallEps;
        r = rsqrtf(s2);
        r = kSmall * fmaf(0.5f * r, fmaf(-s2 * r, r, 1.f), r);  // a Newton step: the last bits
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

// A number as the unrounded sum of two floats.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two sum2(Two a, Two b) {
  const float s = __fadd_rn(a.h, b.h), c = __fsub_rn(s, a.h);
  const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.h, __fsub_rn(s, c)), __fsub_rn(b.h, c)), __fadd_rn(a.l, b.l));
  const float h = __fadd_rn(s, e);
  return {h, __fsub_rn(e, __fsub_rn(h, s))};
}

// Operands of 16 x 16 pieces of fp32 tiles, as pairs at a common scale: load,
// largest of the warp, split.
struct Raw {
  float v[8];
  // A[m][k] = s[m0 + m][k0 + k]
  __device__ __forceinline__ void a(const float* s, int m0, int k0, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = *reinterpret_cast<const float2*>(s + (m0 + (lane >> 2) + 8 * (i & 1)) * kLd + k0 + 2 * (lane & 3) + 8 * (i >> 1));
      v[2 * i] = x.x, v[2 * i + 1] = x.y;
    }
  }
  // B[k][n] = s[k0 + k][n0 + n]
  __device__ __forceinline__ void b(const float* s, int k0, int n0, int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = s[(k0 + 2 * (lane & 3) + (i & 1) + 8 * ((i >> 1) & 1)) * kLd + n0 + (lane >> 2) + 8 * (i >> 2)];
  }
  __device__ __forceinline__ float largest() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
  }
  __device__ __forceinline__ void split(Frag<2>& f, float s) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<2>(v[2 * i] * s, v[2 * i + 1] * s, f.h[i], f.l[i]);
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

// Blocks that an SM's shared memory takes; registers are shared out for as many.
template <typename T, int KP>
constexpr int kBlocks = 227 * 1024 / (sizeof(PrepSmem<T, KP>) + 1024) < 4 ? 227 * 1024 / (sizeof(PrepSmem<T, KP>) + 1024) : 4;

// kOne: each key head has one value head, and the grams end with its P and L.
template <typename T, int KP, bool kOne>
__global__ void __launch_bounds__(kThreads, kBlocks<T, KP>) prep_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  PrepSmem<T, KP>& sm = *reinterpret_cast<PrepSmem<T, KP>*>(raw);
  constexpr int P = In<T>::kParts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x % a.s.Hk;
  int slot = blockIdx.x / a.s.Hk;
  if (a.segn) slot = slot / a.segn * ((a.s.T + kC - 1) / kC) + a.seg0 + slot % a.segn;
  if (a.small) grid_go();
  ChunkAt c;
  if (!chunk_at(a.s, slot, c)) return;
  const size_t at_k = (size_t)slot * a.s.Hk + hk;
  const int g4 = lane >> 2, t4 = lane & 3, group = kOne ? 1 : a.s.Hv / a.s.Hk;
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
      const float x[2] = {gin[0] < -200.f ? -200.f : gin[0], gin[1] < -200.f ? -200.f : gin[1]};
      Two s = sum2({x[0], 0.f}, {x[1], 0.f});
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two y = {__shfl_up_sync(0xffffffffu, s.h, o), __shfl_up_sync(0xffffffffu, s.l, o)};
        if (lane >= o) s = sum2(s, y);
      }
      const Two G[2] = {sum2(s, {-x[1], 0.f}), s}, Gc = {__shfl_sync(0xffffffffu, s.h, 31), __shfl_sync(0xffffffffu, s.l, 31)};
      float top = fmaxf(G[0].h, G[1].h), low = fminf(G[0].h, G[1].h);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
      }
      const float mid = 0.5f * (top + low);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const Two tail = sum2(Gc, {-G[e].h, -G[e].l}), m = sum2(G[e], {-mid, 0.f});
        const float b = bin[e], eg = expf(G[e].h) * (1.f + G[e].l), w = expf(tail.h) * (1.f + tail.l) * b;
        const float fa = expf(m.h) * (1.f + m.l), fb = expf(-m.h) * (1.f - m.l);
        const float qs = sm.rows.qs[i], ks = sm.rows.ks[i];
        Scal& o = sm.scal;
        o.beta[i] = b, o.gh[i] = G[e].h, o.gl[i] = G[e].l, o.eg[i] = eg, o.fa[i] = fa, o.fb[i] = fb;
        o.ek[i] = eg * ks, o.wk[i] = w * ks, o.eq[i] = a.s.scale * eg * qs;
        sm.pa[i] = a.s.scale * qs * fa, sm.la[i] = ks * fa, sm.cb[i] = b * ks * fb;
      }
      if (lane == 31) {
        sm.scal.egc = expf(Gc.h) * (1.f + Gc.l);
        sm.scal.near = top - low <= kNear ? 1.f : 0.f;
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
    if (warp < 2) {  // 16 wide: T21 = -(T2 L21) T1 of rows and columns 32 warp ..
      float* T1 = sm.L + 32 * warp * (kLd + 1);
      Raw ra, rb, rc;
      ra.a(T1, 16, 16, lane), rb.b(T1, 16, 0, lane), rc.b(T1, 0, 0, lane);
      const float sa = pow2_scale(warp_max_abs(ra.largest())), sb = pow2_scale(warp_max_abs(rb.largest())),
                  sc = pow2_scale(warp_max_abs(rc.largest()));
      Frag<2> fa, fb, fc;
      ra.split(fa, sa), rb.split(fb, sb), rc.split(fc, sc);
      float x[2][4], y[2][4];
      mma_parts_first<2, 2>(x[0], x[1], fa, fb);
      const float sx = pow2_scale(warp_max(x));
      to_a(fa, x[0], x[1], sx);
      mma_parts_first<2, 2>(y[0], y[1], fa, fc);
      const float f = -pow2_inverse(sa) * pow2_inverse(sb) * pow2_inverse(sx) * pow2_inverse(sc);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(T1 + (16 + g4 + 8 * h) * kLd + 8 * n + 2 * t4) = make_float2(f * y[n][2 * h], f * y[n][2 * h + 1]);
    }
    __syncthreads();
    {  // 32 wide: a warp has 16 rows (block mb) of T2 L21, and 16 columns (nh) of its product with T1
      const int mb = warp >> 1, nh = warp & 1;
      float* L21 = sm.L + 32 * kLd;
      float x[4][4], y[2][4];
      float inv_x;
      {
        Raw ra[2], rb[2][2];
        float ma = 0.f, mx = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k <= mb) {
            ra[k].a(L21, 16 * mb, 32 + 16 * k, lane);
            ma = fmaxf(ma, ra[k].largest());
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              rb[k][n].b(L21, 16 * k, 16 * n, lane);
              mx = fmaxf(mx, rb[k][n].largest());
            }
          }
        const float sa = pow2_scale(warp_max_abs(ma)), sb = pow2_scale(warp_max_abs(mx));
        inv_x = pow2_inverse(sa) * pow2_inverse(sb);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k <= mb) {
            Frag<2> fa, fb[2];
            ra[k].split(fa, sa);
#pragma unroll
            for (int n = 0; n < 2; ++n) rb[k][n].split(fb[n], sb);
            if (k == 0)
              mma_row<2, true>(x, fa, fb);
            else
              mma_row<2>(x, fa, fb);
          }
      }
      const float sx = pow2_scale(warp_max(x));
      Raw rc[2];
      float mc = 0.f;
#pragma unroll
      for (int k = 1; k >= 0; --k)
        if (k >= nh) rc[k].b(sm.L, 16 * k, 16 * nh, lane), mc = fmaxf(mc, rc[k].largest());
      const float sc = pow2_scale(warp_max_abs(mc)), f = -inv_x * pow2_inverse(sx) * pow2_inverse(sc);
#pragma unroll
      for (int k = 1; k >= 0; --k)
        if (k >= nh) {
          Frag<2> fx, fc;
          to_a(fx, x[2 * k], x[2 * k + 1], sx);
          rc[k].split(fc, sc);
          if (k == 1)
            mma_parts_first<2, 2>(y[0], y[1], fx, fc);
          else
            mma_parts<2, 2>(y[0], y[1], fx, fc);
        }
      __syncthreads();  // every warp has read L21
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(L21 + (16 * mb + g4 + 8 * h) * kLd + 16 * nh + 8 * n + 2 * t4) = make_float2(f * y[n][2 * h], f * y[n][2 * h + 1]);
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
  // begun beside the chain of the segment before: over only when that is, for the next chain
  if (a.seg0 && blockIdx.x == 0) grid_wait();
}

// Zeros where no sequence is, contiguous in each output: before the first and behind
// the last. (In warps of the chains that have nothing else to do it took no launch,
// 2 us of a packed call, but code between theirs: 5 % of every backward chain.)
__global__ void __launch_bounds__(256) gaps_kernel(const Args a, const Gaps g) {
  const int2 in = covered(a.s);
  const long long first = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
#pragma unroll
  for (int b = 0; b < 5; ++b) {
    const long long w = g.words[b];
    for (long long i = first; i < in.x * w; i += step) g.at[b][i] = 0;
    for (long long i = in.y * w + first; i < a.s.T * w; i += step) g.at[b][i] = 0;
  }
  grid_wait();  // over only when the kernel before is
}

template <typename T, int KP, bool kOne>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(PrepSmem<T, KP>);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(prep_kernel<T, KP, kOne>), smem, done);
  if (e != cudaSuccess) return e;
  const size_t slots = a.segn ? (size_t)a.s.B * a.segn : a.s.slots;
  return launch_after(a.seg0 > 0, prep_kernel<T, KP, kOne>, (unsigned)(slots * a.s.Hk), kThreads, smem, stream, a);
}

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  return a.s.Hv == a.s.Hk ? launch<T, KP, true>(a, stream) : launch<T, KP, false>(a, stream);
}

}  // namespace

cudaError_t launch_gaps(const Args& a, const Gaps& g, cudaStream_t stream) {
  return launch_after(true, gaps_kernel, 152u, 256u, 0, stream, a, g);
}

cudaError_t launch_prep(const Args& a, bool bf16, cudaStream_t stream) {
  const bool wide = padded_k(a.s.K) == 128;
  if (bf16) return wide ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
  return wide ? launch<float, 128>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace gdr
