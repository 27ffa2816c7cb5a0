// The gated delta rule's forward chain: the states from chunk to chunk, and o.
//
// Eight warps per sequence, value head and tile of 32 value columns (rows of
// the state [value][key]: they do not meet) walk the chunks in order. With T,
// P, the decays and the images of q and k from the parallel pass (gdr_prep.cu):
//   u  = T (v - e^G k S0^T)
//   S1 = e^Gc S0 + sum_j wr_j u_j k_j^T
//   o  = scale e^G q S0^T + P u
// Each is a product of a 64-row tile: the state is an accumulator in registers,
// its fp16 pair image in shared memory the operand of the next chunk. Warp
// (wr, wc) makes rows 16 wr.. of the chunk by columns 16 wc.. of the tile, and
// of the state rows 16 wc.. by a quarter of the keys. T and P have their lower
// blocks only, so a warp's work grows with wr; the two halves count wr in
// opposite order, which gives every scheduler (warp % 4) the same work.
//
// The chain from S0 to S1 is k S0^T, T r and u^T k, a barrier after each. What
// is not on it runs beside it: q S0^T next to T r, and P u with the stores of o
// after the last barrier, next to the following step's k S0^T.
//
// Scales. An image is written before anyone can know its largest value without
// one more barrier, so it takes a bound instead: |v - e^G k S0| <= max|v| +
// k_read max|S0|, |u| <= t_sum max|r|, |S1| <= e^Gc max|S0| + k_write max|u|,
// where the right sides hold the true maxima of the step before, published at
// the barrier that publishes the image itself. Bounds are loose by 2^10 at most
// in a well-posed chunk, which the pairs' 2^-39 floor leaves room for.
#include "gdr_chain.cuh"

namespace gdr {
namespace {

template <int KP>
struct alignas(128) FwdTile {
  __half s[2 * kVt * KP];
  __half r[2 * kC * kVt], u[2 * kC * kVt], w[2 * kC * kVt];
  float m_s[8], m_r[8], m_u[8], m_v[8];
};
template <typename T, int KP, int kTiles>
struct FwdSmem {
  Images<In<T>::kParts, KP> im;
  FwdTile<KP> tile[kTiles];
};

template <typename T, int KP, int kTiles, bool kSave>
__global__ void __launch_bounds__(kTiles * kGroupThreads, kTiles == 1 && sizeof(FwdSmem<T, KP, 1>) <= 113 * 1024 ? 2 : 1)
    fwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = FwdSmem<T, KP, kTiles>;
  constexpr int P = In<T>::kParts, kNt = KP / 32;  // n8 tiles of a warp's quarter of the keys
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + kTiles - 1) / kTiles;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  const SeqRange sq = seq_range(a.s, seq);
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V;
  const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads, lane = tid & 31, warp = tid >> 5;
  const Filler<P, KP> fill{sm.im, a, sq.slot, 1, n, hk, hv, min(kTiles, vts - set * kTiles)};
  if (threadIdx.x == 0) fill.start();
  __syncthreads();
  const int vt = set * kTiles + group;
  if (vt >= vts) return;
  Images<P, KP>& im = sm.im;
  FwdTile<KP>& tl = sm.tile[group];
  const int wc = warp >> 2, wr = wc ? 3 - (warp & 3) : warp & 3, g4 = lane >> 2, t4 = lane & 3;
  const int bar = group + 1;

  // the warp's part of the state: value rows 16 wc + g4 (+ 8), keys key0 + 8 nt + 2 t4 (+ 1)
  const int key0 = wr * (KP / 4), i0 = 16 * wr + g4;
  const size_t state_at = ((size_t)seq * a.s.Hv + hv) * V;
  float S[kNt][4];
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = vt * kVt + 16 * wc + g4 + 8 * h, key = key0 + 8 * nt + 2 * t4;
      float2 x = make_float2(0.f, 0.f);
      if (a.s_init && row < V && key < K) x = *reinterpret_cast<const float2*>(a.s_init + (state_at + row) * K + key);
      S[nt][2 * h] = x.x, S[nt][2 * h + 1] = x.y;
    }

  // v of the next chunk: rows 16 wr + g4 (+ 8), columns 16 wc + 8 nt + 2 t4 (+ 1)
  const T* v_at = static_cast<const T*>(a.v) + sq.b * a.s.v_b + (size_t)hv * V + vt * kVt;
  float2 v[2][2];
  auto load_v = [&](int c, float2 (&x)[2][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int t = sq.t0 + c * kC + i0 + 8 * h, col = 16 * wc + 8 * nt + 2 * t4;
        x[h][nt] = make_float2(0.f, 0.f);
        if (t < sq.t1 && vt * kVt + col < V) x[h][nt] = load2(v_at + t * a.s.v_t + col);
      }
  };
  auto max_v = [&](const float2 (&x)[2][2]) {
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) m = abs_max(abs_max(m, x[h][nt].x), x[h][nt].y);
    m = warp_max_abs(m);
    if (lane == 0) tl.m_v[warp] = m;
  };
  load_v(0, v);
  ask_rows(v_at, a.s.v_t, sq.t0 + kC, sq.t1, tid);
  ask_rows(v_at, a.s.v_t, sq.t0 + 2 * kC, sq.t1, tid);
  max_v(v);

  float s_max = 0.f;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) s_max = abs_max(s_max, max_of(S[nt]));
  s_max = warp_max_abs(s_max);
  if (lane == 0) tl.m_s[warp] = s_max;
  group_barrier(bar);
  float sS = pow2_scale(max_of(tl.m_s));
  auto put_state = [&](float scale) {
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        put2<true>(tl.s, kVt, kVt * KP, 16 * wc + g4 + 8 * h, key0 + 8 * nt + 2 * t4, S[nt][2 * h] * scale,
                   S[nt][2 * h + 1] * scale);
  };
  put_state(sS);
  if (kSave) wkv7::fence_proxy_async_smem();
  group_barrier(bar);

  for (int c = 0; c < n; ++c) {
    const size_t slot = sq.slot + c, at_t = (slot * a.s.Hv + hv) * vts + vt;
    const uint32_t use = c & 1;
    float2 vn[2][2];
    if (c + 1 < n) load_v(c + 1, vn);
    ask_rows(v_at, a.s.v_t, sq.t0 + (c + 3) * kC, sq.t1, tid);
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (c >> 1) & 1)) return;
    if (kSave && tid == 0) {
      bulk_store(a.b.s_img + at_t * sizeof(tl.s), tl.s, sizeof(tl.s));
      bulk_commit();
    }
    const Scal& sc = im.scal[use];
    const Rows& rows = im.rows[use];
    const __half* kimg = im.k[use];
    const float mS = max_of(tl.m_s), mV = max_of(tl.m_v), inv_s = pow2_inverse(sS);

    // r = v - e^G k S0^T
    float x[2][4];
    {
      float y[2][4];
      zero(x), zero(y);
#pragma unroll
      for (int kt = 0; kt < KP / 16; ++kt) {
        Frag<P> fk;
        Frag<2> fs;
        a_mk<P, true>(fk, kimg, kC, kC * KP, 16 * wr, 16 * kt, lane);
        b_nk<2, true>(fs, tl.s, kVt, kVt * KP, 16 * wc, 16 * kt, lane);
        if (kt & 1)
          mma_parts<P, 2>(y[0], y[1], fk, fs);
        else
          mma_parts<P, 2>(x[0], x[1], fk, fs);
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] += y[nt][e];
    }
    const float sR = pow2_scale(mV + sc.k_read * mS);
    float r_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = -sc.eg[i0 + 8 * h] * rows.ks[i0 + 8 * h] * inv_s;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float r0 = fmaf(f, x[nt][2 * h], v[h][nt].x), r1 = fmaf(f, x[nt][2 * h + 1], v[h][nt].y);
        r_max = abs_max(abs_max(r_max, r0), r1);
        put2<false>(tl.r, kC, kC * kVt, i0 + 8 * h, 16 * wc + 8 * nt + 2 * t4, r0 * sR, r1 * sR);
      }
    }
    r_max = warp_max_abs(r_max);
    if (lane == 0) tl.m_r[warp] = r_max;
    group_barrier(bar);
    if (tid == 0 && c > 0 && fill.last(im.done_p)) fill.p(c);  // every warp is past P u of the step before

    // u = T r, and q S0^T beside it
    float u[2][4], xq[2][4];
    zero(u), zero(xq);
    if (!mbar_wait_bounded(a.status, &im.full_t, use)) return;
    if (!mbar_wait_bounded(a.status, &im.full_q, use)) return;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      if (kt <= wr) {
        Frag<2> ft, fr;
        a_tri(ft, im.t, wr, kt, lane);
        b_kn<2, false>(fr, tl.r, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, 2>(u[0], u[1], ft, fr);
      }
#pragma unroll
      for (int q = kt * (KP / 64); q < (kt + 1) * (KP / 64); ++q) {
        Frag<P> fq;
        Frag<2> fs;
        a_mk<P, true>(fq, im.q, kC, kC * KP, 16 * wr, 16 * q, lane);
        b_nk<2, true>(fs, tl.s, kVt, kVt * KP, 16 * wc, 16 * q, lane);
        mma_parts<P, 2>(xq[0], xq[1], fq, fs);
      }
    }
    const float ft = sc.inv_t * pow2_inverse(sR), bound = sc.t_sum * max_of(tl.m_r);
    const float sU = pow2_scale(bound), sW = pow2_scale(bound * sc.wk_max);
    float u_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w = sc.wr[i0 + 8 * h] * rows.ks[i0 + 8 * h];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float u0 = u[nt][2 * h] * ft, u1 = u[nt][2 * h + 1] * ft;
        u_max = abs_max(abs_max(u_max, u0), u1);
        const int col = 16 * wc + 8 * nt + 2 * t4;
        put2<false>(tl.u, kC, kC * kVt, i0 + 8 * h, col, u0 * sU, u1 * sU);
        put2<false>(tl.w, kC, kC * kVt, i0 + 8 * h, col, (u0 * w) * sW, (u1 * w) * sW);
      }
    }
    u_max = warp_max_abs(u_max);
    if (lane == 0) tl.m_u[warp] = u_max;
    if (kSave) {
      wkv7::fence_proxy_async_smem();
      if (tid == 0) bulk_wait_read();  // the state's image is written anew after this barrier
    }
    group_barrier(bar);
    if (tid == 0 && c + 1 < n && fill.last(im.done_t)) {
      fill.t(c + 1);
      fill.q(c + 1);
      fill.ask(c + 3);
    }
    if (kSave && tid == 0) {
      bulk_store(a.b.u_img + at_t * sizeof(tl.u), tl.u, sizeof(tl.u));
      bulk_commit();
      a.b.su[at_t] = make_float2(inv_s, pow2_inverse(sU));
    }

    // S1 = e^Gc S0 + (wr u)^T k
    {
      float d[kNt][4];
      zero(d);
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        Frag<2> fw;
        a_km<2, false>(fw, tl.w, kC, kC * kVt, 16 * wc, 16 * kt, lane);
#pragma unroll
        for (int nt = 0; nt < kNt; nt += 2) {
          Frag<P> fk;
          b_kn<P, true>(fk, kimg, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
          mma_parts<2, P>(d[nt], d[nt + 1], fw, fk);
        }
      }
      const float inv_w = pow2_inverse(sW);
      s_max = 0.f;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[nt][e] = fmaf(d[nt][e], inv_w, sc.egc * S[nt][e]);
          s_max = abs_max(s_max, S[nt][e]);
        }
    }
    sS = pow2_scale(sc.egc * mS + sc.k_write * max_of(tl.m_u));
    put_state(sS);
    s_max = warp_max_abs(s_max);
    if (lane == 0) tl.m_s[warp] = s_max;
    if (c + 1 < n) max_v(vn);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) v[h][nt] = vn[h][nt];
    const float fo = sc.inv_p * pow2_inverse(sU);
    const float fq[2] = {a.s.scale * sc.eg[i0] * rows.qs[i0] * inv_s, a.s.scale * sc.eg[i0 + 8] * rows.qs[i0 + 8] * inv_s};
    if (kSave) {
      wkv7::fence_proxy_async_smem();
      if (tid == 0) bulk_wait_read();  // the image of u is written anew after the next step's first barrier
    }
    group_barrier(bar);
    if (tid == 0 && c + 2 < n && fill.last(im.done_k[use])) fill.k(c + 2);

    // o = scale e^G q S0^T + P u
    float o[2][4];
    zero(o);
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt <= wr) {
        Frag<2> fp, fu;
        a_tri(fp, im.p, wr, kt, lane);
        b_kn<2, false>(fu, tl.u, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, 2>(o[0], o[1], fp, fu);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = sq.t0 + c * kC + i0 + 8 * h;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int col = vt * kVt + 16 * wc + 8 * nt + 2 * t4;
        if (t < sq.t1 && col < V)
          store2(static_cast<T*>(a.o) + (((size_t)sq.b * a.s.T + t) * a.s.Hv + hv) * V + col,
                 fmaf(fq[h], xq[nt][2 * h], fo * o[nt][2 * h]), fmaf(fq[h], xq[nt][2 * h + 1], fo * o[nt][2 * h + 1]));
      }
    }
  }
  if (kSave && tid == 0) bulk_wait_all();

  if (a.s_final) {
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = vt * kVt + 16 * wc + g4 + 8 * h, key = key0 + 8 * nt + 2 * t4;
        if (row < V && key < K)
          *reinterpret_cast<float2*>(a.s_final + (state_at + row) * K + key) = make_float2(S[nt][2 * h], S[nt][2 * h + 1]);
      }
  }
}

template <typename T, int KP, int kTiles, bool kSave>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(FwdSmem<T, KP, kTiles>);
  auto kernel = fwd_kernel<T, KP, kTiles, kSave>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int sets = (v_tiles(a.s.V) + kTiles - 1) / kTiles;
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), kTiles * kGroupThreads, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int KP, bool kSave>
cudaError_t pick(const Args& a, cudaStream_t s) {
  return two_tiles(a.s) ? launch<T, KP, 2, kSave>(a, s) : launch<T, KP, 1, kSave>(a, s);
}
template <typename T>
cudaError_t pick(const Args& a, bool save, cudaStream_t s) {
  if (padded_k(a.s.K) == 128) return save ? pick<T, 128, true>(a, s) : pick<T, 128, false>(a, s);
  return save ? pick<T, 64, true>(a, s) : pick<T, 64, false>(a, s);
}

}  // namespace

cudaError_t launch_fwd(const Args& a, bool bf16, bool save, cudaStream_t stream) {
  return bf16 ? pick<__nv_bfloat16>(a, save, stream) : pick<float>(a, save, stream);
}

}  // namespace gdr
