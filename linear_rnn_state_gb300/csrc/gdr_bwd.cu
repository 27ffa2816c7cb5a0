// The gated delta rule's backward chain: the carried gradient dS of the state,
// from the last chunk to the first, and dv.
//
// Eight warps per sequence, value head and tile of 32 value columns, as in the
// forward chain (gdr_fwd.cu), whose images of q, k, T and P it reads again:
//   y   = P^T do + wr k dS1^T          (the gradient of u)
//   lam = T^T y = dv
//   dS0 = e^Gc dS1 + sum_i scale e^Gi do_i q_i^T - sum_i e^Gi lam_i k_i^T
// It leaves the images of dS1, lam and do for the gradients of q, k, g and beta
// (gdr_grad.cu). Scales come from bounds, as in the forward:
// |y| <= p_sum max|do| + k_back max|dS1|, |lam| <= t_sum max|y|,
// |dS0| <= e^Gc max|dS1| + q_sum max|do| + k_sum max|lam|.
// The next chunk's do is fetched a step ahead and its image written before the
// step's last barrier; that of scale e^G do, needed late, at the step's start.
#include "gdr_chain.cuh"

namespace gdr {
namespace {

template <int P, int KP>
struct alignas(128) BwdTile {
  __half s[2 * kVt * KP];
  __half y[2 * kC * kVt], lw[2 * kC * kVt], dw[2 * kC * kVt];
  __half d[P * kC * kVt];
  float m_s[8], m_y[8], m_l[8], m_d[8];
};
template <typename T, int KP, int kTiles>
struct BwdSmem {
  Images<In<T>::kParts, KP> im;
  BwdTile<In<T>::kParts, KP> tile[kTiles];
};

template <typename T, int KP, int kTiles>
__global__ void __launch_bounds__(kTiles * kGroupThreads, kTiles == 1 && sizeof(BwdSmem<T, KP, 1>) <= 113 * 1024 ? 2 : 1)
    bwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = BwdSmem<T, KP, kTiles>;
  constexpr int P = In<T>::kParts, kNt = KP / 32;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + kTiles - 1) / kTiles;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  const SeqRange sq = seq_range(a.s, seq);
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V;
  const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads, lane = tid & 31, warp = tid >> 5;
  // step s works on chunk n - 1 - s
  const Filler<P, KP> fill{sm.im, a, sq.slot + n - 1, -1, n, hk, hv, min(kTiles, vts - set * kTiles)};
  if (threadIdx.x == 0) fill.start();
  __syncthreads();
  const int vt = set * kTiles + group;
  if (vt >= vts) return;
  Images<P, KP>& im = sm.im;
  BwdTile<P, KP>& tl = sm.tile[group];
  const int wc = warp >> 2, wr = wc ? 3 - (warp & 3) : warp & 3, g4 = lane >> 2, t4 = lane & 3;
  const int bar = group + 1;

  const int key0 = wr * (KP / 4), i0 = 16 * wr + g4;
  const size_t state_at = ((size_t)seq * a.s.Hv + hv) * V;
  float S[kNt][4];
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = vt * kVt + 16 * wc + g4 + 8 * h, key = key0 + 8 * nt + 2 * t4;
      float2 x = make_float2(0.f, 0.f);
      if (a.dS_final && row < V && key < K) x = *reinterpret_cast<const float2*>(a.dS_final + (state_at + row) * K + key);
      S[nt][2 * h] = x.x, S[nt][2 * h + 1] = x.y;
    }

  // do of a chunk: rows 16 wr + g4 (+ 8), columns 16 wc + 8 nt + 2 t4 (+ 1)
  const long long row_t = (long long)a.s.Hv * V;
  const T* do_at = static_cast<const T*>(a.d_o) + (size_t)sq.b * a.s.T * row_t + (size_t)hv * V + vt * kVt;
  T* dv_at = static_cast<T*>(a.dv) + (size_t)sq.b * a.s.T * row_t + (size_t)hv * V + vt * kVt;
  float2 d[2][2];
  auto load_do = [&](int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int t = sq.t0 + c * kC + i0 + 8 * h, col = 16 * wc + 8 * nt + 2 * t4;
        d[h][nt] = make_float2(0.f, 0.f);
        if (t < sq.t1 && vt * kVt + col < V) d[h][nt] = load2(do_at + t * row_t + col);
      }
  };
  auto ask_do = [&](int c) {
    if (c >= 0) ask_rows(do_at, row_t, sq.t0 + c * kC, sq.t1, tid);
  };
  auto max_do = [&] {
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) m = abs_max(abs_max(m, d[h][nt].x), d[h][nt].y);
    m = warp_max_abs(m);
    if (lane == 0) tl.m_d[warp] = m;
  };
  float mD = 0.f, sD = 1.f;  // of the do whose image is in place
  auto put_do = [&] {
    mD = max_of(tl.m_d);
    sD = pow2_scale(mD);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        put2_p<P, false>(tl.d, kC, kC * kVt, i0 + 8 * h, 16 * wc + 8 * nt + 2 * t4, d[h][nt].x * sD, d[h][nt].y * sD);
  };
  float s_max = 0.f;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) s_max = abs_max(s_max, max_of(S[nt]));
  s_max = warp_max_abs(s_max);
  if (lane == 0) tl.m_s[warp] = s_max;
  if (n > 0) {
    load_do(n - 1);
    ask_do(n - 2);
    ask_do(n - 3);
    max_do();
  }
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
  if (n > 0) put_do();
  wkv7::fence_proxy_async_smem();
  group_barrier(bar);

  for (int s = 0; s < n; ++s) {
    const int c = n - 1 - s;
    const size_t slot = sq.slot + c, at_t = (slot * a.s.Hv + hv) * vts + vt;
    const uint32_t use = s & 1;
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (s >> 1) & 1)) return;
    const Scal& sc = im.scal[use];
    const Rows& rows = im.rows[use];
    const __half* kimg = im.k[use];
    const float mS = max_of(tl.m_s), mDo = mD, inv_s = pow2_inverse(sS), inv_d = pow2_inverse(sD);
    if (tid == 0) {
      bulk_store(a.b.ds_img + at_t * sizeof(tl.s), tl.s, sizeof(tl.s));
      bulk_store(a.b.do_img + at_t * sizeof(tl.d), tl.d, sizeof(tl.d));
      bulk_commit();
    }

    // y = P^T do + wr k dS1^T
    float x[2][4], y[2][4];
    zero(x), zero(y);
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<P> fk;
      Frag<2> fs;
      a_mk<P, true>(fk, kimg, kC, kC * KP, 16 * wr, 16 * kt, lane);
      b_nk<2, true>(fs, tl.s, kVt, kVt * KP, 16 * wc, 16 * kt, lane);
      mma_parts<P, 2>(x[0], x[1], fk, fs);
    }
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt >= wr) {
        Frag<2> fp;
        Frag<P> fd;
        a_tri_t(fp, im.p, kt, wr, lane);
        b_kn<P, false>(fd, tl.d, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, P>(y[0], y[1], fp, fd);
      }
    const float sY = pow2_scale(sc.p_sum * mDo + sc.k_back * mS), sDW = pow2_scale(mDo * sc.eq_max);
    float y_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = sc.wr[i0 + 8 * h] * rows.ks[i0 + 8 * h] * inv_s, fp = sc.inv_p * inv_d;
      const float df = a.s.scale * sc.eg[i0 + 8 * h] * rows.qs[i0 + 8 * h];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int col = 16 * wc + 8 * nt + 2 * t4;
        const float y0 = fmaf(f, x[nt][2 * h], fp * y[nt][2 * h]), y1 = fmaf(f, x[nt][2 * h + 1], fp * y[nt][2 * h + 1]);
        y_max = abs_max(abs_max(y_max, y0), y1);
        put2<false>(tl.y, kC, kC * kVt, i0 + 8 * h, col, y0 * sY, y1 * sY);
        put2<false>(tl.dw, kC, kC * kVt, i0 + 8 * h, col, (d[h][nt].x * df) * sDW, (d[h][nt].y * df) * sDW);
      }
    }
    y_max = warp_max_abs(y_max);
    if (lane == 0) tl.m_y[warp] = y_max;
    group_barrier(bar);
    if (tid == 0 && s + 1 < n && fill.last(im.done_p)) fill.p(s + 1);
    if (s + 1 < n) load_do(c - 1);
    ask_do(c - 3);

    // lam = T^T y
    float l[2][4];
    zero(l);
    if (!mbar_wait_bounded(a.status, &im.full_t, use)) return;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt >= wr) {
        Frag<2> ft, fy;
        a_tri_t(ft, im.t, kt, wr, lane);
        b_kn<2, false>(fy, tl.y, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, 2>(l[0], l[1], ft, fy);
      }
    const float fl = sc.inv_t * pow2_inverse(sY), bound = sc.t_sum * max_of(tl.m_y);
    const float sL = pow2_scale(bound), sLW = pow2_scale(bound * sc.ek_max);
    float l_max = 0.f;
    __half* l_at = reinterpret_cast<__half*>(a.b.l_img + at_t * (2 * kC * kVt * 2));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w = sc.eg[i0 + 8 * h] * rows.ks[i0 + 8 * h];
      const int t = sq.t0 + c * kC + i0 + 8 * h;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float l0 = l[nt][2 * h] * fl, l1 = l[nt][2 * h + 1] * fl;
        l_max = abs_max(abs_max(l_max, l0), l1);
        const int col = 16 * wc + 8 * nt + 2 * t4;
        put2<false>(tl.lw, kC, kC * kVt, i0 + 8 * h, col, (l0 * w) * sLW, (l1 * w) * sLW);
        put2<false>(l_at, kC, kC * kVt, i0 + 8 * h, col, l0 * sL, l1 * sL);  // in global memory
        if (t < sq.t1 && vt * kVt + col < V) store2(dv_at + t * row_t + col, l0, l1);
      }
    }
    l_max = warp_max_abs(l_max);
    if (lane == 0) tl.m_l[warp] = l_max;
    if (s + 1 < n) max_do();
    if (tid == 0) {
      a.b.dsl[at_t] = make_float4(inv_s, pow2_inverse(sL), inv_d, 0.f);
      bulk_wait_read();  // the images of dS and do are written anew after this barrier
    }
    group_barrier(bar);
    if (tid == 0 && s + 1 < n && fill.last(im.done_t)) {
      fill.t(s + 1);
      fill.ask(s + 3);
    }

    // dS0
    {
      float d1[kNt][4], d2[kNt][4];
      zero(d1), zero(d2);
      if (!mbar_wait_bounded(a.status, &im.full_q, use)) return;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        Frag<2> fd, fw;
        a_km<2, false>(fd, tl.dw, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        a_km<2, false>(fw, tl.lw, kC, kC * kVt, 16 * wc, 16 * kt, lane);
#pragma unroll
        for (int nt = 0; nt < kNt; nt += 2) {
          Frag<P> fq, fk;
          b_kn<P, true>(fq, im.q, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
          b_kn<P, true>(fk, kimg, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
          mma_parts<2, P>(d1[nt], d1[nt + 1], fd, fq);
          mma_parts<2, P>(d2[nt], d2[nt + 1], fw, fk);
        }
      }
      const float inv_dw = pow2_inverse(sDW), inv_lw = pow2_inverse(sLW);
      s_max = 0.f;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[nt][e] = fmaf(d1[nt][e], inv_dw, fmaf(-d2[nt][e], inv_lw, sc.egc * S[nt][e]));
          s_max = abs_max(s_max, S[nt][e]);
        }
    }
    sS = pow2_scale(sc.egc * mS + sc.q_sum * mDo + sc.k_sum * max_of(tl.m_l));
    put_state(sS);
    if (s + 1 < n) put_do();
    s_max = warp_max_abs(s_max);
    if (lane == 0) tl.m_s[warp] = s_max;
    wkv7::fence_proxy_async_smem();
    group_barrier(bar);
    if (tid == 0 && s + 1 < n && fill.last(im.done_k[use])) {
      fill.q(s + 1);
      if (s + 2 < n) fill.k(s + 2);
    }
  }
  if (tid == 0) bulk_wait_all();

  if (a.dS_init) {
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = vt * kVt + 16 * wc + g4 + 8 * h, key = key0 + 8 * nt + 2 * t4;
        if (row < V && key < K)
          *reinterpret_cast<float2*>(a.dS_init + (state_at + row) * K + key) = make_float2(S[nt][2 * h], S[nt][2 * h + 1]);
      }
  }
}

template <typename T, int KP, int kTiles>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(BwdSmem<T, KP, kTiles>);
  auto kernel = bwd_kernel<T, KP, kTiles>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int sets = (v_tiles(a.s.V) + kTiles - 1) / kTiles;
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), kTiles * kGroupThreads, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int KP>
cudaError_t pick(const Args& a, cudaStream_t s) {
  return two_tiles(a.s) ? launch<T, KP, 2>(a, s) : launch<T, KP, 1>(a, s);
}
template <typename T>
cudaError_t pick(const Args& a, cudaStream_t s) {
  return padded_k(a.s.K) == 128 ? pick<T, 128>(a, s) : pick<T, 64>(a, s);
}

}  // namespace

cudaError_t launch_bwd(const Args& a, bool bf16, cudaStream_t stream) {
  return bf16 ? pick<__nv_bfloat16>(a, stream) : pick<float>(a, stream);
}

}  // namespace gdr
