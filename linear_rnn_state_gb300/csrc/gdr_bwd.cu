// The gated delta rule's backward chain: the carried gradient dS of the state,
// from the last chunk to the first, and dv.
//
// One block per sequence, value head and tile of 32 value columns, as the
// forward chain (gdr_fwd.cu), whose images of q, k, T and P it reads again:
//   y   = P^T do + wr k dS1^T          (the gradient of u)
//   lam = T^T y = dv
//   dS0 = e^Gc dS1 + sum_i scale e^Gi do_i q_i^T - sum_i e^Gi lam_i k_i^T
// It leaves the images of dS1, lam and do for the gradients of q, k, g and beta
// (gdr_grad.cu). Scales come from bounds, as in the forward:
// |y| <= p_sum max|do| + k_back max|dS1|, |lam| <= t_sum max|y|,
// |dS0| <= e^Gc max|dS1| + q_sum max|do| + k_sum max|lam|.
// The next chunk's do (with its rows' factors, read straight from global
// memory) is fetched a step ahead, so its images cost no barrier.
#include "gdr_common.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

template <int P, int KP>
struct Stage {
  __half k[P * kC * KP], q[P * kC * KP];
  __half t[2 * kC * kC], p[2 * kC * kC];
  Scal scal;
  Rows rows;
};

template <typename T, int KP, int kStages>
struct BwdSmem {
  static constexpr int P = In<T>::kParts;
  Stage<P, KP> st[kStages];
  __half s[2 * kVt * KP];
  __half y[2 * kC * kVt], l[2 * kC * kVt], lw[2 * kC * kVt], dw[2][2 * kC * kVt];
  __half d[P * kC * kVt];
  float m_s[8], m_y[8], m_l[8], m_d[8];
  uint64_t bar[kStages];
};

template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = abs_max(m, x[i]);
  return m;
}

template <typename T, int KP, int kStages>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = BwdSmem<T, KP, kStages>;
  constexpr int P = In<T>::kParts, kNt = KP / 32;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wr = warp & 3, wc = warp >> 2;
  const int g4 = lane >> 2, t4 = lane & 3;
  const int vts = (a.s.V + kVt - 1) / kVt;
  const int vt = blockIdx.x % vts, hv = blockIdx.x / vts % a.s.Hv, seq = blockIdx.x / (vts * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  const SeqRange sq = seq_range(a.s, seq);
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V;

  constexpr int image = P * kC * KP * 2;
  constexpr uint32_t kBytes = 2 * image + 2 * Layout::tp_img + sizeof(Scal) + sizeof(Rows);
  // step s works on chunk n - 1 - s
  auto load = [&](int s) {
    Stage<P, KP>& st = sm.st[s % kStages];
    uint64_t* bar = &sm.bar[s % kStages];
    const size_t slot = sq.slot + (n - 1 - s), at_k = slot * a.s.Hk + hk, at_v = slot * a.s.Hv + hv;
    mbar_arrive_expect_tx(bar, kBytes);
    bulk_load(st.k, a.b.k_img + at_k * image, image, bar);
    bulk_load(&st.rows, a.b.rows + at_k, sizeof(Rows), bar);
    bulk_load(&st.scal, a.b.scal + at_v, sizeof(Scal), bar);
    bulk_load(st.p, a.b.p_img + at_v * Layout::tp_img, Layout::tp_img, bar);
    bulk_load(st.t, a.b.t_img + at_v * Layout::tp_img, Layout::tp_img, bar);
    bulk_load(st.q, a.b.q_img + at_k * image, image, bar);
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.bar[s], 1);
    wkv7::fence_mbar_init();
    for (int s = 0; s < kStages && s < n; ++s) load(s);
  }

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

  float2 d[2][2];      // do of the next step's chunk
  float df[2], eq_max = 0.f;  // scale e^G qs of its two rows, and their bound
  auto load_do = [&](int s) {
    const int c = n - 1 - s;
    const size_t slot = sq.slot + c;
    const Scal* sc = a.b.scal + slot * a.s.Hv + hv;
    const Rows* rows = a.b.rows + slot * a.s.Hk + hk;
    eq_max = sc->eq_max;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      df[h] = a.s.scale * sc->eg[i0 + 8 * h] * rows->qs[i0 + 8 * h];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int t = sq.t0 + c * kC + i0 + 8 * h, col = vt * kVt + 16 * wc + 8 * nt + 2 * t4;
        d[h][nt] = make_float2(0.f, 0.f);
        if (t < sq.t1 && col < V)
          d[h][nt] = load2(static_cast<const T*>(a.d_o) + (((size_t)sq.b * a.s.T + t) * a.s.Hv + hv) * V + col);
      }
    }
  };
  auto max_do = [&] {
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) m = abs_max(abs_max(m, d[h][nt].x), d[h][nt].y);
    m = warp_max_abs(m);
    if (lane == 0) sm.m_d[warp] = m;
  };
  float mD = 0.f, sD = 1.f, sDW = 1.f;  // of the step whose images of do are in place
  auto put_do = [&](int s) {
    mD = max_of(sm.m_d);
    sD = pow2_scale(mD), sDW = pow2_scale(mD * eq_max);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int col = 16 * wc + 8 * nt + 2 * t4;
        put2_p<P, false>(sm.d, kC, kC * kVt, i0 + 8 * h, col, d[h][nt].x * sD, d[h][nt].y * sD);
        // the factors in this order: e^G or a bound of it may be far from 1
        put2<false>(sm.dw[s & 1], kC, kC * kVt, i0 + 8 * h, col, (d[h][nt].x * df[h]) * sDW, (d[h][nt].y * df[h]) * sDW);
      }
  };
  float s_max = 0.f;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) s_max = abs_max(s_max, max_of(S[nt]));
  s_max = warp_max_abs(s_max);
  if (lane == 0) sm.m_s[warp] = s_max;
  if (n > 0) {
    load_do(0);
    max_do();
  }
  __syncthreads();
  float sS = pow2_scale(max_of(sm.m_s));
  auto put_state = [&](float scale) {
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        put2<true>(sm.s, kVt, kVt * KP, 16 * wc + g4 + 8 * h, key0 + 8 * nt + 2 * t4, S[nt][2 * h] * scale,
                   S[nt][2 * h + 1] * scale);
  };
  put_state(sS);
  if (n > 0) put_do(0);
  wkv7::fence_proxy_async_smem();
  __syncthreads();

  for (int s = 0; s < n; ++s) {
    const int c = n - 1 - s;
    Stage<P, KP>& st = sm.st[s % kStages];
    const size_t slot = sq.slot + c, at_t = (slot * a.s.Hv + hv) * vts + vt;
    if (!mbar_wait_bounded(a.status, &sm.bar[s % kStages], (s / kStages) & 1)) return;
    const Scal& sc = st.scal;
    const float mS = max_of(sm.m_s), mDo = mD, inv_s = pow2_inverse(sS), inv_d = pow2_inverse(sD),
                inv_dw = pow2_inverse(sDW);
    if (tid == 0) {
      bulk_store(a.b.ds_img + at_t * sizeof(sm.s), sm.s, sizeof(sm.s));
      bulk_store(a.b.do_img + at_t * sizeof(sm.d), sm.d, sizeof(sm.d));
      bulk_commit();
    }

    // y = P^T do + wr k dS1^T
    float x[2][4], y[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = y[nt][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<P> fk;
      Frag<2> fs;
      a_mk<P, true>(fk, st.k, kC, kC * KP, 16 * wr, 16 * kt, lane);
      b_nk<2, true>(fs, sm.s, kVt, kVt * KP, 16 * wc, 16 * kt, lane);
      mma_parts<P, 2>(x[0], x[1], fk, fs);
    }
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt >= wr) {
        Frag<2> fp;
        Frag<P> fd;
        a_km<2, true>(fp, st.p, kC, kC * kC, 16 * wr, 16 * kt, lane);
        b_kn<P, false>(fd, sm.d, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, P>(y[0], y[1], fp, fd);
      }
    const float sY = pow2_scale(sc.p_sum * mDo + sc.k_back * mS);
    float y_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = sc.wr[i0 + 8 * h] * st.rows.ks[i0 + 8 * h] * inv_s, fp = sc.inv_p * inv_d;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float y0 = fmaf(f, x[nt][2 * h], fp * y[nt][2 * h]), y1 = fmaf(f, x[nt][2 * h + 1], fp * y[nt][2 * h + 1]);
        y_max = abs_max(abs_max(y_max, y0), y1);
        put2<false>(sm.y, kC, kC * kVt, i0 + 8 * h, 16 * wc + 8 * nt + 2 * t4, y0 * sY, y1 * sY);
      }
    }
    y_max = warp_max_abs(y_max);
    if (lane == 0) sm.m_y[warp] = y_max;
    __syncthreads();
    if (s + 1 < n) load_do(s + 1);

    // lam = T^T y
    float l[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) l[nt][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt >= wr) {
        Frag<2> ft, fy;
        a_km<2, true>(ft, st.t, kC, kC * kC, 16 * wr, 16 * kt, lane);
        b_kn<2, false>(fy, sm.y, kC, kC * kVt, 16 * wc, 16 * kt, lane);
        mma_parts<2, 2>(l[0], l[1], ft, fy);
      }
    const float fl = sc.inv_t * pow2_inverse(sY), bound = sc.t_sum * max_of(sm.m_y);
    const float sL = pow2_scale(bound), sLW = pow2_scale(bound * sc.ek_max);
    float l_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w = sc.eg[i0 + 8 * h] * st.rows.ks[i0 + 8 * h];
      const int t = sq.t0 + c * kC + i0 + 8 * h;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float l0 = l[nt][2 * h] * fl, l1 = l[nt][2 * h + 1] * fl;
        l_max = abs_max(abs_max(l_max, l0), l1);
        const int col = 16 * wc + 8 * nt + 2 * t4;
        put2<false>(sm.l, kC, kC * kVt, i0 + 8 * h, col, l0 * sL, l1 * sL);
        put2<false>(sm.lw, kC, kC * kVt, i0 + 8 * h, col, (l0 * w) * sLW, (l1 * w) * sLW);
        if (t < sq.t1 && vt * kVt + col < V)
          store2(static_cast<T*>(a.dv) + (((size_t)sq.b * a.s.T + t) * a.s.Hv + hv) * V + vt * kVt + col, l0, l1);
      }
    }
    l_max = warp_max_abs(l_max);
    if (lane == 0) sm.m_l[warp] = l_max;
    if (s + 1 < n) max_do();
    wkv7::fence_proxy_async_smem();
    if (tid == 0) bulk_wait_read();  // the images of dS and do are written anew after this barrier
    __syncthreads();
    if (tid == 0) {
      bulk_store(a.b.l_img + at_t * sizeof(sm.l), sm.l, sizeof(sm.l));
      bulk_commit();
      a.b.dsl[at_t] = make_float4(inv_s, pow2_inverse(sL), inv_d, 0.f);
    }
    if (s + 1 < n) put_do(s + 1);

    // dS0
    float d1[kNt][4], d2[kNt][4];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) d1[nt][e] = d2[nt][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      Frag<2> fd, fw;
      a_km<2, false>(fd, sm.dw[s & 1], kC, kC * kVt, 16 * wc, 16 * kt, lane);
      a_km<2, false>(fw, sm.lw, kC, kC * kVt, 16 * wc, 16 * kt, lane);
#pragma unroll
      for (int nt = 0; nt < kNt; nt += 2) {
        Frag<P> fq, fk;
        b_kn<P, true>(fq, st.q, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
        b_kn<P, true>(fk, st.k, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
        mma_parts<2, P>(d1[nt], d1[nt + 1], fd, fq);
        mma_parts<2, P>(d2[nt], d2[nt + 1], fw, fk);
      }
    }
    const float inv_lw = pow2_inverse(sLW);
    s_max = 0.f;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[nt][e] = fmaf(d1[nt][e], inv_dw, fmaf(-d2[nt][e], inv_lw, sc.egc * S[nt][e]));
        s_max = abs_max(s_max, S[nt][e]);
      }
    sS = pow2_scale(sc.egc * mS + sc.q_sum * mDo + sc.k_sum * max_of(sm.m_l));
    put_state(sS);
    s_max = warp_max_abs(s_max);
    if (lane == 0) sm.m_s[warp] = s_max;
    wkv7::fence_proxy_async_smem();
    if (tid == 0) bulk_wait_read();  // the image of lam is written anew after the next step's first barrier
    __syncthreads();
    if (tid == 0 && s + kStages < n) load(s + kStages);
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

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr int kStages = sizeof(BwdSmem<T, KP, 2>) <= 227 * 1024 ? 2 : 1;  // as the forward chain
  constexpr size_t smem = sizeof(BwdSmem<T, KP, kStages>);
  auto kernel = bwd_kernel<T, KP, kStages>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * v_tiles(a.s.V)), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd(const Args& a, bool bf16, cudaStream_t stream) {
  const bool wide = padded_k(a.s.K) == 128;
  if (bf16) return wide ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
  return wide ? launch<float, 128>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace gdr
