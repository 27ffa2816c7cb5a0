// The gated delta rule's forward chain: the states from chunk to chunk, and o.
//
// One block per sequence, value head and tile of 32 value columns (rows of the
// state [value][key]: they do not meet), walking the chunks in order. With T,
// P, the decays and the images of q and k from the parallel pass (gdr_prep.cu):
//   u  = T (v - e^G k S0^T)
//   o  = scale e^G q S0^T + P u
//   S1 = e^Gc S0 + sum_j wr_j u_j k_j^T
// Each is a product of a 64-row tile: the state is an accumulator in registers,
// its fp16 pair image in shared memory the operand of the next chunk. Warp
// (wr, wc) makes rows 16 wr.. of the chunk by columns 16 wc.. of the tile, and
// of the state rows 16 wc.. by a quarter of the keys.
//
// Scales. An image is written before anyone can know its largest value without
// one more barrier, so it takes a bound instead: |v - e^G k S0| <= max|v| +
// k_read max|S0|, |u| <= t_sum max|r|, |S1| <= e^Gc max|S0| + k_write max|u|,
// where the right sides hold the true maxima of the step before, published at
// the barrier that publishes the image itself. Bounds are loose by 2^10 at most
// in a well-posed chunk, which the pairs' 2^-39 floor leaves room for.
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
struct FwdSmem {
  Stage<In<T>::kParts, KP> st[kStages];
  __half s[2 * kVt * KP];
  __half r[2 * kC * kVt], u[2 * kC * kVt], w[2 * kC * kVt];
  float m_s[8], m_r[8], m_u[8], m_v[8];
  uint64_t bar[kStages];
};

template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = abs_max(m, x[i]);
  return m;
}

template <typename T, int KP, int kStages, bool kSave>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = FwdSmem<T, KP, kStages>;
  constexpr int P = In<T>::kParts, kNt = KP / 32;  // n8 tiles of a warp's quarter of the keys
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
  auto load = [&](int c) {
    Stage<P, KP>& st = sm.st[c % kStages];
    uint64_t* bar = &sm.bar[c % kStages];
    const size_t slot = sq.slot + c, at_k = slot * a.s.Hk + hk, at_v = slot * a.s.Hv + hv;
    mbar_arrive_expect_tx(bar, kBytes);
    bulk_load(st.k, a.b.k_img + at_k * image, image, bar);
    bulk_load(&st.rows, a.b.rows + at_k, sizeof(Rows), bar);
    bulk_load(&st.scal, a.b.scal + at_v, sizeof(Scal), bar);
    bulk_load(st.q, a.b.q_img + at_k * image, image, bar);
    bulk_load(st.t, a.b.t_img + at_v * Layout::tp_img, Layout::tp_img, bar);
    bulk_load(st.p, a.b.p_img + at_v * Layout::tp_img, Layout::tp_img, bar);
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.bar[s], 1);
    wkv7::fence_mbar_init();
    for (int c = 0; c < kStages && c < n; ++c) load(c);
  }

  // the warp's part of the state: value rows 16 wc + g4 (+ 8), keys key0 + 8 nt + 2 t4 (+ 1)
  const int key0 = wr * (KP / 4);
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
  float2 v[2][2];
  float v_max = 0.f;
  auto load_v = [&](int c) {
    v_max = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int t = sq.t0 + c * kC + 16 * wr + g4 + 8 * h, col = vt * kVt + 16 * wc + 8 * nt + 2 * t4;
        v[h][nt] = make_float2(0.f, 0.f);
        if (t < sq.t1 && col < V)
          v[h][nt] = load2(static_cast<const T*>(a.v) + sq.b * a.s.v_b + t * a.s.v_t + (size_t)hv * V + col);
      }
  };
  auto max_v = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) v_max = abs_max(abs_max(v_max, v[h][nt].x), v[h][nt].y);
    v_max = warp_max_abs(v_max);
    if (lane == 0) sm.m_v[warp] = v_max;
  };
  load_v(0);
  max_v();

  float s_max = 0.f;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) s_max = abs_max(s_max, max_of(S[nt]));
  s_max = warp_max_abs(s_max);
  if (lane == 0) sm.m_s[warp] = s_max;
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
  if (kSave) wkv7::fence_proxy_async_smem();
  __syncthreads();

  for (int c = 0; c < n; ++c) {
    Stage<P, KP>& st = sm.st[c % kStages];
    const size_t slot = sq.slot + c, at_t = (slot * a.s.Hv + hv) * vts + vt;
    if (!mbar_wait_bounded(a.status, &sm.bar[c % kStages], (c / kStages) & 1)) return;
    if (kSave && tid == 0) {
      bulk_store(a.b.s_img + at_t * sizeof(sm.s), sm.s, sizeof(sm.s));
      bulk_commit();
    }
    const Scal& sc = st.scal;
    const float mS = max_of(sm.m_s), mV = max_of(sm.m_v);

    // k S0^T and q S0^T
    float x[2][4], xq[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = xq[nt][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<P> fk, fq;
      Frag<2> fs;
      a_mk<P, true>(fk, st.k, kC, kC * KP, 16 * wr, 16 * kt, lane);
      a_mk<P, true>(fq, st.q, kC, kC * KP, 16 * wr, 16 * kt, lane);
      b_nk<2, true>(fs, sm.s, kVt, kVt * KP, 16 * wc, 16 * kt, lane);
      mma_parts<P, 2>(x[0], x[1], fk, fs);
      mma_parts<P, 2>(xq[0], xq[1], fq, fs);
    }
    const int i0 = 16 * wr + g4;
    const float inv_s = pow2_inverse(sS);
    // r = v - e^G k S0^T
    {
      const float sR = pow2_scale(mV + sc.k_read * mS);
      float r_max = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = -sc.eg[i0 + 8 * h] * st.rows.ks[i0 + 8 * h] * inv_s;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float r0 = fmaf(f, x[nt][2 * h], v[h][nt].x), r1 = fmaf(f, x[nt][2 * h + 1], v[h][nt].y);
          r_max = abs_max(abs_max(r_max, r0), r1);
          put2<false>(sm.r, kC, kC * kVt, i0 + 8 * h, 16 * wc + 8 * nt + 2 * t4, r0 * sR, r1 * sR);
        }
      }
      r_max = warp_max_abs(r_max);
      if (lane == 0) sm.m_r[warp] = r_max;
      __syncthreads();
      if (c + 1 < n) load_v(c + 1);

      // u = T r
      float u[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[nt][e] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt)
        if (kt <= wr) {
          Frag<2> ft, fr;
          a_mk<2, true>(ft, st.t, kC, kC * kC, 16 * wr, 16 * kt, lane);
          b_kn<2, false>(fr, sm.r, kC, kC * kVt, 16 * wc, 16 * kt, lane);
          mma_parts<2, 2>(u[0], u[1], ft, fr);
        }
      const float f = sc.inv_t * pow2_inverse(sR), bound = sc.t_sum * max_of(sm.m_r);
      const float sU = pow2_scale(bound), sW = pow2_scale(bound * sc.wk_max);
      float u_max = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float w = sc.wr[i0 + 8 * h] * st.rows.ks[i0 + 8 * h];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float u0 = u[nt][2 * h] * f, u1 = u[nt][2 * h + 1] * f;
          u_max = abs_max(abs_max(u_max, u0), u1);
          const int col = 16 * wc + 8 * nt + 2 * t4;
          put2<false>(sm.u, kC, kC * kVt, i0 + 8 * h, col, u0 * sU, u1 * sU);
          put2<false>(sm.w, kC, kC * kVt, i0 + 8 * h, col, (u0 * w) * sW, (u1 * w) * sW);
        }
      }
      u_max = warp_max_abs(u_max);
      if (lane == 0) sm.m_u[warp] = u_max;
      if (kSave) {
        wkv7::fence_proxy_async_smem();
        if (tid == 0) bulk_wait_read();  // the state's image is written anew after this barrier
      }
      __syncthreads();
      if (kSave && tid == 0) {
        bulk_store(a.b.u_img + at_t * sizeof(sm.u), sm.u, sizeof(sm.u));
        bulk_commit();
        a.b.su[at_t] = make_float2(inv_s, pow2_inverse(sU));
      }

      // o = scale e^G q S0^T + P u
      float o[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt)
        if (kt <= wr) {
          Frag<2> fp, fu;
          a_mk<2, true>(fp, st.p, kC, kC * kC, 16 * wr, 16 * kt, lane);
          b_kn<2, false>(fu, sm.u, kC, kC * kVt, 16 * wc, 16 * kt, lane);
          mma_parts<2, 2>(o[0], o[1], fp, fu);
        }
      const float fo = sc.inv_p * pow2_inverse(sU);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float fq = a.s.scale * sc.eg[i0 + 8 * h] * st.rows.qs[i0 + 8 * h] * inv_s;
        const int t = sq.t0 + c * kC + i0 + 8 * h;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int col = vt * kVt + 16 * wc + 8 * nt + 2 * t4;
          if (t < sq.t1 && col < V)
            store2(static_cast<T*>(a.o) + (((size_t)sq.b * a.s.T + t) * a.s.Hv + hv) * V + col,
                   fmaf(fq, xq[nt][2 * h], fo * o[nt][2 * h]), fmaf(fq, xq[nt][2 * h + 1], fo * o[nt][2 * h + 1]));
        }
      }

      // S1 = e^Gc S0 + (wr u)^T k
      float d[kNt][4];
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[nt][e] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        Frag<2> fw;
        a_km<2, false>(fw, sm.w, kC, kC * kVt, 16 * wc, 16 * kt, lane);
#pragma unroll
        for (int nt = 0; nt < kNt; nt += 2) {
          Frag<P> fk;
          b_kn<P, true>(fk, st.k, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
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
      sS = pow2_scale(sc.egc * mS + sc.k_write * max_of(sm.m_u));
    }
    put_state(sS);
    s_max = warp_max_abs(s_max);
    if (lane == 0) sm.m_s[warp] = s_max;
    max_v();
    if (kSave) {
      wkv7::fence_proxy_async_smem();
      if (tid == 0) bulk_wait_read();  // the image of u is written anew after the next step's first barrier
    }
    __syncthreads();
    if (tid == 0 && c + kStages < n) load(c + kStages);
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

template <typename T, int KP, bool kSave>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  // two stages of images where they fit the 227 KB beside the rest; fp32 q and k of 128 take one
  constexpr int kStages = sizeof(FwdSmem<T, KP, 2>) <= 227 * 1024 ? 2 : 1;
  constexpr size_t smem = sizeof(FwdSmem<T, KP, kStages>);
  auto kernel = fwd_kernel<T, KP, kStages, kSave>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * v_tiles(a.s.V)), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int KP>
cudaError_t pick(const Args& a, bool save, cudaStream_t s) {
  return save ? launch<T, KP, true>(a, s) : launch<T, KP, false>(a, s);
}

}  // namespace

cudaError_t launch_fwd(const Args& a, bool bf16, bool save, cudaStream_t stream) {
  const bool wide = padded_k(a.s.K) == 128;
  if (bf16) return wide ? pick<__nv_bfloat16, 128>(a, save, stream) : pick<__nv_bfloat16, 64>(a, save, stream);
  return wide ? pick<float, 128>(a, save, stream) : pick<float, 64>(a, save, stream);
}

}  // namespace gdr
