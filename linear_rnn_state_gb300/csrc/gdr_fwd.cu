// The gated delta rule's forward chain: the states from chunk to chunk, and o.
//
// With T, P, the decays and the images of q and k from the parallel pass
// (gdr_prep.cu), for the 16 rows of the state that a warp owns (gdr_chain.cuh),
// all transposed (rows: value columns):
//   r^T = v^T - e^G (S0 k^T)                    chain
//   u^T = r^T T^T                               chain
//   S1  = e^Gc S0 + (wk u)^T k                  chain
//   o^T = scale e^G (S0 q^T) + u^T P^T          helper
// T and P have their lower blocks only: a block (i, j) meets only the tokens j
// of r and the tokens i of the result.
//
// Arithmetic: fp16 pairs in everything that the states depend on. o of
// bfloat16 calls takes S0, u and P with their hi part alone (11 bits against
// the 8 that o is rounded to: 0.0003 of o's error of 0.0017), which saves 72 of
// 312 mma a step at 64 keys.
#include "gdr_chain.cuh"

namespace gdr {
namespace {

// What a chain and its helper share.
template <typename T, int KP>
struct alignas(128) FwdPair {
  unsigned char v[2][kRowsBytes<T>];
  union {  // the helper's ways to memory
    unsigned char o[kRowsBytes<T>];
    __half u_img[2 * kVt * kC];
  };
  __half s[2 * kVt * KP];  // the image of S0
  float4 u[8 * 32];        // u as accumulator tiles
  float inv_s;
  uint64_t full_s, full_u, full_v[2], free_s, free_u;
};
template <typename T, int KP>
constexpr int kFwdChains = 4;
template <typename T, int KP>
struct FwdSmem {
  Images<In<T>::kParts, KP, In<T>::kParts> im;
  FwdPair<T, KP> pair[kFwdChains<T, KP>];
};

template <typename T, int KP, bool kSave>
__global__ void __launch_bounds__((2 * kFwdChains<T, KP> + 1) * 32, 1) fwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  constexpr int P = In<T>::kParts, kNt = KP / 8;
  FwdSmem<T, KP>& sm = *reinterpret_cast<FwdSmem<T, KP>*>(raw);
  const int chains = blockDim.x / 64, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3;
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + chains - 1) / chains;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  const SeqRange sq = seq_range(a.s, seq);
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V;
  auto& im = sm.im;
  if (threadIdx.x == 0) {
    init_images(im, min(chains, vts - set * chains));
    for (int i = 0; i < chains; ++i) {
      FwdPair<T, KP>& p = sm.pair[i];
      for (uint64_t* b : {&p.full_s, &p.full_u, &p.free_s, &p.free_u}) mbar_init(b, 1);
      mbar_init(&p.full_v[0], 32), mbar_init(&p.full_v[1], 32);
    }
    wkv7::fence_mbar_init();
  }
  grid_wait();
  __syncthreads();
  if (warp == 2 * chains) {
    if (lane == 0) fill_images(im, a, sq.slot, 1, n, hk, hv);
    return;
  }
  const int own = warp % chains, vt = set * chains + own;
  if (vt >= vts) return;
  FwdPair<T, KP>& pr = sm.pair[own];
  const int cols = V - vt * kVt, tokens = sq.t1 - sq.t0;
  const T* v_at = static_cast<const T*>(a.v) + sq.b * a.s.v_b + sq.t0 * a.s.v_t + (size_t)hv * V + vt * kVt;

  if (warp < chains) {  // ------------------------------------------------ chain
    const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
    float S[kNt][4];
    load_state(S, a.s_init ? a.s_init + state_at : nullptr, cols, K, lane);
    float s_max = warp_max(S);
    Asked has_k(&im.full_k[0], 0);
    for (int c = 0; c < n; ++c) {
      const int use = c & 1;
      const Scal& sc = im.sc(use);
      const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);
      // S0 k^T
      float x[8][4];
      const Asked has_s(&pr.free_s, use ^ 1), has_v(&pr.full_v[use], c >> 1), has_t(&im.full_t, use);
      if (!has_k.wait(a.status)) return;
      if (c > 0 && !has_s.wait(a.status)) return;
#pragma unroll
      for (int kt = 0; kt < KP / 16; ++kt) {
        Frag<2> fs;
        to_a(fs, S[2 * kt], S[2 * kt + 1], sS);
        put_a(pr.s, kVt * KP, 16 * kt, fs, lane);
        Frag<P> fk[4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) b_nk<P>(fk[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * kt, lane);
        if (kt == 0)
          mma_row<4, true>(x, fs, fk);
        else
          mma_row<4>(x, fs, fk);
      }
      if (lane == 0) pr.inv_s = inv_s;
      if (kSave) wkv7::fence_proxy_async_smem();
      signal(&pr.full_s, lane);

      // r
      if (!has_v.wait(a.status)) return;
      {
        float v[8][4];
        rows_get(v, pr.v[use], lane, v_at);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          const float2 f = *reinterpret_cast<const float2*>(sc.ek + 8 * nt + 2 * t4);
          const float f0 = -f.x * inv_s, f1 = -f.y * inv_s;
#pragma unroll
          for (int h = 0; h < 4; h += 2) {
            x[nt][h] = fmaf(f0, x[nt][h], v[nt][h]), x[nt][h + 1] = fmaf(f1, x[nt][h + 1], v[nt][h + 1]);
          }
        }
      }
      const float sR = pow2_scale(warp_max(x));

      // u = T r
      float u[8][4];
      if (!has_t.wait(a.status)) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Frag<2> fr, ft[4];
        to_a(fr, x[2 * j], x[2 * j + 1], sR);
#pragma unroll
        for (int i = j; i < 4; ++i) b_tri_nk<2>(ft[i], im.t, i, j, lane);
        if (j == 0)
          mma_row<4, true>(u, fr, ft);
        else
          mma_row<4>(u, fr, ft, j);
      }
      const Asked has_u(&pr.free_u, use ^ 1);
      const float fu = sc.inv_t * pow2_inverse(sR);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[nt][e] *= fu;
      if (c > 0 && !has_u.wait(a.status)) return;
      tiles_put(pr.u, u, 1.f, lane);
      signal(&pr.full_u, lane);

      // S1: the products are added to S0 at their own scale, which is kept
      // below 2^60 of S0's so that S0 stays finite in it
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 f = *reinterpret_cast<const float2*>(sc.wk + 8 * nt + 2 * t4);
#pragma unroll
        for (int h = 0; h < 4; h += 2) u[nt][h] *= f.x, u[nt][h + 1] *= f.y;
      }
      const float sW = fminf(pow2_scale(warp_max(u)), sS * 0x1p60f), egc = sc.egc * sW;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= egc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Frag<2> fw;
        to_a(fw, u[2 * j], u[2 * j + 1], sW);
        Frag<P> fk[KP / 16];
#pragma unroll
        for (int nb = 0; nb < KP / 16; ++nb) b_kn<P>(fk[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * j, lane);
        mma_row<KP / 16>(S, fw, fk);
      }
      has_k = Asked(&im.full_k[use ^ 1], (c + 1) >> 1);
      signal(&im.free_k[use], lane);
      const float inv_w = pow2_inverse(sW);
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= inv_w;
      s_max = warp_max(S);
    }
    if (a.s_final) store_state(S, a.s_final + state_at, cols, K, lane);
    return;
  }

  // ------------------------------------------------------------------- helper
  T* o_at = static_cast<T*>(a.o) + (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + vt * kVt;
  const long long o_t = (long long)a.s.Hv * V;
  auto fetch = [&](int c) {  // v of chunk c, and a request for a later one
    if (c < n) {
      rows_in(pr.v[c & 1], v_at + c * kC * a.s.v_t, a.s.v_t, tokens - c * kC, cols, lane);
      copy_arrive(&pr.full_v[c & 1]);
    }
    if (c + 2 < n) rows_ask(v_at + (c + 2) * kC * a.s.v_t, a.s.v_t, tokens - (c + 2) * kC, lane);
  };
  fetch(0), fetch(1);
  for (int c = 0; c < n; ++c) {
    const int use = c & 1;
    constexpr Record rec = f_record(KP, P);
    char* record = a.b.f_rec + (((sq.slot + c) * a.s.Hv + hv) * vts + vt) * rec.size;
    const Scal& sc = im.sc(use);
    // S0 q^T
    float o[8][4], x[8][4];
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (c >> 1) & 1)) return;
    if (!mbar_wait_bounded(a.status, &im.full_q, use)) return;
    if (!mbar_wait_bounded(a.status, &pr.full_s, use)) return;
    if (kSave && lane == 0) {
      bulk_store(record, pr.s, sizeof(pr.s));
      bulk_commit();
    }
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<P> fs, fq[4];
      a_mk<P>(fs, pr.s, kVt, kVt * KP, 0, 16 * kt, lane);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) b_nk<P>(fq[nb], im.q, kC, kC * KP, 16 * nb, 16 * kt, lane);
      if (kt == 0)
        mma_row<4, true>(o, fs, fq);
      else
        mma_row<4>(o, fs, fq);
    }
    signal(&im.free_q, lane);
    const float inv_s = pr.inv_s, inv_p = sc.inv_p;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 f = *reinterpret_cast<const float2*>(sc.eq + 8 * nt + 2 * t4);
#pragma unroll
      for (int h = 0; h < 4; h += 2) o[nt][h] *= f.x * inv_s, o[nt][h + 1] *= f.y * inv_s;
    }
    signal(&im.free_k[use], lane);
    if (kSave && lane == 0) bulk_wait_read();
    signal(&pr.free_s, lane);

    // P u
    if (!mbar_wait_bounded(a.status, &pr.full_u, use)) return;
    float u[8][4];
    tiles_get(u, pr.u, lane);
    signal(&pr.free_u, lane);
    fetch(c + 2);  // the chain is past v of this step
    const float sU = pow2_scale(warp_max(u)), inv_u = pow2_inverse(sU);
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<kSave ? 2 : P> fu;
      Frag<P> fp[4];
      to_a(fu, u[2 * j], u[2 * j + 1], sU);
      if constexpr (kSave) put_a(pr.u_img, kVt * kC, 16 * j, fu, lane);
#pragma unroll
      for (int i = j; i < 4; ++i) b_tri_nk<P>(fp[i], im.p, i, j, lane);
      constexpr bool kHi = P == 1;
      if (j == 0)
        mma_row<4, true, kHi>(x, fu, fp);
      else
        mma_row<4, false, kHi>(x, fu, fp, j);
    }
    signal(&im.free_p, lane);
    if (kSave) {
      wkv7::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        bulk_store(record + rec.u, pr.u_img, sizeof(pr.u_img));
        bulk_commit();
        *reinterpret_cast<float4*>(record + rec.scales) = make_float4(inv_s, inv_u, 0.f, 0.f);
      }
    }
    const float fo = inv_p * inv_u;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = fmaf(fo, x[nt][e], o[nt][e]);
    if (kSave && lane == 0) bulk_wait_read();
    __syncwarp();
    rows_out(o, pr.o, o_at + (size_t)c * kC * o_t, o_t, tokens - c * kC, cols, lane);
  }
  if (kSave && lane == 0) bulk_wait_all();
}

template <typename T, int KP, bool kSave>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr int most = kFwdChains<T, KP>;
  constexpr size_t all = sizeof(FwdSmem<T, KP>);
  static_assert(all <= 227 * 1024, "shared memory of a block");
  auto kernel = fwd_kernel<T, KP, kSave>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), all, done);
  if (e != cudaSuccess) return e;
  const int chains = chain_warps(a.s, most), sets = (v_tiles(a.s.V) + chains - 1) / chains;
  const size_t smem = all - (most - chains) * sizeof(FwdPair<T, KP>);
  return launch_after(a.small, kernel, (unsigned)((size_t)a.s.nseq * a.s.Hv * sets), (2 * chains + 1) * 32, smem, stream, a);
}
template <typename T>
cudaError_t pick(const Args& a, bool save, cudaStream_t s) {
  if (padded_k(a.s.K) == 128) return save ? launch<T, 128, true>(a, s) : launch<T, 128, false>(a, s);
  return save ? launch<T, 64, true>(a, s) : launch<T, 64, false>(a, s);
}

}  // namespace

cudaError_t launch_fwd(const Args& a, bool bf16, bool save, cudaStream_t stream) {
  return bf16 ? pick<__nv_bfloat16>(a, save, stream) : pick<float>(a, save, stream);
}

}  // namespace gdr
