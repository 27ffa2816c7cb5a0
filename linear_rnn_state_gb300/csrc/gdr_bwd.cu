// The gated delta rule's backward chain: the carried gradient dS of the state,
// from the last chunk to the first, and dv.
//
// For the 16 rows of the state that a warp owns (gdr_chain.cuh), with the
// images of q, k, T and P that the forward used, all transposed:
//   y^T   = do^T P (helper) + wk (dS1 k^T)          the gradient of u
//   lam^T = y^T T = dv^T
//   dS0   = e^Gc dS1 + (scale e^G do)^T q (helper) - (e^G lam)^T k
// The helper's two products do not wait for the chain: it makes them a step
// ahead. It leaves the images of dS1, lam and do for the gradients of q, k, g
// and beta (gdr_grad.cu). fp16 pairs throughout: dS, lam and do enter fp32
// results.
#include "gdr_chain.cuh"

namespace gdr {
namespace {

// What a chain and its helper share.
template <typename T, int KP>
struct alignas(128) BwdPair {
  unsigned char d[2][kRowsBytes<T>];
  union {  // the helper's ways to memory
    unsigned char dv[kRowsBytes<T>];
    __half l_img[2 * kVt * kC];
  };
  __half s[2 * kVt * KP], d_img[In<T>::kParts * kVt * kC];  // images of dS1 and do
  float4 l[8 * 32], y[8 * 32], g[KP / 8 * 32];  // lam, do^T P and (scale e^G do)^T q, as accumulator tiles
  float inv_s;
  uint64_t full_s, full_l, full_y, full_g, free_s, free_l, free_y, free_g;
};
// fp32 images of 128 keys leave room for two
template <typename T, int KP>
constexpr int kBwdChains = sizeof(T) * KP <= 256 ? 4 : 2;
template <typename T, int KP>
struct BwdSmem {
  Images<In<T>::kParts, KP, 2> im;
  BwdPair<T, KP> pair[kBwdChains<T, KP>];
};

template <typename T, int KP>
__global__ void __launch_bounds__((2 * kBwdChains<T, KP> + 1) * 32, 1) bwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  constexpr int P = In<T>::kParts, kNt = KP / 8;
  BwdSmem<T, KP>& sm = *reinterpret_cast<BwdSmem<T, KP>*>(raw);
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
      BwdPair<T, KP>& p = sm.pair[i];
      for (uint64_t* b : {&p.full_s, &p.full_l, &p.full_y, &p.full_g, &p.free_s, &p.free_l, &p.free_y, &p.free_g}) mbar_init(b, 1);
    }
    wkv7::fence_mbar_init();
  }
  __syncthreads();
  if (a.small) grid_go();
  if (warp == 2 * chains) {
    if (lane == 0) fill_images(im, a, sq.slot + n - 1, -1, n, hk, hv);
    return;
  }
  const int own = warp % chains, vt = set * chains + own;
  if (vt >= vts) return;
  BwdPair<T, KP>& pr = sm.pair[own];
  const int cols = V - vt * kVt, tokens = sq.t1 - sq.t0;

  // step s works on chunk n - 1 - s
  if (warp < chains) {  // ------------------------------------------------ chain
    const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
    float S[kNt][4];
    load_state(S, a.dS_final ? a.dS_final + state_at : nullptr, cols, K, lane);
    float s_max = warp_max(S);
    Asked has_k(&im.full_k[0], 0);
    for (int s = 0; s < n; ++s) {
      const int use = s & 1;
      const Scal& sc = im.sc(use);
      const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);
      // dS1 k^T
      float x[8][4];
      const Asked has_s(&pr.free_s, use ^ 1), has_y(&pr.full_y, use), has_t(&im.full_t, use);
      if (!has_k.wait(a.status)) return;
      if (s > 0 && !has_s.wait(a.status)) return;
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
      wkv7::fence_proxy_async_smem();
      signal(&pr.full_s, lane);

      // y
      if (!has_y.wait(a.status)) return;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 f = *reinterpret_cast<const float2*>(sc.wk + 8 * nt + 2 * t4);
        const float4 y = pr.y[nt * 32 + lane];
        const float f0 = f.x * inv_s, f1 = f.y * inv_s;
        x[nt][0] = fmaf(f0, x[nt][0], y.x), x[nt][1] = fmaf(f1, x[nt][1], y.y);
        x[nt][2] = fmaf(f0, x[nt][2], y.z), x[nt][3] = fmaf(f1, x[nt][3], y.w);
      }
      signal(&pr.free_y, lane);
      const float sY = pow2_scale(warp_max(x));

      // lam = T^T y
      float l[8][4];
      if (!has_t.wait(a.status)) return;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        Frag<2> fy, ft[4];
        to_a(fy, x[2 * i], x[2 * i + 1], sY);
#pragma unroll
        for (int j = 0; j <= i; ++j) b_tri_kn<2>(ft[j], im.t, i, j, lane);
        if (i == 3)
          mma_row<4, true>(l, fy, ft);
        else
          mma_row<4>(l, fy, ft, 0, i + 1);
      }
      const Asked has_l(&pr.free_l, use ^ 1), has_g(&pr.full_g, use);
      const float fl = sc.inv_t * pow2_inverse(sY);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) l[nt][e] *= fl;
      if (s > 0 && !has_l.wait(a.status)) return;
      tiles_put(pr.l, l, 1.f, lane);
      signal(&pr.full_l, lane);

      // dS0, the product at its own scale, kept below 2^60 of dS1's
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 f = *reinterpret_cast<const float2*>(sc.ek + 8 * nt + 2 * t4);
#pragma unroll
        for (int h = 0; h < 4; h += 2) l[nt][h] *= -f.x, l[nt][h + 1] *= -f.y;
      }
      const float sW = fminf(pow2_scale(warp_max(l)), sS * 0x1p60f), egc = sc.egc * sW;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] *= egc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Frag<2> fw;
        to_a(fw, l[2 * j], l[2 * j + 1], sW);
        Frag<P> fk[KP / 16];
#pragma unroll
        for (int nb = 0; nb < KP / 16; ++nb) b_kn<P>(fk[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * j, lane);
        mma_row<KP / 16>(S, fw, fk);
      }
      has_k = Asked(&im.full_k[use ^ 1], (s + 1) >> 1);
      signal(&im.free_k[use], lane);
      const float inv_w = pow2_inverse(sW);
      if (!has_g.wait(a.status)) return;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        const float4 g = pr.g[nt * 32 + lane];
        S[nt][0] = fmaf(S[nt][0], inv_w, g.x), S[nt][1] = fmaf(S[nt][1], inv_w, g.y);
        S[nt][2] = fmaf(S[nt][2], inv_w, g.z), S[nt][3] = fmaf(S[nt][3], inv_w, g.w);
      }
      signal(&pr.free_g, lane);
      s_max = warp_max(S);
    }
    if (a.dS_init) store_state(S, a.dS_init + state_at, cols, K, lane);
    return;
  }

  // ------------------------------------------------------------------- helper
  const size_t first = (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + vt * kVt;
  const T* do_at = static_cast<const T*>(a.d_o) + first;
  T* dv_at = static_cast<T*>(a.dv) + first;
  const long long row_t = (long long)a.s.Hv * V;
  auto fetch = [&](int s) {  // do of step s, and a request for a later one
    const int c = n - 1 - s;
    if (c >= 0) rows_in(pr.d[s & 1], do_at + c * kC * row_t, row_t, tokens - c * kC, cols, lane);
    copy_commit();
    if (c >= 2) rows_ask(do_at + (c - 2) * kC * row_t, row_t, kC, lane);
  };
  constexpr Record rec = b_record(KP, P);
  auto record_of = [&](int s) { return a.b.b_rec + (((sq.slot + n - 1 - s) * a.s.Hv + hv) * vts + vt) * rec.size; };
  float inv_d = 0.f;
  // What step s needs of do: its image, do^T P and (scale e^G do)^T q.
  auto ahead = [&](int s) {
    const int use = s & 1;
    const Scal& sc = im.sc(use);
    char* record = record_of(s);
    copy_wait<1>();
    __syncwarp();
    float d[8][4], x[8][4];
    rows_get(d, pr.d[use], lane, do_at);
    __syncwarp();
    fetch(s + 2);
    const float sD = pow2_scale(warp_max(d));
    inv_d = pow2_inverse(sD);
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (s >> 1) & 1)) return false;
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return false;
    if (lane == 0) bulk_wait_read();  // the images of dS and do of the step before are out
    __syncwarp();
    if (s > 0) signal(&pr.free_s, lane);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      Frag<P> fd;
      Frag<2> fp[4];
      to_a(fd, d[2 * i], d[2 * i + 1], sD);
      put_a(pr.d_img, kVt * kC, 16 * i, fd, lane);
#pragma unroll
      for (int j = 0; j <= i; ++j) b_tri_kn<2>(fp[j], im.p, i, j, lane);
      if (i == 3)
        mma_row<4, true>(x, fd, fp);
      else
        mma_row<4>(x, fd, fp, 0, i + 1);
    }
    signal(&im.free_p, lane);
    wkv7::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      bulk_store(record + rec.d, pr.d_img, sizeof(pr.d_img));
      bulk_commit();
    }
    if (s > 0 && !mbar_wait_bounded(a.status, &pr.free_y, use ^ 1)) return false;
    tiles_put(pr.y, x, sc.inv_p * inv_d, lane);
    signal(&pr.full_y, lane);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 f = *reinterpret_cast<const float2*>(sc.eq + 8 * nt + 2 * t4);
#pragma unroll
      for (int h = 0; h < 4; h += 2) d[nt][h] *= f.x, d[nt][h + 1] *= f.y;
    }
    const float sW = pow2_scale(warp_max(d));
    float g[kNt][4];
    if (!mbar_wait_bounded(a.status, &im.full_q, use)) return false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<2> fd;
      to_a(fd, d[2 * j], d[2 * j + 1], sW);
      Frag<P> fq[KP / 16];
#pragma unroll
      for (int nb = 0; nb < KP / 16; ++nb) b_kn<P>(fq[nb], im.q, kC, kC * KP, 16 * nb, 16 * j, lane);
      if (j == 0)
        mma_row<KP / 16, true>(g, fd, fq);
      else
        mma_row<KP / 16>(g, fd, fq);
    }
    signal(&im.free_q, lane);
    signal(&im.free_k[use], lane);
    if (s > 0 && !mbar_wait_bounded(a.status, &pr.free_g, use ^ 1)) return false;
    tiles_put(pr.g, g, pow2_inverse(sW), lane);
    signal(&pr.full_g, lane);
    return true;
  };
  fetch(0), fetch(1);
  if (n > 0 && !ahead(0)) return;
  for (int s = 0; s < n; ++s) {
    const int c = n - 1 - s, use = s & 1;
    char* record = record_of(s);
    const float inv_do = inv_d;
    if (!mbar_wait_bounded(a.status, &pr.full_s, use)) return;
    const float inv_s = pr.inv_s;
    if (lane == 0) {
      bulk_store(record, pr.s, sizeof(pr.s));
      bulk_commit();
    }
    if (s + 1 < n && !ahead(s + 1)) return;

    if (!mbar_wait_bounded(a.status, &pr.full_l, use)) return;
    float x[8][4];
    tiles_get(x, pr.l, lane);
    signal(&pr.free_l, lane);
    const float sL = pow2_scale(warp_max(x));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<2> f;
      to_a(f, x[2 * j], x[2 * j + 1], sL);
      put_a(pr.l_img, kVt * kC, 16 * j, f, lane);
    }
    wkv7::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      bulk_store(record + rec.u, pr.l_img, sizeof(pr.l_img));
      bulk_commit();
      *reinterpret_cast<float4*>(record + rec.scales) = make_float4(inv_s, pow2_inverse(sL), inv_do, 0.f);
      bulk_wait_read();
    }
    __syncwarp();
    rows_out(x, pr.dv, dv_at + (size_t)c * kC * row_t, row_t, tokens - c * kC, cols, lane);
  }
  if (lane == 0) bulk_wait_all();
}

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr int most = kBwdChains<T, KP>;
  constexpr size_t all = sizeof(BwdSmem<T, KP>);
  static_assert(all <= 227 * 1024, "shared memory of a block");
  auto kernel = bwd_kernel<T, KP>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), all, done);
  if (e != cudaSuccess) return e;
  const int chains = chain_warps(a.s, most), sets = (v_tiles(a.s.V) + chains - 1) / chains;
  const size_t smem = all - (most - chains) * sizeof(BwdPair<T, KP>);
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), (2 * chains + 1) * 32, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t pick(const Args& a, cudaStream_t s) {
  return padded_k(a.s.K) == 128 ? launch<T, 128>(a, s) : launch<T, 64>(a, s);
}

}  // namespace

cudaError_t launch_bwd(const Args& a, bool bf16, cudaStream_t stream) {
  return bf16 ? pick<__nv_bfloat16>(a, stream) : pick<float>(a, stream);
}

}  // namespace gdr
