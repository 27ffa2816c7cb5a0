// The gated delta rule's backward chain: the carried gradient dS of the state,
// from the last chunk to the first, and dv.
//
// For the 16 rows of the state that a warp owns (gdr_chain.cuh), with the
// images of q, k, T and P that the forward used, all transposed:
//   y^T   = do^T P + wk (dS1 k^T)              (the gradient of u)
//   lam^T = y^T T = dv^T
//   dS0   = e^Gc dS1 + (scale e^G do)^T q - (e^G lam)^T k
// It leaves the images of dS1, lam and do for the gradients of q, k, g and beta
// (gdr_grad.cu). fp16 pairs throughout: dS, lam and do enter fp32 results.
//
// Bound, as the forward, by the tensor pipe: 292 mma of 8 cycles a step, warp
// and scheduler at 64 keys (bfloat16).
#include "gdr_chain.cuh"

namespace gdr {
namespace {

template <typename T, int KP>
struct alignas(128) BwdWarp {
  unsigned char rows[2][kRowsBytes<T>];  // do of this and the next chunk; then dv
  __half s[2 * kVt * KP], l[2 * kVt * kC], d[In<T>::kParts * kVt * kC];  // images on their way out
};
template <typename T, int KP>
struct BwdSmem {
  Images<In<T>::kParts, KP, 2> im;
  BwdWarp<T, KP> w[kMaxWarps];
};

template <typename T, int KP>
__global__ void __launch_bounds__((kMaxWarps + 1) * 32, sizeof(BwdSmem<T, KP>) <= 113 * 1024 ? 2 : 1) bwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = BwdSmem<T, KP>;
  constexpr int P = In<T>::kParts, kNt = KP / 8;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int warps = blockDim.x / 32 - 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3;
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + warps - 1) / warps;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  const SeqRange sq = seq_range(a.s, seq);
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V;
  auto& im = sm.im;
  if (threadIdx.x == 0) init_images(im, min(warps, vts - set * warps));
  __syncthreads();
  if (warp == warps) {
    if (lane == 0) fill_images(im, a, sq.slot + n - 1, -1, n, hk, hv);
    return;
  }
  const int vt = set * warps + warp;
  if (vt >= vts) return;
  BwdWarp<T, KP>& mine = sm.w[warp];
  const int cols = V - vt * kVt;
  const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
  const size_t first = (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + vt * kVt;
  const T* do_at = static_cast<const T*>(a.d_o) + first;
  T* dv_at = static_cast<T*>(a.dv) + first;
  const long long row_t = (long long)a.s.Hv * V;
  const int tokens = sq.t1 - sq.t0;
  // chunk c's rows: where they start and how many there are
  auto ask = [&](int c) {
    if (c >= 0) rows_ask(do_at + c * kC * row_t, row_t, tokens - c * kC, lane);
  };

  float S[kNt][4];
  load_state(S, a.dS_final ? a.dS_final + state_at : nullptr, cols, K, lane);
  float s_max = warp_max(S);
  if (n > 0) rows_in(mine.rows[0], do_at + (n - 1) * kC * row_t, row_t, tokens - (n - 1) * kC, cols, lane);
  copy_commit();
  ask(n - 2), ask(n - 3);

  for (int s = 0; s < n; ++s) {
    const int c = n - 1 - s, use = s & 1, len = tokens - c * kC;
    const size_t at_t = ((sq.slot + c) * a.s.Hv + hv) * vts + vt;
    if (c > 0) rows_in(mine.rows[use ^ 1], do_at + (c - 1) * kC * row_t, row_t, kC, cols, lane);
    copy_commit();
    ask(c - 3);
    if (lane == 0) bulk_wait_read();  // the images of the step before are out
    __syncwarp();
    const Scal& sc = im.sc(use);
    const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);

    // dS1 k^T
    float y[8][4];
    zero(y);
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (s >> 1) & 1)) return;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<2> fs;
      to_a(fs, S[2 * kt], S[2 * kt + 1], sS);
      put_a(mine.s, kVt * KP, 16 * kt, fs, lane);
      Frag<P> fk[4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) b_nk<P>(fk[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * kt, lane);
      mma_row<4>(y, fs, fk);
    }
    copy_wait<1>();
    __syncwarp();
    float d[8][4];
    rows_get(d, mine.rows[use], lane, do_at);
    const float sD = pow2_scale(warp_max(d)), inv_d = pow2_inverse(sD);

    // y = P^T do + wk k dS1^T
    float x[8][4];
    zero(x);
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Frag<P> fd;
      to_a(fd, d[2 * i], d[2 * i + 1], sD);
      put_a(mine.d, kVt * kC, 16 * i, fd, lane);
      Frag<2> fp[4];
#pragma unroll
      for (int j = 0; j <= i; ++j) b_tri_kn<2>(fp[j], im.p, i, j, lane);
      mma_row<4>(x, fd, fp, 0, i + 1);
    }
    give_up(&im.free_p, lane);
    const float fp = sc.inv_p * inv_d;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 f = *reinterpret_cast<const float2*>(sc.wk + 8 * nt + 2 * t4);
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        y[nt][h] = fmaf(f.x * inv_s, y[nt][h], fp * x[nt][h]);
        y[nt][h + 1] = fmaf(f.y * inv_s, y[nt][h + 1], fp * x[nt][h + 1]);
      }
    }
    const float sY = pow2_scale(warp_max(y));

    // lam = T^T y
    zero(x);
    if (!mbar_wait_bounded(a.status, &im.full_t, use)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Frag<2> fy;
      to_a(fy, y[2 * i], y[2 * i + 1], sY);
      Frag<2> ft[4];
#pragma unroll
      for (int j = 0; j <= i; ++j) b_tri_kn<2>(ft[j], im.t, i, j, lane);
      mma_row<4>(x, fy, ft, 0, i + 1);
    }
    give_up(&im.free_t, lane);
    const float fl = sc.inv_t * pow2_inverse(sY);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] *= fl;
    const float sL = pow2_scale(warp_max(x));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<2> f;
      to_a(f, x[2 * j], x[2 * j + 1], sL);
      put_a(mine.l, kVt * kC, 16 * j, f, lane);
    }
    wkv7::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      bulk_store(a.b.ds_img + at_t * sizeof(mine.s), mine.s, sizeof(mine.s));
      bulk_store(a.b.do_img + at_t * sizeof(mine.d), mine.d, sizeof(mine.d));
      bulk_store(a.b.l_img + at_t * sizeof(mine.l), mine.l, sizeof(mine.l));
      bulk_commit();
      a.b.dsl[at_t] = make_float4(inv_s, pow2_inverse(sL), inv_d, 0.f);
    }
    rows_out(x, mine.rows[use], dv_at + (size_t)c * kC * row_t, row_t, len, cols, lane);

    // dS0, both products at one scale, kept below 2^60 of dS1's
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 f = *reinterpret_cast<const float2*>(sc.ek + 8 * nt + 2 * t4), fd = *reinterpret_cast<const float2*>(sc.eq + 8 * nt + 2 * t4);
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        x[nt][h] *= -f.x, x[nt][h + 1] *= -f.y;
        d[nt][h] *= fd.x, d[nt][h + 1] *= fd.y;
      }
    }
    const float sW = fminf(pow2_scale(abs_max(warp_max(x), warp_max(d))), sS * 0x1p60f), egc = sc.egc * sW;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] *= egc;
    if (!mbar_wait_bounded(a.status, &im.full_q, use)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<2> fl2, fd;
      to_a(fl2, x[2 * j], x[2 * j + 1], sW);
      to_a(fd, d[2 * j], d[2 * j + 1], sW);
      Frag<P> fb[KP / 16];
#pragma unroll
      for (int nb = 0; nb < KP / 16; ++nb) b_kn<P>(fb[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * j, lane);
      mma_row<KP / 16>(S, fl2, fb);
#pragma unroll
      for (int nb = 0; nb < KP / 16; ++nb) b_kn<P>(fb[nb], im.q, kC, kC * KP, 16 * nb, 16 * j, lane);
      mma_row<KP / 16>(S, fd, fb);
    }
    give_up(&im.free_q, lane);
    give_up(&im.free_k[use], lane);
    const float inv_w = pow2_inverse(sW);
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] *= inv_w;
    s_max = warp_max(S);
  }
  if (lane == 0) bulk_wait_all();
  if (a.dS_init) store_state(S, a.dS_init + state_at, cols, K, lane);
}

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const int warps = chain_warps(a.s);
  constexpr size_t most = sizeof(BwdSmem<T, KP>);
  static_assert(most <= 227 * 1024, "shared memory of a block");
  auto kernel = bwd_kernel<T, KP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  const int sets = (v_tiles(a.s.V) + warps - 1) / warps;
  const size_t smem = most - (kMaxWarps - warps) * sizeof(BwdWarp<T, KP>);
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), (warps + 1) * 32, smem, stream>>>(a);
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
