// The gated delta rule's forward chain: the states from chunk to chunk, and o.
//
// With T, P, the decays and the images of q and k from the parallel pass
// (gdr_prep.cu), for the 16 rows of the state that a warp owns (gdr_chain.cuh),
// all transposed (rows: value columns):
//   r^T = v^T - e^G (S0 k^T)
//   u^T = r^T T^T
//   o^T = scale e^G (S0 q^T) + u^T P^T
//   S1  = e^Gc S0 + (wk u)^T k
// T and P have their lower blocks only: a block (i, j) meets only the tokens j
// of r and the tokens i of the result.
//
// Arithmetic: fp16 pairs in everything that the states depend on. o of
// bfloat16 calls takes S0, u and P with their hi part alone (11 bits against
// the 8 that o is rounded to: 0.0003 of o's error of 0.0017), which saves 72 of
// 312 mma a step at 64 keys.
//
// Bound by the tensor pipe of the four schedulers, one warp each: 240 mma of 8
// cycles a step and 64 keys, with the conversions between products beside them.
#include "gdr_chain.cuh"

namespace gdr {
namespace {

template <typename T, int KP, bool kSave>
struct alignas(128) FwdWarp {
  unsigned char rows[2][kRowsBytes<T>];       // v of this and the next chunk; then o
  __half s[kSave ? 2 * kVt * KP : 64], u[kSave ? 2 * kVt * kC : 64];  // images on their way out
};
template <typename T, int KP, bool kSave>
struct FwdSmem {
  Images<In<T>::kParts, KP, In<T>::kParts> im;
  FwdWarp<T, KP, kSave> w[kMaxWarps];
};

template <typename T, int KP, bool kSave>
__global__ void __launch_bounds__((kMaxWarps + 1) * 32, sizeof(FwdSmem<T, KP, kSave>) <= 113 * 1024 ? 2 : 1) fwd_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = FwdSmem<T, KP, kSave>;
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
    if (lane == 0) fill_images(im, a, sq.slot, 1, n, hk, hv);
    return;
  }
  const int vt = set * warps + warp;
  if (vt >= vts) return;
  FwdWarp<T, KP, kSave>& mine = sm.w[warp];
  const int cols = V - vt * kVt;
  const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
  const T* v_at = static_cast<const T*>(a.v) + sq.b * a.s.v_b + sq.t0 * a.s.v_t + (size_t)hv * V + vt * kVt;
  T* o_at = static_cast<T*>(a.o) + (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + vt * kVt;
  const long long o_t = (long long)a.s.Hv * V;
  const int tokens = sq.t1 - sq.t0;

  float S[kNt][4];
  load_state(S, a.s_init ? a.s_init + state_at : nullptr, cols, K, lane);
  float s_max = warp_max(S);
  if (n > 0) rows_in(mine.rows[0], v_at, a.s.v_t, tokens, cols, lane);
  copy_commit();
  if (n > 1) rows_ask(v_at + kC * a.s.v_t, a.s.v_t, tokens - kC, lane);
  if (n > 2) rows_ask(v_at + 2 * kC * a.s.v_t, a.s.v_t, tokens - 2 * kC, lane);

  for (int c = 0; c < n; ++c) {
    const int use = c & 1, len = tokens - c * kC;
    const size_t at_t = ((sq.slot + c) * a.s.Hv + hv) * vts + vt;
    if (c + 1 < n) rows_in(mine.rows[use ^ 1], v_at + (c + 1) * kC * a.s.v_t, a.s.v_t, len - kC, cols, lane);
    copy_commit();
    if (c + 3 < n) rows_ask(v_at + (c + 3) * kC * a.s.v_t, a.s.v_t, len - 3 * kC, lane);
    if constexpr (kSave) {
      if (lane == 0) bulk_wait_read();  // the images of the step before are out
      __syncwarp();
    }
    const Scal& sc = im.sc(use);
    const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);

    // S0 k^T and S0 q^T
    float x[8][4], o[8][4];
    zero(x), zero(o);
    if (!mbar_wait_bounded(a.status, &im.full_k[use], (c >> 1) & 1)) return;
    if (!mbar_wait_bounded(a.status, &im.full_q, use)) return;
#pragma unroll
    for (int kt = 0; kt < KP / 16; ++kt) {
      Frag<2> fs;
      to_a(fs, S[2 * kt], S[2 * kt + 1], sS);
      if constexpr (kSave) put_a(mine.s, kVt * KP, 16 * kt, fs, lane);
      Frag<P> fb[4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) b_nk<P>(fb[nb], im.k[use], kC, kC * KP, 16 * nb, 16 * kt, lane);
      mma_row<4>(x, fs, fb);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) b_nk<P>(fb[nb], im.q, kC, kC * KP, 16 * nb, 16 * kt, lane);
      mma_row_out<4>(o, fs, fb);
    }
    give_up(&im.free_q, lane);
    if constexpr (kSave) {
      wkv7::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        bulk_store(a.b.s_img + at_t * sizeof(mine.s), mine.s, sizeof(mine.s));
        bulk_commit();
      }
    }

    // r
    copy_wait<1>();
    __syncwarp();
    {
      float v[8][4];
      rows_get(v, mine.rows[use], lane, v_at);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 f = *reinterpret_cast<const float2*>(sc.ek + 8 * nt + 2 * t4), fo = *reinterpret_cast<const float2*>(sc.eq + 8 * nt + 2 * t4);
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
          x[nt][h] = fmaf(-f.x * inv_s, x[nt][h], v[nt][h]), x[nt][h + 1] = fmaf(-f.y * inv_s, x[nt][h + 1], v[nt][h + 1]);
          o[nt][h] *= fo.x * inv_s, o[nt][h + 1] *= fo.y * inv_s;
        }
      }
    }
    const float sR = pow2_scale(warp_max(x));

    // u = T r
    float u[8][4];
    zero(u);
    if (!mbar_wait_bounded(a.status, &im.full_t, use)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<2> fr;
      to_a(fr, x[2 * j], x[2 * j + 1], sR);
      Frag<2> ft[4];
#pragma unroll
      for (int i = j; i < 4; ++i) b_tri_nk<2>(ft[i], im.t, i, j, lane);
      mma_row<4>(u, fr, ft, j);
    }
    give_up(&im.free_t, lane);
    const float fu = sc.inv_t * pow2_inverse(sR);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[nt][e] *= fu;
    const float sU = pow2_scale(warp_max(u));
    if constexpr (kSave)
      if (lane == 0) a.b.su[at_t] = make_float2(inv_s, pow2_inverse(sU));

    // P u
    zero(x);
    if (!mbar_wait_bounded(a.status, &im.full_p, use)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Frag<(kSave || P == 2) ? 2 : 1> fp;
      to_a(fp, u[2 * j], u[2 * j + 1], sU);
      if constexpr (kSave) put_a(mine.u, kVt * kC, 16 * j, fp, lane);
      Frag<P> ft[4];
#pragma unroll
      for (int i = j; i < 4; ++i) b_tri_nk<P>(ft[i], im.p, i, j, lane);
      mma_row_out<4>(x, fp, ft, j);
    }
    give_up(&im.free_p, lane);
    if constexpr (kSave) {
      wkv7::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        bulk_store(a.b.u_img + at_t * sizeof(mine.u), mine.u, sizeof(mine.u));
        bulk_commit();
      }
    }
    const float fo = sc.inv_p * pow2_inverse(sU);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 f = *reinterpret_cast<const float2*>(sc.wk + 8 * nt + 2 * t4);
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        o[nt][h] = fmaf(fo, x[nt][h], o[nt][h]), o[nt][h + 1] = fmaf(fo, x[nt][h + 1], o[nt][h + 1]);
        u[nt][h] *= f.x, u[nt][h + 1] *= f.y;
      }
    }

    // S1: the products are added to S0 at their own scale, which is kept below
    // 2^60 of S0's so that S0 stays finite in it
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
    give_up(&im.free_k[use], lane);
    const float inv_w = pow2_inverse(sW);
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] *= inv_w;
    s_max = warp_max(S);
    rows_out(o, mine.rows[use], o_at + (size_t)c * kC * o_t, o_t, len, cols, lane);
  }
  if (kSave && lane == 0) bulk_wait_all();
  if (a.s_final) store_state(S, a.s_final + state_at, cols, K, lane);
}

template <typename T, int KP, bool kSave>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const int warps = chain_warps(a.s);
  constexpr size_t most = sizeof(FwdSmem<T, KP, kSave>);
  static_assert(most <= 227 * 1024, "shared memory of a block");
  auto kernel = fwd_kernel<T, KP, kSave>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  const int sets = (v_tiles(a.s.V) + warps - 1) / warps;
  const size_t smem = most - (kMaxWarps - warps) * sizeof(FwdWarp<T, KP, kSave>);
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), (warps + 1) * 32, smem, stream>>>(a);
  return cudaGetLastError();
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
