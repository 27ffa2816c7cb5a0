// The gated delta rule's gradients of q, k, g and beta, every chunk and value
// head at once, from the images the chains left: the state before the chunk
// (S0) and u, the carried gradient after it (dS1), lam and do.
//
// With r_ij = e^(G_i - G_j), F_ij = scale r_ij do_i.u_j, E_ij = r_ij lam_i.u_j
// (j < i), f_i = scale do_i.u_i and the columns' beta:
//   dq   = scale e^G do S0 + (F beta) k          + f beta k
//   read = -e^G lam S0 - (E beta) k              (k where it reads the state)
//   w    = F^T q - E^T k + e^(Gc - G) u dS1      + f q
//   dk   = read + beta w,   dbeta = k.w          (k where it writes)
//   dG   = q.dq + k.read - beta k.w, Gc's own + <S1, dS1>; dg = its suffix sum
// The terms with f cancel in dG and are left out of the sums that form it: a
// sequence of one token has dg = 0 exactly, as it should. The terms of a pair
// (i, j) cancel in dg_t for t outside (j, i], and do so to fp32 rounding,
// because both sums are formed from the same images of F and E.
// <S1, dS1> = e^Gc <S0, dS1> + sum_j beta_j k_j.(e^(Gc - G_j) u_j dS1).
//
// Value heads that share a key head: a block takes them one after the other and
// adds their terms in shared memory where that has room (bfloat16, 128 keys, and
// enough key heads to fill the SMs: 2 x 4095 tokens of 16 key and 32 value heads
// 537 -> 461 us); otherwise each writes fp32 terms that a second kernel adds in the
// order of the heads. No atomics.
//
// Bound by the SM's shared-memory pipe and issue (57 % and 47 % at two blocks of
// eight warps, the tensor pipe 35 %): fragments by ldmatrix, four warps of a block
// reading the same columns. Measured: 4 x 4096 tokens x 32 heads of 64 bfloat16
// 329 us, 2.7 TB/s; 8 x 4032 x 12 x 64 fp32 415 us, 2.4 TB/s; 2 x 4095 x 16 and 32
// x 128 bfloat16 495 us. mma.sync and not tcgen05: every tile of 16 value columns
// has scales of its own, which products over several tiles would have to share.
#include <type_traits>

#include "gdr_common.cuh"

namespace gdr {
namespace {

// Warps: four times 16 rows by a warp for every 32 keys.
template <int KP>
constexpr int kThreads = KP / 32 * 128;

template <int P, int KP>
struct alignas(128) Tile {  // of 16 value columns: the forward's record, the backward's
  __half s[2 * kVt * KP], u[2 * kVt * kC];
  float4 su, pad0[7];  // inverse scales: of S0, of u
  __half ds[2 * kVt * KP], l[2 * kVt * kC], d[P * kVt * kC];
  float4 dsl, pad1[7];  // of dS1, of lam, of do
};
// How the gradients of q and k leave a block: its one value head's, that head's
// terms for the second kernel, or the sum over its key head's value heads.
enum Out { kAlone, kTerms, kSum };
constexpr int stages_of(Out out) { return out == kSum ? 3 : 4; }
// Rows of fp32 gradients on their way out, 32 bytes apart from a multiple of 128,
// so that the eight rows of an accumulator's store fall into different banks.
template <int KP>
constexpr int kRow = KP + 8;
struct alignas(128) Pairs {  // F and E as operands: columns times beta ks, and rows times qs or ks
  __half fb[2 * kTriPart], eb[2 * kTriPart], f[2 * kTriPart], e[2 * kTriPart];
};
template <typename T, int KP, Out kOut>
struct alignas(128) GradSmem {
  static constexpr int P = In<T>::kParts, kStages = stages_of(kOut);
  __half q[P * kC * KP], k[P * kC * KP];
  struct Apart {  // the next head's tiles come in while this one's pairs are in use
    Tile<P, KP> tile[kStages];
    Pairs pairs;
    float out[2][kC][kRow<KP>];
  };
  union Shared {
    Tile<P, KP> tile[kStages];
    Pairs pairs;  // once the tiles are used up
    float out[2][kC][kRow<KP>];  // once the pairs are
  };
  std::conditional_t<kOut == kSum, Apart, Shared> m;
  Scal scal;
  Rows rows;
  float fd[kC];               // f_i
  float dot[4][KP / 32][kC];  // row sums of 32 keys each: q.dq, k.read, k.w, k.(e^(Gc - G) u dS1)
  float sdot[KP / 8];
  float4 most[KP / 8];        // the warps' largest values of the four pairs
  uint64_t bar[kStages], bar_k, bar_s;
};

template <int P, int KP>
__device__ __forceinline__ float2 pick2(const __half* s, int row, int col) {
  const int at = img(kC, row, col);
  float2 x = unpack_f16(*reinterpret_cast<const uint32_t*>(s + at));
  if constexpr (P == 2) {
    const float2 y = unpack_f16(*reinterpret_cast<const uint32_t*>(s + kC * KP + at));
    x.x += y.x, x.y += y.y;
  }
  return x;
}

template <int N>
__device__ __forceinline__ float row_sum(const float (&x)[N][kC], int i) {
  float s = x[0][i];
#pragma unroll
  for (int n = 1; n < N; ++n) s += x[n][i];
  return s;
}

template <typename T, int KP, Out kOut>
__global__ void __launch_bounds__(kThreads<KP>, KP == 64 ? 2 : 1) grad_kernel(const Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = GradSmem<T, KP, kOut>;
  constexpr int P = In<T>::kParts, kWc = KP / 32, kNt = 4, kNf = 4 / kWc;  // n8 tiles of keys, 16-blocks of F's columns
  constexpr int kStages = Smem::kStages;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  auto& tiles = sm.m.tile;
  auto& pairs = sm.m.pairs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wc = warp >> 2, wr = wc & 1 ? 3 - (warp & 3) : warp & 3;
  const int g4 = lane >> 2, t4 = lane & 3, group = a.s.Hv / a.s.Hk;
  const int heads = kOut == kSum ? group : 1, per_slot = a.s.Hv / heads;
  int slot = blockIdx.x / per_slot;
  if (a.segn) slot = slot / a.segn * ((a.s.T + kC - 1) / kC) + a.seg0 + slot % a.segn;
  const int hv0 = blockIdx.x % per_slot * heads, hk = hv0 / group;
  ChunkAt c;
  if (a.small) grid_go();
  // in segments begun beside the chain of the segment before, of which nothing is read; elsewhere
  // every block waits for the chain, those without a chunk too: this kernel's end is the chain's
  if (!a.segn) grid_wait();
  if (!chunk_at(a.s, slot, c)) return;
  const int vts = (a.s.V + kVt - 1) / kVt, K = a.s.K;
  const size_t at_k = (size_t)slot * a.s.Hk + hk, at_v0 = (size_t)slot * a.s.Hv + hv0;
  constexpr int image = P * kC * KP * 2;

  // tile n of the block: of value head hv0 + n / vts; the heads' records follow one another
  const int n_tiles = heads * vts;
  auto load = [&](int n) {
#ifdef WKV7_DEBUG
    if (n + 1 == a.skip_tile) return;
#endif
    Tile<P, KP>& t = tiles[n % kStages];
    uint64_t* bar = &sm.bar[n % kStages];
    constexpr uint32_t f = f_record(KP, P).size, b = b_record(KP, P).size;
    static_assert(sizeof(Tile<P, KP>) == f + b, "a tile is its two records");
    const size_t at = at_v0 * vts + n;
    mbar_arrive_expect_tx(bar, f + b);
    bulk_load(t.s, a.b.f_rec + at * f, f, bar);
    bulk_load(t.ds, a.b.b_rec + at * b, b, bar);
  };
  auto load_scal = [&](int hg) {
    mbar_arrive_expect_tx(&sm.bar_s, sizeof(Scal));
    bulk_load(&sm.scal, a.b.scal + at_v0 + hg, sizeof(Scal), &sm.bar_s);
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.bar[s], 1);
    mbar_init(&sm.bar_k, 1), mbar_init(&sm.bar_s, 1);
    wkv7::fence_mbar_init();
  }
  __syncthreads();
  // an issue of a bulk copy takes some 80 cycles of its thread: a warp a tile
  if (lane == 0 && warp < kStages && warp < n_tiles) load(warp);
  if (lane == 0 && warp == kStages) {
    load_scal(0);
    mbar_arrive_expect_tx(&sm.bar_k, 2 * image + sizeof(Rows));
    bulk_load(sm.q, a.b.q_img + at_k * image, image, &sm.bar_k);
    bulk_load(sm.k, a.b.k_img + at_k * image, image, &sm.bar_k);
    bulk_load(&sm.rows, a.b.rows + at_k, sizeof(Rows), &sm.bar_k);
  }
  __syncwarp();
  const Scal& sc = sm.scal;
  const Rows& rows = sm.rows;
  const size_t tok = (size_t)c.b * a.s.T + c.t0;
  // A wait that this thread gives up on once: from then on it goes on without waiting
  // (all accesses are in bounds whatever the data), so that the block's barriers are
  // kept and nobody leaves while copies are in flight.
  bool ok = true;
  auto wait = [&](uint64_t* bar, int parity) {
    if (ok) ok = mbar_wait_bounded(a.status, bar, parity);
  };

  for (int hg = 0; hg < heads; ++hg) {
  const int hv = hv0 + hg;
  const int key0 = wc * 32;
  float dq[kNt][4], rd[kNt][4], w[kNt][4], F[2 * kNf][4], E[2 * kNf][4];
  zero(dq), zero(rd), zero(w), zero(F), zero(E);
  float sdot = 0.f;
  for (int v = 0; v < vts; ++v) {
    const int n = hg * vts + v;
    Tile<P, KP>& t = tiles[n % kStages];
    wait(&sm.bar[n % kStages], (n / kStages) & 1);
    const float4 su = t.su, dsl = t.dsl;
    Frag<P> fd;
    Frag<2> fl, fu;
    a_km<P>(fd, t.d, kVt, kVt * kC, 16 * wr, 0, lane);
    a_km<2>(fl, t.l, kVt, kVt * kC, 16 * wr, 0, lane);
    a_km<2>(fu, t.u, kVt, kVt * kC, 16 * wr, 0, lane);
    const float f1 = dsl.z * su.x, f2 = dsl.y * su.x, f3 = su.y * dsl.x;
#pragma unroll
    for (int nt = 0; nt < kNt; nt += 2) {
      Frag<2> fs, fds;
      float x[6][4];
      b_kn<2>(fs, t.s, kVt, kVt * KP, key0 + 8 * nt, 0, lane);
      b_kn<2>(fds, t.ds, kVt, kVt * KP, key0 + 8 * nt, 0, lane);
      mma_parts_first<P, 2>(x[0], x[1], fd, fs);
      mma_parts_first<2, 2>(x[2], x[3], fl, fs);
      mma_parts_first<2, 2>(x[4], x[5], fu, fds);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dq[nt + h][e] = fmaf(f1, x[h][e], dq[nt + h][e]);
          rd[nt + h][e] = fmaf(f2, x[2 + h][e], rd[nt + h][e]);
          w[nt + h][e] = fmaf(f3, x[4 + h][e], w[nt + h][e]);
        }
    }
#pragma unroll
    for (int b = 0; b < kNf; ++b) {
      const int jb = kNf * wc + b;
      if (jb <= wr) {
        float x[4][4];
        Frag<2> fj;
        b_kn<2>(fj, t.u, kVt, kVt * kC, 16 * jb, 0, lane);
        mma_parts_first<P, 2>(x[0], x[1], fd, fj);
        mma_parts_first<2, 2>(x[2], x[3], fl, fj);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            F[2 * b + h][e] = fmaf(dsl.z * su.y, x[h][e], F[2 * b + h][e]);
            E[2 * b + h][e] = fmaf(dsl.y * su.y, x[2 + h][e], E[2 * b + h][e]);
          }
      }
    }
    {  // <S0, dS1>: the same four values of both images
      static_assert(kVt * KP == 4 * kThreads<KP>, "four values a thread");
      const uint2 x0 = *reinterpret_cast<const uint2*>(t.s + 4 * tid), x1 = *reinterpret_cast<const uint2*>(t.s + kVt * KP + 4 * tid);
      const uint2 y0 = *reinterpret_cast<const uint2*>(t.ds + 4 * tid), y1 = *reinterpret_cast<const uint2*>(t.ds + kVt * KP + 4 * tid);
      const uint32_t xs[4] = {x0.x, x0.y, x1.x, x1.y}, ys[4] = {y0.x, y0.y, y1.x, y1.y};
      float sd = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 xh = unpack_f16(xs[e]), xl = unpack_f16(xs[2 + e]), yh = unpack_f16(ys[e]), yl = unpack_f16(ys[2 + e]);
        sd = fmaf(xh.x + xl.x, yh.x + yl.x, sd);
        sd = fmaf(xh.y + xl.y, yh.y + yl.y, sd);
      }
      sdot = fmaf(sd, su.x * dsl.x, sdot);
    }
    if (n + kStages < n_tiles) {
      __syncthreads();
      if (tid == 0 && ok) load(n + kStages);
    }
  }
  wait(&sm.bar_k, 0);
  wait(&sm.bar_s, hg & 1);

  // F and E with their decays, the diagonal of F apart, and the largest value of
  // each of the four operands that they become. (A bound by the largest decay ratio,
  // do, lam and u has no maximum to wait for and saved 4 to 6 % of a backward. But
  // these may belong to different tokens; then it is loose without limit, and pairs
  // at its scale lose bits, or all.)
  const int i0 = 16 * wr + g4;
  sdot = wkv7::group_allreduce<32>(sdot);
  const bool near = sc.near != 0.f;
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < 2 * kNf; ++n) {
    const int jb = kNf * wc + n / 2;
    if (jb > wr) continue;  // above the diagonal blocks
    const int j = 16 * kNf * wc + 8 * n + 2 * t4;
    const float c0 = sc.beta[j] * rows.ks[j], c1 = sc.beta[j + 1] * rows.ks[j + 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + 8 * h;
      float r0, r1;
      if (near) {
        r0 = sc.fa[i] * sc.fb[j], r1 = sc.fa[i] * sc.fb[j + 1];
      } else {
        r0 = j <= i ? expf((sc.gh[i] - sc.gh[j]) + (sc.gl[i] - sc.gl[j])) : 0.f;
        r1 = j + 1 <= i ? expf((sc.gh[i] - sc.gh[j + 1]) + (sc.gl[i] - sc.gl[j + 1])) : 0.f;
      }
      float x0 = a.s.scale * r0 * F[n][2 * h], x1 = a.s.scale * r1 * F[n][2 * h + 1], y0 = r0 * E[n][2 * h], y1 = r1 * E[n][2 * h + 1];
      if (jb == wr) {
        if (j == i) sm.fd[i] = a.s.scale * F[n][2 * h];
        if (j + 1 == i) sm.fd[i] = a.s.scale * F[n][2 * h + 1];
        x0 = j < i ? x0 : 0.f, x1 = j + 1 < i ? x1 : 0.f, y0 = j < i ? y0 : 0.f, y1 = j + 1 < i ? y1 : 0.f;
      }
      F[n][2 * h] = x0, F[n][2 * h + 1] = x1, E[n][2 * h] = y0, E[n][2 * h + 1] = y1;
      m[0] = fmaxf(m[0], fmaxf(fabsf(x0 * c0), fabsf(x1 * c1))), m[1] = fmaxf(m[1], fmaxf(fabsf(y0 * c0), fabsf(y1 * c1)));
      m[2] = fmaxf(m[2], fmaxf(fabsf(x0), fabsf(x1)) * rows.qs[i]), m[3] = fmaxf(m[3], fmaxf(fabsf(y0), fabsf(y1)) * rows.ks[i]);
    }
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) m[p] = warp_max_abs(m[p]);
  if (lane == 0) sm.sdot[warp] = sdot, sm.most[warp] = make_float4(m[0], m[1], m[2], m[3]);
  __syncthreads();  // and the tiles are used up
#pragma unroll
  for (int w = 0; w < KP / 8; ++w) {
    const float4 x = sm.most[w];
    m[0] = fmaxf(m[0], x.x), m[1] = fmaxf(m[1], x.y), m[2] = fmaxf(m[2], x.z), m[3] = fmaxf(m[3], x.w);
  }
  const float scale[4] = {pow2_scale(m[0]), pow2_scale(m[1]), pow2_scale(m[2]), pow2_scale(m[3])};
#pragma unroll
  for (int n = 0; n < 2 * kNf; ++n) {
    if (kNf * wc + n / 2 > wr) continue;
    const int j = 16 * kNf * wc + 8 * n + 2 * t4;
    const float c0 = sc.beta[j] * rows.ks[j], c1 = sc.beta[j + 1] * rows.ks[j + 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + 8 * h;
      const float q = rows.qs[i], k = rows.ks[i], x0 = F[n][2 * h], x1 = F[n][2 * h + 1], y0 = E[n][2 * h], y1 = E[n][2 * h + 1];
      // the factor first: with its scale it may pass fp32
      put2_tri(pairs.fb, i, j, x0 * c0 * scale[0], x1 * c1 * scale[0]);
      put2_tri(pairs.eb, i, j, y0 * c0 * scale[1], y1 * c1 * scale[1]);
      put2_tri(pairs.f, i, j, x0 * q * scale[2], x1 * q * scale[2]);
      put2_tri(pairs.e, i, j, y0 * k * scale[3], y1 * k * scale[3]);
    }
  }
  __syncthreads();

  // of the thread's two rows: e^(Gc - G), e^G, scale e^G, beta, f, f beta, qs, ks
  float ex[2], eg[2], sg[2], beta[2], fdi[2], fb[2], qs[2], ks[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = i0 + 8 * h;
    ex[h] = expf((sc.gh[kC - 1] - sc.gh[i]) + (sc.gl[kC - 1] - sc.gl[i]));
    eg[h] = sc.eg[i], sg[h] = a.s.scale * eg[h], beta[h] = sc.beta[i], fdi[h] = sm.fd[i], fb[h] = fdi[h] * beta[h];
    qs[h] = rows.qs[i], ks[h] = rows.ks[i];
  }
  const float inv[4] = {pow2_inverse(scale[0]), pow2_inverse(scale[1]), pow2_inverse(scale[2]), pow2_inverse(scale[3])};
  // (F beta) k and (E beta) k: the tokens up to the warp's rows
  {
    float x[kNt][4], y[kNt][4];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
      if (kt <= wr) {
        Frag<2> f, e;
        a_tri(f, pairs.fb, wr, kt, lane);
        a_tri(e, pairs.eb, wr, kt, lane);
#pragma unroll
        for (int nt = 0; nt < kNt; nt += 2) {
          Frag<P> fk;
          b_kn<P>(fk, sm.k, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
          if (kt == 0) {
            mma_parts_first<2, P>(x[nt], x[nt + 1], f, fk);
            mma_parts_first<2, P>(y[nt], y[nt + 1], e, fk);
          } else {
            mma_parts<2, P>(x[nt], x[nt + 1], f, fk);
            mma_parts<2, P>(y[nt], y[nt + 1], e, fk);
          }
        }
      }
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dq[nt][e] = fmaf(x[nt][e], inv[0], sg[e >> 1] * dq[nt][e]);
        rd[nt][e] = fmaf(y[nt][e], -inv[1], -eg[e >> 1] * rd[nt][e]);
      }
  }
  // F^T q and E^T k: the tokens from the warp's rows on
  float q[kNt][4], z[kNt][4];
#pragma unroll
  for (int kt = 3; kt >= 0; --kt)
    if (kt >= wr) {
      Frag<2> f, e;
      a_tri_t(f, pairs.f, kt, wr, lane);
      a_tri_t(e, pairs.e, kt, wr, lane);
#pragma unroll
      for (int nt = 0; nt < kNt; nt += 2) {
        Frag<P> fq, fk;
        b_kn<P>(fq, sm.q, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
        b_kn<P>(fk, sm.k, kC, kC * KP, key0 + 8 * nt, 16 * kt, lane);
        if (kt == 3) {
          mma_parts_first<2, P>(q[nt], q[nt + 1], f, fq);
          mma_parts_first<2, P>(z[nt], z[nt + 1], e, fk);
        } else {
          mma_parts<2, P>(q[nt], q[nt + 1], f, fq);
          mma_parts<2, P>(z[nt], z[nt + 1], e, fk);
        }
      }
    }
  float dot[4][2];
#pragma unroll
  for (int m = 0; m < 4; ++m) dot[m][0] = dot[m][1] = 0.f;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + 8 * h, col = key0 + 8 * nt + 2 * t4;
      const float2 qh = pick2<P, KP>(sm.q, i, col), kh = pick2<P, KP>(sm.k, i, col);
      const float qq[2] = {qh.x * qs[h], qh.y * qs[h]}, kk[2] = {kh.x * ks[h], kh.y * ks[h]};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = 2 * h + e;
        const float tail = ex[h] * w[nt][at], d = dq[nt][at], r = rd[nt][at];
        const float ww = fmaf(q[nt][at], inv[2], fmaf(z[nt][at], -inv[3], tail));
        dot[0][h] = fmaf(qq[e], d, dot[0][h]);
        dot[1][h] = fmaf(kk[e], r, dot[1][h]);
        dot[2][h] = fmaf(kk[e], ww, dot[2][h]);
        dot[3][h] = fmaf(kk[e], tail, dot[3][h]);
        dq[nt][at] = fmaf(fb[h], kk[e], d);
        rd[nt][at] = fmaf(beta[h], fmaf(fdi[h], qq[e], ww), r);  // dk
      }
    }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = wkv7::group_allreduce<4>(dot[m][h]);
      if (t4 == 0) sm.dot[m][wc][i0 + 8 * h] = x;
    }
  __syncthreads();
  if (warp == 0) {  // dbeta, and dg as suffix sums, two tokens a lane
    float dG[2], x = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      const float b = sc.beta[i], kw = row_sum(sm.dot[2], i);
      dG[e] = row_sum(sm.dot[0], i) + row_sum(sm.dot[1], i) - b * kw;
      x = fmaf(b, row_sum(sm.dot[3], i), x);
      if (i < c.len) a.dbeta[(tok + i) * a.s.Hv + hv] = fmaf(sm.fd[i], rows.qk[i], kw);
    }
    x = wkv7::group_allreduce<32>(x);
    float s0 = sm.sdot[0];
#pragma unroll
    for (int i = 1; i < KP / 8; ++i) s0 += sm.sdot[i];
    const float d0 = dG[0], d1 = dG[1] + (lane == 31 ? fmaf(sc.egc, s0, x) : 0.f);
    float s = d0 + d1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, s, o);
      if (lane + o < 32) s += y;
    }
    const float after = __shfl_down_sync(0xffffffffu, s, 1);
    const float s1 = d1 + (lane < 31 ? after : 0.f);
    // where e^g is 0 in fp32 (-inf, a reset) so is dg, without the sums' rounding
    const int i = 2 * lane;
    const float g0 = i ? (sc.gh[i] - sc.gh[i - 1]) + (sc.gl[i] - sc.gl[i - 1]) : sc.gh[0];
    const float g1 = (sc.gh[i + 1] - sc.gh[i]) + (sc.gl[i + 1] - sc.gl[i]);
    if (i < c.len) a.dg[(tok + i) * a.s.Hv + hv] = g0 < -150.f ? 0.f : s;
    if (i + 1 < c.len) a.dg[(tok + i + 1) * a.s.Hv + hv] = g1 < -150.f ? 0.f : s1;
  }
  // the rows in fp32; the pairs are used up (the barrier above)
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + 8 * h, col = key0 + 8 * nt + 2 * t4;
      float2* x = reinterpret_cast<float2*>(&sm.m.out[0][i][col]);
      float2* y = reinterpret_cast<float2*>(&sm.m.out[1][i][col]);
      float2 p = make_float2(dq[nt][2 * h], dq[nt][2 * h + 1]), r = make_float2(rd[nt][2 * h], rd[nt][2 * h + 1]);
      if (kOut == kSum && hg > 0) p.x += x->x, p.y += x->y, r.x += y->x, r.y += y->y;
      *x = p, *y = r;
    }
  if (kOut == kSum && hg + 1 < heads) {
    __syncthreads();  // warp 0 is past the scalars
    if (tid == 0 && ok) load_scal(hg + 1);
  }
  }
  __syncthreads();
  if (tid == 0 && !ok) {  // the thread that waits for every copy
    for (uint64_t& b : sm.bar) drain(&b);
    drain(&sm.bar_k), drain(&sm.bar_s);
  }

  // eight keys a lane: the gradient of the normalisation, and out. fp32 rows by
  // halves, four keys of each, so that a store writes whole sectors (8 x 4096
  // tokens of 12 heads of 64: 430 -> 409 us).
  using Stored = std::conditional_t<kOut == kTerms, float, T>;
  constexpr int kLanes = KP / 8, kPass = kThreads<KP> / kLanes;
  constexpr bool kHalves = sizeof(Stored) == 4;
  const int cl = tid % kLanes, c0 = kHalves ? 4 * cl : 8 * cl, c1 = kHalves ? KP / 2 + 4 * cl : 8 * cl + 4;
#pragma unroll
  for (int id = tid / kLanes; id < 2 * kC; id += kPass) {
    const bool is_k = id >= kC;
    const int i = id % kC;
    float d[8];
    const float4 lo = *reinterpret_cast<const float4*>(&sm.m.out[is_k][i][c0]), hi = *reinterpret_cast<const float4*>(&sm.m.out[is_k][i][c1]);
    d[0] = lo.x, d[1] = lo.y, d[2] = lo.z, d[3] = lo.w, d[4] = hi.x, d[5] = hi.y, d[6] = hi.z, d[7] = hi.w;
    if (kOut != kTerms && a.s.l2norm) {
      const __half* im = is_k ? sm.k : sm.q;
      float x[8], xd = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = pick2<P, KP>(im, i, (e < 2 ? c0 : c1) + 2 * (e & 1));
        x[2 * e] = y.x, x[2 * e + 1] = y.y;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) xd = fmaf(x[e], d[e], xd);
      xd = wkv7::group_allreduce<kLanes>(xd);
      const float s = is_k ? rows.ks[i] : rows.qs[i], r = is_k ? rows.rk[i] : rows.rq[i], f = -s * s * xd;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = r * fmaf(f, x[e], d[e]);
    }
    if (i < c.len) {
      Stored* out = kOut == kTerms ? reinterpret_cast<Stored*>(is_k ? a.b.dk_part : a.b.dq_part) + ((tok + i) * a.s.Hv + hv0) * K
                                   : static_cast<Stored*>(is_k ? a.dk : a.dq) + ((tok + i) * a.s.Hk + hk) * K;
      if constexpr (kHalves) {
        if (c0 < K) *reinterpret_cast<float4*>(out + c0) = make_float4(d[0], d[1], d[2], d[3]);
        if (c1 < K) *reinterpret_cast<float4*>(out + c1) = make_float4(d[4], d[5], d[6], d[7]);
      } else if (c0 < K) {
        store8(out + c0, d);
      }
    }
  }
  if (a.segn && blockIdx.x == 0) grid_wait();  // over only when that chain is, for what comes next
}

// dq and dk of a key head: its value heads' terms in order, then the gradient
// of the normalisation. 16 lanes a row of q or k, eight keys a lane.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  grid_wait();
  const size_t rows = (size_t)a.s.B * a.s.T * a.s.Hk;
  const size_t id = ((size_t)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int cl = threadIdx.x & 15, group = a.s.Hv / a.s.Hk, K = a.s.K;
  const bool is_k = id >= rows, in = id < 2 * rows && cl * 8 < K;
  const size_t row = is_k ? id - rows : id;
  // tokens in no sequence have no terms
  bool none = false;
  if (a.s.packed && in) {
    const int2 some = covered(a.s);
    const int t = (int)(row / a.s.Hk);
    none = t < some.x || t >= some.y;
  }
  float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in && !none) {
    const float* part = (is_k ? a.b.dk_part : a.b.dq_part) + row * group * K + cl * 8;
    for (int g = 0; g < group; ++g) {
      float y[8];
      load8(y, part + (size_t)g * K);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += y[e];
    }
  }
  if (a.s.l2norm) {
    if (in) {
      const size_t tok = row / a.s.Hk, b = tok / a.s.T, t = tok % a.s.T, h = row % a.s.Hk;
      load8(x, static_cast<const T*>(is_k ? a.k : a.q) + b * (is_k ? a.s.k_b : a.s.q_b) + t * (is_k ? a.s.k_t : a.s.q_t) + h * K + cl * 8);
    }
    float s2 = 0.f, xd = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= kSmall, s2 = fmaf(x[e], x[e], s2), xd = fmaf(x[e], d[e], xd);
    s2 = wkv7::group_allreduce<16>(s2), xd = wkv7::group_allreduce<16>(xd);
    const float r = 1.f / sqrtf(s2 + kSmallEps), f = r * (r * xd);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = r * kSmall * fmaf(-f, x[e], d[e]);
  }
  if (in && !none) {
    T* out = static_cast<T*>(is_k ? a.dk : a.dq) + row * K + cl * 8;
    store8(out, d);
  }
}

template <typename T, int KP, Out kOut>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(GradSmem<T, KP, kOut>);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  auto kernel = grad_kernel<T, KP, kOut>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  const size_t blocks = (a.segn ? (size_t)a.s.B * a.segn : a.s.slots) * (kOut == kSum ? a.s.Hk : a.s.Hv);
  const bool more = a.segn && a.seg0 > 0;  // segments
  e = launch_after(a.small || more, kernel, (unsigned)blocks, kThreads<KP>, smem, stream, a);
  if (e != cudaSuccess || kOut != kTerms || more) return e;
  const size_t rows = 2 * (size_t)a.s.B * a.s.T * a.s.Hk;
  return launch_after(a.small, join_kernel<T>, (unsigned)((rows * 16 + 255) / 256), 256, 0, stream, a);
}
template <typename T, int KP>
cudaError_t pick(const Args& a, cudaStream_t s) {
  if (a.s.Hv == a.s.Hk) return launch<T, KP, kAlone>(a, s);
  if constexpr (sums_in_block(In<T>::kParts, KP))
    if (!needs_terms(a.s, In<T>::kParts)) return launch<T, KP, kSum>(a, s);
  return launch<T, KP, kTerms>(a, s);
}

}  // namespace

cudaError_t launch_grad(const Args& a, bool bf16, cudaStream_t stream) {
  const bool wide = padded_k(a.s.K) == 128;
  if (bf16) return wide ? pick<__nv_bfloat16, 128>(a, stream) : pick<__nv_bfloat16, 64>(a, stream);
  return wide ? pick<float, 128>(a, stream) : pick<float, 64>(a, stream);
}

}  // namespace gdr
