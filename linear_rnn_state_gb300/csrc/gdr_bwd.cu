// The gated delta rule's backward chain: the carried gradient dS of the state,
// from the last chunk to the first, and dv.
//
// For 64 rows of the state a block, with the images of q, k, T and P that the
// forward used, all transposed:
//   y^T   = do^T P (helpers) + wk (dS1 k^T)          the gradient of u
//   lam^T = y^T T = dv^T
//   dS0   = e^Gc dS1 + (scale e^G do)^T q (helpers) - (e^G lam)^T k
// Built as the forward chain (gdr_fwd.cu): three batches of tcgen05 products a
// step that wait for one another, the rows in registers between them. The
// helpers' two products do not wait for the chain: they are a step ahead. The
// helpers leave the images of dS1, lam and do for the gradients of q, k, g and
// beta (gdr_grad.cu). fp16 pairs throughout: dS, lam and do enter fp32 results.
//
// Two helper warps for each 16 rows, as the chain has: one took 5800 cycles over
// its step, and the chain waited for 1100 to 2200 of them (200 to 162 us).
//
// Bound by a step's latency, some 4700 cycles, and at 4.7 TB/s by memory in part
// (stores wait). Measured (64 steps): 4 x 4096 x 32 heads of 64 bfloat16 160 us, 4.7
// TB/s; 8 x 4032 x 12 x 64 fp32 207 us, 3.9 TB/s; 2 x 4095 x 32 x 128 bfloat16 189
// us, 4.8 TB/s. Measured and dropped, at the first size: four warps apart for dv and
// the images of dS1 and lam (201 to 193 us, at 128 keys 201 to 220); products issued
// in rolled loops, for less code (210 to 218).
#include "gdr_chain.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace {

// Warps: the chain's eight, eight helpers, and those without rows and one more to
// make them four. Registers of a thread of each, and what it is launched with.
constexpr int kHelpers = 2 * kWarps, kFiller = kChains + kHelpers, kThreads = (kFiller + 4) * 32;
enum { kIssuer = kFiller + 1, kHelpersIssuer };
constexpr int kRegChain = 120, kRegHelper = 96, kRegRest = 48, kRegLaunch = 96;
static_assert(2 * kRegChain + 2 * kRegHelper + kRegRest <= 5 * kRegLaunch, "a request for more would wait forever");

template <typename T, int KP>
struct alignas(1024) BwdSmem {
  static constexpr int P = In<T>::kParts, kPlaces = P * KP >= 256 ? 1 : 2;  // of do: what fits
  __half k[2][P * kC * KP], q[P * kC * KP];
  __half t[2 * kSpreadPart], p[2 * kSpreadPart];
  __half s[kWarps][2 * kVt * KP];  // images of dS1 on their way to memory
  float4 l[kWarps][8 * 32];        // lam as accumulator tiles
  union {                          // the helpers' ways to memory
    __half image[2 * kVt * kC];
    unsigned char dv[kRowsBytes<T>];
  } out[kWarps];
  unsigned char d[kWarps][kPlaces][kRowsBytes<T>];
  unsigned char scal[2][kChainScal];
  float most[6][kWarps][2];  // of the chain warps' dS, y and e^G lam, of the helpers' do, scale e^G do and lam
  float inv_s[kWarps], inv_d[2][kWarps], inv_g[2][kWarps];  // inverse scales of the warps' rows
  uint64_t full[5], free_k[2], free_q, free_t, free_p;
  uint64_t done_x, done_y, done_l, done_w, done_g, end[2];    // products
  uint64_t ready_s, ready_y, ready_w, ready_d, ready_e;       // operands in tensor memory
  uint64_t full_s[kWarps], free_s[kWarps], full_l[kWarps], free_l[kWarps], full_d[kWarps], free_y, free_g;
  uint32_t tmem;
  __device__ __forceinline__ const Scal& sc(int place) const { return *reinterpret_cast<const Scal*>(scal[place]); }
};

// Tensor memory, columns: the products x (and then the state's), do P, lam (which
// for 128 keys lies behind x, where the state's product comes later) and
// (scale e^G do) q; the operands dS1 (and then y, and then e^G lam) and do (and
// then scale e^G do), hi and lo.
template <int KP>
struct Columns {
  static constexpr uint32_t x = 0, y = KP, g = KP + 64, l = KP == 64 ? 2 * KP + 64 : 64;
  static constexpr uint32_t s_in = KP == 64 ? 256 : 320, d_in = s_in + KP, all = 512;
};

// The warp that fills the chunk's images; lane 0 of it. Step s is chunk slot - s.
template <typename T, int KP>
__device__ __forceinline__ void fill(BwdSmem<T, KP>& m, const Args& a, long long slot, int n, int hk, int hv) {
  constexpr int P = In<T>::kParts, image = P * kC * KP * 2, tri = kTriPart * 2;
  auto at_k = [&](int s) { return (size_t)(slot - s) * a.s.Hk + hk; };
  auto at_v = [&](int s) { return (size_t)(slot - s) * a.s.Hv + hv; };
  auto k = [&](int s) {
    uint64_t* bar = &m.full[s & 1];
    mbar_arrive_expect_tx(bar, image + kChainScal);
    bulk_load(m.k[s & 1], a.b.k_img + at_k(s) * image, image, bar);
    bulk_load(m.scal[s & 1], a.b.scal + at_v(s), kChainScal, bar);
  };
  auto spread = [&](__half* to, const char* from, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 2 * tri);
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bulk_load(to + part * kSpreadPart + 5 * j * 256, from + 2 * (part * kTriPart + tri_block(j, j)), (4 - j) * 512, bar);
  };
  auto q = [&](int s) {
    mbar_arrive_expect_tx(&m.full[kQ], image);
    bulk_load(m.q, a.b.q_img + at_k(s) * image, image, &m.full[kQ]);
  };
  auto t = [&](int s) {
#ifdef WKV7_DEBUG
    if (s + 1 == a.skip_t) return;
#endif
    spread(m.t, a.b.t_img + at_v(s) * Layout::tp_img, &m.full[kT]);
  };
  auto p = [&](int s) { spread(m.p, a.b.p_img + at_v(s) * Layout::tp_img, &m.full[kP]); };
  auto ask = [&](int s) {  // into L2
    if (s >= n) return;
    bulk_prefetch(a.b.k_img + at_k(s) * image, image);
    bulk_prefetch(a.b.q_img + at_k(s) * image, image);
    bulk_prefetch(a.b.t_img + at_v(s) * Layout::tp_img, 2 * tri);
    bulk_prefetch(a.b.p_img + at_v(s) * Layout::tp_img, 2 * tri);
    bulk_prefetch(a.b.scal + at_v(s), kChainScal);
  };
  k(0), p(0), q(0), t(0);
  if (n > 1) k(1);
  ask(2);
  int s = 1;
  for (; s < n; ++s) {  // in the order in which step s - 1 gives the places up
    if (!mbar_wait_bounded(a.status, &m.free_p, (s - 1) & 1)) break;
    p(s);
    if (!mbar_wait_bounded(a.status, &m.free_q, (s - 1) & 1)) break;
    q(s);
    if (!mbar_wait_bounded(a.status, &m.free_t, (s - 1) & 1)) break;
    t(s);
    if (!mbar_wait_bounded(a.status, &m.free_k[(s - 1) & 1], ((s - 1) >> 1) & 1)) break;
    if (s + 1 < n) k(s + 1);
    ask(s + 2);
  }
  if (s < n)
    for (uint64_t& b : m.full) drain(&b);
  else
    drain_last(m.full, n);
}

// An image to memory, half of it by each of two warps. (By loads and stores: the
// proxy fence that a bulk copy wants before it took 400 to 1400 cycles beside
// running products.)
template <int kHalves>
__device__ __forceinline__ void image_out(char* to, const __half* image, int half, int lane) {
  constexpr int kEach = kHalves / 512;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = (half * kEach + i) * 32 + lane;
    reinterpret_cast<uint4*>(to)[at] = reinterpret_cast<const uint4*>(image)[at];
  }
}
// The columns 32 half .. of an image of 16 rows of 64, which the warp itself wrote.
template <int kParts>
__device__ __forceinline__ void columns_out(char* to, const __half* image, int half, int lane) {
#pragma unroll
  for (int i = 0; i < 2 * kParts; ++i) {
    const int row = (i & 1) * 8 + (lane >> 2), at = (i >> 1) * kVt * kC + img(16, row, 32 * half + 8 * (lane & 3));
    *reinterpret_cast<uint4*>(to + 2 * at) = *reinterpret_cast<const uint4*>(image + at);
  }
}

template <typename T, int KP>
__global__ void __launch_bounds__(kThreads, 1) bwd_kernel(const Args a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  using Smem = BwdSmem<T, KP>;
  using Col = Columns<KP>;
  constexpr int P = In<T>::kParts, kPlaces = Smem::kPlaces;
  Smem& sm = *reinterpret_cast<Smem*>(raw + (-smem_addr(raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, t4 = lane & 3, own = warp & 3;
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + kWarps - 1) / kWarps;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&sm.full[0], &sm.full[1], &sm.full[kQ], &sm.full[kT], &sm.full[kP], &sm.free_q, &sm.free_t, &sm.free_p,
                        &sm.done_x, &sm.done_y, &sm.done_l, &sm.done_w, &sm.done_g, &sm.end[0], &sm.end[1]})
      mbar_init(b, 1);
    for (uint64_t* b : {&sm.free_k[0], &sm.free_k[1]}) mbar_init(b, kChains + kHelpers + 1);
    for (uint64_t* b : {&sm.free_y, &sm.free_g, &sm.ready_s, &sm.ready_y, &sm.ready_w}) mbar_init(b, kChains);
    for (uint64_t* b : {&sm.ready_d, &sm.ready_e}) mbar_init(b, kHelpers);
    for (int i = 0; i < kWarps; ++i)
      for (uint64_t* b : {&sm.full_s[i], &sm.full_l[i], &sm.free_s[i], &sm.free_l[i], &sm.full_d[i]}) mbar_init(b, 2);
    wkv7::fence_mbar_init();
  }
  if (warp == kFiller) wkv7::tmem_alloc(&sm.tmem, Col::all);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (a.small || a.segn) grid_go();  // the gradients, of the segment before
  SeqRange sq = seq_range(a.s, seq);
  if (a.segn) sq.t0 += a.seg0 * kC, sq.t1 = min(sq.t1, sq.t0 + a.segn * kC), sq.slot += a.seg0;
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V, vt = set * kWarps + own;
  const int cols = V - vt * kVt, tokens = sq.t1 - sq.t0;  // cols <= 0: this warp's rows are zeros
  const uint32_t tmem = sm.tmem, mine = tmem + ((uint32_t)own << 21);  // this warp's lanes
  const int half = warp / kWarps & 1, token0 = half * (kC / 2);  // of the two warps of the same rows
  Patience wait{a.status};
  auto ready = [&](uint64_t* bar) {  // what was stored to tensor memory is there
    tc_stored();
    tmem_fence_before_sync();
    signal(bar, lane);
  };

  // step s works on chunk n - 1 - s
  if (warp >= kFiller) {
    fewer_registers<kRegRest>();
    if (warp == kFiller) {
      if (lane == 0 && n > 0) fill(sm, a, sq.slot + n - 1, n, hk, hv);
    } else if (warp == kIssuer) {
      for (int s = 0; s < n; ++s) {
        const int use = s & 1;
        wait(&sm.full[use], s >> 1);
        wait(&sm.ready_s, use);
        tmem_fence_after_sync();
        if (elected()) {
          tc_rows<2, P, KP>(tmem + Col::x, tmem + Col::s_in, sm.k[use]);
          tc_commit(&sm.done_x);
        }
        wait(&sm.full[kT], use);
        wait(&sm.ready_y, use);
        tmem_fence_after_sync();
        if (elected()) {
          tc_tri_columns<2, 2>(tmem + Col::l, tmem + Col::s_in, sm.t);
          tc_commit(&sm.done_l);
          tc_commit(&sm.free_t);
        }
        wait(&sm.ready_w, use);
        tmem_fence_after_sync();
        if (elected()) {
          tc_columns<2, P, KP>(tmem + Col::x, tmem + Col::s_in, sm.k[use]);
          tc_commit(&sm.done_w);
          tc_commit(&sm.free_k[use]);
        }
      }
      if (elected()) tc_commit(&sm.end[0]);
      mbar_wait_bounded(a.status, &sm.end[0], 0);
    } else if (warp == kHelpersIssuer) {
      for (int s = 0; s < n; ++s) {
        const int use = s & 1;
        wait(&sm.full[kP], use);
        if (s > 0) wait(&sm.free_y, use ^ 1);
        wait(&sm.ready_d, use);
        tmem_fence_after_sync();
        if (elected()) {
          tc_tri_columns<P, 2>(tmem + Col::y, tmem + Col::d_in, sm.p);
          tc_commit(&sm.done_y);
          tc_commit(&sm.free_p);
        }
        wait(&sm.full[kQ], use);
        if (s > 0) wait(&sm.free_g, use ^ 1);
        wait(&sm.ready_e, use);
        tmem_fence_after_sync();
        if (elected()) {
          tc_columns<2, P, KP>(tmem + Col::g, tmem + Col::d_in, sm.q);
          tc_commit(&sm.done_g);
          tc_commit(&sm.free_q);
        }
      }
      if (elected()) tc_commit(&sm.end[1]);
      mbar_wait_bounded(a.status, &sm.end[1], 0);
    }
  } else if (warp < kChains) {  // ----------------------------------------- chain
    more_registers<kRegChain>();
    constexpr int kS = KP / 16;                // n8 tiles of the warp's half of the keys
    const int key0 = half * (KP / 2);
    const uint32_t s_in = mine + Col::s_in + half * (KP / 4), y_in = mine + Col::s_in + half * (kC / 4);
    const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
    auto both = [&](float m, int which) { return both_max(m, sm.most[which][own], half, 1 + own, lane); };
    float S[kS][4];
    load_state(S, a.dS_final ? a.dS_final + state_at : nullptr, cols, key0, K, lane);
    float s_max = both(warp_max(S), 0);
    for (int s = 0; s < n; ++s) {
      const int use = s & 1;
      const Scal& sc = sm.sc(use);
      // dS1 k^T
      const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);
      const Asked has_s(&sm.free_s[own], use ^ 1);
      Operand<2, kS / 2> f;
      f.split(S, sS), f.store(s_in, KP / 2);
      ready(&sm.ready_s);
      const Asked has_k(&sm.full[use], s >> 1), has_d(&sm.full_d[own], use);
      if (s > 0) wait(has_s);
      if (lane == 0 && half == 0) sm.inv_s[own] = inv_s;
      f.put(sm.s[own], kVt * KP, key0, lane);
      signal(&sm.full_s[own], lane);

      // y
      float x[4][4], y[4][4];
      wait(has_k);
      wait(has_d);
      const float fy = sc.inv_p * sm.inv_d[use][own], inv_g = sm.inv_g[use][own];
      float2 wk[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        wk[nt] = mul2(*reinterpret_cast<const float2*>(sc.wk + token0 + 8 * nt + 2 * t4), make_float2(inv_s, inv_s));
      wait(&sm.done_y, use);
      tmem_fence_after_sync();
      tc_load(y, mine + Col::y + token0);
      tc_loaded(y);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(y[nt], h, mul2(pair_of(y[nt], h), make_float2(fy, fy)));
      wait(&sm.done_x, use);
      tmem_fence_after_sync();
      tc_load(x, mine + Col::x + token0);
      tc_loaded(x);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(y[nt], h, fma2(wk[nt], pair_of(x[nt], h), pair_of(y[nt], h)));
      const float sY = pow2_scale(both(warp_max(y), 1)), fl = sc.inv_t * pow2_inverse(sY);
      {
        Operand<2, 2> f2;
        f2.split(y, sY), f2.store(y_in, 32);
      }
      ready(&sm.ready_y);
      signal(&sm.free_y, lane);

      // lam = T^T y
      const Asked has_l(&sm.free_l[own], use ^ 1);
      float2 ek[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        ek[nt] = mul2(*reinterpret_cast<const float2*>(sc.ek + token0 + 8 * nt + 2 * t4), make_float2(-fl, -fl));
      const float egc = sc.egc;
      wait(&sm.done_l, use);
      tmem_fence_after_sync();
      tc_load(x, mine + Col::l + token0);
      tc_loaded(x);

      // e^G lam, and the state's gradient
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(y[nt], h, mul2(pair_of(x[nt], h), ek[nt]));
      const float sW = pow2_scale(both(warp_max(y), 2)), inv_w = pow2_inverse(sW);
      {
        Operand<2, 2> fw;
        fw.split(y, sW), fw.store(y_in, 32);
      }
      ready(&sm.ready_w);
      if (s > 0) wait(has_l);
      tiles_put(sm.l[own] + token0 / 8 * 32, x, fl, lane);
      signal(&sm.full_l[own], lane);
      signal(&sm.free_k[use], lane);
#pragma unroll
      for (int nt = 0; nt < kS; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(S[nt], h, mul2(pair_of(S[nt], h), make_float2(egc, egc)));
      auto add = [&](uint32_t at, float f) {
        float z[kS][4];
        tc_load(z, at);
        tc_loaded(z);
#pragma unroll
        for (int nt = 0; nt < kS; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) set_pair(S[nt], h, fma2(make_float2(f, f), pair_of(z[nt], h), pair_of(S[nt], h)));
      };
      wait(&sm.done_g, use);
      tmem_fence_after_sync();
      add(mine + Col::g + key0, inv_g);
      tmem_fence_before_sync();
      signal(&sm.free_g, lane);
      wait(&sm.done_w, use);
      tmem_fence_after_sync();
      add(mine + Col::x + key0, inv_w);
      s_max = both(warp_max(S), 0);
    }
    if (a.dS_init && cols > 0) store_state(S, a.dS_init + state_at, cols, key0, K, lane);
  } else {  // -------------------------------------------------------------- helper
    const size_t first = (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + (cols > 0 ? vt * kVt : 0);
    const T* do_at = static_cast<const T*>(a.d_o) + first;
    T* dv_at = static_cast<T*>(a.dv) + first;
    const long long row_t = (long long)a.s.Hv * V;
    const uint32_t d_in = mine + Col::d_in + half * (kC / 4);
    const int meet = 1 + kWarps + own;
    auto both = [&](float m, int which) { return both_max(m, sm.most[which][own], half, meet, lane); };
    auto fetch = [&](int s) {  // do of step s, and a request for a later one
      const int c = n - 1 - s;
      if (c >= 0)
        rows_in<4>(sm.d[own][s % kPlaces], do_at + c * kC * row_t, row_t, cols > 0 ? tokens - c * kC : 0, cols, token0 / 8, lane);
      copy_commit();
      if (c >= 2 && cols > 0) rows_ask<4>(do_at + (c - 2) * kC * row_t, row_t, kC, token0 / 8, lane);
    };
    constexpr Record rec = b_record(KP, P);
    auto record_of = [&](int s) { return a.b.b_rec + (((sq.slot + n - 1 - s) * a.s.Hv + hv) * vts + vt) * rec.size; };
    float inv_d = 0.f;
    // What step s needs of do: its image, do^T P and (scale e^G do)^T q.
    auto ahead = [&](int s) {
      const int use = s & 1;
      const Scal& sc = sm.sc(use);
      float d[4][4];
      copy_wait<kPlaces - 1>();
      __syncwarp();
      rows_get(d, sm.d[own][s % kPlaces], token0 / 8, lane, do_at);
      __syncwarp();
      const float sD = pow2_scale(both(warp_max(d), 3));
      inv_d = pow2_inverse(sD);
      if (s > 0) wait(&sm.done_g, use ^ 1);
      tmem_fence_after_sync();
      {
        Operand<P, 2> f;
        f.split(d, sD), f.store(d_in, 32);
        ready(&sm.ready_d);
        f.put(sm.out[own].image, kVt * kC, token0, lane);
      }
      __syncwarp();
      if (cols > 0) columns_out<P>(record_of(s) + rec.d, sm.out[own].image, half, lane);
      __syncwarp();
      wait(&sm.full[use], s >> 1);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float2 eq = *reinterpret_cast<const float2*>(sc.eq + token0 + 8 * nt + 2 * t4);
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(d[nt], h, mul2(pair_of(d[nt], h), eq));
      }
      signal(&sm.free_k[use], lane);
      const float sE = pow2_scale(both(warp_max(d), 4));
      Operand<2, 2> f;
      f.split(d, sE);
      wait(&sm.done_y, use);  // do's place is free
      tmem_fence_after_sync();
      f.store(d_in, 32);
      ready(&sm.ready_e);
      // the chain has taken do P of the step before, and with it these of that step
      if (lane == 0 && half == 0) sm.inv_d[use][own] = inv_d, sm.inv_g[use][own] = pow2_inverse(sE);
      signal(&sm.full_d[own], lane);
      fetch(s + kPlaces);
    };
    fetch(0);
    if (kPlaces == 2) fetch(1);
    if (n > 0) ahead(0);
    for (int s = 0; s < n; ++s) {
      const int c = n - 1 - s, use = s & 1;
      char* record = record_of(s);
      const float inv_do = inv_d;
      wait(&sm.full_s[own], use);
      const float inv_s = sm.inv_s[own];
      if (cols > 0) image_out<2 * kVt * KP>(record, sm.s[own], half, lane);
      signal(&sm.free_s[own], lane);
      if (s + 1 < n) ahead(s + 1);

      wait(&sm.full_l[own], use);
      float x[4][4];
      tiles_get(x, sm.l[own] + token0 / 8 * 32, lane);
      signal(&sm.free_l[own], lane);
      const float sL = pow2_scale(both(warp_max(x), 5));
      {
        Operand<2, 2> f;
        f.split(x, sL), f.put(sm.out[own].image, kVt * kC, token0, lane);
      }
      __syncwarp();
      if (cols > 0) {
        columns_out<2>(record + rec.u, sm.out[own].image, half, lane);
        if (lane == 0 && half == 0) *reinterpret_cast<float4*>(record + rec.scales) = make_float4(inv_s, pow2_inverse(sL), inv_do, 0.f);
      }
      both_sync(meet);  // dv takes the place of the image
      rows_out(x, sm.out[own].dv, dv_at + (size_t)c * kC * row_t, row_t, tokens - c * kC, cols, token0 / 8, lane);
    }
    copy_wait_all();
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == kFiller) wkv7::tmem_dealloc(tmem, Col::all);
}

template <typename T, int KP>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(BwdSmem<T, KP>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  auto kernel = bwd_kernel<T, KP>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  static const bool enough = [kernel] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, reinterpret_cast<const void*>(kernel)) == cudaSuccess && f.numRegs >= kRegLaunch;
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  const int sets = (v_tiles(a.s.V) + kWarps - 1) / kWarps;
  kernel<<<(unsigned)((size_t)a.s.nseq * a.s.Hv * sets), kThreads, smem, stream>>>(a);
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
