// The gated delta rule's forward chain: the states from chunk to chunk, and o.
//
// With T, P, the decays and the images of q and k from the parallel pass
// (gdr_prep.cu), for 64 rows of the state (value columns) a block, all
// transposed (rows: value columns):
//   r^T = v^T - e^G (S0 k^T)                    chain
//   u^T = r^T T^T                               chain
//   S1  = e^Gc S0 + (wk u)^T k                  chain
//   o^T = scale e^G (S0 q^T) + u^T P^T          helpers
// Every product has the 64 rows as its m and goes to the tensor cores as one
// batch of tcgen05 instructions (gdr_tc.cuh). Between two batches a warp has 16
// of the rows in registers: it reads its accumulator tiles from tensor memory,
// scales them, splits them to fp16 pairs at the exact maximum of its own values,
// and writes them back as rows of the next batch's operand.
//
// What bounds it is the latency of a step, some 3700 cycles: three batches that
// wait for one another, each 300 to 450 cycles until its products are back and
// some 500 to scale, split and store the next operand. So the chain's warps, two
// for each 16 rows with half of the columns each, make only what the next state
// waits for; four helper warps beside them (which reach the same rows) make o and
// move the rows and images to and from memory. Two warps wait for operands and
// issue the products, one fills the chunk's images.
// kSave: the images of S0 and u go to memory for the backward.
//
// Arithmetic: fp16 pairs in every product, those of o too: a bfloat16 o is an
// fp32 result rounded once.
//
// Measured (64 steps; time, traffic): 4 x 4096 x 32 heads of 64 bfloat16 133 us,
// 4.5 TB/s; 8 x 4032 x 12 x 64 fp32 160 us, 3.6 TB/s; 2 x 4095 x 32 x 128 bfloat16
// 159 us, 4.3 TB/s. 65536 tokens of 40 heads (1024 steps on 40 of 152 SMs) 2.09 ms.
// (bfloat16 with 11 bits of S0, u and P in o: 127 and 155 us, and o 1.1e-3 from the
// rounded fp32 result.)
// Measured and dropped, at the first size: 128 rows, the hi and lo parts as one
// operand (twice the reads of tensor memory; 183 to 202 us); v by a warp of its own
// (145 to 156, it comes later); v and o by whole rows of 64 columns instead of 16 a
// warp (139 to 144); the images to memory by loads and stores instead of bulk copies
// (137 to 145); two helper warps for each 16 rows (128 to 133).
#include "gdr_chain.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace {

// Warps: the chain's eight, four helpers, and those without rows.
constexpr int kFiller = kChains + kWarps, kIssuer = kFiller + 1, kHelpersIssuer = kIssuer + 1, kThreads = (kHelpersIssuer + 1) * 32;

template <typename T, int KP, bool kSave>
struct alignas(1024) FwdSmem {
  static constexpr int P = In<T>::kParts, kPlaces = P * KP >= 256 ? 1 : 2;  // of v: what fits
  __half k[2][P * kC * KP], q[P * kC * KP];
  __half s[kSave ? kWarps : 1][2 * kVt * KP];  // images of S0 on their way to memory
  union {
    __half u[2 * kVt * kC];  // and of u
    unsigned char o[kRowsBytes<T>];
  } out[kWarps];
  __half t[2 * kTriPart], p[2 * kTriPart];
  unsigned char v[kWarps][kPlaces][kRowsBytes<T>];
  unsigned char scal[2][kChainScal];
  float most[3][kWarps][2];  // of the chain warps' S, r and u
  float inv_s[kWarps], inv_r[kWarps];  // inverse scales of the warps' rows
  uint64_t full[5], free_k[2], free_q, free_t, free_p;
  uint64_t done_x, done_q, done_u, done_w, done_o, end[2];  // products
  uint64_t ready_s, ready_r, ready_w, ready_u;  // operands in tensor memory
  uint64_t full_s[kWarps], full_u[kWarps], full_v[kWarps][2], free_v[kWarps], free_s, free_u;
  uint32_t tmem;
  __device__ __forceinline__ const Scal& sc(int place) const { return *reinterpret_cast<const Scal*>(scal[place]); }
};

// Tensor memory, columns: the products x (and then the state's), S0 q^T, u and
// u P^T (which for 128 keys takes u's place); the operands S0, r (and then wk u)
// and u, hi and lo.
template <int KP>
struct Columns {
  static constexpr uint32_t x = 0, q = KP, u = KP + 64, o = KP == 64 ? u + 64 : u;
  static constexpr uint32_t s_in = 256, r_in = s_in + KP, u_in = r_in + 64, all = 512;
};

// The warp that fills the chunk's images; lane 0 of it.
template <typename T, int KP, bool kSave>
__device__ __forceinline__ void fill(FwdSmem<T, KP, kSave>& m, const Args& a, long long slot, int n, int hk, int hv) {
  constexpr int P = In<T>::kParts, image = P * kC * KP * 2, tri = kTriPart * 2;
  auto at_k = [&](int c) { return (size_t)(slot + c) * a.s.Hk + hk; };
  auto at_v = [&](int c) { return (size_t)(slot + c) * a.s.Hv + hv; };
  auto k = [&](int c) {
    uint64_t* bar = &m.full[c & 1];
    mbar_arrive_expect_tx(bar, image + kChainScal);
    bulk_load(m.k[c & 1], a.b.k_img + at_k(c) * image, image, bar);
    bulk_load(m.scal[c & 1], a.b.scal + at_v(c), kChainScal, bar);
  };
  auto one = [&](void* to, const char* from, uint32_t bytes, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(to, from, bytes, bar);
  };
  auto q = [&](int c) { one(m.q, a.b.q_img + at_k(c) * image, image, &m.full[kQ]); };
  auto t = [&](int c) {
#ifdef WKV7_DEBUG
    if (c + 1 == a.skip_t) return;
#endif
    one(m.t, a.b.t_img + at_v(c) * Layout::tp_img, 2 * tri, &m.full[kT]);
  };
  auto p = [&](int c) { one(m.p, a.b.p_img + at_v(c) * Layout::tp_img, 2 * tri, &m.full[kP]); };
  auto ask = [&](int c) {  // into L2
    if (c >= n) return;
    bulk_prefetch(a.b.k_img + at_k(c) * image, image);
    bulk_prefetch(a.b.q_img + at_k(c) * image, image);
    bulk_prefetch(a.b.t_img + at_v(c) * Layout::tp_img, 2 * tri);
    bulk_prefetch(a.b.p_img + at_v(c) * Layout::tp_img, 2 * tri);
    bulk_prefetch(a.b.scal + at_v(c), kChainScal);
  };
  k(0), t(0), q(0), p(0);
  if (n > 1) k(1);
  ask(2);
  int c = 1;
  for (; c < n; ++c) {  // in the order in which step c - 1 gives the places up
    if (!mbar_wait_bounded(a.status, &m.free_q, (c - 1) & 1)) break;
    q(c);
    if (!mbar_wait_bounded(a.status, &m.free_t, (c - 1) & 1)) break;
    t(c);
    if (!mbar_wait_bounded(a.status, &m.free_k[(c - 1) & 1], ((c - 1) >> 1) & 1)) break;
    if (c + 1 < n) k(c + 1);
    if (!mbar_wait_bounded(a.status, &m.free_p, (c - 1) & 1)) break;
    p(c);
    ask(c + 2);
  }
  if (c < n)
    for (uint64_t& b : m.full) drain(&b);
  else
    drain_last(m.full, n);
}

template <typename T, int KP, bool kSave>
__global__ void __launch_bounds__(kThreads, 1) fwd_kernel(const Args a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  constexpr int P = In<T>::kParts, kPlaces = FwdSmem<T, KP, kSave>::kPlaces;
  using Col = Columns<KP>;
  using Smem = FwdSmem<T, KP, kSave>;
  Smem& sm = *reinterpret_cast<Smem*>(raw + (-smem_addr(raw) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, t4 = lane & 3, own = warp & 3;
  const int vts = (a.s.V + kVt - 1) / kVt, sets = (vts + kWarps - 1) / kWarps;
  const int set = blockIdx.x % sets, hv = blockIdx.x / sets % a.s.Hv, seq = blockIdx.x / (sets * a.s.Hv);
  const int hk = hv / (a.s.Hv / a.s.Hk);
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&sm.full[0], &sm.full[1], &sm.full[kQ], &sm.full[kT], &sm.full[kP], &sm.free_q, &sm.free_t, &sm.free_p,
                        &sm.done_x, &sm.done_q, &sm.done_u, &sm.done_w, &sm.done_o, &sm.end[0], &sm.end[1]})
      mbar_init(b, 1);
    for (uint64_t* b : {&sm.free_k[0], &sm.free_k[1]}) mbar_init(b, kChains + kWarps + 1);
    for (uint64_t* b : {&sm.ready_s, &sm.ready_r, &sm.ready_w}) mbar_init(b, kChains);
    for (uint64_t* b : {&sm.free_s, &sm.free_u, &sm.ready_u}) mbar_init(b, kWarps);
    for (int i = 0; i < kWarps; ++i) {
      for (uint64_t* b : {&sm.full_s[i], &sm.full_u[i], &sm.free_v[i]}) mbar_init(b, 2);
      mbar_init(&sm.full_v[i][0], 32), mbar_init(&sm.full_v[i][1], 32);
    }
    wkv7::fence_mbar_init();
  }
  if (warp == kFiller) wkv7::tmem_alloc(&sm.tmem, Col::all);
  grid_wait();
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (a.segn) grid_go();  // the next segment's preparation
  SeqRange sq = seq_range(a.s, seq);
  if (a.segn) sq.t0 += a.seg0 * kC, sq.t1 = min(sq.t1, sq.t0 + a.segn * kC), sq.slot += a.seg0;
  const int n = (sq.t1 - sq.t0 + kC - 1) / kC;
  const int K = a.s.K, V = a.s.V, vt = set * kWarps + own;
  const int cols = V - vt * kVt, tokens = sq.t1 - sq.t0;  // cols <= 0: this warp's rows are zeros
  const uint32_t tmem = sm.tmem, mine = tmem + ((uint32_t)own << 21);  // this warp's lanes
  const T* v_at = static_cast<const T*>(a.v) + sq.b * a.s.v_b + sq.t0 * a.s.v_t + (size_t)hv * V + (cols > 0 ? vt * kVt : 0);
  Patience wait{a.status};

  if (warp == kFiller) {
    if (lane == 0 && n > 0) fill(sm, a, sq.slot, n, hk, hv);
  } else if (warp == kIssuer) {
    for (int c = 0; c < n; ++c) {
      const int use = c & 1;
      wait(&sm.full[use], c >> 1);
      wait(&sm.ready_s, use);
      tmem_fence_after_sync();
      if (elected()) {
        tc_rows<2, P, KP>(tmem + Col::x, tmem + Col::s_in, sm.k[use]);
        tc_commit(&sm.done_x);
      }
      wait(&sm.full[kQ], use);
      if (elected()) {
        tc_rows<2, P, KP>(tmem + Col::q, tmem + Col::s_in, sm.q);
        tc_commit(&sm.done_q);
        tc_commit(&sm.free_q);
      }
      wait(&sm.full[kT], use);
      if (c > 0) wait(&sm.free_u, use ^ 1);
      wait(&sm.ready_r, use);
      tmem_fence_after_sync();
      if (elected()) {
        tc_tri_rows<2, 2>(tmem + Col::u, tmem + Col::r_in, sm.t);
        tc_commit(&sm.done_u);
        tc_commit(&sm.free_t);
      }
      wait(&sm.ready_w, use);
      tmem_fence_after_sync();
      if (elected()) {
        tc_columns<2, P, KP>(tmem + Col::x, tmem + Col::r_in, sm.k[use]);
        tc_commit(&sm.done_w);
        tc_commit(&sm.free_k[use]);
      }
    }
    if (elected()) tc_commit(&sm.end[0]);
    mbar_wait_bounded(a.status, &sm.end[0], 0);
  } else if (warp == kHelpersIssuer) {
    for (int c = 0; c < n; ++c) {
      const int use = c & 1;
      wait(&sm.full[kP], use);
      wait(&sm.ready_u, use);
      tmem_fence_after_sync();
      if (elected()) {
        tc_tri_rows<2, 2>(tmem + Col::o, tmem + Col::u_in, sm.p);
        tc_commit(&sm.done_o);
        tc_commit(&sm.free_p);
      }
    }
    if (elected()) tc_commit(&sm.end[1]);
    mbar_wait_bounded(a.status, &sm.end[1], 0);
  } else if (warp < kChains) {  // ----------------------------------------- chain
    constexpr int kS = KP / 16;                // n8 tiles of the warp's half of the keys
    const int half = warp / kWarps, key0 = half * (KP / 2), token0 = half * (kC / 2);
    const uint32_t s_in = mine + Col::s_in + half * (KP / 4), r_in = mine + Col::r_in + half * (kC / 4);
    const size_t state_at = (((size_t)seq * a.s.Hv + hv) * V + vt * kVt) * K;
    auto both = [&](float m, int which) { return both_max(m, sm.most[which][own], half, 1 + own, lane); };
    float S[kS][4];
    load_state(S, a.s_init ? a.s_init + state_at : nullptr, cols, key0, K, lane);
    float s_max = both(warp_max(S), 0);
    Asked has_s(&sm.free_s, 1);
    auto ready = [&](uint64_t* bar) {  // what was stored to tensor memory is there
      tc_stored();
      tmem_fence_before_sync();
      signal(bar, lane);
    };
    for (int c = 0; c < n; ++c) {
      const int use = c & 1, place = kPlaces == 2 ? use : 0;
      const Scal& sc = sm.sc(use);
      // S0 k^T and S0 q^T
      const float sS = pow2_scale(s_max), inv_s = pow2_inverse(sS);
      Operand<2, kS / 2> f;
      f.split(S, sS);
      if (c > 0) wait(has_s);
      f.store(s_in, KP / 2);
      ready(&sm.ready_s);
      const Asked has_k(&sm.full[use], c >> 1), has_v(&sm.full_v[own][place], kPlaces == 2 ? c >> 1 : c);
      if (lane == 0 && half == 0) sm.inv_s[own] = inv_s;
      if constexpr (kSave) {
        f.put(sm.s[own], kVt * KP, key0, lane);
        wkv7::fence_proxy_async_smem();
      }
      signal(&sm.full_s[own], lane);

      // r
      float x[4][4];
      {
        wait(has_k);
        float2 ek[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
          ek[nt] = mul2(*reinterpret_cast<const float2*>(sc.ek + token0 + 8 * nt + 2 * t4), make_float2(-inv_s, -inv_s));
        wait(has_v);
        float v[4][4];
        rows_get(v, sm.v[own][place], token0 / 8, lane, v_at);
        if (kPlaces == 1) signal(&sm.free_v[own], lane);
        wait(&sm.done_x, use);
        tmem_fence_after_sync();
        tc_load(x, mine + Col::x + token0);
        tc_loaded(x);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) set_pair(x[nt], h, fma2(ek[nt], pair_of(x[nt], h), pair_of(v[nt], h)));
      }
      const float sR = pow2_scale(both(warp_max(x), 1));
      const float fu = sc.inv_t * pow2_inverse(sR);
      {
        Operand<2, 2> fr;
        fr.split(x, sR), fr.store(r_in, 32);
      }
      ready(&sm.ready_r);

      // u = T r
      float2 wk[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        wk[nt] = mul2(*reinterpret_cast<const float2*>(sc.wk + token0 + 8 * nt + 2 * t4), make_float2(fu, fu));
      const float egc = sc.egc;
      wait(&sm.done_u, use);
      tmem_fence_after_sync();
      if (lane == 0 && half == 0) sm.inv_r[own] = fu;  // the helpers are past the one before
      tc_load(x, mine + Col::u + token0);
      tc_loaded(x);

      // wk u, and the state
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(x[nt], h, mul2(pair_of(x[nt], h), wk[nt]));
      const float sW = pow2_scale(both(warp_max(x), 2)), inv_w = pow2_inverse(sW);
      {
        Operand<2, 2> fw;
        fw.split(x, sW), fw.store(r_in, 32);
      }
      ready(&sm.ready_w);
      signal(&sm.full_u[own], lane);  // only now: the helper beside has its work while this warp waits
      signal(&sm.free_k[use], lane);
      has_s = Asked(&sm.free_s, use);
#pragma unroll
      for (int nt = 0; nt < kS; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(S[nt], h, mul2(pair_of(S[nt], h), make_float2(egc, egc)));
      wait(&sm.done_w, use);
      tmem_fence_after_sync();
      float y[kS][4];
      tc_load(y, mine + Col::x + key0);
      tc_loaded(y);
#pragma unroll
      for (int nt = 0; nt < kS; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(S[nt], h, fma2(make_float2(inv_w, inv_w), pair_of(y[nt], h), pair_of(S[nt], h)));
      s_max = both(warp_max(S), 0);
    }
    if (a.s_final && cols > 0) store_state(S, a.s_final + state_at, cols, key0, K, lane);
  } else {  // -------------------------------------------------------------- helper
    T* o_at = static_cast<T*>(a.o) + (((size_t)sq.b * a.s.T + sq.t0) * a.s.Hv + hv) * V + vt * kVt;
    const long long o_t = (long long)a.s.Hv * V;
    auto fetch = [&](int c) {  // v of chunk c, and a request for a later one
      const int place = kPlaces == 2 ? c & 1 : 0;
      if (c < n) {
        rows_in<8>(sm.v[own][place], v_at + c * kC * a.s.v_t, a.s.v_t, cols > 0 ? tokens - c * kC : 0, cols, 0, lane);
        copy_arrive(&sm.full_v[own][place]);
      }
      if (c + 2 < n && cols > 0) rows_ask<8>(v_at + (c + 2) * kC * a.s.v_t, a.s.v_t, tokens - (c + 2) * kC, 0, lane);
    };
    fetch(0);
    if (kPlaces == 2) fetch(1);
    for (int c = 0; c < n; ++c) {
      const int use = c & 1;
      constexpr Record rec = f_record(KP, P);
      char* record = a.b.f_rec + (((sq.slot + c) * a.s.Hv + hv) * vts + vt) * rec.size;
      const Scal& sc = sm.sc(use);
      if (kPlaces == 1 && c + 1 < n) {
        wait(&sm.free_v[own], c);
        fetch(c + 1);
      }
      // S0 q^T
      float o[8][4], x[8][4];
      wait(&sm.full_s[own], use);
      if (kSave && lane == 0 && cols > 0) {
        bulk_store(record, sm.s[own], sizeof(sm.s[own]));
        bulk_commit();
      }
      const float inv_s = sm.inv_s[own];
      wait(&sm.done_q, use);
      tmem_fence_after_sync();
      tc_load(o, mine + Col::q);
      tc_loaded(o);
      if (kSave && lane == 0) bulk_wait_read();
      tmem_fence_before_sync();
      signal(&sm.free_s, lane);

      // u P^T
      wait(&sm.full_u[own], use);
      tmem_fence_after_sync();
      tc_load(x, mine + Col::u);
      tc_loaded(x);
      const float fu = sm.inv_r[own];
      const float sU = pow2_scale(warp_max(x)), inv_u = pow2_inverse(sU) * fu;
      Operand<2, 4> f;
      f.split(x, sU), f.store(mine + Col::u_in, 32);
      tc_stored();
      tmem_fence_before_sync();
      signal(&sm.ready_u, lane);
      if (kPlaces == 2) fetch(c + 2);  // the chain is past v of this step
      if constexpr (kSave) {
        f.put(sm.out[own].u, kVt * kC, 0, lane);
        wkv7::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && cols > 0) {
          bulk_store(record + rec.u, sm.out[own].u, sizeof(sm.out[own].u));
          bulk_commit();
          *reinterpret_cast<float4*>(record + rec.scales) = make_float4(inv_s, inv_u, 0.f, 0.f);
        }
      }
      wait(&sm.full[use], c >> 1);
      const float fo = sc.inv_p * inv_u;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 eq = mul2(*reinterpret_cast<const float2*>(sc.eq + 8 * nt + 2 * t4), make_float2(inv_s, inv_s));
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(o[nt], h, mul2(pair_of(o[nt], h), eq));
      }
      signal(&sm.free_k[use], lane);
      wait(&sm.done_o, use);
      tmem_fence_after_sync();
      tc_load(x, mine + Col::o);
      tc_loaded(x);
      tmem_fence_before_sync();
      signal(&sm.free_u, lane);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) set_pair(o[nt], h, fma2(make_float2(fo, fo), pair_of(x[nt], h), pair_of(o[nt], h)));
      if (kSave && lane == 0) bulk_wait_read();
      __syncwarp();
      rows_out(o, sm.out[own].o, o_at + (size_t)c * kC * o_t, o_t, tokens - c * kC, cols, 0, lane);
    }
    if (kSave && lane == 0) bulk_wait_all();
    copy_wait_all();
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == kFiller) wkv7::tmem_dealloc(tmem, Col::all);
}

template <typename T, int KP, bool kSave>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(FwdSmem<T, KP, kSave>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  auto kernel = fwd_kernel<T, KP, kSave>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  const int sets = (v_tiles(a.s.V) + kWarps - 1) / kWarps;
  return launch_after(a.small, kernel, (unsigned)((size_t)a.s.nseq * a.s.Hv * sets), kThreads, smem, stream, a);
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
