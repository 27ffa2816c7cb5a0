// Linear attention with a decay, fp32 with heads of up to 64: o, and backward dv, from chunk to chunk on tcgen05.
//
// As linattn_chain.cu, with every operand in three bfloat16 parts (24 bits) and six products of parts for each
// product. The tiles of a chunk (a, b, x and u . x, 192 KB) leave room for one stage: threads split the values of
// the next chunk when the products that read the places are done (P x runs beside it); they ask for them while the
// products before run, and a warp has brought them to L2. Sums alone need b and u . x only, and have two places for each.
//
// Bound by the products: the tensor cores of a block's SM are busy 68 % of the time. 8 x 4096 x 12 x 64 takes 201 us (96
// blocks, 6.2 us a chunk); 65536 x 40 x 64 in segments 384 us for the sums (1.3 GB, 3.5 TB/s) and 790 us for the
// rest (2.7 GB, 3.4 TB/s; 490 of products at the rate of the largest ones).
//
// Tensor memory: the scores (128 columns, later the rows' P x), P (192), a S^T (64), the state's sum (64).
#include "linattn_tc.cuh"

namespace linattn {
namespace {

constexpr int kWorkers = 512, kMembers = kWorkers + 64, kThreads = kWorkers + 128;  // (registers go by four warps)
constexpr int kHelpWarp = 16;                                                          // and 17 issues

struct Smem {
  bf16_t a[3 * kCT * 64], b[3 * kCT * 64], x[3 * kCT * 64], xt[3 * kCT * 64];
  bf16_t s[3 * 64 * 64];
  Decays d[3];
  uint64_t scored, summed, out, end;
  uint32_t tmem;
};
static_assert(sizeof(Smem) <= 232448, "shared memory of a block");

struct Plan {
  int chunks;  // of a segment
  Way way;
  int keep;
};

template <bool kUpper, bool kSumsOnly>
__global__ void __launch_bounds__(kThreads, 1) chain32_kernel(const Args a, const Plan plan) {
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  enum { kScore = 0, kP = 128, kIn = 320, kU = 384, kO = 0, kCols = 512 };
  enum { kBarP = 1, kBarOut, kBarFree, kBarRows };
  constexpr int kPair = kWorkers + 32, kPart = kCT * 64;
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), sub = warp & 3, quarter = warp >> 2;
  const int hv = blockIdx.x % s.Hv, slot = blockIdx.x / s.Hv, hk = hv / (s.Hv / s.Hk);
  ChunkAt seg;
  constexpr bool sums = kSumsOnly;
  if (plan.way != kWhole) {
    if (!chunk_at(s, slot, kCT * plan.chunks, seg)) return;
  } else {  // a whole sequence, which may be empty: its state passes through
    const SeqRange r = seq_range(s, slot, kCT);
    seg.b = r.b, seg.t0 = seg.first = r.t0, seg.len = r.t1 - r.t0, seg.seq = slot;
  }
  if (warp == 0) wkv7::tmem_alloc(&sm.tmem, kCols);
  if (tid == 0) {
    for (uint64_t* b : {&sm.scored, &sm.summed, &sm.out, &sm.end}) mbar_init(b, 1);
    wkv7::fence_mbar_init();
  }
  const int n = (seg.len + kCT - 1) / kCT;
  const size_t tok = (size_t)seg.b * s.T + seg.t0;
  auto begin = [&](int i) { return (kUpper ? n - 1 - i : i) * kCT; };  // first token of the i-th chunk, from the segment's
  auto length = [&](int i) { return min(kCT, seg.len - begin(i)); };
  const long long st_a = kUpper ? s.k_t : s.q_t, st_b = kUpper ? s.q_t : s.k_t, st_x = kUpper ? (long long)s.Hv * s.V : s.v_t;
  const float* q = static_cast<const float*>(a.q) + seg.b * s.q_b + seg.t0 * s.q_t + (size_t)hk * s.K;
  const float* k = static_cast<const float*>(a.k) + seg.b * s.k_b + seg.t0 * s.k_t + (size_t)hk * s.K;
  const float* pa = kUpper ? k : q;
  const float* pb = kUpper ? q : k;
  const float* px = kUpper ? static_cast<const float*>(a.d_o) + (tok * s.Hv + hv) * s.V
                           : static_cast<const float*>(a.v) + seg.b * s.v_b + seg.t0 * s.v_t + (size_t)hv * s.V;

  if (warp >= kHelpWarp) fewer_registers<40>();
  if (warp > kHelpWarp + 1) return;
  if (warp == kHelpWarp) {
    const float* g = s.fixed ? a.g + hv : a.g + tok * s.Hv + hv;
    float r[4];
    auto ask = [&](int i) {
      if (i < n) load_decays(r, s.fixed ? g : g + (size_t)begin(i) * s.Hv, s.fixed ? 0 : s.Hv, length(i), lane);
    };
    auto make = [&](int i) {  // and the next chunk's are asked for
      if (i < n) {
        float x[4] = {r[0], r[1], r[2], r[3]};
        ask(i + 1);
        make_decays<true>(sm.d[i % 3], x, s.scale, lane);
      }
    };
    auto prefetch = [&](const float* p, long long stride, int cols, int len) {
      for (int r = lane; r < len; r += 32)
        for (int c = 0; c < cols; c += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + r * stride + c));
    };
    char* to = static_cast<char*>(kUpper ? a.dimages : a.images) +
               ((size_t)(n ? chunk_slot(s, seg, seg.t0 + begin(0)) : 0) * s.Hv + hv) * image_bytes(s.K, s.V);
    const long long next = (kUpper ? -1 : 1) * (long long)(s.Hv * image_bytes(s.K, s.V));
    auto leave = [&](int i) {  // the state before chunk i
      if (plan.keep && i < n && lane == 0) {
#pragma unroll
        for (int part = 0; part < 3; ++part) bulk_store(to + (size_t)part * kImagePiece, sm.s + part * 64 * 64, kImagePiece);
        bulk_commit();
        to += next;
      }
    };
    ask(0), make(0);
    meet(0, kMembers);
    make(1);
    meet(0, kMembers);
    leave(0);
    for (int i = 0; i < n; ++i) {
      if (!sums) {
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        announce(kBarFree, kPair);
      }
      make(i + 2);
      constexpr int kLead = sums ? 3 : 2;
      if (i + kLead < n) {
        const int t = begin(i + kLead), len = length(i + kLead);
        if (!sums) prefetch(pa + t * st_a, st_a, s.K, len);
        prefetch(pb + t * st_b, st_b, s.K, len), prefetch(px + t * st_x, st_x, s.V, len);
      }
      if (!sums) {
        meet(kBarOut, kPair);
        leave(i + 1);
      }
      meet(0, kMembers);
    }
    if (lane == 0) bulk_wait_all();
    meet(0, kMembers);
    return;
  }
  if (warp > kHelpWarp) {
    meet(0, kMembers);
    meet(0, kMembers);
    tmem_fence_after_sync();
    const uint32_t tm = sm.tmem;
    for (int i = 0; i < n; ++i) {
      if (elected()) {
        const uint64_t da = desc(sm.a), db = desc(sums && i & 1 ? sm.a : sm.b), ds = desc(sm.s), du = desc(sums && i & 1 ? sm.x : sm.xt);
        if (!sums) {
          terms<3, 3>([&](int p, int r, bool first) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma(tm + kScore, da + along<kCT>(ks) + p * (kRowPanel >> 4), db + along<kCT>(ks) + r * (kRowPanel >> 4),
                     product_of(128, 128, false, false), !first || ks > 0);
          });
          if (!LINATTN_SKIPPED(LINATTN_SKIP_SCORES, i + 1)) tc_commit(&sm.scored);
          terms<3, 3>([&](int p, int r, bool first) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma(tm + kIn, da + along<kCT>(ks) + p * (kRowPanel >> 4), ds + along<64>(ks) + r * (64 * 128 >> 4),
                     product_of(128, 64, false, false), !first || ks > 0);
          });
        }
        terms<3, 3>([&](int p, int r, bool first) {
#pragma unroll
          for (int ks = 0; ks < kCT / 16; ++ks)
            tc_mma(tm + kU, du + across(ks) + p * (kRowPanel >> 4), db + across(ks) + r * (kRowPanel >> 4), product_of(64, 64, true, true),
                   !first || ks > 0);
        });
        tc_commit(&sm.summed);
      }
      __syncwarp();
      if (!sums) meet(kBarP, kPair);
      tmem_fence_after_sync();
      if (!sums && elected()) {
        const uint64_t dx = desc(sm.x);
        terms<3, 3>([&](int p, int r, bool first) {
#pragma unroll
          for (int ks = 0; ks < kCT / 16; ++ks)
            tc_mma_t(tm + kO, tm + kP + part_at<3>(ks, p), dx + across(ks) + r * (kRowPanel >> 4), product_of(128, 64, false, true), !first || ks > 0);
        });
        tc_commit(&sm.out);
      }
      __syncwarp();
      meet(0, kMembers);
      tmem_fence_after_sync();
    }
    finish_products(&sm.end);
    meet(0, kMembers);
    return;
  }

  // ------------------------------------------------------------------ rows ---
  more_registers<104>();
  const int row = sub * 32 + lane;
  float* out = static_cast<float*>(kUpper ? a.dv : a.o) + (tok * s.Hv + hv) * s.V;
  // A chunk's values: two pieces of eight of each of a, b and x a thread.
  float va[sums ? 1 : 2][8], vb[2][8];
  const int piece = (tid & 7) * 8;
  auto ask = [&](int i) {
    const int t0 = begin(i), len = length(i);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = (e * kWorkers + tid) >> 3;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!sums) va[e][j] = 0.f;
        vb[e][j] = 0.f;
      }
      if (r < len && piece < s.K) {
        if (!sums) load8(va[e], pa + (t0 + r) * st_a + piece);
        load8(vb[e], pb + (t0 + r) * st_b + piece);
      }
    }
  };
  auto ask_x = [&](int i, float (&vx)[2][8]) {
    const int t0 = begin(i), len = length(i);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = (e * kWorkers + tid) >> 3;
#pragma unroll
      for (int j = 0; j < 8; ++j) vx[e][j] = 0.f;
      if (r < len && piece < s.V) load8(vx[e], px + (t0 + r) * st_x + piece);
    }
  };
  auto fill = [&](int i) {  // a and b
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int o = at(kCT, (e * kWorkers + tid) >> 3, piece);
      if (!sums) put8<3>(sm.a + o, kPart, va[e]);
      put8<3>((sums && i & 1 ? sm.a : sm.b) + o, kPart, vb[e]);
    }
  };
  auto fill_x = [&](const float (&vx)[2][8]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) put8<3>(sm.x + at(kCT, (e * kWorkers + tid) >> 3, piece), kPart, vx[e]);
  };
  auto fill_u = [&](int i, const float (&vx)[2][8]) {  // u . x
    const float* u = kUpper ? sm.d[i % 3].head : sm.d[i % 3].tail;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = (e * kWorkers + tid) >> 3;
      const float f = u[r];
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = vx[e][j] * f;
      put8<3>((sums && i & 1 ? sm.x : sm.xt) + at(kCT, r, piece), kPart, y);
    }
  };
  if (n) ask(0);
  // The state: rows 16 sub .., keys 16 quarter .. in accumulator tiles.
  float S[2][4];
  const int s_row = 16 * sub + (lane >> 2), s_col = quarter * 16 + 2 * (lane & 3);
  float* const states = (kUpper ? a.dstates : a.states) + ((size_t)s_row * s.K + s_col);
  const size_t state = (size_t)s.V * s.K;
  auto each = [&](float* m, auto f) {  // pairs of the state's numbers that exist; m is where its first is
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (s_row + 8 * h < s.V && s_col + 8 * t < s.K) f(reinterpret_cast<float2*>(m + (h ? 8 * s.K : 0) + 8 * t), S[t][2 * h], S[t][2 * h + 1]);
  };
  auto load = [](float2* p, float& x, float& y) {
    const float2 v = *p;
    x = v.x, y = v.y;
  };
  auto store = [](float2* p, float& x, float& y) { *p = make_float2(x, y); };
  auto planes = [&] {
    Frag<3> f;
    to_a(f, S[0], S[1]);
    const int o = at(64, 16 * sub + (lane & 15), quarter * 16 + (lane >> 4) * 8);
#pragma unroll
    for (int p = 0; p < 3; ++p) stsm4(sm.s + p * 64 * 64 + o, f.p[p]);
  };
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[t][e] = 0.f;
  const size_t ends = ((size_t)seg.seq * s.Hv + hv) * state + (size_t)s_row * s.K + s_col;
  float* init = const_cast<float*>(kUpper ? a.dS_final : a.s_init);
  if (plan.way == kResume)
    each(states + ((size_t)slot * s.Hv + hv) * state, load);
  else if (plan.way == kWhole && init)
    each(init + ends, load);
  planes();
  meet(0, kMembers);  // the first decays
  float vx[2][8];
  if (n) {
    ask_x(0, vx);
    fill(0), fill_u(0, vx);
    if (!sums) fill_x(vx);
    if (sums && n > 1) ask(1), ask_x(1, vx);
  }
  fence_proxy_async_smem();
  tmem_fence_before_sync();
  meet(0, kMembers);
  tmem_fence_after_sync();
  const uint32_t tm = sm.tmem, mine = tm + ((uint32_t)(sub * 32) << 16);
  Patience wait{a.status};
  float passed = 1.f;  // the decay of the segment so far
  for (int i = 0; i < n; ++i) {
    const Decays& d = sm.d[i % 3];
    if (!sums) {
      wait(&sm.scored, i);
      tmem_fence_after_sync();
      if (kUpper ? quarter >= sub : quarter <= sub) {
        float x[32];
        tc_read(x, mine + kScore + 32 * quarter);
        decayed<kUpper, true>(x, d, row, quarter, s.scale);
        store_parts<3>(mine + kP + 48 * quarter, x);
      } else {
        store_zeros<3>(mine + kP + 48 * quarter);
      }
      wkv7::tmem_wait_st();
      tmem_fence_before_sync();
      announce(kBarP, kPair);
    }
    const bool more = i + 1 < n;
    if (sums) {  // the next chunk's places beside the products, and the one's after it on their way
      if (more) fill(i + 1), fill_u(i + 1, vx);
      if (i + 2 < n) ask(i + 2), ask_x(i + 2, vx);
    } else if (more) {  // (on their way while the products run)
      ask(i + 1), ask_x(i + 1, vx);
    }
    wait(&sm.summed, i);
    tmem_fence_after_sync();
    {
      float x[2][4];
      tc_load_tiles(x, mine + kU + 16 * quarter);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = fmaf(d.whole, S[j][e], x[j][e]);
    }
    passed *= d.whole;
    if (sums) {
      fence_proxy_async_smem();
      tmem_fence_before_sync();
      meet(0, kMembers);
      tmem_fence_after_sync();
      continue;
    }
    meet(kBarFree, kPair);  // the last state has left
    planes();
    if (more) fill(i + 1), fill_u(i + 1, vx);
    wait(&sm.out, i);
    tmem_fence_after_sync();
    // rows through shared memory (x's place): 16 pieces of four values, permuted by the row
    float4* stage = reinterpret_cast<float4*>(sm.x);
    {
      float x[16], y[16];
      tc_read(x, mine + kIn + 16 * quarter);
      tc_read(y, mine + kO + 16 * quarter);
      const float w = (kUpper ? d.tail : d.head)[row];
#pragma unroll
      for (int p = 0; p < 4; ++p)
        stage[row * 16 + ((4 * quarter + p) ^ (row & 15))] =
            make_float4(fmaf(w, x[4 * p], y[4 * p]), fmaf(w, x[4 * p + 1], y[4 * p + 1]), fmaf(w, x[4 * p + 2], y[4 * p + 2]), fmaf(w, x[4 * p + 3], y[4 * p + 3]));
    }
    fence_proxy_async_smem();
    meet(kBarOut, kPair);
    {
      const int len = length(i);
      float* p = out + (size_t)begin(i) * s.Hv * s.V;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (e * kWorkers + tid) >> 4, c = tid & 15;
        const float4 v = stage[r * 16 + (c ^ (r & 15))];
        if (r < len && 4 * c < s.V) *reinterpret_cast<float4*>(p + (size_t)r * s.Hv * s.V + 4 * c) = v;
      }
    }
    meet(kBarRows, kWorkers);
    if (more) fill_x(vx);
    fence_proxy_async_smem();
    tmem_fence_before_sync();
    meet(0, kMembers);
    tmem_fence_after_sync();
  }
  float* last = kUpper ? a.dS_init : a.s_final;
  if (plan.way == kWhole && last) each(last + ends, store);
  if (sums) {
    each(states + ((size_t)slot * s.Hv + hv) * state, store);
    if (tid == 0) a.decay[(size_t)slot * s.Hv + hv] = passed;
  }
  meet(0, kMembers);
  if (warp == 0) wkv7::tmem_dealloc(tm, kCols);
}

template <bool kUpper, bool kSumsOnly>
cudaError_t launch(const Args& a, const Plan& plan, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(chain32_kernel<kUpper, kSumsOnly>), sizeof(Smem), done);
  if (e != cudaSuccess) return e;
  const Shape& s = a.s;
  const long long segs = plan.way != kWhole ? slot_count(s.B, s.T, s.nseq, s.packed, kCT * plan.chunks) : s.nseq;
  chain32_kernel<kUpper, kSumsOnly><<<(unsigned)(segs * s.Hv), kThreads, sizeof(Smem), stream>>>(a, plan);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chain32(const Args& a, bool backward, int chunks, Way way, bool keep, cudaStream_t stream) {
  const Plan plan{chunks, way, keep};
  if (way == kSums) return backward ? launch<true, true>(a, plan, stream) : launch<false, true>(a, plan, stream);
  return backward ? launch<true, false>(a, plan, stream) : launch<false, false>(a, plan, stream);
}

}  // namespace linattn
