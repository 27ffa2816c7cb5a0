// Linear attention with a decay, bfloat16: o, and backward dv, from chunk to chunk on tcgen05.
//
// A block takes a sequence (or a segment of one), a value head and 64 of its values, and goes through
// its chunks of 128 tokens with the state in registers. With a, b, x = q, k, v forward and k, q, do
// backward (there in reverse, the state being the gradient D of the state after the chunk):
//   P = mask . decay . (a b^T),  out = P x + w . (a S^T),  S <- e^{Gc} S + (u . x)^T b
// P x and a S^T end as bfloat16 values, so P and S enter them as pairs of bfloat16 (16 bits); u . x enters
// the state, an fp32 result, in three parts (24 bits).
//
// Eight warps make P and the rows that leave, eight at the same time u . x and the state; one brings the tiles of a chunk
// to come (TMA), one forms its decays, one issues the products.
// For the gradients (linattn_grad.cu) the state before each chunk leaves as the tiles that products read, its pair
// and a third part, by bulk copies. With up to 64 keys
// the scores of chunk i + 1 are made and decayed while the other products of chunk i run (three stages of
// tiles, two places for the scores); wider keys leave room for two stages, and u . x goes by halves of the tokens.
#include "linattn_tc.cuh"

namespace linattn {
namespace {

constexpr int kTeam = 256, kThreads = 2 * kTeam + 96;
constexpr int kBringWarp = 16, kDecayWarp = 17;  // and 18 issues

template <int KP>
struct Smem {
  static constexpr bool kEarly = KP == 64;
  static constexpr int kStages = kEarly ? 3 : 2, kHalves = kEarly ? 1 : 2, kXt = kCT / kHalves;
  struct Stage {
    bf16_t a[kCT * KP], b[kCT * KP], x[kCT * 64];
  };
  Stage stage[kStages];
  bf16_t xt[3 * kXt * 64];  // u . x
  bf16_t s[2 * 64 * KP];    // the state's pair
  bf16_t third[kEarly ? 64 * KP : 8];  // its third part; wider keys: in the place of the keys of the chunk before
  Decays d[3];
  uint64_t full[kStages];               // the tiles are there
  uint64_t end;                         // nothing is in flight
  uint64_t scored, first, summed, out;  // the scores; the first half of the state's sum, all of it; the rows
  uint32_t tmem;
};

struct Plan {
  int chunks;  // of a segment
  Way way;
  int keep;
};

template <int KP, bool kUpper>
__global__ void __launch_bounds__(kThreads, 1) chain_kernel(const __grid_constant__ Maps maps, const Args a, const Plan plan) {
  extern __shared__ __align__(1024) unsigned char raw[];
  using M = Smem<KP>;
  M& sm = *reinterpret_cast<M*>(raw);
  constexpr int kTiles = KP / 16;  // n8 tiles of a warp's half of the keys
  constexpr bool kEarly = M::kEarly;
  constexpr int kSt = M::kStages, kXt = M::kXt;
  enum { kP = 0, kIn = kEarly ? 256 : 128, kO = kIn + 64, kU = kO + 64, kCols = 512 };
  enum { kBarX = 1, kBarP, kBarX2, kBarPlanes, kBarFree, kBarOut };
  constexpr int kPair = kTeam + 32;  // a team and a warp beside it
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), sub = warp & 3, half = warp >> 2 & 1;
  const int slices = (s.V + 63) >> 6, slice = blockIdx.x % slices, hv = blockIdx.x / slices % s.Hv, slot = blockIdx.x / slices / s.Hv;
  const int hk = hv / (s.Hv / s.Hk), v0 = slice * 64, vn = min(64, s.V - v0);
  ChunkAt seg;
  const bool sums = plan.way == kSums;
  if (plan.way != kWhole) {
    if (!chunk_at(s, slot, kCT * plan.chunks, seg)) return;
  } else {  // a whole sequence, which may be empty: its state passes through
    const SeqRange r = seq_range(s, slot, kCT);
    seg.b = r.b, seg.t0 = seg.first = r.t0, seg.len = r.t1 - r.t0, seg.seq = slot;
  }
  if (warp == 0) wkv7::tmem_alloc(&sm.tmem, kCols);
  if (tid == 0) {
    for (uint64_t* b : {&sm.scored, &sm.first, &sm.summed, &sm.out, &sm.end}) mbar_init(b, 1);
    for (uint64_t& b : sm.full) mbar_init(&b, 1);
    wkv7::fence_mbar_init();
  }
  __syncthreads();
  const int n = (seg.len + kCT - 1) / kCT;
  const size_t tok = (size_t)seg.b * s.T + seg.t0;
  auto begin = [&](int i) { return (kUpper ? n - 1 - i : i) * kCT; };  // first token of the i-th chunk, from the segment's
  auto length = [&](int i) { return min(kCT, seg.len - begin(i)); };

  if (warp >= kBringWarp) {
    Patience wait{a.status};
    if (warp == kDecayWarp) {
      const float* g = s.fixed ? a.g + hv : a.g + tok * s.Hv + hv;
      float r[4];
      auto ask = [&](int i) {
        if (i < n) load_decays(r, s.fixed ? g : g + (size_t)begin(i) * s.Hv, s.fixed ? 0 : s.Hv, length(i), lane);
      };
      auto make = [&](int i) {  // and the next chunk's are asked for
        if (i < n) {
          float x[4] = {r[0], r[1], r[2], r[3]};
          ask(i + 1);
          make_decays(sm.d[i % 3], x, s.scale, lane);
        }
      };
      ask(0), make(0);
      __syncthreads();
      make(1);
      if (kEarly) __syncthreads();
      for (int i = 0; i < n; ++i) {
        make(i + 2);
        __syncthreads();
      }
      __syncthreads();
      return;
    }
    if (warp == kBringWarp) {
      constexpr int kLead = kEarly ? 2 : 1;  // chunks ahead
      const CUtensorMap *ma = kUpper ? &maps.k : &maps.q, *mb = kUpper ? &maps.q : &maps.k, *mx = kUpper ? &maps.d : &maps.v;
      const int b_a = kUpper ? s.k_b != 0 : s.q_b != 0, b_b = kUpper ? s.q_b != 0 : s.k_b != 0, b_x = kUpper || s.v_b != 0;
      auto bring = [&](int i, bool keys) {  // b, or a and x
        if (i < n && lane == 0) {
          auto& st = sm.stage[i % kSt];
          uint64_t* bar = &sm.full[i % kSt];
          const int t = seg.t0 + begin(i);
          if (keys) {
            load_tile<KP>(st.b, mb, bar, 0, hk, t, seg.b * b_b);
          } else {
            wkv7::mbar_arrive_expect_tx(bar, sums ? sizeof st.b + sizeof st.x : sizeof st);
            if (!sums) load_tile<KP>(st.a, ma, bar, 0, hk, t, seg.b * b_a);
            load_tile<64>(st.x, mx, bar, v0, hv, t, seg.b * b_x);
          }
        }
      };
      auto brought = [&](int i) {
        if (i >= n) return;
        wait(&sm.full[i % kSt], i / kSt);
        if (s.packed && length(i) < kCT) {
          auto& st = sm.stage[i % kSt];
          if (!sums) clear_rows<KP>(st.a, length(i), lane, 32);
          clear_rows<KP>(st.b, length(i), lane, 32);
          clear_rows<64>(st.x, length(i), lane, 32);
          fence_proxy_async_smem();
        }
      };
      // the state before chunk i: its pair, and the third part in the place of the keys of the chunk before
      char* const images = static_cast<char*>(kUpper ? a.dimages : a.images);
      char* to = images + ((size_t)(n ? chunk_slot(s, seg, seg.t0 + begin(0)) : 0) * s.Hv + hv) * image_bytes(s.K, s.V) + slice * kImagePiece;
      const long long next = (kUpper ? -1 : 1) * (long long)(s.Hv * image_bytes(s.K, s.V));
      auto leave = [&](int i) {
        if (plan.keep && i < n && lane == 0) {
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int c = 0; c < KP / 64; ++c)
              bulk_store(to + (size_t)(part * (KP / 64) + c) * slices * kImagePiece,
                         (part < 2 ? sm.s + part * 64 * KP : kEarly ? sm.third : sm.stage[(i + kSt - 1) % kSt].b) + c * 64 * 64, kImagePiece);
          bulk_commit();
          to += next;
        }
      };
      bring(0, false), bring(0, true);
      if (kEarly) bring(1, false), bring(1, true);
      brought(0);
      __syncthreads();
      leave(0);
      if (kEarly) {
        brought(1);
        __syncthreads();
      }
      for (int i = 0; i < n; ++i) {
        bring(i + kLead, false);
        if (kEarly) bring(i + kLead, true);
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        if (!kEarly) bring(i + kLead, true);
        if (!sums) announce(kBarFree, kPair);
        brought(i + kLead);
        if (!sums) {
          meet(kBarPlanes, kPair);
          leave(i + 1);
        }
        __syncthreads();
      }
      if (lane == 0) bulk_wait_all();
      if (!wait.ok)
        for (int st = 0; st < kSt; ++st) finish_copies(&sm.full[st], (n - st + kSt - 1) / kSt);
      __syncthreads();
      return;
    }
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = sm.tmem;
    auto scores = [&](int i) {
      const uint64_t da = desc(sm.stage[i % kSt].a), db = desc(sm.stage[i % kSt].b);
#pragma unroll
      for (int ks = 0; ks < KP / 16; ++ks)
        tc_mma(tm + kP + (kEarly ? i % 2 * 128 : 0), da + along<kCT>(ks), db + along<kCT>(ks), product_of(128, 128, false, false), ks > 0);
      tc_commit(&sm.scored);
    };
    auto from_state = [&](int i) {
      const uint64_t da = desc(sm.stage[i % kSt].a), ds = desc(sm.s);
#pragma unroll
      for (int part = 1; part >= 0; --part)
#pragma unroll
        for (int ks = 0; ks < KP / 16; ++ks)
          tc_mma(tm + kIn, da + along<kCT>(ks), ds + along<64>(ks) + part * (64 * KP * 2 >> 4), product_of(128, 64, false, false), part == 0 || ks > 0);
    };
    auto from_chunk = [&](int i) {
      const uint64_t dx = desc(sm.stage[i % kSt].x);
#pragma unroll
      for (int part = 1; part >= 0; --part)
#pragma unroll
        for (int ks = 0; ks < kCT / 16; ++ks)
          tc_mma_t(tm + kO, tm + kP + (kEarly ? i % 2 * 128 : 0) + part_at<2>(ks, part), dx + across(ks), product_of(128, 64, false, true), part == 0 || ks > 0);
    };
    auto sum = [&](int i, int h) {  // of half h of the tokens
      const uint64_t dx = desc(sm.xt), db = desc(sm.stage[i % kSt].b, kRowPanel) + across(h * (kXt / 16));
#pragma unroll
      for (int part = 2; part >= 0; --part)
#pragma unroll
        for (int ks = 0; ks < kXt / 16; ++ks)
          tc_mma(tm + kU, dx + across(ks) + part * (kXt * 128 >> 4), db + across(ks), product_of(64, KP, true, true), h > 0 || part < 2 || ks > 0);
    };
    if (kEarly) {
      if (n && !sums && elected()) scores(0);
      __syncwarp();
      __syncthreads();
      tmem_fence_after_sync();
    }
    for (int i = 0; i < n; ++i) {
      if (!sums && elected()) {
        if (!kEarly) scores(i);
        if (kEarly && i + 1 < n) scores(i + 1);
        from_state(i);
        if (kEarly) {
          from_chunk(i);
          tc_commit(&sm.out);
        }
      }
      __syncwarp();
      meet(kBarX, kPair);
      if (elected()) {
        sum(i, 0);
        tc_commit(kEarly ? &sm.summed : &sm.first);
      }
      __syncwarp();
      if (!kEarly) {
        if (!sums) {
          meet(kBarP, kPair);
          tmem_fence_after_sync();
          if (elected()) {
            from_chunk(i);
            tc_commit(&sm.out);
          }
          __syncwarp();
        }
        meet(kBarX2, kPair);
        if (elected()) {
          sum(i, 1);
          tc_commit(&sm.summed);
        }
        __syncwarp();
      }
      __syncthreads();
      tmem_fence_after_sync();
    }
    finish_products(&sm.end);
    __syncthreads();
    return;
  }

  Patience wait{a.status};
  const int team_tid = tid & (kTeam - 1);
  auto turn = [&] {  // every role's end of a chunk
    fence_proxy_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
  };
  if (warp < kTeam / 32) {  // ------------------------------------------------ P, and the rows that leave ---
    const int row = sub * 32 + lane;
    bf16_t* out = static_cast<bf16_t*>(kUpper ? a.dv : a.o) + (tok * s.Hv + hv) * s.V + v0;
    turn();
    const uint32_t mine = sm.tmem + ((uint32_t)(sub * 32) << 16);
    // The scores of chunk i, decayed, as pairs.
    auto score = [&](int i) {
      const uint32_t at_p = mine + kP + (kEarly ? i % 2 * 128 : 0);
      wait(&sm.scored, i);
      tmem_fence_after_sync();
#pragma unroll 1
      for (int blk = half; blk < 4; blk += 2) {
        if (kUpper ? blk >= sub : blk <= sub) {
          float x[32];
          tc_read(x, at_p + 32 * blk);
          decayed<kUpper>(x, sm.d[i % 3], row, blk, s.scale);
          store_parts<2>(at_p + 32 * blk, x);
        } else {
          store_zeros<2>(at_p + 32 * blk);
        }
      }
      wkv7::tmem_wait_st();
      tmem_fence_before_sync();
    };
    for (int i = kEarly ? -1 : 0; i < n; ++i) {
      if (!sums) {
        if (kEarly) {
          if (i + 1 < n) score(i + 1);
        } else {
          score(i);
          announce(kBarP, kPair);
        }
      }
      if (!sums && i >= 0) {
        const Decays& d = sm.d[i % 3];
        bf16_t* stage = sm.stage[i % kSt].a;
        wait(&sm.out, i);
        tmem_fence_after_sync();
        const float w = (kUpper ? d.tail : d.head)[row];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[16], y[16];
          tc_read(x, mine + kIn + 32 * half + 16 * h);
          tc_read(y, mine + kO + 32 * half + 16 * h);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = pack2(fmaf(w, x[8 * p + 2 * j], y[8 * p + 2 * j]), fmaf(w, x[8 * p + 2 * j + 1], y[8 * p + 2 * j + 1]));
            *reinterpret_cast<uint4*>(stage + at(kCT, row, 32 * half + 16 * h + 8 * p)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        meet(kBarOut, kTeam);
        const int len = length(i);
        bf16_t* p = out + (size_t)begin(i) * s.Hv * s.V;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = (e * kTeam + team_tid) >> 3, c = (team_tid & 7) * 8;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + at(kCT, r, c));
          if (r < len && c < vn) *reinterpret_cast<uint4*>(p + (size_t)r * s.Hv * s.V + c) = v;
        }
      }
      turn();
    }
    __syncthreads();
    if (warp == 0) wkv7::tmem_dealloc(sm.tmem, kCols);
    return;
  }

  // ------------------------------------------------------------------ u . x, and the state ---
  // The state: rows 16 sub .., keys KP / 2 half .. in accumulator tiles.
  float S[kTiles][4];
  const int s_row = v0 + 16 * sub + (lane >> 2), s_col = half * (KP / 2) + 2 * (lane & 3);
  float* const states = (kUpper ? a.dstates : a.states) + ((size_t)s_row * s.K + s_col);
  const size_t state = (size_t)s.V * s.K;
  auto each = [&](float* m, auto f) {  // pairs of the state's numbers that exist; m is where its first is
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (s_row + 8 * h < s.V && s_col + 8 * t < s.K) f(reinterpret_cast<float2*>(m + (h ? 8 * s.K : 0) + 8 * t), S[t][2 * h], S[t][2 * h + 1]);
  };
  auto load = [](float2* p, float& x, float& y) {
    const float2 v = *p;
    x = v.x, y = v.y;
  };
  auto store = [](float2* p, float& x, float& y) { *p = make_float2(x, y); };
  auto planes = [&](bf16_t* third) {
#pragma unroll
    for (int t = 0; t < kTiles; t += 2) {
      Frag<3> f;
      to_a(f, S[t], S[t + 1]);
      const int o = at(64, 16 * sub + (lane & 15), half * (KP / 2) + 8 * t + (lane >> 4) * 8);
      stsm4(sm.s + o, f.p[0]);
      stsm4(sm.s + 64 * KP + o, f.p[1]);
      if (plan.keep) stsm4(third + o, f.p[2]);
    }
  };
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[t][e] = 0.f;
  const size_t ends = ((size_t)seg.seq * s.Hv + hv) * state + (size_t)s_row * s.K + s_col;
  float* init = const_cast<float*>(kUpper ? a.dS_final : a.s_init);
  if (plan.way == kResume)
    each(states + ((size_t)slot * s.Hv + hv) * state, load);
  else if (plan.way == kWhole && init)
    each(init + ends, load);
  planes(kEarly ? sm.third : sm.stage[kSt - 1].b);
  turn();
  const uint32_t mine = sm.tmem + ((uint32_t)(sub * 32) << 16);
  // u . x of half h of the tokens
  auto scaled = [&](int i, int h) {
    const bf16_t* x0 = sm.stage[i % kSt].x;
    const float* u = kUpper ? sm.d[i % 3].head : sm.d[i % 3].tail;
#pragma unroll 2
    for (int e = team_tid; e < kXt * 8; e += kTeam) {
      const int r = e >> 3;
      float x[8];
      load8(x, x0 + at(kCT, h * kXt + r, (e & 7) * 8));
      const float f = u[h * kXt + r];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 y = times2(make_float2(x[j], x[j + 1]), make_float2(f, f));
        x[j] = y.x, x[j + 1] = y.y;
      }
      put8<3>(sm.xt + at(kXt, r, (e & 7) * 8), kXt * 64, x);
    }
    fence_proxy_async_smem();
  };
  if (kEarly) __syncthreads();
  float passed = 1.f;  // the decay of the segment so far
  for (int i = 0; i < n; ++i) {
    const Decays& d = sm.d[i % 3];
    wait(&sm.full[i % kSt], i / kSt);
    scaled(i, 0);
    announce(kBarX, kPair);
    if (!kEarly) {
      wait(&sm.first, i);
      scaled(i, 1);
      announce(kBarX2, kPair);
    }
    wait(&sm.summed, i);
    tmem_fence_after_sync();
#pragma unroll
    for (int t = 0; t < kTiles; t += 4) {
      float x[4][4];
      tc_load_tiles(x, mine + kU + half * (KP / 2) + 8 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t + j][e] = fmaf(d.whole, S[t + j][e], x[j][e]);
    }
    passed *= d.whole;
    if (!sums) {
      // (the state's products and copies have read it: the sum was issued after the former)
      meet(kBarFree, kPair);
      planes(kEarly ? sm.third : sm.stage[i % kSt].b);
      fence_proxy_async_smem();
      announce(kBarPlanes, kPair);
    }
    turn();
  }
  float* last = kUpper ? a.dS_init : a.s_final;
  if (plan.way == kWhole && last) each(last + ends, store);
  if (sums) {
    each(states + ((size_t)slot * s.Hv + hv) * state, store);
    if (team_tid == 0 && slice == 0) a.decay[(size_t)slot * s.Hv + hv] = passed;
  }
  __syncthreads();
}

template <int KP, bool kUpper>
cudaError_t launch(const Maps& maps, const Args& a, const Plan& plan, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<KP>);
  static_assert(sizeof(Smem<KP>) <= 232448, "shared memory of a block");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(chain_kernel<KP, kUpper>), smem, done);
  if (e != cudaSuccess) return e;
  const Shape& s = a.s;
  const long long segs = plan.way != kWhole ? slot_count(s.B, s.T, s.nseq, s.packed, kCT * plan.chunks) : s.nseq;
  chain_kernel<KP, kUpper><<<(unsigned)(segs * s.Hv * ((s.V + 63) / 64)), kThreads, smem, stream>>>(maps, a, plan);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chain(const Maps& maps, const Args& a, bool backward, int chunks, Way way, bool keep, cudaStream_t stream) {
  const Plan plan{chunks, way, keep};
  if (a.s.K <= 64) return backward ? launch<64, true>(maps, a, plan, stream) : launch<64, false>(maps, a, plan, stream);
  return backward ? launch<128, true>(maps, a, plan, stream) : launch<128, false>(maps, a, plan, stream);
}

}  // namespace linattn
