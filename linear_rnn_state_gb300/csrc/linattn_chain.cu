// Linear attention with a decay, bfloat16: o, and backward dv, from chunk to chunk on tcgen05.
//
// A block takes a sequence (or a segment of one), a value head and 64 of its values, and goes through
// its chunks of 128 tokens with the state in registers. With a, b, x = q, k, v forward and k, q, do
// backward (there in reverse, the state being the gradient D of the state after the chunk):
//   P = mask . decay . (a b^T),  out = P x + w . (a S^T),  S <- e^{Gc} S + (u . x)^T b
// P, S and u . x enter the products in three parts of bfloat16 (24 bits), so that o and dv are fp32 results rounded once. (P and S
// in pairs, 16 bits, gave another neighbour of the exact value in 2 of 1000 places: 1e-4 in the 2-norm for 2e-5, at 4 % less of a chain's
// time with 64 keys and 10 % with 128.)
//
// Eight warps make P and the rows that leave, eight at the same time u . x and the state; one brings the tiles of a chunk
// to come (TMA), one forms its decays and says which chunks follow, one issues the products.
// For the gradients (linattn_grad.cu) the state before each chunk leaves as the tiles that products read, by bulk copies. With
// up to 64 keys
// the scores of chunk i + 1 are made and decayed while the other products of chunk i run (three stages of
// tiles, two places for the scores); wider keys leave room for two stages, and u . x goes by halves of the tokens.
//
// A block that is done takes the place of one that has not begun and goes on with its chunks as if they were its own, a
// list of steps ahead of the roles: no pause between short sequences (8191 tokens in 24 sequences, 32 heads of 128: 121 us for 147 when
// it was measured, 133 since the operands have three parts).
// The first chunks of a block are slow (10 thousand cycles, then 6), for its code is cold: each role has one copy of what it does.
//
// Bound by the steps' latency, 5600 cycles a chunk with 64 keys and 6700 with 128, of which the products take 1500 to 2200
// and shared memory's traffic 3100. Measured: 4 x 4096 x 32 x 64 94 us, backward 92 (369 MB with the images, 3.9 TB/s), 2 x 4095 x 32 x
// 128 119 us (403 MB, 3.4 TB/s; 128 blocks of 64 values). One team of warps for all of it took 101 for 95 us when that was tried.
#include "linattn_tc.cuh"

namespace linattn {
namespace {

// A block that has not begun gives its place up: `reply` gets its number, or that there is none, and `bar` 16 bytes.
__device__ __forceinline__ void claim_block(uint4* reply, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_addr(reply)),
               "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ bool claimed_block(const uint4* reply, unsigned& block) {
  uint32_t there;
  asm volatile("{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
               " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
               " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}"
               : "=r"(there), "=r"(block)
               : "r"(smem_addr(reply))
               : "memory");
  return there;
}

constexpr int kTeam = 256, kThreads = 2 * kTeam + 96;
constexpr int kBringWarp = 16, kDecayWarp = 17;  // and 18 issues

// A chunk of the block's run, as the warp of the decays tells all others, four ahead.
struct alignas(16) Step {
  int live, last, len;   // there is one; of its sequence or segment (for this head and slice); its tokens, 0 for a sequence of none
  int b, t;              // batch row, first token
  int hv, hk, slice;     // value and key head, which 64 values
  int ends;              // whose states at the ends (the sequence or segment)
  long long image;       // bytes from the first image to the piece of the state before it
};
constexpr int kSteps = 8, kAhead = 4;
constexpr int kSorted = 256;  // packed sequences that are taken by length

template <int KP>
struct Smem {
  static constexpr bool kEarly = KP == 64;
  static constexpr int kStages = kEarly ? 3 : 2, kHalves = kEarly ? 1 : 2, kXt = kCT / kHalves;
  struct Stage {
    bf16_t a[kCT * KP], b[kCT * KP], x[kCT * 64];
  };
  Stage stage[kStages];
  bf16_t xt[3 * kXt * 64];  // u . x
  bf16_t s[2 * 64 * KP];    // two parts of the state
  bf16_t third[kEarly ? 64 * KP : 8];  // its third; wider keys: in the place of the keys of the chunk before
  Decays d[3];
  Step step[kSteps];
  uint8_t order[kSorted];               // packed sequences, the longest first
  uint4 reply;                          // to a claim
  uint64_t claimed;                     // it is there
  uint64_t full[kStages];               // the tiles are there
  uint64_t end;                         // nothing is in flight
  uint64_t scored, first, summed, out;  // the scores; the first half of the state's sum, all of it; the rows
  uint64_t fed;                         // wider keys: the state before the chunk has been multiplied
  uint32_t tmem;
};

struct Plan {
  int chunks;  // of a segment
  Way way;
  int keep;
};

// kLate: the state's product comes behind the first half of the sum. (128 keys where images leave: 2 x 4095 x 32 x 128 132 -> 124 us; where
// they do not, before it: 24 sequences in 8191 tokens 138 -> 132.)
template <int KP, bool kUpper, bool kLate>
__global__ void __launch_bounds__(kThreads, 1) chain_kernel(const __grid_constant__ Maps maps, const Args a, const Plan plan) {
  extern __shared__ __align__(1024) unsigned char raw[];
  using M = Smem<KP>;
  M& sm = *reinterpret_cast<M*>(raw);
  constexpr int kTiles = KP / 16;  // n8 tiles of a warp's half of the keys
  constexpr bool kEarly = M::kEarly;
  constexpr int kSt = M::kStages, kXt = M::kXt;
  enum { kP = 0, kIn = kEarly ? 256 : 128, kO = kIn + 64, kU = kO + 64, kThird = 448, kCols = 512 };
  enum { kBarX = 1, kBarP, kBarX2, kBarPlanes, kBarFree, kBarOut };
  constexpr int kPair = kTeam + 32;  // a team and a warp beside it
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), sub = warp & 3, half = warp >> 2 & 1;
  const int slices = (s.V + 63) >> 6, group = s.Hv / s.Hk;
  const bool sums = plan.way == kSums;
  // More packed sequences than fit the GPU at once: long ones first, so that none is begun when the others end (24 in 8191
  // tokens, 32 heads of 128, eight draws: 127 us for 130 when it was measured).
  const bool sorted = plan.way == kWhole && s.starts && s.nseq <= kSorted && gridDim.x > kSms;
  int* const lengths = reinterpret_cast<int*>(sm.xt);
  if (sorted && tid < s.nseq) {
    const SeqRange r = seq_range(s, tid, kCT);
    lengths[tid] = (r.t1 - r.t0 + kCT - 1) / kCT;
  }
  if (warp == 0) wkv7::tmem_alloc(&sm.tmem, kCols);
  if (tid == 0) {
    for (uint64_t* b : {&sm.scored, &sm.first, &sm.summed, &sm.out, &sm.fed, &sm.end, &sm.claimed}) mbar_init(b, 1);
    for (uint64_t& b : sm.full) mbar_init(&b, 1);
    wkv7::fence_mbar_init();
  }
  auto step = [&](int i) -> const Step& { return sm.step[i & (kSteps - 1)]; };
  // The run of a block's chunks: of its own sequence or segment, head and slice, then of those of blocks that have not begun.
  Patience wait{a.status};
  ChunkAt seg;
  int run_hv = 0, run_slice = 0, run_ends = 0, run_n = 0, run_i = 0, claims = 0;
  bool more = true;
  auto begin_run = [&](unsigned block) {
    run_slice = block % slices, run_hv = block / slices % s.Hv, run_ends = block / slices / s.Hv;
    if (sorted) run_ends = sm.order[run_ends];
    if (plan.way != kWhole) {
      if (!chunk_at(s, run_ends, kCT * plan.chunks, seg)) return false;
    } else {  // a whole sequence, which may be empty: its state passes through a chunk of no tokens
      const SeqRange r = seq_range(s, run_ends, kCT);
      seg.b = r.b, seg.t0 = seg.first = r.t0, seg.len = r.t1 - r.t0, seg.seq = run_ends;
    }
    run_n = max(1, (seg.len + kCT - 1) / kCT), run_i = 0;
    return true;
  };
  auto claim = [&] {
    __syncwarp();
    ++claims;
    if (lane == 0 && !LINATTN_SKIPPED(LINATTN_SKIP_CLAIM, claims)) {
      fence_proxy_async_smem();
      wkv7::mbar_arrive_expect_tx(&sm.claimed, sizeof sm.reply);
      claim_block(&sm.reply, &sm.claimed);
    }
  };
  auto taken = [&](unsigned& block) {
    wait(&sm.claimed, claims - 1);
    return wait.ok && claimed_block(&sm.reply, block);
  };
  auto next_step = [&] {
    Step x{};
    const int off = (kUpper ? run_n - 1 - run_i : run_i) * kCT;
    x.live = 1, x.last = ++run_i == run_n, x.len = min(kCT, seg.len - off), x.b = seg.b, x.t = seg.t0 + off;
    x.hv = run_hv, x.hk = run_hv / group, x.slice = run_slice, x.ends = run_ends;
    x.image = x.len ? (chunk_slot(s, seg, x.t) * s.Hv + x.hv) * (long long)image_bytes(s.K, s.V) + x.slice * kImagePiece : 0;
    return x;
  };
  auto produce = [&](int j) {  // step j, by one warp
    while (more && run_i == run_n) {
      unsigned block;
      more = taken(block);
      if (more && !begin_run(block)) claim();
    }
    Step x{};
    if (more) {
      x = next_step();
      if (x.last) claim();
    }
    if (lane == 0) sm.step[j & (kSteps - 1)] = x;
    __syncwarp();
  };
  __syncthreads();
  if (sorted) {
    if (tid < s.nseq) {
      const int own = lengths[tid];
      int rank = 0;
      for (int j = 0; j < s.nseq; ++j) rank += lengths[j] > own || (lengths[j] == own && j < tid);
      sm.order[rank] = (uint8_t)tid;
    }
    __syncthreads();
  }
  if (warp != kBringWarp && warp != kDecayWarp) {
    __syncthreads();  // the first steps
    if (!step(0).live) {
      if (warp == 0) wkv7::tmem_dealloc(sm.tmem, kCols);
      return;
    }
  }

  if (warp >= kBringWarp) {
    if (warp == kDecayWarp) {
      float r[4];
      auto ask = [&](int i) {
        const Step& x = step(i);
        if (x.live) load_decays(r, a.g + x.hv + (s.fixed ? 0 : ((size_t)x.b * s.T + x.t) * s.Hv), s.fixed ? 0 : s.Hv, x.len, lane);
      };
      auto make = [&](int i) {  // and the next chunk's are asked for
        if (step(i).live) {
          const float x[4] = {r[0], r[1], r[2], r[3]};
          ask(i + 1);
          make_decays<false>(sm.d[i % 3], x, s.scale, lane);
        }
      };
      if (!begin_run(blockIdx.x)) claim();
      // (one loop for what comes before the first chunk and after: code runs cold once)
#pragma unroll 1
      for (int k = -kAhead;; ++k) {
        if (k >= 0) make(k);
        if (k < 0 || k >= 2) produce(k < 0 ? k + kAhead : k - 2 + kAhead);
        if (k >= 0 ? kEarly || k != 1 : k == -1) __syncthreads();
        if (k == -1) {
          if (!step(0).live) {
            if (!wait.ok) finish_copies(&sm.claimed);
            return;
          }
          ask(0);
        }
        if (k >= 2 && !step(k - 1).live) break;
      }
      if (!wait.ok) finish_copies(&sm.claimed);
      __syncthreads();
      return;
    }
    if (warp == kBringWarp) {
      constexpr int kLead = kEarly ? 2 : 1;  // chunks ahead
      const CUtensorMap *ma = kUpper ? &maps.k : &maps.q, *mb = kUpper ? &maps.q : &maps.k, *mx = kUpper ? &maps.d : &maps.v;
      const int b_a = kUpper ? s.k_b != 0 : s.q_b != 0, b_b = kUpper ? s.q_b != 0 : s.k_b != 0, b_x = kUpper || s.v_b != 0;
      auto bring_of = [&](const Step& w, int i, bool keys) {  // b, or a and x
        if (w.live && (wait.ok & (lane == 0)) && !LINATTN_SKIPPED(LINATTN_SKIP_TILES, i + 1)) {
          auto& st = sm.stage[i % kSt];
          uint64_t* bar = &sm.full[i % kSt];
          if (keys) {
            load_tile<KP>(st.b, mb, bar, 0, w.hk, w.t, w.b * b_b);
          } else {
            wkv7::mbar_arrive_expect_tx(bar, sums ? sizeof st.b + sizeof st.x : sizeof st);
            if (!sums) load_tile<KP>(st.a, ma, bar, 0, w.hk, w.t, w.b * b_a);
            load_tile<64>(st.x, mx, bar, 64 * w.slice, w.hv, w.t, w.b * b_x);
          }
        }
      };
      auto bring = [&](int i, bool keys) { bring_of(step(i), i, keys); };
      auto brought = [&](int i) {
        const Step& w = step(i);
        if (!w.live) return;
        wait(&sm.full[i % kSt], i / kSt);
        if (s.packed && w.len < kCT) {
          auto& st = sm.stage[i % kSt];
          if (!sums) clear_rows<KP>(st.a, w.len, lane, 32);
          clear_rows<KP>(st.b, w.len, lane, 32);
          clear_rows<64>(st.x, w.len, lane, 32);
          fence_proxy_async_smem();
        }
      };
      // the state before chunk i
      char* const images = static_cast<char*>(kUpper ? a.dimages : a.images);
      auto place_of = [&](int i) {
        const Step& w = step(i);
        return plan.keep && w.live && w.len && lane == 0 ? images + w.image : nullptr;
      };
      auto leave = [&](int i, char* to) {
        if (to) {
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int c = 0; c < KP / 64; ++c)
              bulk_store(to + (size_t)(part * (KP / 64) + c) * slices * kImagePiece,
                         (part < 2 ? sm.s + part * 64 * KP : kEarly ? sm.third : sm.stage[(i + kSt - 1) % kSt].b) + c * 64 * 64, kImagePiece);
          bulk_commit();
        }
      };
      const bool own = begin_run(blockIdx.x);
      if (own) {  // (the first tiles before the steps are there)
        const Step x = next_step();
        bring_of(x, 0, false), bring_of(x, 0, true);
      }
      __syncthreads();
      if (!step(0).live) return;
      if (!own) bring(0, false), bring(0, true);
      if (kEarly) bring(1, false), bring(1, true);
      brought(0);
      __syncthreads();
      leave(0, place_of(0));
      if (kEarly) {
        brought(1);
        __syncthreads();
      }
      for (int i = 0, live = 1; live; ++i) {
        bring(i + kLead, false);
        if (kEarly) bring(i + kLead, true);
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        if (!kEarly) {  // (where the state's third part has been until now)
          if (!sums) wait(&sm.fed, i);
          bring(i + kLead, true);
        }
        if (!sums) announce(kBarFree, kPair);
        brought(i + kLead);
        live = step(i + 1).live;
        char* const to = place_of(i + 1);
        if (!sums) {
          meet(kBarPlanes, kPair);
          leave(i + 1, to);
        }
        __syncthreads();
      }
      if (lane == 0) bulk_wait_all();
      if (!wait.ok)
        for (uint64_t& full : sm.full) finish_copies(&full);
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
      if (!LINATTN_SKIPPED(LINATTN_SKIP_SCORES, i + 1)) tc_commit(&sm.scored);
    };
    auto from_state = [&](int i) {
      const uint64_t da = desc(sm.stage[i % kSt].a), ds = desc(sm.s), dt = desc(kEarly ? sm.third : sm.stage[(i + kSt - 1) % kSt].b);
#pragma unroll 1
      for (int part = 2; part >= 0; --part) {
        const uint64_t d = part == 2 ? dt : ds + part * (64 * KP * 2 >> 4);
#pragma unroll
        for (int ks = 0; ks < KP / 16; ++ks) tc_mma(tm + kIn, da + along<kCT>(ks), d + along<64>(ks), product_of(128, 64, false, false), part < 2 || ks > 0);
      }
    };
    auto from_chunk = [&](int i) {
      const uint64_t dx = desc(sm.stage[i % kSt].x);
#pragma unroll 1
      for (int part = 2; part >= 0; --part)
#pragma unroll
        for (int ks = 0; ks < kCT / 16; ++ks) {
          const int place = kP + (kEarly ? i % 2 * 128 : 0);
          tc_mma_t(tm + kO, tm + place + two_and_third(ks, part, kThird - place + (ks >> 1) * 16), dx + across(ks), product_of(128, 64, false, true), part < 2 || ks > 0);
        }
    };
    auto sum = [&](int i, int h) {  // of half h of the tokens
      const uint64_t dx = desc(sm.xt), db = desc(sm.stage[i % kSt].b, kRowPanel) + across(h * (kXt / 16));
#pragma unroll 1
      for (int part = 2; part >= 0; --part)
#pragma unroll
        for (int ks = 0; ks < kXt / 16; ++ks)
          tc_mma(tm + kU, dx + across(ks) + part * (kXt * 128 >> 4), db + across(ks), product_of(64, KP, true, true), h > 0 || part < 2 || ks > 0);
    };
    if (kEarly) {
      if (!sums && elected()) scores(0);
      __syncwarp();
      __syncthreads();
      tmem_fence_after_sync();
    }
    for (int i = 0, live = 1, next = step(1).live; live; ++i) {
      if (!sums && elected()) {
        if (!kEarly) scores(i);
        if (kEarly && next) scores(i + 1);
        if (!kLate) from_state(i);
        if (!kEarly && !kLate) tc_commit(&sm.fed);
        if (kEarly) {
          from_chunk(i);
          tc_commit(&sm.out);
        }
      }
      __syncwarp();
      live = next, next = step(i + 2).live;
#pragma unroll 1
      for (int h = 0; h < M::kHalves; ++h) {
        if (h && !sums) {
          meet(kBarP, kPair);
          tmem_fence_after_sync();
          if (elected()) {
            from_chunk(i);
            tc_commit(&sm.out);
          }
          __syncwarp();
        }
        meet(h ? kBarX2 : kBarX, kPair);
        if (elected()) {
          sum(i, h);
          tc_commit(h == M::kHalves - 1 ? &sm.summed : &sm.first);
          if (kLate && !h && !sums) {
            from_state(i);
            tc_commit(&sm.fed);
          }
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

  const int team_tid = tid & (kTeam - 1);
  auto turn = [&] {  // every role's end of a chunk
    fence_proxy_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
  };
  if (warp < kTeam / 32) {  // ------------------------------------------------ P, and the rows that leave ---
    const int row = sub * 32 + lane;
    turn();
    const uint32_t mine = sm.tmem + ((uint32_t)(sub * 32) << 16);
    // The scores of chunk i, decayed, in three parts. Where there are two places for the scores, there is one for the third parts,
    // which the chunk before still reads: they are held until its rows are done.
    uint32_t held[kEarly ? 2 : 1][16];
    auto score = [&](int i) {
      const uint32_t at_p = mine + kP + (kEarly ? i % 2 * 128 : 0);
      wait(&sm.scored, i);
      tmem_fence_after_sync();
#pragma unroll 1
      for (int blk = half; blk < 4; blk += 2) {
        uint32_t(&third)[16] = held[kEarly];
#pragma unroll
        for (int j = 0; j < 16; ++j) held[0][j] = third[j], third[j] = 0;
        if (kUpper ? blk >= sub : blk <= sub) {
          float x[32];
          tc_read(x, at_p + 32 * blk);
          decayed<kUpper, false>(x, sm.d[i % 3], row, blk, s.scale);
          store_two(at_p + 32 * blk, x, third);
        } else {
          store_zeros<2>(at_p + 32 * blk);
        }
        if (!kEarly) tc_store16(mine + kThird + 16 * blk, third);
      }
    };
    auto stored = [&] {
      if (kEarly) {
#pragma unroll
        for (int b = 0; b < 2; ++b) tc_store16(mine + kThird + 16 * (half + 2 * b), held[kEarly && b]);
      }
      wkv7::tmem_wait_st();
      tmem_fence_before_sync();
    };
    for (int i = kEarly ? -1 : 0, live = 1; live; ++i) {
      live = step(i + 1).live;
      if (!sums) {
        if (kEarly) {
          if (live) score(i + 1);
          if (i < 0) stored();
        } else {
          score(i), stored();
          announce(kBarP, kPair);
        }
      }
      if (!sums && i >= 0) {
        const Decays& d = sm.d[i % 3];
        bf16_t* stage = sm.stage[i % kSt].a;
        const Step& to = step(i);
        const int len = to.len, vn = s.V - 64 * to.slice;
        bf16_t* p = static_cast<bf16_t*>(kUpper ? a.dv : a.o) + (((size_t)to.b * s.T + to.t) * s.Hv + to.hv) * s.V + 64 * to.slice;
        wait(&sm.out, i);
        tmem_fence_after_sync();
        if (kEarly && live) stored();
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
  const int s_row = 16 * sub + (lane >> 2), s_col = half * (KP / 2) + 2 * (lane & 3);
  auto each = [&](float* m, const Step& of, auto f) {  // pairs of the state's numbers that exist; m: [ends][Hv][V][K]
    const int v0 = 64 * of.slice + s_row;
    m += (((size_t)of.ends * s.Hv + of.hv) * s.V + v0) * s.K + s_col;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (v0 + 8 * h < s.V && s_col + 8 * t < s.K) f(reinterpret_cast<float2*>(m + (h ? 8 * s.K : 0) + 8 * t), S[t][2 * h], S[t][2 * h + 1]);
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
      stsm4(third + o, f.p[2]);
    }
  };
  float* const states = kUpper ? a.dstates : a.states;
  float* const init = plan.way == kResume ? states : plan.way == kWhole ? const_cast<float*>(kUpper ? a.dS_final : a.s_init) : nullptr;
  float* const last = sums ? states : plan.way == kWhole ? (kUpper ? a.dS_init : a.s_final) : nullptr;
  auto start = [&](const Step& of) {  // the state that a sequence or segment begins with
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = 0.f;
    if (init) each(init, of, load);
  };
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
  float passed = 1.f;  // the decay of the segment so far
#pragma unroll 1
  for (int i = -1, live = 1; live; ++i) {  // from -1, where the first state begins
    const Step &now = step(max(i, 0)), &next = step(i + 1);
    const bool ends = i < 0 || now.last;
    live = next.live;
    if (i >= 0) {
      const Decays& d = sm.d[i % 3];
      wait(&sm.full[i % kSt], i / kSt);
#pragma unroll 1
      for (int h = 0; h < M::kHalves; ++h) {
        if (h) wait(&sm.first, i);
        scaled(i, h);
        announce(h ? kBarX2 : kBarX, kPair);
      }
      if (ends && live && init) {  // the next state's 64 rows, one piece after the other
        const size_t from = (((size_t)next.ends * s.Hv + next.hv) * s.V + 64 * next.slice) * s.K + 32 * team_tid;
        if (32 * team_tid < min(64, s.V - 64 * next.slice) * s.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(init + from));
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
    }
    if (ends) {
      if (i >= 0) {
        if (last) each(last, now, store);
        if (sums && team_tid == 0 && now.slice == 0) a.decay[(size_t)now.ends * s.Hv + now.hv] = passed;
        passed = 1.f;
      }
      if (live) start(next);
    }
    if (!sums) {
      // (the state's products and copies have read it: the sum was issued after the former)
      if (i >= 0) meet(kBarFree, kPair);
      planes(kEarly ? sm.third : sm.stage[(i + kSt) % kSt].b);
      if (i >= 0) {
        fence_proxy_async_smem();
        announce(kBarPlanes, kPair);
      }
    }
    turn();
    if (kEarly && i < 0) __syncthreads();
  }
  __syncthreads();
}

template <int KP, bool kUpper, bool kLate>
cudaError_t launch(const Maps& maps, const Args& a, const Plan& plan, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<KP>);
  static_assert(sizeof(Smem<KP>) <= 232448, "shared memory of a block");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(chain_kernel<KP, kUpper, kLate>), smem, done);
  if (e != cudaSuccess) return e;
  const Shape& s = a.s;
  const long long segs = plan.way != kWhole ? slot_count(s.B, s.T, s.nseq, s.packed, kCT * plan.chunks) : s.nseq;
  chain_kernel<KP, kUpper, kLate><<<(unsigned)(segs * s.Hv * ((s.V + 63) / 64)), kThreads, smem, stream>>>(maps, a, plan);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chain(const Maps& maps, const Args& a, bool backward, int chunks, Way way, bool keep, cudaStream_t stream) {
  const Plan plan{chunks, way, keep};
  if (a.s.K <= 64) return backward ? launch<64, true, false>(maps, a, plan, stream) : launch<64, false, false>(maps, a, plan, stream);
  if (backward) return launch<128, true, true>(maps, a, plan, stream);
  return keep ? launch<128, false, true>(maps, a, plan, stream) : launch<128, false, false>(maps, a, plan, stream);
}

}  // namespace linattn
