// Linear attention with a decay: dq, dk and dg of every chunk, all chunks at once, on tcgen05 (bfloat16, and fp32
// with heads of up to 64).
//
// With G the running sum of the chunk's log decays, Gc the whole sum, S the state before the chunk and D the
// gradient of the state after it:
//   dq_i = sum_{j<=i} A_ij k_j + scale e^{G_i} S^T do_i,   A_ij = scale e^{G_i - G_j} (do_i.v_j)
//   dk_j = sum_{i>=j} A_ij q_i + e^{Gc - G_j} D^T v_j
// A log decay g_t moves whatever passes it: pairs j < t <= i of the chunk, the state's part that is read
// from t on, what is written before t and read after the chunk, and what passes the whole chunk,
//   dg_t = sum_{j<t<=i} A_ij (q_i.k_j) + sum_{i>=t} q_i.(scale e^{G_i} S^T do_i) + sum_{j<t} k_j.(e^{Gc - G_j} D^T v_j)
//          + e^{Gc} <S, D>,
// all of them sums: no differences of large ones.
//
// A block takes a chunk and a key head, one of its value heads after the other. A thread has a row of the
// products, a half or (kQ = 4) a quarter of its columns. A, S and D enter in three parts (24 bits), S and D 64 keys of them
// at a time, and fp32 inputs too. (A as a pair, for bfloat16 results: 1e-4 from the exact values rounded for 2e-5, at 7 % less of the
// gradients' time.)
//
// Bound by latency: a chunk's tiles and states come, are multiplied, decayed, multiplied again and read out, twice, one
// step after the other, with one block an SM but for bfloat16's heads of 64. Measured: 4 x 4096 x 32 x 64 bfloat16 183 us
// (605 MB with the states' images: 3.3 TB/s), 2 x 4095 x 16 and 32 x 128 234 us (670 MB, 2.9 TB/s), fp32 8 x 4096 x 12 x 64
// 362 us (755 MB, 2.1 TB/s; six products of parts for each product, 105 us of them at the tensor cores' rate).
#include <type_traits>

#include "linattn_tc.cuh"

namespace linattn {
namespace {

template <typename T, int KP, int VP, int kQ, int kDecays>
struct Smem {
  static constexpr int kN = In<T>::kParts;
  bf16_t q[kN * kCT * KP], k[kN * kCT * KP], v[kN * kCT * VP], d[kN * kCT * VP];
  bf16_t s[3 * VP * 64];  // 64 keys of S or D; then (bfloat16) rows on their way out
  Decays dec[kDecays];
  float total[3][kCT];     // of a row's A_ij (q_i.k_j), by blocks of 32 columns
  float pairs[4][kCT];     // of a block of 32 rows: the sums over j < t
  float dots[2][kQ][kCT];  // q.(S's part of dq), k.(D's part of dk), by parts of the columns
  float whole[4 * kQ];
  // Products: scores, rows, of the state's first 64 keys (two blocks an SM: of A's third part), each twice a value head, for dq and for dk; q k^T,
  // once. Copies: the tiles, once a head; the state and its gradient, 64 keys at a time.
  uint64_t done[4], end, full[2];
  uint32_t tmem;
};

// The sums of 32 values over a warp: lane l ends with that of value l.
__device__ __forceinline__ float warp_columns(float (&y)[32], int lane) {
#pragma unroll
  for (int n = 16; n >= 1; n /= 2) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] = (up ? y[i + n] : y[i]) + __shfl_xor_sync(0xffffffffu, up ? y[i] : y[i + n], n);
  }
  return y[0];
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Of heads that share keys the next one's decays are made while dg of the last is added up, where a second set of
// them fits.
template <typename T, bool kShared>
constexpr int kDecaySets = kShared && sizeof(T) == 2 ? 2 : 1;

template <typename T, int KP, int VP, bool kShared, int kQ>
__global__ void __launch_bounds__(128 * kQ, kQ == 2 ? 2 : 1) grad_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  using M = Smem<T, KP, VP, kQ, kDecaySets<T, kShared>>;
  M& sm = *reinterpret_cast<M*>(raw);
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kThreads = 128 * kQ, kSlices = KP / 64, kN = In<T>::kParts, kW = 64 / kQ;
  constexpr int kCols = kQ == 2 ? 256 : 512;
  // E of dq and of dk; A (bfloat16: two parts in its place, the third from kThird on); q k^T; then, where what was there has been
  // read, the chunk's and the state's products
  enum { kE = 0, kQk = kF32 ? 320 : 128, kE2 = kF32 ? kQk : kE, kAt = kF32 ? 128 : 0, kOut = kF32 ? 0 : 128, kIn = kF32 ? 64 : 128 + KP, kThird = kQ == 2 ? kIn : kIn + KP };
  constexpr bool kHold = kQ == 2;  // registers for S's numbers, so that <S, D> need not read D from global memory (4 x 4096 x 32 x 64: 177 -> 168 us when it was measured)
  // A block's columns when two share an SM: A's third part is where q k^T was (a thread stores it when it has read that, its
  // last columns first) and where the state's products come to be: those wait for its own, which are the chunk's first.
  constexpr bool kTight = kQ == 2;
  auto third_of = [](int blk) { return kThird + (kTight ? 32 * (blk & 1) + 16 * (blk >> 1) : 16 * blk); };
  constexpr bool kEarlyIn = !kF32 && KP == 128;  // the state's products have columns of their own
  static_assert(!kF32 || (KP == 64 && VP == 64 && kQ == 4), "fp32 tiles of 64 columns fill shared memory");
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), sub = warp & 3, part_of = warp >> 2;
  const int hk = blockIdx.x % s.Hk, slot = blockIdx.x / s.Hk, group = kShared ? s.Hv / s.Hk : 1, row = 32 * sub + lane;
  ChunkAt c;
  if (!chunk_at(s, slot, kCT, c)) return;
  const size_t tok = (size_t)c.b * s.T + c.t0;
  const bool dg = a.dg != nullptr;
  if (warp == 0) wkv7::tmem_alloc(&sm.tmem, kCols);
  if (tid == 0) {
    for (uint64_t* b : {sm.done, sm.done + 1, sm.done + 2, sm.done + 3, &sm.end, sm.full, sm.full + 1}) mbar_init(b, 1);
    wkv7::fence_mbar_init();
  }
  float acc[2][kShared ? kW * kSlices : 1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < (kShared ? kW * kSlices : 1); ++j) acc[i][j] = 0.f;
  Patience wait{a.status};
  uint32_t tm = 0;
  __syncthreads();
  // The thread's kW columns of 64 to dq or dk (called by all threads). fp32: four lanes exchange four columns each, and a
  // store is of 64 bytes of eight rows instead of 16 of 32. bfloat16: through shared memory.
  auto leave = [&](T* to, int sl, float* x) {
    T* p = to + (tok * s.Hk + hk) * s.K + 64 * sl;
    if constexpr (kF32) {
#pragma unroll
      for (int n = 1; n < 4; n *= 2)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!(j & 4 * n)) {
            const bool up = lane & n;
            float &lo = x[j], &hi = x[j + 4 * n];
            const float got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, n);
            (up ? lo : hi) = got;
          }
      const int col = 16 * part_of + 4 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (row & ~3) + j;
        if (r < c.len && col < s.K) *reinterpret_cast<float4*>(p + (size_t)r * s.Hk * s.K + col) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kW; j += 8)
        *reinterpret_cast<uint4*>(sm.s + at(kCT, row, kW * part_of + j)) =
            make_uint4(pack2(x[j], x[j + 1]), pack2(x[j + 2], x[j + 3]), pack2(x[j + 4], x[j + 5]), pack2(x[j + 6], x[j + 7]));
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8 / kQ; ++e) {
        const int r = (e * kThreads + tid) >> 3, col = (tid & 7) * 8;
        if (r < c.len && 64 * sl + col < s.K)
          *reinterpret_cast<uint4*>(p + (size_t)r * s.Hk * s.K + col) = *reinterpret_cast<const uint4*>(sm.s + at(kCT, r, col));
      }
      fence_proxy_async_smem();
      __syncthreads();
    }
  };
  const int first = hk * group, last = first + group - 1;
  auto image_of = [&](const void* images, int hv) {
    return static_cast<const char*>(images) + ((size_t)slot * s.Hv + hv) * image_bytes(s.K, s.V);
  };
  // 64 keys of a state. (What was there has been read: the products that did are waited for.)
  auto fetch = [&](const char* from, int sl, int who = 0) {
    if (wait.ok & (tid == who)) {
      wkv7::mbar_arrive_expect_tx(&sm.full[1], sizeof sm.s);
#pragma unroll
      for (int part = 0; part < 3; ++part)
        bulk_load(sm.s + part * VP * 64, from + (size_t)(part * kSlices + sl) * VP * 128, VP * 128, &sm.full[1]);
    }
  };
  // The state before the chunk and (bfloat16) the tiles of a value head.
  auto begin = [&](int hv) {
    if (!LINATTN_SKIPPED(LINATTN_SKIP_STATE, hv - first + 1)) fetch(image_of(a.images, hv), 0);
    if (!kF32 && (wait.ok & (tid == 0)) && !LINATTN_SKIPPED(LINATTN_SKIP_TILES, hv - first + 1)) {
      wkv7::mbar_arrive_expect_tx(&sm.full[0], (hv == first ? sizeof sm.q + sizeof sm.k : 0) + sizeof sm.v + sizeof sm.d);
      load_tile<VP>(sm.v, &maps.v, &sm.full[0], 0, hv, c.t0, s.v_b ? c.b : 0);
      load_tile<VP>(sm.d, &maps.d, &sm.full[0], 0, hv, c.t0, c.b);
      if (hv == first) {
        load_tile<KP>(sm.q, &maps.q, &sm.full[0], 0, hk, c.t0, s.q_b ? c.b : 0);
        load_tile<KP>(sm.k, &maps.k, &sm.full[0], 0, hk, c.t0, s.k_b ? c.b : 0);
      }
    }
  };
  // fp32: what the block that takes this one's place will read first, into the L2, by one of `of` warps: the memory is
  // read while the products run instead of by all blocks of the next wave at once (8 x 4096 x 12 x 64: 386 -> 362 us;
  // bfloat16, with half the bytes a chunk, loses by it: 4 x 4096 x 32 x 64 176 -> 186).
  auto ahead = [&](int who, int of) {
    const unsigned next = blockIdx.x + kSms;  // (one block an SM)
    ChunkAt n;
    if (next >= gridDim.x || !chunk_at(s, (int)(next / s.Hk), kCT, n)) return;
    const int k_head = (int)(next % s.Hk), v_head = k_head * group;
    auto rows = [&](const void* base, long long offset, long long stride, int cols) {
      for (int r = 32 * who + lane; r < n.len; r += 32 * of)
        for (int x = 0; x < cols; x += 128 / (int)sizeof(T))
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(base) + offset + r * stride + x));
    };
    rows(a.v, n.b * s.v_b + n.t0 * s.v_t + (long long)v_head * s.V, s.v_t, s.V);
    rows(a.d_o, (((long long)n.b * s.T + n.t0) * s.Hv + v_head) * s.V, (long long)s.Hv * s.V, s.V);
    rows(a.q, n.b * s.q_b + n.t0 * s.q_t + (long long)k_head * s.K, s.q_t, s.K);
    rows(a.k, n.b * s.k_b + n.t0 * s.k_t + (long long)k_head * s.K, s.k_t, s.K);
    const char* S = static_cast<const char*>(a.images) + ((size_t)(next / s.Hk) * s.Hv + v_head) * image_bytes(s.K, s.V);
    for (int i = 32 * who + lane; i < 3 * VP; i += 32 * of)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(S + ((size_t)(i / VP) * kSlices * VP + i % VP) * 128));
  };
  begin(first);
  for (int hv = first; hv <= last; ++hv) {
    const char *S = image_of(a.images, hv), *D = image_of(a.dimages, hv);
    Decays& dec = sm.dec[(hv - first) % kDecaySets<T, kShared>];
    // fp32: all values on their way at once, 16 of a tile a thread
    float4 raw_q[4], raw_k[4], raw_v[4], raw_d[4];
    auto bring = [&](float4 (&x)[4], const void* base, long long offset, long long stride, int cols) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (tid >> 3) + 64 * e, col = (tid & 7) * 8;
        const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(base) + offset + r * stride + col);
        const bool in = r < c.len && col < cols;
        x[2 * e] = in ? __ldg(from) : make_float4(0.f, 0.f, 0.f, 0.f), x[2 * e + 1] = in ? __ldg(from + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    auto place = [&](bf16_t* tile, const float4 (&x)[4]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 lo = x[2 * e], hi = x[2 * e + 1];
        const float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        put8<3>(tile + at(kCT, (tid >> 3) + 64 * e, (tid & 7) * 8), kCT * 64, y);
      }
    };
    if constexpr (kF32) {
      bring(raw_v, a.v, c.b * s.v_b + c.t0 * s.v_t + (long long)hv * s.V, s.v_t, s.V);
      bring(raw_d, a.d_o, (tok * s.Hv + hv) * s.V, (long long)s.Hv * s.V, s.V);
      if (hv == first) {
        bring(raw_q, a.q, c.b * s.q_b + c.t0 * s.q_t + (long long)hk * s.K, s.q_t, s.K);
        bring(raw_k, a.k, c.b * s.k_b + c.t0 * s.k_t + (long long)hk * s.K, s.k_t, s.K);
      }
    }
    if (warp == 4 * kQ - 1) {
      float r[4];
      load_decays(r, s.fixed ? a.g + hv : a.g + tok * s.Hv + hv, s.fixed ? 0 : s.Hv, c.len, lane);
      make_decays<kF32>(dec, r, s.scale, lane);
    }
    // A product of two tiles along their rows, in tensor memory from column `to` on.
    auto scores = [&](uint32_t to, const bf16_t* ta, const bf16_t* tb, auto cols) {
      constexpr int D = decltype(cols)::value;
      const uint64_t da = desc(ta), db = desc(tb);
      terms<kN, kN>([&](int p, int r, bool start) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma(tm + to, da + along<kCT>(ks) + p * (kCT * D * 2 >> 4), db + along<kCT>(ks) + r * (kCT * D * 2 >> 4),
                 product_of(128, 128, false, false), !start || ks > 0);
      });
    };
    using Keys = std::integral_constant<int, KP>;
    using Values = std::integral_constant<int, VP>;
    auto first_products = [&] {
      if (warp == 0) {
        if (elected()) {
          scores(kE, sm.d, sm.v, Values{});
          if (!LINATTN_SKIPPED(LINATTN_SKIP_SCORES, 2 * (hv - first) + 1)) tc_commit(&sm.done[0]);
        }
        __syncwarp();
      }
    };
    const bool ready = !kF32 && !(s.packed && c.len < kCT);  // the tiles are as they came: the first products need not wait for the decays
    if constexpr (kF32) {
      place(sm.v, raw_v), place(sm.d, raw_d);
      fence_proxy_async_smem();
      tmem_fence_before_sync();
      __syncthreads();
      tmem_fence_after_sync();
      tm = sm.tmem;
      first_products();
      if (hv == first) place(sm.q, raw_q), place(sm.k, raw_k);
    } else {
      wait(&sm.full[0], hv - first);
      if (!ready) {
        if (hv == first) clear_rows<KP>(sm.q, c.len, tid, kThreads), clear_rows<KP>(sm.k, c.len, tid, kThreads);
        clear_rows<VP>(sm.v, c.len, tid, kThreads);
        clear_rows<VP>(sm.d, c.len, tid, kThreads);
      }
    }
    fence_proxy_async_smem();
    tmem_fence_before_sync();
    if (!ready) __syncthreads();
    tmem_fence_after_sync();
    tm = sm.tmem;
    const uint32_t mine = tm + ((uint32_t)(32 * sub) << 16);
    float whole = 0.f, held[kHold ? VP * 8 / kThreads : 1][8];  // kHold: S, until D is there
    auto phase = [&](auto upper) {
      constexpr bool kUpper = decltype(upper)::value;
      const bf16_t *ta = kUpper ? sm.v : sm.d, *tx = kUpper ? sm.q : sm.k, *td = kUpper ? sm.k : sm.q;
      if (!kUpper) {
        if (!kF32) first_products();
        if (dg && warp == 0) {
          if (elected()) {
            scores(kQk, sm.q, sm.k, Keys{});
            tc_commit(&sm.done[3]);
          }
          __syncwarp();
        }
      }
      // They are there; their part of <S, D>.
      auto fetched = [&](int sl) {
        wait(&sm.full[1], kEarlyIn ? sl : kUpper);
        if (kHold && dg) {
#pragma unroll
          for (int e = 0; e < VP * 8 / kThreads; ++e) {
            const bf16_t* at = sm.s + 8 * (e * kThreads + tid);
            float x[8], t[8];
            load8(x, at);
#pragma unroll
            for (int part = 1; part < 3; ++part) {
              load8(t, at + part * VP * 64);
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] += t[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (kUpper)
                whole = fmaf(x[j], held[e][j], whole);
              else
                held[e][j] = x[j];
            }
          }
          fence_proxy_async_smem();
        }
        if (!kHold && !kUpper && dg) {
          const bf16_t* other = reinterpret_cast<const bf16_t*>(D + (size_t)sl * VP * 128);
#pragma unroll 2
          for (int i = tid; i < VP * 8; i += kThreads) {
            float x[8], y[8], t[8];
            load8(x, sm.s + 8 * i), load8(y, other + 8 * i);
#pragma unroll
            for (int part = 1; part < 3; ++part) {
              load8(t, sm.s + part * VP * 64 + 8 * i);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] += t[e];
              load8(t, other + part * kSlices * VP * 64 + 8 * i);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] += t[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) whole = fmaf(x[e], y[e], whole);
          }
          fence_proxy_async_smem();
        }
      };
      auto inter = [&](int sl) {
        const uint64_t da = desc(ta), ds = desc(sm.s);
        terms<kN, 3>([&](int p, int r, bool first) {
#pragma unroll
          for (int ks = 0; ks < VP / 16; ++ks)
            tc_mma(tm + kIn + 64 * sl, da + along<kCT>(ks) + p * (kCT * VP * 2 >> 4), ds + across(ks) + r * (VP * 128 >> 4),
                   product_of(128, 64, false, true), !first || ks > 0);
        });
      };
      if (kEarlyIn && warp == 0) {
        wait(&sm.full[1], 0);
        if (elected()) {
          inter(0);
          tc_commit(&sm.done[2]);
        }
        __syncwarp();
      }
      if (!kUpper && kF32) fetched(0);  // (while the products of parts run)
      if (!kUpper && ready) __syncthreads();  // the decays
      // The other 64 keys come while the scores are decayed: brought by a warp that has none (S: once <S, D> has read its first half).
      if (kEarlyIn) {
        if (!kUpper) {  // (D: the products that read it wait for it, and who brings the rest for them)
          fetched(0);
          __syncthreads();
        }
        constexpr int kWho = kUpper ? 1 : 4;
        if (warp == kWho) {
          wait(&sm.done[2], kUpper);
          fetch(kUpper ? D : S, 1, 32 * kWho);
        }
      }
      wait(&sm.done[0], kUpper);
      tmem_fence_after_sync();
      if (kF32 && !kUpper && hv == first && sub == 0 && part_of) ahead(part_of - 1, kQ - 1);  // (these have nothing else to do now)
#pragma unroll 1
      for (int blk = part_of + 4 - kQ; blk >= 0; blk -= kQ) {
        if (kUpper ? blk >= sub : blk <= sub) {
          float x[32];
          tc_read(x, mine + (kUpper ? kE2 : kE) + 32 * blk);
          decayed<kUpper, kF32>(x, dec, row, blk, s.scale);
          if (kF32) store_parts<3>(mine + kAt + 48 * blk, x);
          if (!kUpper && dg) {
            float y[32], run = 0.f;
            wait(&sm.done[3], hv - first);
            tmem_fence_after_sync();
            tc_read(y, mine + kQk + 32 * blk);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int col = 32 * blk + j;
              const float z = col < row ? x[j] * y[j] : 0.f;
              y[j] = col <= row ? run : 0.f;
              run += z;
            }
            if (blk < 3) sm.total[blk][row] = run;
            sm.pairs[sub][32 * blk + lane] = warp_columns(y, lane);
          }
          if (!kF32) {
            uint32_t third[16];
            store_two(mine + kAt + 32 * blk, x, third);
            tc_store16(mine + third_of(blk), third);
          }
        } else if (kF32) {
          store_zeros<3>(mine + kAt + 48 * blk);
        } else {
          if (kTight && !kUpper && dg) {  // (q k^T comes to be where the third part goes)
            wait(&sm.done[3], hv - first);
            tmem_fence_after_sync();
          }
          const uint32_t third[16] = {};
          store_zeros<2>(mine + kAt + 32 * blk), tc_store16(mine + third_of(blk), third);
        }
      }
      if (!kEarlyIn && (kUpper || !kF32)) fetched(0);
      wkv7::tmem_wait_st();
      tmem_fence_before_sync();
      __syncthreads();
      if (warp == 0) {
        tmem_fence_after_sync();
        if (elected()) {
          const uint64_t dx = desc(tx);
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
            terms<3, kN>([&](int p, int r, bool first) {
#pragma unroll
              for (int ks = 0; ks < kCT / 16; ++ks)
                tc_mma_t(tm + kOut + 64 * sl, tm + kAt + (kF32 ? part_at<3>(ks, p) : two_and_third(ks, p, third_of(ks >> 1) - kAt)),
                         dx + across(ks) + sl * (kRowPanel >> 4) + r * (kCT * KP * 2 >> 4), product_of(128, 64, false, true), !first || ks > 0);
              if (kTight && first) tc_commit(&sm.done[2]);  // (the third part)
            });
          if (!kEarlyIn && !kTight) {
            inter(0);
            tc_commit(&sm.done[1]);
          }
        }
        __syncwarp();
        if (kTight) {
          wait(&sm.done[2], kUpper);
          tmem_fence_after_sync();
          if (elected()) {
            inter(0);
            tc_commit(&sm.done[1]);
          }
          __syncwarp();
        }
        if (kEarlyIn) {
          wait(&sm.full[1], 1);
          if (elected()) {
            inter(1);
            tc_commit(&sm.done[1]);
          }
          __syncwarp();
        }
      }
      if (kEarlyIn) {
        // (Shared heads' upper phase: who reads D are the products, and warp 0 has waited for it. A wait of the others here
        // could come after the next head's S has been asked for, and would then see neither copy's phase.)
        if (!kUpper || !kShared) fetched(1);
        if (!kShared) __syncthreads();  // <S, D> has been read: rows take its place
      }
      wait(&sm.done[1], kUpper);
      tmem_fence_after_sync();
      const bool back = !LINATTN_SKIPPED(LINATTN_SKIP_BACK, hv - first + 1);
      if (!kUpper && back && !kEarlyIn && (kShared || kF32)) fetch(D, 0);
      if (!kUpper && warp == 0) {  // (where A was, or q k^T: both have been read)
        if (elected()) {
          scores(kE2, sm.v, sm.d, Values{});
          if (!LINATTN_SKIPPED(LINATTN_SKIP_SCORES, 2 * (hv - first) + 2)) tc_commit(&sm.done[0]);
        }
        __syncwarp();
      }
      if (kUpper && kShared && hv < last) begin(hv + 1);  // (the products that read v, do and D are done)
      const float w = (kUpper ? dec.tail : dec.head)[row];
      float dot = 0.f;
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) {
        float x[kW], y[kW];
        tc_read(x, mine + kIn + 64 * sl + kW * part_of);
        tc_read(y, mine + kOut + 64 * sl + kW * part_of);
#pragma unroll
        for (int j = 0; j < kW; ++j) x[j] *= w;
        if (dg) {
#pragma unroll
          for (int j = 0; j < kW; j += 8) {
            const bf16_t* z0 = td + at(kCT, row, 64 * sl + kW * part_of + j);
            float z[8];
            load8(z, z0);
#pragma unroll
            for (int p = 1; p < kN; ++p) {
              float t[8];
              load8(t, z0 + p * kCT * KP);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] += t[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(z[e], x[j + e], dot);
          }
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
          if (kShared)
            acc[kUpper][kW * sl + j] += x[j] + y[j];
          else
            x[j] += y[j];
        }
        if (!kShared) leave(static_cast<T*>(kUpper ? a.dk : a.dq), sl, x);
      }
      if (dg) sm.dots[kUpper][part_of][row] = dot;
      tmem_fence_before_sync();
      __syncthreads();
      tmem_fence_after_sync();
      if (!kUpper && back && (kEarlyIn || !(kShared || kF32))) fetch(D, 0);  // (all threads are done with the place)
    };
    phase(std::false_type{});
    phase(std::true_type{});
    if (dg) {
      whole = warp_sum(whole);
      if (lane == 0) sm.whole[warp] = whole;
      __syncthreads();
      if (warp < 4) {  // 32 tokens, one a lane
        const int b = warp, t = 32 * b + lane;
        auto rows_of = [&](int which, int i) {
          float x = sm.dots[which][0][i];
#pragma unroll
          for (int q = 1; q < kQ; ++q) x += sm.dots[which][q][i];
          return x;
        };
        // terms of rows from t on: the state's part, and pairs with columns of the blocks before t's
        auto term = [&](int i) {
          float x = rows_of(0, i);
          for (int q = 0; q < b; ++q) x += sm.total[q][i];
          return x;
        };
        float later = 0.f, before = 0.f, pairs = 0.f;
        for (int q = b + 1; q < 4; ++q) later += term(32 * q + lane);
        for (int q = 0; q < b; ++q) before += rows_of(1, 32 * q + lane);
        for (int q = b; q < 4; ++q) pairs += sm.pairs[q][t];
        later = warp_sum(later), before = warp_sum(before);
        float from = term(t), upto = rows_of(1, t);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_down_sync(0xffffffffu, from, o), y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane + o < 32) from += x;
          if (lane >= o) upto += y;
        }
        upto = __shfl_up_sync(0xffffffffu, upto, 1);
        if (lane == 0) upto = 0.f;
        float pass = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * kQ; ++i) pass += sm.whole[i];
        if (t < c.len) a.dg[(tok + t) * s.Hv + hv] = ((from + later) + (upto + before)) + (pairs + dec.whole * pass);
      }
      if (kShared && kDecaySets<T, kShared> == 1) __syncthreads();
    }
  }
  if (kShared) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) leave(static_cast<T*>(i ? a.dk : a.dq), sl, acc[i] + kW * sl);
  }
  if (warp == 0) {
    if (!__all_sync(0xffffffffu, wait.ok)) {
      finish_products(&sm.end);
      if (lane == 0) finish_copies(&sm.full[0]), finish_copies(&sm.full[1]);
    }
  }
  __syncthreads();
  if (warp == 0) wkv7::tmem_dealloc(tm, kCols);
}

template <typename T, int KP, int VP, bool kShared>
cudaError_t launch(const Maps& maps, const Args& a, cudaStream_t stream) {
  // two blocks of 256 threads an SM where they fit, else one of 512 (4 x 4096 x 32 x 64: 176 us for 281 when it was measured)
  constexpr int kQ = sizeof(T) == 2 && KP == 64 && VP == 64 && !kShared ? 2 : 4;
  using M = Smem<T, KP, VP, kQ, kDecaySets<T, kShared>>;
  static_assert(sizeof(M) <= 232448, "shared memory of a block");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(grad_kernel<T, KP, VP, kShared, kQ>), sizeof(M), done);
  if (e != cudaSuccess) return e;
  grad_kernel<T, KP, VP, kShared, kQ><<<(unsigned)((size_t)a.s.slots * a.s.Hk), 128 * kQ, sizeof(M), stream>>>(maps, a);
  return cudaGetLastError();
}
template <typename T, int KP, int VP>
cudaError_t shared(const Maps& maps, const Args& a, cudaStream_t stream) {
  return a.s.Hv > a.s.Hk ? launch<T, KP, VP, true>(maps, a, stream) : launch<T, KP, VP, false>(maps, a, stream);
}

}  // namespace

cudaError_t launch_grad(const Maps& maps, const Args& a, bool bf16, cudaStream_t stream) {
  if (!bf16) return shared<float, 64, 64>(maps, a, stream);
  if (a.s.K <= 64) return a.s.V <= 64 ? shared<bf16_t, 64, 64>(maps, a, stream) : shared<bf16_t, 64, 128>(maps, a, stream);
  return a.s.V <= 64 ? shared<bf16_t, 128, 64>(maps, a, stream) : shared<bf16_t, 128, 128>(maps, a, stream);
}

}  // namespace linattn
