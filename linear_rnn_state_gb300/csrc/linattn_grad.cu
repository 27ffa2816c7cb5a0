// Linear attention with a decay, bfloat16: dq, dk and dg of every chunk, all chunks at once, on tcgen05.
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
// products, half of its columns; A enters as a pair of bfloat16 (16 bits, for bfloat16 results), S and D in
// three parts, 64 keys of them at a time (24 bits: dg is an fp32 result).
#include <type_traits>

#include "linattn_tc.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256;

template <int KP, int VP>
struct Smem {
  bf16_t q[kCT * KP], k[kCT * KP], v[kCT * VP], d[kCT * VP];
  bf16_t s[3 * VP * 64];  // 64 keys of S or D; then rows on their way out
  Decays dec;
  float total[4][kCT];    // of a row's A_ij (q_i.k_j), by blocks of 32 columns
  float pairs[4][kCT];    // of a block of 32 rows: the sums over j < t
  float dots[2][2][kCT];  // q.(S's part of dq), k.(D's part of dk), by halves of the columns
  float whole[8];
  uint64_t done[2], full[2];  // products; tiles of q and k or of v and do, the state
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

template <int KP, int VP, bool kShared>
__global__ void __launch_bounds__(kThreads, KP == 64 && VP == 64 && !kShared ? 2 : 1) grad_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  Smem<KP, VP>& sm = *reinterpret_cast<Smem<KP, VP>*>(raw);
  constexpr int kSlices = KP / 64, kCols = KP == 64 ? 256 : 512;
  enum { kE = 0, kQk = 128, kOut = 128, kIn = 128 + KP };
  const Shape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), sub = warp & 3, half = warp >> 2;
  const int hk = blockIdx.x % s.Hk, slot = blockIdx.x / s.Hk, group = kShared ? s.Hv / s.Hk : 1, row = 32 * sub + lane;
  ChunkAt c;
  if (!chunk_at(s, slot, kCT, c)) return;
  const size_t tok = (size_t)c.b * s.T + c.t0;
  const bool dg = a.dg != nullptr;
  if (warp == 0) wkv7::tmem_alloc(&sm.tmem, kCols);
  if (tid == 0) {
    mbar_init(&sm.done[0], 1), mbar_init(&sm.done[1], 1), mbar_init(&sm.full[0], 1), mbar_init(&sm.full[1], 1);
    wkv7::fence_mbar_init();
  }
  float acc[2][kShared ? 32 * kSlices : 1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < (kShared ? 32 * kSlices : 1); ++j) acc[i][j] = 0.f;
  Patience wait{a.status};
  uint32_t turn0 = 0, turn1 = 0, turn2 = 0, turn3 = 0, tm = 0;
  __syncthreads();
  // 64 columns of rows from shared memory to dq or dk
  auto leave = [&](bf16_t* to, int sl) {
    __syncthreads();
    bf16_t* p = to + (tok * s.Hk + hk) * s.K + 64 * sl;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = (e * kThreads + tid) >> 3, col = (tid & 7) * 8;
      if (r < c.len && 64 * sl + col < s.K)
        *reinterpret_cast<uint4*>(p + (size_t)r * s.Hk * s.K + col) = *reinterpret_cast<const uint4*>(sm.s + at(kCT, r, col));
    }
    fence_proxy_async_smem();
    __syncthreads();
  };
  auto put_row = [&](const float* x) {  // the thread's 32 columns
#pragma unroll
    for (int p = 0; p < 4; ++p)
      *reinterpret_cast<uint4*>(sm.s + at(kCT, row, 32 * half + 8 * p)) =
          make_uint4(pack2(x[8 * p], x[8 * p + 1]), pack2(x[8 * p + 2], x[8 * p + 3]), pack2(x[8 * p + 4], x[8 * p + 5]),
                     pack2(x[8 * p + 6], x[8 * p + 7]));
  };
  for (int hv = hk * group; hv < hk * group + group; ++hv) {
    if (tid == 0) {
      const bool all = hv == hk * group;
      wkv7::mbar_arrive_expect_tx(&sm.full[0], (all ? sizeof sm.q + sizeof sm.k : 0) + sizeof sm.v + sizeof sm.d);
      if (all) {
        load_tile<KP>(sm.q, &maps.q, &sm.full[0], 0, hk, c.t0, s.q_b ? c.b : 0);
        load_tile<KP>(sm.k, &maps.k, &sm.full[0], 0, hk, c.t0, s.k_b ? c.b : 0);
      }
      load_tile<VP>(sm.v, &maps.v, &sm.full[0], 0, hv, c.t0, s.v_b ? c.b : 0);
      load_tile<VP>(sm.d, &maps.d, &sm.full[0], 0, hv, c.t0, c.b);
    }
    if (warp == 7) {
      float r[4];
      load_decays(r, s.fixed ? a.g + hv : a.g + tok * s.Hv + hv, s.fixed ? 0 : s.Hv, c.len, lane);
      make_decays(sm.dec, r, s.scale, lane);
    }
    const size_t image = ((size_t)slot * s.Hv + hv) * image_bytes(s.K, s.V);
    const char *S = static_cast<const char*>(a.images) + image, *D = static_cast<const char*>(a.dimages) + image;
    wait(&sm.full[0], turn2++);
    if (s.packed && c.len < kCT) {
      if (hv == hk * group) clear_rows<KP>(sm.q, c.len, tid, kThreads), clear_rows<KP>(sm.k, c.len, tid, kThreads);
      clear_rows<VP>(sm.v, c.len, tid, kThreads);
      clear_rows<VP>(sm.d, c.len, tid, kThreads);
    }
    fence_proxy_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    tm = sm.tmem;
    const uint32_t mine = tm + ((uint32_t)(32 * sub) << 16);
    float whole = 0.f;
    auto phase = [&](auto upper) {
      constexpr bool kUpper = decltype(upper)::value;
      const bf16_t *ta = kUpper ? sm.v : sm.d, *tb = kUpper ? sm.d : sm.v, *tx = kUpper ? sm.q : sm.k, *td = kUpper ? sm.k : sm.q;
      if (warp == 0) {
        if (elected()) {
          const uint64_t da = desc(ta), db = desc(tb);
#pragma unroll
          for (int ks = 0; ks < VP / 16; ++ks) tc_mma(tm + kE, da + along<kCT>(ks), db + along<kCT>(ks), product_of(128, 128, false, false), ks > 0);
          if (!kUpper && dg) {
            const uint64_t dq = desc(sm.q), dk = desc(sm.k);
#pragma unroll
            for (int ks = 0; ks < KP / 16; ++ks) tc_mma(tm + kQk, dq + along<kCT>(ks), dk + along<kCT>(ks), product_of(128, 128, false, false), ks > 0);
          }
          tc_commit(&sm.done[0]);
        }
        __syncwarp();
      }
      // 64 keys of the state. (What was there has been read: the products that did are waited for.)
      auto fetch = [&](int sl) {
        if (tid == 0) {
          wkv7::mbar_arrive_expect_tx(&sm.full[1], sizeof sm.s);
#pragma unroll
          for (int part = 0; part < 3; ++part)
            bulk_load(sm.s + part * VP * 64, (kUpper ? D : S) + (size_t)(part * kSlices + sl) * VP * 128, VP * 128, &sm.full[1]);
        }
      };
      // and their part of <S, D>
      auto fetched = [&](int sl) {
        wait(&sm.full[1], turn3++);
        if (!kUpper && dg) {
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
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int ks = 0; ks < VP / 16; ++ks)
            tc_mma(tm + kIn + 64 * sl, da + along<kCT>(ks), ds + across(ks) + part * (VP * 128 >> 4), product_of(128, 64, false, true), part < 2 || ks > 0);
      };
      fetch(0);
      wait(&sm.done[0], turn0++);
      tmem_fence_after_sync();
#pragma unroll 1
      for (int blk = half; blk < 4; blk += 2) {
        if (kUpper ? blk >= sub : blk <= sub) {
          float x[32];
          tc_load32(x, mine + kE + 32 * blk);
          tc_loaded32(x);
          decayed<kUpper>(x, sm.dec, row, blk, s.scale);
          store_pairs(mine + kE + 32 * blk, x);
          if (!kUpper && dg) {
            float y[32], run = 0.f;
            tc_load32(y, mine + kQk + 32 * blk);
            tc_loaded32(y);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int col = 32 * blk + j;
              const float z = col < row ? x[j] * y[j] : 0.f;
              y[j] = col <= row ? run : 0.f;
              run += z;
            }
            sm.total[blk][row] = run;
            sm.pairs[sub][32 * blk + lane] = warp_columns(y, lane);
          }
        } else {
          store_zeros(mine + kE + 32 * blk);
        }
      }
      fetched(0);
      wkv7::tmem_wait_st();
      tmem_fence_before_sync();
      __syncthreads();
      if (warp == 0) {
        tmem_fence_after_sync();
        if (elected()) {
          const uint64_t dx = desc(tx);
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int ks = 0; ks < kCT / 16; ++ks)
                tc_mma_t(tm + kOut + 64 * sl, tm + kE + pair_at(ks, part), dx + across(ks) + sl * (kRowPanel >> 4), product_of(128, 64, false, true),
                         part == 0 || ks > 0);
          inter(0);
          tc_commit(&sm.done[1]);
        }
        __syncwarp();
      }
      wait(&sm.done[1], turn1++);
      if (kSlices == 2) {
        __syncthreads();  // <S, D> has been read
        fetch(1);
        fetched(1);
        tmem_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          tmem_fence_after_sync();
          if (elected()) {
            inter(1);
            tc_commit(&sm.done[1]);
          }
          __syncwarp();
        }
        wait(&sm.done[1], turn1++);
      }
      tmem_fence_after_sync();
      const float w = (kUpper ? sm.dec.tail : sm.dec.head)[row];
      float dot = 0.f;
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) {
        float x[32], y[32];
        tc_load32(x, mine + kIn + 64 * sl + 32 * half);
        tc_load32(y, mine + kOut + 64 * sl + 32 * half);
        tc_loaded32(x);
        tc_loaded32(y);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] *= w;
        if (dg) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            float z[8];
            load8(z, td + at(kCT, row, 64 * sl + 32 * half + 8 * p));
#pragma unroll
            for (int j = 0; j < 8; ++j) dot = fmaf(z[j], x[8 * p + j], dot);
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (kShared)
            acc[kUpper][32 * sl + j] += x[j] + y[j];
          else
            x[j] += y[j];
        }
        if (!kShared) {
          put_row(x);
          leave(static_cast<bf16_t*>(kUpper ? a.dk : a.dq), sl);
        }
      }
      if (dg) sm.dots[kUpper][half][row] = dot;
      tmem_fence_before_sync();
      __syncthreads();
      tmem_fence_after_sync();
    };
    phase(std::false_type{});
    phase(std::true_type{});
    if (dg) {
      whole = warp_sum(whole);
      if (lane == 0) sm.whole[warp] = whole;
      __syncthreads();
      if (warp < 4) {  // 32 tokens, one a lane
        const int b = warp, t = 32 * b + lane;
        // terms of rows from t on: the state's part, and pairs with columns of the blocks before t's
        auto term = [&](int i) {
          float x = sm.dots[0][0][i] + sm.dots[0][1][i];
          for (int q = 0; q < b; ++q) x += sm.total[q][i];
          return x;
        };
        float later = 0.f, before = 0.f, pairs = 0.f;
        for (int q = b + 1; q < 4; ++q) later += term(32 * q + lane);
        for (int q = 0; q < b; ++q) before += sm.dots[1][0][32 * q + lane] + sm.dots[1][1][32 * q + lane];
        for (int q = b; q < 4; ++q) pairs += sm.pairs[q][t];
        later = warp_sum(later), before = warp_sum(before);
        float from = term(t), upto = sm.dots[1][0][t] + sm.dots[1][1][t];
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
        for (int i = 0; i < 8; ++i) pass += sm.whole[i];
        if (t < c.len) a.dg[(tok + t) * s.Hv + hv] = ((from + later) + (upto + before)) + (pairs + sm.dec.whole * pass);
      }
      if (kShared) __syncthreads();
    }
  }
  if (kShared) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int sl = 0; sl < kSlices; ++sl) {
        put_row(acc[i] + 32 * sl);
        leave(static_cast<bf16_t*>(i ? a.dk : a.dq), sl);
      }
  }
  __syncthreads();
  if (warp == 0) wkv7::tmem_dealloc(tm, kCols);
}

template <int KP, int VP, bool kShared>
cudaError_t launch(const Maps& maps, const Args& a, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<KP, VP>);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(grad_kernel<KP, VP, kShared>), smem, done);
  if (e != cudaSuccess) return e;
  grad_kernel<KP, VP, kShared><<<(unsigned)((size_t)a.s.slots * a.s.Hk), kThreads, smem, stream>>>(maps, a);
  return cudaGetLastError();
}
template <int KP, int VP>
cudaError_t shared(const Maps& maps, const Args& a, cudaStream_t stream) {
  return a.s.Hv > a.s.Hk ? launch<KP, VP, true>(maps, a, stream) : launch<KP, VP, false>(maps, a, stream);
}

}  // namespace

cudaError_t launch_grad(const Maps& maps, const Args& a, cudaStream_t stream) {
  if (a.s.K <= 64) return a.s.V <= 64 ? shared<64, 64>(maps, a, stream) : shared<64, 128>(maps, a, stream);
  return a.s.V <= 64 ? shared<128, 64>(maps, a, stream) : shared<128, 128>(maps, a, stream);
}

}  // namespace linattn
