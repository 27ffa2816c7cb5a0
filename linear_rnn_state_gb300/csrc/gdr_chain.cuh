// What the forward and the backward chain of the gated delta rule share: the
// images of a chunk in shared memory, read by one or two groups of eight warps,
// each with a tile of 32 value columns.
//
// q, T and P have one place each and k two: each is filled again as soon as
// every group is past its last use in the step, which leaves half a step or
// more for the copy, and a block of one group with 64-wide keys in 113 KB, so
// that two share an SM. The thread that finds its group to be the last issues
// the copy, so nobody waits to fill.
#pragma once

#include "gdr_common.cuh"

namespace gdr {

constexpr int kGroupThreads = 256;

template <int P, int KP>
struct alignas(128) Images {
  __half k[2][P * kC * KP];
  __half q[P * kC * KP];
  __half t[2 * kTriPart], p[2 * kTriPart];
  Scal scal[2];
  Rows rows[2];
  uint64_t full_k[2], full_q, full_t, full_p;
  // groups past their last use, ever. k has a count a place: a group may be a step ahead in it
  unsigned done_k[2], done_t, done_p;
};

// Fills the images of steps 0 .. n - 1, whose chunk slots are slot0 + s or,
// backwards, slot0 - s.
template <int P, int KP>
struct Filler {
  static constexpr int image = P * kC * KP * 2, tri = Layout::tp_img;
  Images<P, KP>& m;
  const Args& a;
  long long slot0;
  int direction, n, hk, hv, groups;

  __device__ __forceinline__ size_t at_k(int s) const { return (size_t)(slot0 + (long long)direction * s) * a.s.Hk + hk; }
  __device__ __forceinline__ size_t at_v(int s) const { return (size_t)(slot0 + (long long)direction * s) * a.s.Hv + hv; }
  __device__ __forceinline__ void k(int s) const {
    uint64_t* bar = &m.full_k[s & 1];
    mbar_arrive_expect_tx(bar, image + sizeof(Rows) + sizeof(Scal));
    bulk_load(m.k[s & 1], a.b.k_img + at_k(s) * image, image, bar);
    bulk_load(&m.rows[s & 1], a.b.rows + at_k(s), sizeof(Rows), bar);
    bulk_load(&m.scal[s & 1], a.b.scal + at_v(s), sizeof(Scal), bar);
  }
  __device__ __forceinline__ void q(int s) const {
    mbar_arrive_expect_tx(&m.full_q, image);
    bulk_load(m.q, a.b.q_img + at_k(s) * image, image, &m.full_q);
  }
  __device__ __forceinline__ void t(int s) const {
    mbar_arrive_expect_tx(&m.full_t, tri);
    bulk_load(m.t, a.b.t_img + at_v(s) * tri, tri, &m.full_t);
  }
  __device__ __forceinline__ void p(int s) const {
    mbar_arrive_expect_tx(&m.full_p, tri);
    bulk_load(m.p, a.b.p_img + at_v(s) * tri, tri, &m.full_p);
  }
  // Asks step s into L2.
  __device__ __forceinline__ void ask(int s) const {
    if (s >= n) return;
    bulk_prefetch(a.b.k_img + at_k(s) * image, image);
    bulk_prefetch(a.b.q_img + at_k(s) * image, image);
    bulk_prefetch(a.b.t_img + at_v(s) * tri, tri);
    bulk_prefetch(a.b.p_img + at_v(s) * tri, tri);
    bulk_prefetch(a.b.scal + at_v(s), sizeof(Scal));
  }
  __device__ __forceinline__ void start() const {
    for (uint64_t* b : {&m.full_k[0], &m.full_k[1], &m.full_q, &m.full_t, &m.full_p}) mbar_init(b, 1);
    m.done_k[0] = m.done_k[1] = m.done_t = m.done_p = 0;
    wkv7::fence_mbar_init();
    if (n <= 0) return;
    k(0), p(0), t(0), q(0);
    if (n > 1) k(1);
    ask(2);
  }
  // One thread of a group calls this after a barrier that every warp of it
  // reaches past its last use: whether the other groups are past theirs too.
  __device__ __forceinline__ bool last(unsigned& done) const {
    if (groups == 1) return true;
    __threadfence_block();
    const bool l = (atomicAdd(&done, 1u) + 1) % groups == 0;
    __threadfence_block();
    return l;
  }
};

// Asks for the rows of v (or do) of one chunk into L2: a thread a row.
template <typename T>
__device__ __forceinline__ void ask_rows(const T* base, long long stride_t, int t0, int t1, int tid) {
  if (tid < kC && t0 + tid < t1) prefetch_l2(base + (t0 + tid) * stride_t);
}

}  // namespace gdr
