// Internal launch interface of the gated delta rule between the C ABI
// (gdr_api.cu) and its kernels, and the layout of what they hand on.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define GDR_BOTH __host__ __device__
#else
#define GDR_BOTH
#endif

namespace gdr {

constexpr int kC = 64;        // tokens of a chunk
constexpr int kVt = 16;       // value columns (rows of the state) of a tile
constexpr int kMaxDim = 128;  // largest head size

// What a call's sequences and heads look like.
struct Shape {
  int B, T, Hk, Hv, K, V;
  int nseq;             // sequences: B, or those packed in the one batch row
  const int* starts;    // device [nseq + 1], or null
  int slots;            // chunk slots: an upper bound of the chunks, see slot_count
  int packed;           // nseq sequences in one batch row
  int l2norm;
  float scale;
  long long q_b, q_t, k_b, k_t, v_b, v_t;  // element strides of a batch row and of a token
};

// Every sequence's chunks get slots of their own. Dense: batch * ceil(T / 64).
// Packed: a sequence that starts at token x is given the slots from x / 64 + s
// on (s its number): x / 64 + ceil(len / 64) <= (x + len) / 64 + 1, so the next
// sequence's slots start after them, and T / 64 + nseq are enough.
inline long long slot_count(int B, int T, int nseq, bool packed) {
  return packed ? (long long)T / kC + nseq : (long long)B * ((T + kC - 1) / kC);
}

inline int padded_k(int K) { return K <= 64 ? 64 : 128; }
inline int v_tiles(int V) { return (V + kVt - 1) / kVt; }

// Scalars of a chunk: per key head (Rows) and per value head (Scal).
struct Rows {        // of the 64 tokens, the actual q is qs * image (and k is ks * image)
  float qs[kC], ks[kC];
  float rq[kC], rk[kC];  // 1 / |q|, 1 / |k| with l2norm, else 1
  float qk[kC];          // q.k
};
struct Scal {
  // with G the running sum of g in the chunk and Gc its whole sum:
  float ek[kC];  // e^G ks
  float wk[kC];  // beta e^(Gc - G) ks
  float eq[kC];  // scale e^G qs
  float inv_t, inv_p;  // the inverse scales of the T and P images
  float egc;           // e^Gc
  float near;          // 1: G spans at most kNear in the chunk, and fa, fb hold
  float pad[28];
  // up to here for the chains, from here on for the gradients
  float eg[kC];          // e^G
  float gh[kC], gl[kC];  // G as an unrounded sum of two floats
  float fa[kC], fb[kC];  // e^(G - m), e^(m - G), m the middle of G's range: e^(G_i - G_j) = fa_i fb_j
  float beta[kC];
};
constexpr float kNear = 60.f;  // e^+-30 leaves the products of fa, fb and any factors far from overflow
constexpr size_t kChainScal = 3 * kC * sizeof(float) + 128;
static_assert(sizeof(Scal) % 128 == 0 && sizeof(Rows) % 128 == 0, "bulk copies");

// Where a record holds its images (the state's or its gradient's first) and its
// scales; pairs of fp16, do in `parts`.
struct Record {
  size_t u, d, scales, size;
};
GDR_BOTH constexpr Record f_record(int Kp, int) {
  const size_t st = 2 * kVt * Kp * 2, u = 2 * kVt * kC * 2;
  return {st, 0, st + u, st + u + 128};
}
GDR_BOTH constexpr Record b_record(int Kp, int parts) {
  const size_t st = 2 * kVt * Kp * 2, u = 2 * kVt * kC * 2, d = (size_t)parts * kVt * kC * 2;
  return {st, st + u, st + u + d, st + u + d + 128};
}

struct Layout {
  int Kp, vt, parts;
  size_t n_k, n_v, n_t;           // (slot, key head), (slot, value head), (slot, value head, tile) counts
  size_t kq_img;         // bytes of one image of q or k
  size_t f_rec, b_rec;   // and of a tile's records
  static constexpr size_t tp_img = 2 * 10 * 16 * 16 * 2;  // T or P: the lower ten blocks of 16 x 16
};
inline Layout layout(const Shape& s, bool bf16) {
  Layout l;
  l.Kp = padded_k(s.K);
  l.vt = v_tiles(s.V);
  l.parts = bf16 ? 1 : 2;
  l.n_k = (size_t)s.slots * s.Hk;
  l.n_v = (size_t)s.slots * s.Hv;
  l.n_t = l.n_v * l.vt;
  l.kq_img = (size_t)l.parts * kC * l.Kp * 2;
  l.f_rec = f_record(l.Kp, l.parts).size;
  l.b_rec = b_record(l.Kp, l.parts).size;
  return l;
}

// The regions of the caller's `saved` buffer (first line: always; second: for a
// backward) and of the backward's workspace.
struct Buffers {
  char *k_img, *q_img, *t_img, *p_img;
  Rows* rows;
  Scal* scal;
  // A record a tile of value columns, which the gradients copy whole. Of the
  // forward: the images of the state before the chunk and of u, their inverse
  // scales; of the backward: of the carried gradient after it, lambda and do.
  char *f_rec, *b_rec;
  float *carry, *carry_back;      // states and their gradients from segment to segment, where the caller wants none
  float *dq_part, *dk_part;       // [B][T][Hv][K] terms of shared heads' gradients, or null
};

struct Args {
  Shape s;
  const void *q, *k, *v, *d_o;
  const float *g, *beta, *s_init, *dS_final;
  void *o, *dq, *dk, *dv;
  float *s_final, *dg, *dbeta, *dS_init;
  Buffers b;
  unsigned* status;
  int seg0, segn;  // the chunks of a sequence that this launch is about (segments_of), segn 0: all
  int small;  // few chunks: a call's kernels may begin while the one before still runs (launch_after).
              // Saves 4 of 31 us for one chunk; 40 heads of 1024 chunks lost 650 of 3900 us to blocks
              // that waited where others could have run.
  // The debug build's: this one (from 1) of the gradients' tiles, or of the chains' images of T, is not
  // copied, and its wait runs out.
  int skip_tile, skip_t;
};
// A forward in segments, the preparation of one beside the chain of the one before,
// and a backward, the gradients of one beside the chain of the next: where the
// chains leave SMs free. us in one segment and in as many as here: 40 heads of 1024
// chunks, fp32, forward 2985 and 2174 (4: 2467, 8: 2399); forward and backward,
// bfloat16, 32 heads of 256 chunks 1580 and 1306, 100 of 256 2568 and 2388, 8 of 256
// 1242 and 1208 (8: 1248), 8 of 64 348 (2: 355), fp32 96 of 64 957 and 925.
inline int segments_of(const Shape& s) {
  const int n = (s.T + kC - 1) / kC;
  const long long chains = (long long)s.nseq * s.Hv * ((v_tiles(s.V) + 3) / 4);
  const int most = n >= 128 ? n / 64 : n >= 64 && chains >= 16 ? 2 : 1;
  return s.packed || chains > 104 ? 1 : most < 16 ? most : 16;
}
inline int is_small(const Shape& s) { return (long long)s.slots * s.Hv <= 152; }

cudaError_t launch_prep(const Args& a, bool bf16, cudaStream_t stream);
cudaError_t launch_fwd(const Args& a, bool bf16, bool save, cudaStream_t stream);
cudaError_t launch_bwd(const Args& a, bool bf16, cudaStream_t stream);
cudaError_t launch_grad(const Args& a, bool bf16, cudaStream_t stream);
// Zeros in up to five outputs of a packed call at the tokens of no sequence; after
// its other kernels.
struct Gaps {
  uint32_t* at[5];
  long long words[5];  // of a token
};
cudaError_t launch_gaps(const Args& a, const Gaps& g, cudaStream_t stream);

// Allows a kernel its dynamic shared memory, once a device; `done` belongs to the kernel.
inline cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A launch that may begin (early) while the kernel before it on the stream, one of
// the same call, is still running: it sees that kernel's results from its wait
// (grid_wait) on.
template <typename... A>
cudaError_t launch_after(bool early, void (*kernel)(A...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = early;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid), c.blockDim = dim3(block), c.dynamicSmemBytes = smem, c.stream = stream, c.attrs = &attr, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}
#ifdef __CUDACC__
// In the kernel launched so, before anything of the kernel before is read; and in
// that kernel, to let the next begin once every block has come this far.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// The gradients of shared heads: summed in the block that makes them all, where
// shared memory has room for the sums and the key heads fill the SMs, or terms.
constexpr bool sums_in_block(int parts, int Kp) { return parts == 1 && Kp == 128; }
inline bool needs_terms(const Shape& s, int parts) {
  return s.Hv != s.Hk && !(sums_in_block(parts, padded_k(s.K)) && (long long)s.slots * s.Hk >= 152);
}

struct StepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  float* state;        // [slots][Hv][V][K]
  const int* slots;    // [R], negative: skip; or null for 0 .. R-1
  void* o;
  int R, T, Hk, Hv, K, V, n_slots, l2norm;
  float scale;
  long long q_b, q_t, k_b, k_t, v_b, v_t;
};
cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t stream);

}  // namespace gdr
