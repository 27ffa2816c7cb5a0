// Internal launch interface of linear attention with a decay between the C ABI
// (linattn_api.cu) and its kernels.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#ifdef WKV7_DEBUG
#include "linattn_debug.h"
#endif

namespace linattn {

// Tokens of a chunk: those that fill the rows of a tcgen05 product, or (mma.sync: fp32 with heads above 64) 64.
constexpr int kCBf16 = 128, kCF32 = 64;
inline bool on_tcgen05(int K, int V, bool bf16) { return bf16 || (K <= 64 && V <= 64); }
constexpr int kMaxDim = 128;  // largest head size
constexpr int kSms = 152;     // of the GPU that plans go by

// What a call's sequences and heads look like.
struct Shape {
  int B, T, Hk, Hv, K, V;
  int nseq;           // sequences: B, or those packed in the one batch row
  const int* starts;  // device [nseq + 1], or null
  int C;              // tokens of a chunk
  int slots;          // chunk slots: an upper bound of the chunks, see slot_count
  int packed;         // nseq sequences in one batch row
  int fixed;          // g is [Hv], one number a head
  float scale;
  long long q_b, q_t, k_b, k_t, v_b, v_t;  // element strides of a batch row and of a token
};

// Every sequence's chunks get slots of their own, and so do segments of several chunks. Dense: batch *
// ceil(T / tokens). Packed: a sequence that starts at token x is given the slots from x / tokens + s
// on (s its number): x / tokens + ceil(len / tokens) <= (x + len) / tokens + 1, so the next
// sequence's slots start after them, and T / tokens + nseq are enough.
inline long long slot_count(int B, int T, int nseq, bool packed, int tokens) {
  return packed ? (long long)T / tokens + nseq : (long long)B * ((T + tokens - 1) / tokens);
}

struct Args {
  Shape s;
  const void *q, *k, *v, *d_o;
  const float *g, *s_init, *dS_final;
  void *o, *dq, *dk, *dv;
  float *s_final, *dS_init;
  float *dg;           // [B][T][Hv] (a workspace where g is fixed)
  float *dg_fixed;     // [Hv], where g is fixed
  float *states;       // [slots][Hv][V][K]: the state before each chunk or segment
  float *dstates;      // the gradient of the state after each
  float *decay;        // [slots][Hv]: the whole decay of each
  void *images, *dimages;  // states and dstates as the gradients' products read them (linattn_tc.cuh)
  double *part;        // [kParts][Hv]: sums of dg over tokens
  unsigned* status;    // the device's status word
  int skip_what, skip_n;   // debug build only: linattn_debug.h
};
constexpr int kParts = 256;

// fp32 with heads above 64: the states before all chunks, or the gradients of those after them, and the last one
// (s_final, dS_init); o; dv, dq, dk and dg of all chunks at once.
cudaError_t launch_states(const Args& a, bool backward, cudaStream_t stream);
cudaError_t launch_rows_o(const Args& a, cudaStream_t stream);
cudaError_t launch_rows_grad(const Args& a, cudaStream_t stream);
// On tcgen05: o (backward: dv), from chunk to chunk.
//   kWhole: whole sequences, from s_init (dS_final) to s_final (dS_init)
//   kSums: segments of `chunks` chunks from zeros: only the sum of each, to `states` (dstates), and its whole decay
//   kResume: segments from `states`, where join has put the state before each
// keep: images (or dimages) of the states before (after) the chunks too.
struct Maps;
enum Way { kWhole, kSums, kResume };
cudaError_t launch_chain(const Maps& maps, const Args& a, bool backward, int chunks, Way way, bool keep, cudaStream_t stream);
cudaError_t launch_chain32(const Args& a, bool backward, int chunks, Way way, bool keep, cudaStream_t stream);  // fp32
// From sums of stretches of `tokens` tokens to the states before (the gradients after) them, and the last one.
cudaError_t launch_join(const Args& a, bool backward, int tokens, cudaStream_t stream);
// dq, dk and dg of all chunks at once, from the images.
cudaError_t launch_grad(const Maps& maps, const Args& a, bool bf16, cudaStream_t stream);
// The tensor maps of q, k, v and (where not null) do; false: the driver has no encoder or refuses.
bool make_maps(Maps& maps, const Args& a);
cudaError_t launch_dg_sums(const Args& a, cudaStream_t stream);          // dg_fixed from dg

// Zeros in the outputs of a packed call (null: none) at the tokens of no sequence.
constexpr int kGapOutputs = 4;
struct Gaps {
  uint32_t* at[kGapOutputs];
  long long words[kGapOutputs];  // of a token
};
cudaError_t launch_gaps(const Args& a, const Gaps& g, cudaStream_t stream);

struct StepArgs {
  const void *q, *k, *v;
  const float* g;
  float* state;
  const int* slots;
  void* o;
  int R, T, Hk, Hv, K, V, n_slots, fixed;
  float scale;
  long long q_b, q_t, k_b, k_t, v_b, v_t;
};
cudaError_t launch_step(const StepArgs& a, bool bf16, cudaStream_t stream);

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

}  // namespace linattn
