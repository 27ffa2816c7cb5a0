/*
 * gdr.h - C ABI of the gated delta rule on one GPU (sm_103a), in the same
 * library as wkv7.h (libwkv7.so). Status codes, the error message
 * (wkv7_last_error), wkv7_status and the stream conventions are those of
 * wkv7.h.
 *
 * The operation. For every sequence and value head a V x K fp32 state S (row =
 * value index, column = key index, as wkv7.h) runs over the tokens with a log
 * decay g_t and a write strength beta_t of one number each:
 *     u_t = v_t - e^{g_t} S k_t          (the value less what S holds for k)
 *     S  <- e^{g_t} S + beta_t u_t k_t^T
 *     o_t = scale S q_t
 * With l2norm != 0, q_t and k_t (of lengths up to 2^115) are first divided by
 * sqrt(|.|^2 + 1e-6), and the gradients are those of the vectors given. g = -inf empties the state.
 * The rule is stable for |k| <= 1, 0 <= beta <= 1 (up to 2), g <= 0; the
 * kernels compute any finite values.
 *
 * Heads: q and k have Hk heads, v, o, g and beta Hv = a multiple of Hk; value
 * head h reads key head h / (Hv / Hk). K and V are multiples of 8 up to 128.
 *
 * Layouts. q, k [B][T][Hk][K]; v, o, d_o, dv [B][T][Hv][V]; g, beta, dg, dbeta
 * [B][T][Hv] fp32; states [n][Hv][V][K] fp32, n = B or the packed sequences.
 * Row-major; q, k and v may be slices of a wider tensor: `strides`, if not
 * NULL, points to six numbers on the host, the elements from one batch row to
 * the next and from one token to the next of q, of k and of v (multiples of 8).
 *
 * Packed sequences: with seq_starts (device int32 [nseq + 1]) B is 1 and
 * sequence s has the tokens seq_starts[s] .. seq_starts[s+1] - 1 of the one
 * batch row, from its own state; it may be empty. The numbers must not
 * decrease (they are clamped into [0, T]); where they do not run from 0 to T, o
 * and the gradients of the tokens before and behind are 0, so that a batch may be
 * padded to a fixed size. Without it nseq is not read.
 *
 * Chunks. The forward and backward work on chunks of 64 tokens: what a chunk
 * needs beyond the state (the inverse of its key Gram matrix, its decays) for
 * all chunks at once, then the states from chunk to chunk, then (backward) the
 * gradients of all chunks at once. Products run on the tensor cores with
 * operands of two fp16 values (22 bits; bfloat16 inputs are exact in one) and
 * fp32 accumulation; states, sums and decays are fp32. Each operand tile (a chunk's
 * 64 tokens by 16 value columns, 16 rows of a state, a chunk's T, P, F or E, a
 * token's q or k) has a scale from its largest value: a value 2^-17 of that has 22
 * bits, smaller ones have fewer, and below 2^-39 it counts as 0. So a state that only
 * decays within a chunk is right to 2^-36 of the chunk's largest input and state, not
 * of itself, and results have fewer bits where g > 0 lets a chunk grow by more than
 * 2^17 from one token to another (1e-4 at e^17). (gdr_step computes in fp32
 * throughout.) A value of infinity or
 * NaN makes its chunk and those after it (before it, for gradients)
 * non-finite in its head.
 *
 * Every pointer is device memory owned by the caller, 16-byte aligned (g, beta,
 * their gradients, seq_starts and slots: 4-byte); outputs are overwritten and
 * must not overlap an input or another output. An invalid argument returns
 * WKV7_ERR_INVALID before anything is enqueued; nothing is allocated. Empty
 * problems (B, T, Hv or a sequence of 0) are valid: states
 * pass through.
 */
#ifndef GDR_H
#define GDR_H

#include <stddef.h>

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the buffer `saved` of a forward call: its workspace, and with
 * for_backward != 0 also what gdr_backward reads. nseq: the packed sequences,
 * or a negative number for dense batches. 0 for sizes that are not supported. */
size_t gdr_saved_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, int for_backward);
/* Bytes of gdr_backward's workspace. */
size_t gdr_backward_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16);

/* Forward. s_init: initial states, or NULL for zeros. o and s_final: outputs,
 * s_final may be NULL. saved: gdr_saved_bytes(..., for_backward). */
int gdr_forward(const float* q, const float* k, const float* v, const float* g, const float* beta, const float* s_init,
                const int* seq_starts, float* o, float* s_final, void* saved, const long long* strides, float scale,
                int l2norm, int for_backward, int B, int T, int Hk, int Hv, int K, int V, int nseq, void* stream);
int gdr_forward_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                     const float* s_init, const int* seq_starts, wkv7_bf16* o, float* s_final, void* saved,
                     const long long* strides, float scale, int l2norm, int for_backward, int B, int T, int Hk, int Hv,
                     int K, int V, int nseq, void* stream);

/* Backward of sum <d_o, o> + <dS_final, s_final>, with the `saved` of a forward
 * call of the same inputs, sizes and options with for_backward. dS_final may be
 * NULL (zeros); dq, dk, dv have the inputs' type and dense layout, dg, dbeta and
 * dS_init (may be NULL) are fp32. workspace: gdr_backward_bytes(...). dq and dk
 * of shared heads are summed in the order of the heads: results are the same
 * bits every time. */
int gdr_backward(const float* q, const float* k, const float* v, const float* g, const float* beta, const float* d_o,
                 const float* dS_final, const int* seq_starts, const void* saved, void* workspace, float* dq, float* dk,
                 float* dv, float* dg, float* dbeta, float* dS_init, const long long* strides, float scale, int l2norm,
                 int B, int T, int Hk, int Hv, int K, int V, int nseq, void* stream);
int gdr_backward_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                      const wkv7_bf16* d_o, const float* dS_final, const int* seq_starts, const void* saved,
                      void* workspace, wkv7_bf16* dq, wkv7_bf16* dk, wkv7_bf16* dv, float* dg, float* dbeta,
                      float* dS_init, const long long* strides, float scale, int l2norm, int B, int T, int Hk, int Hv,
                      int K, int V, int nseq, void* stream);

/* The recurrence itself for T tokens of each of R requests (T = 1 when
 * decoding), states updated in place: q, k [R][T][Hk][K], v, o [R][T][Hv][V],
 * g, beta [R][T][Hv], strides as above; state [n_slots][Hv][V][K]. slots
 * (device int32 [R]) names each request's state, no state twice; NULL: request
 * r has state r. A slot below 0 or not below n_slots is skipped: its o is 0 and
 * no state changes. fp32 arithmetic throughout. */
int gdr_step(const float* q, const float* k, const float* v, const float* g, const float* beta, float* state,
             const int* slots, float* o, const long long* strides, float scale, int l2norm, int R, int T, int Hk, int Hv,
             int K, int V, int n_slots, void* stream);
int gdr_step_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                  float* state, const int* slots, wkv7_bf16* o, const long long* strides, float scale, int l2norm, int R,
                  int T, int Hk, int Hv, int K, int V, int n_slots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
