/*
 * linattn.h - C ABI of linear attention with a decay on one GPU (sm_103a), in
 * the same library as wkv7.h (libwkv7.so). Status codes, the error message
 * (wkv7_last_error) and the stream conventions are those of wkv7.h.
 *
 * The operation. For every sequence and value head a V x K fp32 state S (row =
 * value index, column = key index, as wkv7.h) runs over the tokens with a log
 * decay g_t of one number:
 *     S  <- e^{g_t} S + v_t k_t^T
 *     o_t = scale S q_t
 * g = -inf (or below -1e6) empties the state. The rule is stable for g <= 0; the
 * kernels compute any finite values.
 *
 * Heads: q and k have Hk heads, v, o and g Hv = a multiple of Hk; value head h
 * reads key head h / (Hv / Hk). K and V are multiples of 8 up to 128.
 *
 * Layouts. q, k [B][T][Hk][K]; v, o, d_o, dv [B][T][Hv][V]; states
 * [n][Hv][V][K] fp32, n = B or the packed sequences. g and dg are fp32:
 * [B][T][Hv], or with g_fixed != 0 [Hv], one decay a head for all tokens. Row-major;
 * q, k and v may be slices of a wider tensor: `strides`, if not NULL, points to
 * six numbers on the host, the elements from one batch row to the next and from
 * one token to the next of q, of k and of v (multiples of 8). With bf16 != 0 q, k, v,
 * o and their gradients are bfloat16, else fp32.
 *
 * Packed sequences: with seq_starts (device int32 [nseq + 1]) B is 1 and
 * sequence s has the tokens seq_starts[s] .. seq_starts[s+1] - 1 of the one
 * batch row, from its own state; it may be empty. The numbers must not
 * decrease (they are clamped into [0, T]); where they do not run from 0 to T, o
 * and the gradients of the tokens before and behind are 0, so that a batch may be
 * padded to a fixed size. Without it nseq is not read.
 *
 * Arithmetic. The forward and backward work on chunks of tokens: products run on
 * the tensor cores with operands as sums of bfloat16 parts and fp32 accumulation.
 * bfloat16 inputs are exact in one part, fp32 inputs and what is computed are held in three
 * (24 bits); bfloat16 outputs are fp32 results rounded once. States, sums and decays are
 * fp32. Parts have fp32's exponents: no value loses bits beside a larger one. A value of infinity or
 * NaN makes its chunk and those after it (before it, for gradients) non-finite in its
 * head. (linattn_step computes in fp32 throughout.)
 *
 * Every pointer is device memory owned by the caller, 16-byte aligned (g, dg,
 * seq_starts and slots: 4-byte); outputs are overwritten and must not overlap an
 * input or another output. An invalid argument returns WKV7_ERR_INVALID before
 * anything is enqueued; nothing is allocated. Empty problems (B, T, Hv or a
 * sequence of 0) are valid: states pass through.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the buffer `saved` of a forward call: its workspace, and with
 * for_backward != 0 also what linattn_backward reads. nseq: the packed sequences,
 * or a negative number for dense batches. 0 for sizes that are not supported. */
size_t linattn_saved_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, int for_backward);
/* Bytes of linattn_backward's workspace. */
size_t linattn_backward_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int g_fixed, int bf16);

/* Forward. s_init: initial states, or NULL for zeros. o and s_final: outputs,
 * s_final may be NULL. saved: linattn_saved_bytes(..., for_backward). */
int linattn_forward(const void* q, const void* k, const void* v, const float* g, const float* s_init,
                    const int* seq_starts, void* o, float* s_final, void* saved, const long long* strides, float scale,
                    int g_fixed, int for_backward, int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16,
                    void* stream);

/* Backward of sum <d_o, o> + <dS_final, s_final>, with the `saved` of a forward
 * call of the same inputs, sizes and options with for_backward. dS_final may be
 * NULL (zeros); dq, dk, dv have the inputs' type and dense layout; dg (g's shape)
 * and dS_init may be NULL where they are not wanted. workspace:
 * linattn_backward_bytes(...). dq and dk of shared heads and dg of fixed decays are
 * summed in a fixed order: results are the same bits every time. */
int linattn_backward(const void* q, const void* k, const void* v, const float* g, const void* d_o,
                     const float* dS_final, const int* seq_starts, const void* saved, void* workspace, void* dq,
                     void* dk, void* dv, float* dg, float* dS_init, const long long* strides, float scale, int g_fixed,
                     int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, void* stream);

/* The recurrence itself for T tokens of each of R requests (T = 1 when
 * decoding), states updated in place: q, k [R][T][Hk][K], v, o [R][T][Hv][V],
 * g [R][T][Hv] or [Hv], strides as above; state [n_slots][Hv][V][K]. slots
 * (device int32 [R]) names each request's state, no state twice; NULL: request
 * r has state r. A slot below 0 or not below n_slots is skipped: its o is 0 and
 * no state changes. fp32 arithmetic throughout. */
int linattn_step(const void* q, const void* k, const void* v, const float* g, float* state, const int* slots, void* o,
                 const long long* strides, float scale, int g_fixed, int R, int T, int Hk, int Hv, int K, int V,
                 int n_slots, int bf16, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
