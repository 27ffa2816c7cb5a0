/*
 * qkrope.h - C ABI of the norms of queries and keys with the position rotation
 * on one GPU (sm_103a), in the same library as wkv7.h (libwkv7.so). Status codes,
 * the error message (wkv7_last_error) and the stream conventions are those of wkv7.h.
 *
 * For every token and head of q, and of k with its own weight:
 *     n = x / sqrt(mean(x^2) + eps) * weight
 *     y = n with its first 2 half values turned in pairs by the angles a_j =
 *         position * freq_j, j < half:  (y_a, y_b) = (n_a cos a_j - n_b sin a_j, n_a sin a_j + n_b cos a_j)
 * where pair j is the values (j, half + j), or with interleaved != 0 (2 j, 2 j + 1).
 * The values from 2 half on are not turned. All arithmetic is fp32, but the
 * angles: position * freq_j is formed in turns as an integer of 64 bits (modulo a
 * whole turn), so a far position costs no accuracy (cosines and sines within 2e-7). Rows
 * whose squares leave fp32's range (values from 3e18 on, or below 1e-15 without an eps)
 * are normed times a power of two.
 *
 * Sizes: D a multiple of 8 up to 256, half from 0 to D / 2. q [tokens][Hq][D] and k
 * [tokens][Hk][D] have one type (bfloat16 with bf16 != 0, else fp32), as have the
 * outputs and gradients; a token's heads are dense, q_stride and k_stride are the
 * elements from token to token (multiples of 8). Everything else is dense. Weights
 * and their gradients [D] are fp32, freq [half] is fp64 (finite, radians a position), positions
 * int32 [tokens], or NULL: token t has the position t % T.
 * Every pointer is device memory owned by the caller, 16-byte aligned (positions:
 * 4-byte); outputs are overwritten and must not overlap an input or another output.
 * An invalid argument returns WKV7_ERR_INVALID before anything is enqueued; nothing
 * is allocated. 0 tokens or heads are valid.
 */
#ifndef QKROPE_H
#define QKROPE_H

#include <stddef.h>

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

int qkrope_forward(const void* q, const void* k, const float* q_weight, const float* k_weight, const double* freq,
                   const int* positions, void* q_out, void* k_out, long long q_stride, long long k_stride,
                   long long tokens, long long T, int Hq, int Hk, int D, int half, int interleaved, float eps, int bf16,
                   void* stream);
/* Gradients of sum <dq_out, q_out> + <dk_out, k_out>. part: a workspace of
 * qkrope_part_bytes. The weights' sums are the same bits every time. */
int qkrope_backward(const void* q, const void* k, const float* q_weight, const float* k_weight, const double* freq,
                    const int* positions, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                    float* dk_weight, void* part, long long q_stride, long long k_stride, long long tokens, long long T,
                    int Hq, int Hk, int D, int half, int interleaved, float eps, int bf16, void* stream);
/* Bytes of a backward's workspace. */
size_t qkrope_part_bytes(long long tokens, int Hq, int Hk, int D);

#ifdef __cplusplus
}
#endif

#endif /* QKROPE_H */
