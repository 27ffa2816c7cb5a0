/*
 * blocknorm.h - C ABI of the norms around a block on one GPU (sm_103a), in the
 * same library as wkv7.h (libwkv7.so). Status codes, the error message
 * (wkv7_last_error) and the stream conventions are those of wkv7.h.
 *
 * Before a block, for every row of D values:
 *     h = residual + scale x,   r = 1 / sqrt(mean(h^2) + eps),   n = h r weight
 * x is the block before's output, scale [D] fp32 or NULL for 1. With x NULL, n
 * is the norm of residual itself and h is not written.
 * After it, for every row of D values (a head):
 *     r = 1 / sqrt(mean(o^2) + eps),   y = o r weight z sigmoid(z)
 * All arithmetic is fp32; h enters n before it is rounded to its type. The sigmoid
 * of bfloat16 calls comes from the fast exponential: within (2 + |z|) 2^-24 of
 * itself, and 0 for z below -87.3.
 *
 * Sizes: D from 1 to 8192. x, n and their gradients have one type, residual, h
 * and their gradients another (bfloat16 or fp32; fp32 where x is fp32); weight,
 * scale, their gradients and rstd (one number a row) are fp32. Inputs x,
 * residual (o, z) may have rows wider apart than D: x_stride and
 * residual_stride are the elements from row to row (o_stride and z_stride from
 * token to token, a token's H rows being adjacent). Everything else is dense.
 * Every pointer is device memory owned by the caller, 16-byte aligned; outputs
 * are overwritten and must not overlap an input or another output, except that
 * h may be residual itself (and nothing else). An invalid argument returns
 * WKV7_ERR_INVALID before anything is enqueued; nothing is allocated. 0 rows
 * are valid.
 */
#ifndef BLOCKNORM_H
#define BLOCKNORM_H

#include <stddef.h>

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* rstd: [rows] for the backward, or NULL. */
int blocknorm_add_forward(const void* x, const void* residual, const float* weight, const float* scale, void* h, void* n,
                          float* rstd, long long x_stride, long long residual_stride, long long rows, int D, float eps,
                          int bf16, int residual_bf16, void* stream);
/* dn: gradient of n; dh: gradient of h, or NULL. Outputs dresidual, dx (NULL
 * only with scale NULL, where it equals dresidual up to its type), dweight [D]
 * and dscale [D] (NULL only with scale NULL). part: a workspace of
 * blocknorm_part_bytes. The sums over rows are the same bits every time. */
int blocknorm_add_backward(const void* x, const void* residual, const float* weight, const float* scale,
                           const float* rstd, const void* dn, const void* dh, void* dresidual, void* dx, float* dweight,
                           float* dscale, void* part, long long x_stride, long long residual_stride, long long rows,
                           int D, int bf16, int residual_bf16, void* stream);
int blocknorm_gated_forward(const void* o, const void* z, const float* weight, void* y, float* rstd, long long o_stride,
                            long long z_stride, long long tokens, int H, int D, float eps, int bf16, void* stream);
int blocknorm_gated_backward(const void* o, const void* z, const float* weight, const float* rstd, const void* dy,
                             void* d_o, void* dz, float* dweight, void* part, long long o_stride, long long z_stride,
                             long long tokens, int H, int D, int bf16, void* stream);
/* Bytes of a backward's workspace: rows (tokens * H), and 2 sums for the add
 * norm, 1 for the gated. */
size_t blocknorm_part_bytes(long long rows, int D, int sums);

#ifdef __cplusplus
}
#endif

#endif /* BLOCKNORM_H */
