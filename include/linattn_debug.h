/*
 * linattn_debug.h - extra entry point of the debug build (libwkv7_debug.so,
 * compiled with WKV7_DEBUG) for linear attention. The product library does not
 * export it. It exists to test WKV7_ERR_TIMEOUT of the chains and of the
 * gradients' kernel, whose waits in the debug build end after 1 ms instead of
 * about 2 s.
 */
#ifndef LINATTN_DEBUG_H
#define LINATTN_DEBUG_H

#ifdef __cplusplus
extern "C" {
#endif

/* What a block leaves out from now on, so that the waits for it run out; n counts from 1, 0 restores normal operation:
 *   LINATTN_SKIP_TILES   the copies of q, k, v and d_o (and their expected byte counts) of the n-th chunk of a bfloat16
 *                        chain, of the n-th value head in the bfloat16 gradients
 *   LINATTN_SKIP_SCORES  the arrival of the n-th scores: a chunk's in the chains; dq's and dk's, by turns, in the gradients
 *   LINATTN_SKIP_STATE   the gradients' copy of the n-th value head's first 64 keys of the state
 *   LINATTN_SKIP_BACK    the same of the state's gradient
 *   LINATTN_SKIP_CLAIM   a bfloat16 chain's n-th question for a block that has not begun
 * The call returns WKV7_OK, its results are without meaning and the next wkv7_status() returns WKV7_ERR_TIMEOUT.
 * Process-wide; returns WKV7_OK. */
enum { LINATTN_SKIP_TILES = 1, LINATTN_SKIP_SCORES, LINATTN_SKIP_STATE, LINATTN_SKIP_BACK, LINATTN_SKIP_CLAIM };
int linattn_debug_skip(int what, int n);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_DEBUG_H */
