/*
 * gdr_debug.h - extra entry points of the debug build (libwkv7_debug.so,
 * compiled with WKV7_DEBUG) for the gated delta rule. The product library does
 * not export them. They exist to test WKV7_ERR_TIMEOUT of the chains and of the
 * gradients' kernel, whose waits in the debug build end after 1 ms instead of
 * about 2 s.
 */
#ifndef GDR_DEBUG_H
#define GDR_DEBUG_H

#ifdef __cplusplus
extern "C" {
#endif

/* tile > 0: from now on the gradients' kernel of gdr_backward issues no copy, and
 * no expected byte count, for this one (counted from 1) of every block's tiles of
 * 16 value columns, so that the wait for it runs out; the call returns WKV7_OK, its
 * gradients of q, k, g and beta are without meaning and the next wkv7_status()
 * returns WKV7_ERR_TIMEOUT. tile = 0 restores normal operation. Process-wide;
 * returns WKV7_OK. */
int gdr_debug_skip_tile(int tile);

/* step > 0: from now on the chains of gdr_forward and gdr_backward issue no copy,
 * and no expected byte count, of the image of T in this one (counted from 1) of
 * their steps, a chunk each, of every sequence (or segment) that has it; otherwise as
 * above. step = 0 restores normal operation. */
int gdr_debug_skip_t(int step);

#ifdef __cplusplus
}
#endif

#endif /* GDR_DEBUG_H */
