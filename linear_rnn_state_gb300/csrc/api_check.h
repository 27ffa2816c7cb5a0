// Argument checks shared by the C entry points of gdr.h and blocknorm.h.
#pragma once

#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "wkv7.h"
#include "wkv7_launch.h"

namespace wkv7 {
// The current device's status word, which kernels report a timeout through (wkv7_api.cu).
int api_status_word(unsigned** out);
}  // namespace wkv7

namespace api {

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return wkv7::api_fail(code, buf);
}

// A buffer of a call: where it is, the bytes the call may touch, whether it must be there.
struct Span {
  const void* p;
  unsigned long long bytes;
  const char* name;
  bool required;
  unsigned align = 16;
};

inline bool overlaps(const Span& x, const Span& y) {
  if (!x.p || !y.p || !x.bytes || !y.bytes) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a < b + y.bytes && b < a + x.bytes;
}

template <int kIn, int kOut>
int check_spans(const Span (&ins)[kIn], const Span (&outs)[kOut]) {
  for (int side = 0; side < 2; ++side)
    for (int i = 0; i < (side ? kOut : kIn); ++i) {
      const Span& s = side ? outs[i] : ins[i];
      if (!s.p && s.required && s.bytes) return fail(WKV7_ERR_INVALID, "%s must not be NULL", s.name);
      if (reinterpret_cast<uintptr_t>(s.p) % s.align)
        return fail(WKV7_ERR_INVALID, "%s is not %u-byte aligned", s.name, s.align);
    }
  for (int o = 0; o < kOut; ++o) {
    for (int i = 0; i < kIn; ++i)
      if (overlaps(outs[o], ins[i])) return fail(WKV7_ERR_INVALID, "%s overlaps input %s", outs[o].name, ins[i].name);
    for (int q = 0; q < o; ++q)
      if (overlaps(outs[o], outs[q])) return fail(WKV7_ERR_INVALID, "%s overlaps output %s", outs[o].name, outs[q].name);
  }
  return WKV7_OK;
}

}  // namespace api
