// What the C ABI's entry points share: the thread's last error, argument
// checks and the end of a call.
#pragma once

#include "../../include/gdn.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

namespace gdn {

extern thread_local std::string g_last_error;  // gdn_api.cpp

namespace api {

inline gdn_status fail(gdn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool debug_sync() {
  static const bool on = [] {
    const char* e = std::getenv("GDN_DEBUG");
    return e && e[0] && e[0] != '0';
  }();
  return on;
}

inline gdn_status finish(hipError_t e, hipStream_t stream, const char* what) {
  if (e == hipSuccess && debug_sync()) e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return fail(GDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  g_last_error.clear();
  return GDN_OK;
}

inline bool is_dtype(int32_t d) { return d == GDN_F32 || d == GDN_BF16; }
inline size_t esize(int32_t d) { return d == GDN_BF16 ? 2 : 4; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  size_t rows, width, stride;
  size_t span() const { return p && rows ? (rows - 1) * stride + width : 0; }
};

// Whether two sets of rows share a byte.  Rows of one stride may lie side by
// side in a wider buffer (column slices); of unequal strides the whole spans
// have to be apart.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.rows <= 1 || b.rows <= 1 || a.stride != b.stride || !a.stride) return true;
  // the distance from a row of `a` to the next row of `b`, in [0, stride)
  const intptr_t diff = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
  const intptr_t st = static_cast<intptr_t>(a.stride);
  const size_t off = static_cast<size_t>(((diff % st) + st) % st);
  return off < a.width || a.stride - off < b.width;
}

}  // namespace api
}  // namespace gdn
