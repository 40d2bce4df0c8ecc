// The host side that the kernel files of libselscan share: the error message
// behind ssm_last_error() and the argument checks.
#ifndef SELSCAN_HOST_H
#define SELSCAN_HOST_H

#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "selscan.h"

// one message per host thread, shared by the files
inline thread_local char g_last_error[512] __attribute__((visibility("hidden"))) = "";

namespace {

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return status;
}

struct Span {
  const void* p;
  int64_t bytes;
  const char* name;
};

bool overlaps(const Span& x, const Span& y) {
  if (!x.p || !y.p || x.bytes <= 0 || y.bytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)x.p, a1 = a0 + (uintptr_t)x.bytes;
  const uintptr_t b0 = (uintptr_t)y.p, b1 = b0 + (uintptr_t)y.bytes;
  return a0 < b1 && b0 < a1;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t kMaxExtent = (int64_t)1 << 40;

int check_extent(const char* name, int64_t v) {
  if (v <= 0 || v > kMaxExtent) return fail(SSM_E_SHAPE, "%s = %lld is out of range", name, (long long)v);
  return SSM_OK;
}

// a * b * c * d <= 2^60 (byte sizes of every tensor stay far from overflow)
bool product_ok(int64_t a, int64_t b, int64_t c = 1, int64_t d = 1) {
  const int64_t lim = (int64_t)1 << 60;
  int64_t p = a;
  for (int64_t f : {b, c, d}) {
    if (p > lim / f) return false;
    p *= f;
  }
  return true;
}

int launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SSM_E_HIP, "%s: %s", what, hipGetErrorString(e));
  return SSM_OK;
}

}  // namespace

#endif  // SELSCAN_HOST_H
