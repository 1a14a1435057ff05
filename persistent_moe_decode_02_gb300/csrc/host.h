// What the C entries of the mixture-of-experts operators share on the host:
// errors, and checks of their buffers.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "launch.cuh"
#include "mk.h"

namespace mk {

void set_last_error(const char* msg);

inline int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

inline int fail_cuda(const char* what, cudaError_t e) {
  cudaGetLastError();   // reported here: not to the caller's next question
  allowed = {};
  char buf[224];
  snprintf(buf, sizeof(buf), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  return fail(MK_ERR_CUDA, buf);
}

inline bool aligned(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }

struct Span {
  const void* at;
  size_t n;
};
// Whether any of the first `written` spans meets another one.
inline bool clash(const Span* s, int written, int n) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (s[i].at && s[j].at && meet(s[i].at, s[i].n, s[j].at, s[j].n)) return true;
  return false;
}

// Multiprocessors of the current device, asked for once by each host thread.
inline cudaError_t multiprocessors(int* out) {
  thread_local int device = -1, count = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev != device) {
    e = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) device = dev;
  }
  *out = count;
  return e;
}

}  // namespace mk
