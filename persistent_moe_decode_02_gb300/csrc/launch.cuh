// Launches of the operators' kernels.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mk {

// Before a kernel's first touch of memory that the kernel before it in the
// stream may write or read: its launch does not wait for that one's end, it
// does (launch_kernel).  Such memory is read with plain loads behind it: the
// read-only path (__ldg) is for what nobody writes while a kernel runs, and
// these kernels run before their inputs' last writer has ended.  Tables that
// the host uploads may take it: a stream's copies and kernels never overlap.
__device__ __forceinline__ void await_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be launched; its own await_stream() still waits for this
// one's end.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Whether two ranges of memory meet.
inline bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

// Launches a kernel that begins with await_stream() while the kernel before it
// still runs, so that a chain of short ones does not pay each one's launch
// (one token's attention over 8K cached tokens and its join, call after call:
// 12.3 us, 9.3 so).  Returns the call's own error, none that was left before.
template <class... A, class... B>
cudaError_t launch_kernel(void (*k)(A...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, B&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, static_cast<A>(args)...);
}

// Allocations and releases of this thread while it captures some other stream: without it
// they would fail, and end that capture.
struct BesideCaptures {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Kernels' attributes that this thread of the host has asked for already (asking
// takes as long as a fifth of a launch).  Forgotten after any error, so that a
// device whose context was made anew is asked again.
struct Allowed {
  struct Asked {
    const void* kernel;
    int dev, what;
  } asked[16];
  int n;
};
inline thread_local Allowed allowed = {};

inline cudaError_t allow(const void* kernel, cudaFuncAttribute what, int value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (const Allowed::Asked& a : allowed.asked)
    if (a.kernel == kernel && a.dev == dev && a.what == (int)what) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, what, value);
  if (e == cudaSuccess) allowed.asked[allowed.n++ % 16] = {kernel, dev, (int)what};
  return e;
}

}  // namespace mk
