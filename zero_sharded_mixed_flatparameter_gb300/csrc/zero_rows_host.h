// Host helpers of the operators over rows of activations: argument checks and
// error texts.  Not part of the public ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "zero_flatstep.h"
#include "zero_internal.h"

namespace zfs {

inline zero_status refuse(zero_status st, const char* text) {
  zfs_report_error(nullptr, st, text);
  return st;
}

// As the other calls of every step: NULL and alignment are checked, not where
// the memory lies.
inline bool misplaced(const void* p, int alignment) { return !p || reinterpret_cast<uintptr_t>(p) % alignment != 0; }

inline bool is_dtype(int d) { return d == ZERO_GRAD_BF16 || d == ZERO_GRAD_FP32; }
inline int dtype_bytes(int d) { return d == ZERO_GRAD_FP32 ? 4 : 2; }

// Rows that are written must not share elements: several threads would write them.
inline bool rows_overlap(long long stride, long long rows, long long cols) { return rows > 1 && stride < cols; }

inline zero_status launch_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return ZERO_OK;
  char buf[256];
  std::snprintf(buf, sizeof buf, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return refuse(ZERO_ECUDA, buf);
}

// Whether rows can be read and written in 16-byte accesses.
inline bool rows_aligned(const void* p, long long stride, long long rows, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || stride % (16 / dtype_bytes(dtype)) == 0);
}

inline int power_of_two(int x) {
  int p = 1;
  while (p < x) p *= 2;
  return p;
}

// Lets a kernel have kMostShared bytes of dynamic shared memory, once a context
// (the limit belongs to it); its static part and 1 KB of the system's come on top
// of that, to 228 KB.
template <auto kKernel, int kMostShared>
cudaError_t allow_shared() {
  static std::atomic<unsigned long long> done{~0ull};
  unsigned long long id = 0;
  const bool known = current_context_id(&id);
  if (known && done.load(std::memory_order_relaxed) == id) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
  if (e == cudaSuccess && known) done.store(id, std::memory_order_relaxed);
  return e;
}

// Launches that may become resident while the kernel before them finishes (the
// kernel waits for it before it reads anything).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t shared, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t launch = {};
  launch.gridDim = grid;
  launch.blockDim = block;
  launch.dynamicSmemBytes = shared;
  launch.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  launch.attrs = attr;
  launch.numAttrs = 1;
  return cudaLaunchKernelEx(&launch, kernel, args...);
}

}  // namespace zfs
