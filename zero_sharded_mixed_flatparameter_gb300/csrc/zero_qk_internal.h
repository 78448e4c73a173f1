// Internal interface of the norm and rotation of queries and keys
// (zero_qk_kernels.cu).  Not part of the public ABI.
#pragma once

namespace zfs {

constexpr int kMaxHeadDim = 256;

// Failed index checks of a debug build in zero_qk_kernels.cu (0xFFFFFFFF if
// the counter cannot be read; always 0 in a release build).
unsigned int qk_debug_failures();

}  // namespace zfs
