// Internal interface of the embedding (zero_embedding_kernels.cu).  Not part of
// the public ABI.
#pragma once

namespace zfs {

// Failed index checks of a debug build in zero_embedding_kernels.cu (0xFFFFFFFF if
// the counter cannot be read; always 0 in a release build).
unsigned int embedding_debug_failures();

}  // namespace zfs
