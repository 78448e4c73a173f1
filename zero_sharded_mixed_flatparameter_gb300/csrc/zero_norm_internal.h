// Internal interface of the layer norm (zero_norm_kernels.cu), the 8-bit form
// of activations (zero_pack_kernels.cu) and the embedding
// (zero_embedding_kernels.cu).  Not part of the public ABI.
#pragma once

namespace zfs {

// Failed index checks of a debug build in the file named (0xFFFFFFFF if the
// counter cannot be read; always 0 in a release build).
unsigned int norm_debug_failures();
unsigned int pack_debug_failures();
unsigned int embedding_debug_failures();

}  // namespace zfs
