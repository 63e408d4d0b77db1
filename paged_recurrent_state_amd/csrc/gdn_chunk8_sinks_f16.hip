// Chunks of f16 queries over 8-bit caches, with first tokens that stay visible beside a window.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_chunk8_sinks_f16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return chunk_of_type<Hf, true, true>(p, D, workspace, s);
}

}  // namespace gdn
