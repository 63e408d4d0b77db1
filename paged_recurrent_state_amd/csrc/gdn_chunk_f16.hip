// Chunks of f16 queries over f16 caches.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_chunk_f16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return chunk_of_type<Hf, false, false>(p, D, workspace, s);
}

}  // namespace gdn
