// Chunks of bf16 queries over bf16 caches.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_chunk_bf16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return chunk_of_type<Bf, false, false>(p, D, workspace, s);
}

}  // namespace gdn
