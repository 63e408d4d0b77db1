// Attention of bf16 queries and caches.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_attention_bf16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return launch_type<Bf, false>(p, D, workspace, s);
}

}  // namespace gdn
