// Attention of f16 queries and caches.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_attention_f16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return launch_type<Hf, false>(p, D, workspace, s);
}

}  // namespace gdn
