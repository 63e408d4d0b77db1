// Attention of bf16 queries over 8-bit caches.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_attention8_bf16(const AttnParams& p, int D, void* workspace, hipStream_t s) {
  return launch_type<Bf, true>(p, D, workspace, s);
}

}  // namespace gdn
