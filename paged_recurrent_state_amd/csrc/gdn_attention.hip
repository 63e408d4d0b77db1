// Attention over the paged cache: the kernels' sources by element type, and their
// workspace.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_attention(const AttnParams& p, int D, int dtype, void* workspace, hipStream_t s) {
  if (p.T == 0 || p.kv.B == 0) return hipSuccess;
  if (p.scales.k) return (dtype == 0 ? launch_attention8_bf16 : launch_attention8_f16)(p, D, workspace, s);
  return (dtype == 0 ? launch_attention_bf16 : launch_attention_f16)(p, D, workspace, s);
}

size_t attention_bytes(int D, int64_t T, int64_t B, int64_t G) {
  if (D == 64) return std::max(decode_bytes<64>(), chunk_ws<64>(T, B, G).total);
  if (D == 128) return std::max(decode_bytes<128>(), chunk_ws<128>(T, B, G).total);
  return std::max(decode_bytes<256>(), chunk_ws<256>(T, B, G).total);
}

}  // namespace gdn
