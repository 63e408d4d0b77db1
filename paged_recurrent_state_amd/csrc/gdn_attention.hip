// Attention over the paged cache: decode, the choice of the kernels, which are built by
// element type, and their workspace.
#include "gdn_attention_kernels.h"

namespace gdn {

hipError_t launch_attention(const AttnParams& p, int D, int dtype, void* workspace, hipStream_t s) {
  if (p.T == 0 || p.kv.B == 0) return hipSuccess;
  const bool bf16 = dtype == 0, codes = p.scales.k != nullptr;
  if (!p.cu) {
    if (codes) return bf16 ? decode_of_type<Bf, true>(p, D, workspace, s) : decode_of_type<Hf, true>(p, D, workspace, s);
    return bf16 ? decode_of_type<Bf, false>(p, D, workspace, s) : decode_of_type<Hf, false>(p, D, workspace, s);
  }
  if (codes && p.sinks) return bf16 ? launch_chunk8_sinks_bf16(p, D, workspace, s) : launch_chunk8_sinks_f16(p, D, workspace, s);
  if (codes) return bf16 ? launch_chunk8_bf16(p, D, workspace, s) : launch_chunk8_f16(p, D, workspace, s);
  if (p.sinks) return bf16 ? launch_chunk_sinks_bf16(p, D, workspace, s) : launch_chunk_sinks_f16(p, D, workspace, s);
  return bf16 ? launch_chunk_bf16(p, D, workspace, s) : launch_chunk_f16(p, D, workspace, s);
}

template <int D>
static size_t bytes_of(int64_t T, int64_t B, int64_t G, bool codes) {
  return std::max(codes ? decode_bytes<D, true>(G) : decode_bytes<D, false>(G), chunk_ws<D>(T, B, G).total);
}

size_t attention_bytes(int D, int64_t T, int64_t B, int64_t G, bool codes) {
  return D == 64 ? bytes_of<64>(T, B, G, codes) : D == 128 ? bytes_of<128>(T, B, G, codes) : bytes_of<256>(T, B, G, codes);
}

}  // namespace gdn
