// Attention of drafted trees, single tokens and prompt chunks over the whole paged cache: the instances of
// attention_dev.hpp without a window.
#include "attention_dev.hpp"

namespace srmoe {

size_t attention_workspace_bytes(int S, int max_q, int Hq, int Hkv, int D) {
  (void)S;
  const int M = tile_rows(max_q, Hq / Hkv);
  return parts_of(M) * 2 * (slot_floats(M, D) * 4 + sizeof(PartDesc));
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t stream) { return launch_dims<false>(a, stream); }

}  // namespace srmoe
