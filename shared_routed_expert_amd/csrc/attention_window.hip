// Attention with a sliding window and sinks over the paged cache: the instances of attention_dev.hpp that walk
// the tiles of the sinks and of the window alone.
#include "attention_dev.hpp"

namespace srmoe {

hipError_t launch_window_attention(const AttnArgs& a, hipStream_t stream) { return launch_dims<true>(a, stream); }

}  // namespace srmoe
