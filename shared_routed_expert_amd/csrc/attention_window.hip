// Attention with a sliding window and sinks over the paged cache: the instances of attention_dev.hpp that walk
// the tiles of the sinks and of the window alone. Token i of a sequence of n tokens and ctx = kv - n cached ones before sees
//   j <= ctx + i   and   (j > ctx + i - window   or   j < sinks)
// and the softmax is over what it sees. Pages that hold no such token of any i are not looked up.
//
// What bounds it. A tile of TB tokens sees window + TB + sinks keys, so the line of segments, in which a segment counts what
// it sees (window_keys), is that much shorter and the split, the tiles and the join stay as they are. Masked tiles are those at
// either edge of the window and the last of the sinks. 12 heads of 128 on one: 64 single tokens with a window of 4096 and 4 sinks
// 32 us (135 MB, 4.2 TB/s; the keys' bytes), one sequence of 777 with a window of 512 12 (latency); 16384 tokens in e4m3 behind a window of 4096 476 to
// 495 (860 TFLOP/s; the matrix cores and the vector unit in turn, as without a window); ragged prompts of 96 heads on 8 with a
// window of 1024 and a cap of 30 833 to 848 (610 TFLOP/s: the cap's vector work costs a quarter, and 17% of the scores are of
// rows without a token or outside the mask).
#include "attention_dev.hpp"

namespace srmoe {

hipError_t launch_window_attention(const AttnArgs& a, hipStream_t stream) { return launch_dims<true>(a, stream); }

}  // namespace srmoe
