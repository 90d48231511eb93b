// Attention with a sliding window and sinks over the paged cache: the instances of attention_dev.hpp that walk
// the tiles of the sinks and of the window alone. Token i of a sequence of n tokens and ctx = kv - n cached ones before sees
//   j <= ctx + i   and   (j > ctx + i - window   or   j < sinks)
// and the softmax is over what it sees. Pages that hold no such token of any i are not looked up.
//
// What bounds it. A tile of TB tokens sees window + TB + sinks keys, so the line of segments, in which a segment counts what
// it sees (window_keys), is that much shorter and the split, the tiles and the join stay as they are. Masked tiles are those at
// either edge of the window and the last of the sinks. Measured (times by the card), 12 heads of 128 on one unless named:
//   64 single tokens, window 4096 and 4 sinks: 32 us (135 MB, 4.2 TB/s: the keys' bytes), e4m3 22 (68 MB); 8 heads of 256 55 (269
//   MB, 4.9 TB/s); one sequence of 777, window 512: 12 (latency)
//   16384 tokens behind a window of 4096: e4m3 476 to 510 (810 to 860 TFLOP/s), bf16 502, with a cap of 30 614; the matrix cores
//   and the vector unit in turn, as without a window, but the segments are all alike: 1639 of them on 512 places are 3.2 rounds
//   8192 tokens of 8 heads of 256: 271, e4m3 268 (1020 TFLOP/s; 5 to 21 registers spill)
//   ragged prompts of 96 heads on 8, window 1024, cap 30: 819 to 880 (590 to 630 TFLOP/s: the cap takes an exponential and a
//   reciprocal more for every score, and 14% of the scores are of rows without a token or outside the mask)
#include "attention_dev.hpp"

namespace srmoe {

hipError_t launch_window_attention(const AttnArgs& a, hipStream_t stream) { return launch_dims<true>(a, stream); }

}  // namespace srmoe
