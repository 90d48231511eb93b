// Arguments of the paged-cache kernels (see include/srmoe.h for what each one is).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace srmoe {

struct KvAppendArgs {
  const uint16_t* qkv;
  size_t qkv_stride;
  int T, Hq, Hkv, D, rd;
  bool neox, norm, fp8;
  const float *qw, *kw;
  float eps;
  const int32_t* positions;
  const float* cos_sin;
  int max_pos;
  const int32_t* slots;
  uint16_t* q_out;
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  int num_slots, page_shift;
  size_t page_stride;   // elements
};

struct AttnArgs {
  const uint16_t* q;
  size_t q_stride;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;   // null: a bf16 cache
  int num_pages, page_shift;
  size_t page_stride;   // elements
  const int32_t* block_table;
  int max_pages;
  const int32_t *cu_q, *kv_lens;
  const uint64_t* tree_mask;        // null: causal
  const int32_t* prefix_lens;       // null: no prefix
  int S, T, max_q, Hq, Hkv, G, D;
  float scale, softcap;
  uint16_t* out;
  float* lse;
  void* ws;
};

hipError_t launch_attention(const AttnArgs&, hipStream_t);
size_t attention_workspace_bytes(int S, int max_q, int Hq, int Hkv, int D);

// One sequence of an attention call, with every length taken from device memory held to
// what the arrays can hold: first query row, query tokens (of them the first max_q are computed),
// cached tokens.
struct SeqInfo {
  int row0, tokens, n, kv;
};
__device__ __forceinline__ SeqInfo seq_info(const AttnArgs& a, int s) {
  SeqInfo q;
  const int lo = min(max(a.cu_q[s], 0), a.T), hi = min(max(a.cu_q[s + 1], 0), a.T);
  q.row0 = lo;
  q.tokens = max(hi - lo, 0);
  q.n = min(q.tokens, a.max_q);
  q.kv = min(max(a.kv_lens[s], 0), a.max_pages << a.page_shift);
  return q;
}

}  // namespace srmoe
