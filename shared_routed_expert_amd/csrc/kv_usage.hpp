// Arguments of the kernels that keep the cached tokens' usage and evict by it (see include/srmoe.h).
#pragma once
#include "attention.hpp"

namespace srmoe {

struct UsageArgs {
  AttnArgs a;                  // (v_cache, out, lse and tree_mask are not set)
  const float* lse;
  const float* prev;           // null: nothing is known of the tokens before
  float decay;
  float* usage;
  const int32_t* usage_rows;   // null: row s
  int rows;
};

struct EvictArgs {
  uint8_t *k_cache, *v_cache;
  int num_pages, page_shift;
  size_t page_bytes;
  int row_bytes;               // of a token's head: 64 to 512
  const int32_t* block_table;
  int max_pages;
  const int32_t* kv_lens;
  const float* usage;
  float* new_usage;            // may be usage
  const int32_t* usage_rows;   // null: row s
  int rows, S, Hkv, limit, budget, sinks, recent;
  const int32_t* new_table;
  int new_max_pages;
  int32_t *new_lens, *kept;
};

hipError_t launch_kv_evict(const EvictArgs&, hipStream_t);
hipError_t launch_kv_usage(const UsageArgs&, hipStream_t);
size_t kv_usage_workspace_bytes(int D);

}  // namespace srmoe
