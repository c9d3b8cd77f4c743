// tl_kv_prefill.h -- what tl_kv_attn hands to the kernel for many query rows.
#pragma once

#include "tl_internal.h"
#include "tl_kv.cuh"

namespace tl {

struct PrefillParams {
  KvCacheDev c;
  KvBatch b;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  float* lse;
  uint32_t* counters;  // [CTAs][2], zero between calls
  float* partial;      // [CTAs][2][2][D + 3][128]
  uint64_t timeout_ns;
  int32_t H, group, causal;
  int32_t min_rows;    // sequences of more query rows per kv head than this are this kernel's
  float scale_log2;
  KvTree tree;         // tl_kv_tree_attn (mask not NULL; causal is 0 then)
  uint32_t page_magic; // groups of 16 tokens to pages: the upper half of a product with it (set by launch_kv_prefill)
};

size_t prefill_partial_bytes(int ctas, int D);
tl_status launch_kv_prefill(PrefillParams& p, int D, int ctas, cudaStream_t st);

}  // namespace tl
