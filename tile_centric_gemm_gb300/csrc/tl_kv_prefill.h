// tl_kv_prefill.h -- what tl_kv_attn hands to the kernel for many query rows.
#pragma once

#include "tl_internal.h"
#include "tl_kv.cuh"

namespace tl {

// a / b, in 32 bits where that is enough (a 64-bit division takes about 500 cycles)
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}

// Which of tl_kv_tree_attn's kernels takes the sequences of more rows per kv head than min_rows, all of them: the lengths are
// on the device, so both kernels decide, from the same whole numbers.  In ns, as measured: the kernel for few rows takes
// 8 us and 0.21 us of a CTA for each 32 tokens of 16 rows (and as if each tile had 24 times 32 more); the one for many
// 20 us, 0.95 us for each 64 tokens of a unit of 256 rows and 8 us for the unit, and where units are cut 8 us and 2.2 us for
// each part to join them (all of it with 4 query heads to each of 8 kv heads of 128; heads of 64 go by the same figures,
// though half as much is read and computed for them).  One tree of 26 over 4099 takes 25 us by few and 46 us by many, one
// of 64 over 16000 100 and 71 us, eight of 64 over 500 62 and 25 us, 32 of 12 over 300 29 and 47 us.
constexpr int kFewLead = 24, kManyTiles = 8;
__host__ __device__ __forceinline__ int64_t few_cost(int Hkv, int group, int min_rows, const KvSeq& q) {  // in 32 tokens of 16 rows
  const int64_t rows = int64_t(q.q) * group;
  return rows > min_rows ? (rows + 15) / 16 * Hkv * ((q.len + 31) / 32 + kFewLead) : 0;
}
__host__ __device__ __forceinline__ bool tree_by_many(int ctas, int64_t units, int64_t tiles, int64_t few) {
  if (units == 0) return false;
  const int64_t most = units > tiles / kManyTiles ? units : tiles / kManyTiles, runs = ctas < most ? ctas : most;
  const int64_t join = runs == units ? 0 : 8000 + quotient(2200 * runs, units);
  return quotient(950 * tiles + 8000 * units, ctas) + join + 20000 < quotient(210 * few, ctas) + 8000;
}

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
  int32_t ctas;        // of the launch (set by launch_kv_prefill)
  KvTree tree;         // tl_kv_tree_attn (mask not NULL; causal is 0 then)
  uint32_t page_magic; // groups of 16 tokens to pages: the upper half of a product with it (set by launch_kv_prefill)
};

size_t prefill_partial_bytes(int ctas, int D);
tl_status launch_kv_prefill(PrefillParams& p, int D, int ctas, cudaStream_t st);

}  // namespace tl
