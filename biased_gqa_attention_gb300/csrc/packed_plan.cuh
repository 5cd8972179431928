// packed_plan.cuh -- the work list of a packed prefill: which query tiles there
// are, the dearest first.
#pragma once

#include "common.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace extkv {

// One tile of queries: tokens tok0 .. of the sequence whose first row is
// `row0` and which has `len` tokens; tile_tok of them, or half as many where the
// item is split over its keys (tensor-core kernel for head sizes 64 and 128).
struct PackedItem {
  int row0, len, tok0, split;
};

struct PackedParams {
  void* y;
  const void* q;
  const void* k;
  const void* v;
  const int64_t* cu;
  float c;  // scale * log2(e)
  int causal, window, T, B, Hq, Hkv, g, D;
  int64_t q_stride, k_stride, v_stride;
  int pk;        // query heads of one KV head in a tile (a power of two that divides g)
  int tile_tok;  // tokens of a tile
  int ctas;      // CTAs that share the list where items may be split, or 0
  int heads;     // head groups: Hq / pk
  int max_items;
  int* count;         // items, written by the plan kernel
  PackedItem* items;
  int32_t* status;
  uint32_t wait_limit;
};

// Checked builds: cu_seqlens[b], item `at` of the list.
__device__ __forceinline__ bool cu_in(const PackedParams& p, int64_t b) {
  return EXTKV_IN_KIND(kChkLens, b, 1, static_cast<int64_t>(p.B) + 1, p.status);
}
__device__ __forceinline__ bool item_in(const PackedParams& p, int64_t at) {
  return EXTKV_IN_KIND(kChkItems, at, 1, p.max_items, p.status);
}

// The keys some of `tokens` rows from tok0 on attends, [lo, hi).
__device__ __forceinline__ int2 item_keys(const PackedParams& p, int len, int tok0, int tokens) {
  const int last = min(len, tok0 + tokens);
  return make_int2(p.window > 0 ? max(0, tok0 - p.window + 1) : 0, p.causal ? last : len);
}

constexpr int kPlanThreads = 512;  // the plan kernel's (0.6 us a call better than 1024; 256 and 128 no better)

}  // namespace extkv
