// Launch interface of the attention under per-query key ranges (attn_masked.cu).
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace sfm {

// Query i (at position n_kv - n_q + i of the keys) attends to keys
// [max(key_lo[i], 0), min(key_hi[i], n_kv)); null arrays: 0 and n_kv.
struct MaskedArgs {
  const void* q;          // [n_q][H][D]
  const void* k;          // [n_kv][H_kv][D]
  const void* v;
  void* o;                // [n_q][H][D]
  int n_q, n_kv, heads, kv_heads, head_dim;
  const int* key_lo;
  const int* key_hi;
  float softcap;          // 0: none
  const float* slopes;    // [H], null: no bias
};

// Key splits of a call (a function of the shape alone) and the scratch they need.
int masked_splits(int n_q, int n_kv, int heads, int kv_heads, int head_dim, int dtype);
size_t masked_workspace(int n_q, int n_kv, int heads, int kv_heads, int head_dim, int dtype);
int launch_attention_masked_tc(const MaskedArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                               const CUtensorMap& mv, void* workspace, const Guard& gd, cudaStream_t s);
int launch_attention_masked_f32(const MaskedArgs& a, void* workspace, cudaStream_t s);

struct BoundsArgs {
  int n_q, n_kv;
  const int* doc_starts;   // [n_docs + 1] ascending, null: one document of all keys
  const int* prefixes;     // [n_docs], null: 0
  int n_docs;
  int causal;
  int* key_lo;
  int* key_hi;
};
int launch_attention_bounds(const BoundsArgs& a, cudaStream_t s);

}  // namespace sfm
