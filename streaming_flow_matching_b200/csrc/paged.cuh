// The paged K/V cache shared by its kernels: page lookup, error recording, and the
// launch interface between the C ABI and the kernels.
//
// One layer's cache: K and V pools [n_pages][page_size][H_kv][D]; sequence s keeps
// slot t (its t-th cached token) in row t % page_size of page table[s][t / page_size].
// Page tables and lengths live on the device, so a captured graph follows them; the
// kernels therefore check every entry they use: an entry outside the pool or a
// length outside the table is recorded in the standalone calls' error word and the
// row is left out, never read or written.
#pragma once

#include "common.cuh"
#include "dependent.cuh"

namespace sfm {

constexpr int kErrPage = 0x301;     // a block-table entry outside [0, n_pages)
constexpr int kErrLength = 0x302;   // a length (or slot) the table or state arrays do not hold

struct PagedCache {
  const int* table;       // [n_seq][max_pages]
  const int* lengths;     // [n_seq]
  int n_seq;
  int n_pages;
  int page_size;
  int max_pages;
  int kv_heads;
  int head_dim;
  int max_tokens;         // slots a sequence can have: max_pages * page_size, cut to the
                          // state arrays' capacity where a call has them
  unsigned magic;         // slot / page_size = slot * magic >> shift
  int shift;
};

// Division of 0 <= n < 2^31 by d: shift = 31 + ceil(log2 d), magic = floor(2^shift / d) + 1.
// magic d - 2^shift <= d <= 2^(shift - 31), so the quotient's excess is below 1 / d.
inline void page_divisor(int d, unsigned* magic, int* shift) {
  int l = 0;
  while ((1LL << l) < d) ++l;
  *shift = 31 + l;
  *magic = (unsigned)(((1ULL << *shift) / (unsigned long long)d) + 1);
}

#ifdef __CUDACC__
__device__ __forceinline__ void record_err(int* err, int code) {
  if (err) atomicCAS(err, 0, code);
}

// The length of sequence s, cut to what the cache can hold (and recorded if it had to be).
__device__ __forceinline__ int cache_len(const PagedCache& c, int s, int* err) {
  int n = c.lengths[s];
  if ((unsigned)n > (unsigned)c.max_tokens) {
    record_err(err, kErrLength);
    n = n < 0 ? 0 : c.max_tokens;
  }
  return n;
}

// Pool row (page * page_size + row in page) of slot t of sequence s, t inside the
// table; -1 (recorded) if its page is not one of the pool's.
__device__ __forceinline__ int cache_row(const PagedCache& c, int s, int t, int* err) {
  const int pg = (int)(((unsigned long long)(unsigned)t * c.magic) >> c.shift);
  const int id = load_late(c.table + (size_t)s * c.max_pages + pg);
  if ((unsigned)id >= (unsigned)c.n_pages) {
    record_err(err, kErrPage);
    return -1;
  }
  return id * c.page_size + (t - pg * c.page_size);
}
#endif

// k, v: [n_rows][H_kv][D]; sequence s owns rows [row_starts[s], row_starts[s + 1])
// (null: row s), which go to slots c.lengths[s] + i.  positions / weights (nullable):
// [n_seq][H_kv][cap].
struct AppendArgs {
  PagedCache c;
  const void* k;
  const void* v;
  void* k_pages;
  void* v_pages;
  const int* row_starts;
  int n_rows;
  int* positions;
  const int* pos0;       // null: c.lengths
  float* weights;
  int cap;
  int* err;
};
int launch_paged_append(const AppendArgs& a, int row_bytes, cudaStream_t s);

struct DecodeArgs {
  PagedCache c;
  const void* q;            // [n_seq][H][D]
  const void* k_pages;
  const void* v_pages;
  void* o;                  // [n_seq][H][D]
  int heads;
  float softcap;            // 0: none
  const float* slopes;      // [H], null: no bias
  const int* positions;     // [n_seq][H_kv][cap], null: position = slot
  const int* q_positions;   // [n_seq], null: length - 1
  float* weights;           // [n_seq][H_kv][cap], null: not accumulated
  int cap;
  int* err;
};
size_t paged_attention_workspace(int n_seq, int max_tokens, int heads, int kv_heads, int head_dim,
                                 int dtype, bool weights);
int launch_paged_attention(const DecodeArgs& a, int dtype, void* workspace, cudaStream_t s);

struct EvictArgs {
  PagedCache c;
  void* k_pages;
  void* v_pages;
  float* weights;       // [n_seq][H_kv][cap]
  int* positions;       // [n_seq][H_kv][cap]
  int cap;
  int keep;
  int n_first;
  int n_recent;
  int* err;
};
size_t paged_evict_workspace(int n_seq, int max_tokens, int kv_heads, int keep);
int launch_paged_evict(const EvictArgs& a, int row_bytes_head, void* workspace, cudaStream_t s);

}  // namespace sfm
