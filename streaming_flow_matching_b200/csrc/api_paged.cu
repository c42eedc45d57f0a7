// C ABI of the paged K/V cache and of attention under per-query key ranges: argument
// validation and the launches.  Every error the host can see is returned before any
// launch; what only the device holds (page tables, lengths) is checked by the kernels,
// which record it in the standalone calls' error word and leave the row out.
#include <limits.h>
#include <math.h>

#include "attn_masked.cuh"
#include "paged.cuh"
#include "sm100.cuh"

using namespace sfm;

namespace {

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1u)) == 0; }

int check_heads(int heads, int kv_heads, int head_dim, int dtype) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads) return SFM_EINVAL;
  if (dtype != SFM_DTYPE_BF16 && dtype != SFM_DTYPE_FP32) return SFM_EINVAL;
  if (dtype == SFM_DTYPE_BF16 && head_dim != 128) return SFM_EUNSUPPORTED;
  if (dtype == SFM_DTYPE_FP32 && (head_dim % 32 || head_dim < 32 || head_dim > 128)) return SFM_EUNSUPPORTED;
  return SFM_OK;
}

int elem_bytes(int dtype) { return dtype == SFM_DTYPE_BF16 ? 2 : 4; }

// cap < 0: the call has no state arrays
int fill_cache(PagedCache* c, const void* k_pages, const void* v_pages, const int* table, const int* lengths,
               int n_seq, int n_pages, int page_size, int max_pages, int kv_heads, int head_dim, int cap) {
  if (!k_pages || !v_pages || !table || !lengths) return SFM_EINVAL;
  if (n_seq < 1 || n_pages < 1 || page_size < 1 || max_pages < 1) return SFM_EINVAL;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(table, 4) || !aligned(lengths, 4))
    return SFM_EINVAL;
  // rows and slots are 32-bit numbers in the kernels, byte offsets 64-bit ones
  if ((long long)n_pages * page_size > INT_MAX || (long long)max_pages * page_size > INT_MAX / 2)
    return SFM_EUNSUPPORTED;
  if ((long long)n_seq * ((long long)max_pages * page_size + 64) / 64 > INT_MAX / 2)
    return SFM_EUNSUPPORTED;
  c->table = table;
  c->lengths = lengths;
  c->n_seq = n_seq;
  c->n_pages = n_pages;
  c->page_size = page_size;
  c->max_pages = max_pages;
  c->kv_heads = kv_heads;
  c->head_dim = head_dim;
  c->max_tokens = max_pages * page_size;
  if (cap >= 0 && cap < c->max_tokens) c->max_tokens = cap;
  page_divisor(page_size, &c->magic, &c->shift);
  return SFM_OK;
}

// 0 (none), or a cap whose powers and multiples the kernels' fp32 constants hold
bool cap_ok(float c) { return c == 0.f || (c >= 1e-3f && c <= 1e30f); }

// grids are one-dimensional: every launch's block count has to fit
bool fits_grid(long long blocks) { return blocks >= 1 && blocks <= INT_MAX; }

}  // namespace

extern "C" {

int sfm_paged_append(const void* k, const void* v, void* k_pages, void* v_pages, const int* table,
                     const int* lengths, const int* row_starts, int n_rows, int n_seq, int n_pages, int page_size,
                     int max_pages, int n_kv_heads, int head_dim, int dtype, int* positions, const int* pos0,
                     float* weights, int cap, void* stream) {
  int rc = check_heads(n_kv_heads, n_kv_heads, head_dim, dtype);
  if (rc) return rc;
  if (n_rows < 0 || (n_rows > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16)))) return SFM_EINVAL;
  const bool state = positions || weights;
  if ((state && cap < 1) || (pos0 && !positions) || (!row_starts && n_rows != n_seq)) return SFM_EINVAL;
  if (!aligned(row_starts, 4) || !aligned(positions, 4) || !aligned(pos0, 4) || !aligned(weights, 4))
    return SFM_EINVAL;
  AppendArgs a{};
  rc = fill_cache(&a.c, k_pages, v_pages, table, lengths, n_seq, n_pages, page_size, max_pages, n_kv_heads,
                  head_dim, state ? cap : -1);
  if (rc) return rc;
  const long long row_bytes = (long long)n_kv_heads * head_dim * elem_bytes(dtype);
  if (row_bytes > (1 << 24) || n_rows > INT_MAX - 256) return SFM_EUNSUPPORTED;
  if (k_pages == v_pages) return SFM_EINVAL;        // K and V of a row would go to the same place
  Guard gd;
  if ((rc = call_guard(&gd))) return rc;
  a.k = k;
  a.v = v;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.row_starts = row_starts;
  a.n_rows = n_rows;
  a.positions = positions;
  a.pos0 = pos0;
  a.weights = weights;
  a.cap = cap;
  a.err = gd.err;
  return launch_paged_append(a, (int)row_bytes, (cudaStream_t)stream);
}

size_t sfm_paged_attention_workspace_bytes(int n_seq, int max_tokens, int n_heads, int n_kv_heads, int head_dim,
                                           int dtype, int with_weights) {
  if (n_seq < 1 || max_tokens < 1 || check_heads(n_heads, n_kv_heads, head_dim, dtype)) return 0;
  if (!fits_grid((long long)n_seq * n_heads)) return 0;
  return paged_attention_workspace(n_seq, max_tokens, n_heads, n_kv_heads, head_dim, dtype, with_weights != 0);
}

int sfm_paged_attention(const void* q, const void* k_pages, const void* v_pages, const int* table,
                        const int* lengths, void* o, int n_seq, int n_pages, int page_size, int max_pages,
                        int n_heads, int n_kv_heads, int head_dim, int dtype, float softcap, const float* slopes,
                        const int* positions, const int* q_positions, float* weights, int cap, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check_heads(n_heads, n_kv_heads, head_dim, dtype);
  if (rc) return rc;
  if (!q || !o || o == q || !aligned(q, 16) || !aligned(o, 16)) return SFM_EINVAL;
  if (!cap_ok(softcap)) return SFM_EINVAL;
  const bool state = positions || weights;
  if ((state && cap < 1) || ((positions != nullptr) != (q_positions != nullptr))) return SFM_EINVAL;
  if (!aligned(slopes, 4) || !aligned(positions, 4) || !aligned(q_positions, 4) || !aligned(weights, 4))
    return SFM_EINVAL;
  DecodeArgs a{};
  rc = fill_cache(&a.c, k_pages, v_pages, table, lengths, n_seq, n_pages, page_size, max_pages, n_kv_heads,
                  head_dim, state ? cap : -1);
  if (rc) return rc;
  if (!fits_grid((long long)n_seq * n_heads) || !fits_grid((long long)n_seq * n_kv_heads) ||
      !fits_grid((long long)n_seq * n_heads + (long long)n_seq * n_kv_heads * (a.c.max_tokens / 1024 + 1)))
    return SFM_EUNSUPPORTED;
  const size_t need =
      paged_attention_workspace(n_seq, a.c.max_tokens, n_heads, n_kv_heads, head_dim, dtype, weights != nullptr);
  if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 16)))) return SFM_EINVAL;
  Guard gd;
  if ((rc = call_guard(&gd))) return rc;
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.o = o;
  a.heads = n_heads;
  a.softcap = softcap;
  a.slopes = slopes;
  a.positions = slopes ? positions : nullptr;      // only the bias looks at them
  a.q_positions = slopes ? q_positions : nullptr;
  a.weights = weights;
  a.cap = cap;
  a.err = gd.err;
  return launch_paged_attention(a, dtype, workspace, (cudaStream_t)stream);
}

size_t sfm_paged_evict_workspace_bytes(int n_seq, int max_tokens, int n_kv_heads, int keep) {
  if (n_seq < 1 || max_tokens < 1 || n_kv_heads < 1 || keep < 1) return 0;
  return paged_evict_workspace(n_seq, max_tokens, n_kv_heads, keep);
}

int sfm_paged_evict(void* k_pages, void* v_pages, const int* table, const int* lengths, float* weights,
                    int* positions, int cap, int n_seq, int n_pages, int page_size, int max_pages, int n_kv_heads,
                    int head_dim, int dtype, int keep, int n_first, int n_recent, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc = check_heads(n_kv_heads, n_kv_heads, head_dim, dtype);
  if (rc) return rc;
  if (!weights || !positions || cap < 1 || keep < 1 || n_first < 0 || n_recent < 0 ||
      (long long)n_first + n_recent > keep || !aligned(weights, 4) || !aligned(positions, 4))
    return SFM_EINVAL;
  EvictArgs a{};
  rc = fill_cache(&a.c, k_pages, v_pages, table, lengths, n_seq, n_pages, page_size, max_pages, n_kv_heads,
                  head_dim, cap);
  if (rc) return rc;
  if (!fits_grid((long long)n_seq * n_kv_heads * 4096)) return SFM_EUNSUPPORTED;
  const size_t need = paged_evict_workspace(n_seq, a.c.max_tokens, n_kv_heads, keep);
  if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 16)))) return SFM_EINVAL;
  Guard gd;
  if ((rc = call_guard(&gd))) return rc;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.weights = weights;
  a.positions = positions;
  a.cap = cap;
  a.keep = keep;
  a.n_first = n_first;
  a.n_recent = n_recent;
  a.err = gd.err;
  return launch_paged_evict(a, head_dim * elem_bytes(dtype), workspace, (cudaStream_t)stream);
}

int sfm_attention_bounds(int n_q, int n_kv, const int* doc_starts, const int* prefixes, int n_docs, int causal,
                         int* key_lo, int* key_hi, void* stream) {
  if (n_q < 1 || n_kv < n_q || !key_lo || !key_hi || (causal != 0 && causal != 1)) return SFM_EINVAL;
  if (n_kv > INT_MAX - 256) return SFM_EUNSUPPORTED;
  if (n_docs < 0 || (doc_starts && n_docs < 1) || (!doc_starts && n_docs != (prefixes ? 1 : 0))) return SFM_EINVAL;
  if (!aligned(doc_starts, 4) || !aligned(prefixes, 4) || !aligned(key_lo, 4) || !aligned(key_hi, 4))
    return SFM_EINVAL;
  if (key_lo == key_hi) return SFM_EINVAL;
  BoundsArgs a{n_q, n_kv, doc_starts, prefixes, n_docs, causal, key_lo, key_hi};
  return launch_attention_bounds(a, (cudaStream_t)stream);
}

size_t sfm_attention_masked_workspace_bytes(int n_q, int n_kv, int n_heads, int n_kv_heads, int head_dim,
                                            int dtype) {
  if (n_q < 1 || n_kv < 1 || check_heads(n_heads, n_kv_heads, head_dim, dtype)) return 0;
  if (n_q > INT_MAX - 256 || n_kv > INT_MAX - 256) return 0;
  return masked_workspace(n_q, n_kv, n_heads, n_kv_heads, head_dim, dtype);
}

int sfm_attention_masked(const void* q, const void* k, const void* v, void* o, int n_q, int n_kv, int n_heads,
                         int n_kv_heads, int head_dim, int dtype, const int* key_lo, const int* key_hi,
                         float softcap, const float* slopes, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int rc = check_heads(n_heads, n_kv_heads, head_dim, dtype);
  if (rc) return rc;
  if (!q || !k || !v || !o || o == q || o == k || o == v || n_q < 1 || n_kv < 1) return SFM_EINVAL;
  if (slopes && n_kv < n_q) return SFM_EINVAL;      // the bias needs the queries' positions among the keys
  if (!cap_ok(softcap)) return SFM_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(key_lo, 4) ||
      !aligned(key_hi, 4) || !aligned(slopes, 4))
    return SFM_EINVAL;
  if (n_q > INT_MAX - 256 || n_kv > INT_MAX - 256 || !fits_grid((long long)n_q * n_heads) ||
      !fits_grid(((long long)n_q / 32 + 1) * n_heads * 32)) return SFM_EUNSUPPORTED;
  const size_t need = masked_workspace(n_q, n_kv, n_heads, n_kv_heads, head_dim, dtype);
  if (workspace_bytes < need || (need && (!workspace || !aligned(workspace, 16)))) return SFM_EINVAL;
  MaskedArgs a{q, k, v, o, n_q, n_kv, n_heads, n_kv_heads, head_dim, key_lo, key_hi, softcap, slopes};
  if (dtype == SFM_DTYPE_FP32) return launch_attention_masked_f32(a, workspace, (cudaStream_t)stream);
  CUtensorMap mq, mk, mv;
  rc = make_rows_map(&mq, q, n_q, n_heads, 128);
  if (!rc) rc = make_rows_map(&mk, k, n_kv, n_kv_heads, 128);
  if (!rc) rc = make_rows_map(&mv, v, n_kv, n_kv_heads, 128);
  Guard gd;
  if (!rc) rc = call_guard(&gd);
  if (rc) return rc;
  return launch_attention_masked_tc(a, mq, mk, mv, workspace, gd, (cudaStream_t)stream);
}

}  // extern "C"
