// Writer and eviction of the paged K/V cache.
//
// Append: row i of sequence s goes to slot len_s + i.  A copy: each source row is
// read once and written once (16-byte accesses); the source loads are issued before
// the page lookup, which they do not depend on, so the lookup's chain of small
// loads hides behind them.
//
// Eviction: a sequence of n > keep tokens keeps, for each key head, its `keep` best
// slots by (protected first, accumulated attention weight, lower slot), protected
// being the first n_first positions and the last n_recent.  Attention over a cache
// does not depend on the order of its slots, so nothing is compacted: the kept rows
// that lie at slots >= keep move into the evicted slots < keep, both in ascending
// order, and no other row is touched.  Sources and destinations are disjoint, so
// the moves run in any order.  Two kernels:
//   select  one CTA per (sequence, key head): the keep-th largest rank by radix
//           selection (digits of 11, 11 and 10 bits, a histogram each), then the
//           lists of evicted slots < keep and kept slots >= keep in slot order
//   move    a warp per moved row (K and V rows of one head, weight, position)
#include <limits.h>

#include "paged.cuh"

namespace sfm {

namespace {

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const __grid_constant__ AppendArgs a, int row_vecs, int rows_per_cta) {
  const int r0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.n_rows - r0);
  auto place = [&](int r, int* seq, int* i) -> bool {   // row -> sequence and index in it
    if (!a.row_starts) {
      *seq = r;
      *i = 0;
      return true;
    }
    int lo = 0, hi = a.c.n_seq;      // the last s with row_starts[s] <= r
    if (r < __ldg(a.row_starts) || r >= __ldg(a.row_starts + hi)) return false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.row_starts + mid) <= r) lo = mid;
      else hi = mid;
    }
    *seq = lo;
    *i = r - __ldg(a.row_starts + lo);
    return true;
  };
  auto slot_of = [&](int seq, int i) -> int {           // -1: outside the table (recorded)
    const long long t = (long long)__ldg(a.c.lengths + seq) + i;
    if (t < i || t >= a.c.max_tokens) {
      record_err(a.err, kErrLength);
      return -1;
    }
    return (int)t;
  };
  const uint4* ks = reinterpret_cast<const uint4*>(a.k) + (size_t)r0 * row_vecs;
  const uint4* vs = reinterpret_cast<const uint4*>(a.v) + (size_t)r0 * row_vecs;
  for (int x = threadIdx.x; x < rows * row_vecs; x += kAppendThreads) {
    const uint4 kv = __ldcs(ks + x);
    const uint4 vv = __ldcs(vs + x);
    const int rr = x / row_vecs, c = x - rr * row_vecs;
    int seq, i;
    if (!place(r0 + rr, &seq, &i)) continue;
    const int t = slot_of(seq, i);
    if (t < 0) continue;
    const int row = cache_row(a.c, seq, t, a.err);
    if (row < 0) continue;
    reinterpret_cast<uint4*>(a.k_pages)[(size_t)row * row_vecs + c] = kv;
    reinterpret_cast<uint4*>(a.v_pages)[(size_t)row * row_vecs + c] = vv;
  }
  if (!a.positions && !a.weights) return;
  const int hk = a.c.kv_heads;
  for (int x = threadIdx.x; x < rows * hk; x += kAppendThreads) {
    // consecutive threads take consecutive slots of one head
    const int h = x / rows, rr = x - h * rows;
    int seq, i;
    if (!place(r0 + rr, &seq, &i)) continue;
    const int t = slot_of(seq, i);
    if (t < 0) continue;
    const size_t at = ((size_t)seq * hk + h) * a.cap + t;
    if (a.positions) a.positions[at] = (a.pos0 ? __ldg(a.pos0 + seq) : __ldg(a.c.lengths + seq)) + i;
    if (a.weights) a.weights[at] = 0.f;
  }
}

// ---- eviction ---------------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeldRanks = 48 * 1024;   // ranks in shared memory: 192 KB

// Rank of a token as an unsigned number, larger = kept first: NaN below every number,
// -0 equal to +0, protected tokens above all.
__device__ __forceinline__ unsigned rank_of(float w, int pos, int first, long long recent_from) {
  if (pos < first || pos >= recent_from) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const unsigned b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// lists: per (sequence, key head) `room` evicted slots then `room` moved slots; counts: one each.
// The ranks are made once and kept in shared memory (`held` of them at most; a longer
// sequence makes them again in each of the five passes): 36,000 slots took 90 us when every
// pass read weights and positions from L2.
__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictArgs a, int* __restrict__ counts,
                        int* __restrict__ lists, int room, int held) {
  extern __shared__ unsigned ranks[];
  __shared__ unsigned hist[kBins];
  __shared__ int part[3][kSelWarps];
  __shared__ unsigned sh_digit;
  __shared__ int sh_above;
  const int item = blockIdx.x, seq = item / a.c.kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = cache_len(a.c, seq, a.err), keep = a.keep;
  if (n <= keep) {
    if (tid == 0) counts[item] = 0;
    return;
  }
  const float* w = a.weights + (size_t)item * a.cap;
  const int* pos = a.positions + (size_t)item * a.cap;
  // newest position
  int mx = INT_MIN;
#pragma unroll 8
  for (int t = tid; t < n; t += kSelThreads) mx = max(mx, __ldg(pos + t));
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) part[0][warp] = mx;
  __syncthreads();
  mx = __reduce_max_sync(0xffffffffu, part[0][lane]);
  __syncthreads();
  const long long recent_from = (long long)mx - a.n_recent + 1;
  const bool hold = n <= held;
  auto make_rank = [&](int t) { return rank_of(__ldg(w + t), __ldg(pos + t), a.n_first, recent_from); };
  if (hold) {
#pragma unroll 8
    for (int t = tid; t < n; t += kSelThreads) ranks[t] = make_rank(t);
  }
  auto rank = [&](int t) { return hold ? ranks[t] : make_rank(t); };
  // the keep-th largest rank, digit by digit: `want` of the ranks that match the
  // prefix found so far are still to be taken
  unsigned prefix = 0, mask = 0;
  int want = keep;
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const unsigned bins = d == 2 ? 1024u : 2048u;
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
#pragma unroll 4
    for (int t = tid; t < n; t += kSelThreads) {
      const unsigned r = rank(t);
      if ((r & mask) == prefix) atomicAdd(&hist[(r >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // bins from the top: thread i holds bins (2047 - 2 i), (2046 - 2 i)
    const int c0 = (int)hist[kBins - 1 - 2 * tid], c1 = (int)hist[kBins - 2 - 2 * tid];
    int inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) part[0][warp] = inc;
    __syncthreads();
    int before = 0;
    for (int k = 0; k < warp; ++k) before += part[0][k];
    const int exc = before + inc - c0 - c1;
    if (exc < want && want <= exc + c0) {
      sh_digit = kBins - 1 - 2 * tid;
      sh_above = exc;
    } else if (exc + c0 < want && want <= exc + c0 + c1) {
      sh_digit = kBins - 2 - 2 * tid;
      sh_above = exc + c0;
    }
    __syncthreads();
    prefix |= sh_digit << shift;
    mask |= (bins - 1) << shift;
    want -= sh_above;
    __syncthreads();
  }
  // ranks above `prefix` stay, and of those equal to it the first `want` by slot.
  // Each warp walks a contiguous run of slots: its number of ties first, then the lists.
  const int per = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int t0 = min(n, warp * per), t1 = min(n, t0 + per);
  int ties = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 32) ties += rank(t) == prefix;
  ties = warp_sum(ties);
  if (lane == 0) part[0][warp] = ties;
  __syncthreads();
  int tie_base = 0;
  for (int k = 0; k < warp; ++k) tie_base += part[0][k];
  int n_out = 0, n_mv = 0, out_base = 0, mv_base = 0;
  int* outs = lists + (size_t)item * 2 * room;
  int* mvs = outs + room;
  for (int pass = 0; pass < 2; ++pass) {
    int tie = tie_base, no = out_base, nm = mv_base;
    for (int t = t0; t < t1; t += 32) {
      const int x = t + lane;
      const unsigned r = x < t1 ? rank(x) : 0u;
      const bool eq = x < t1 && r == prefix;
      const unsigned eqs = __ballot_sync(0xffffffffu, eq);
      const unsigned lower = (1u << lane) - 1u;
      const bool stay = x < t1 && (r > prefix || (eq && tie + __popc(eqs & lower) < want));
      const unsigned out_m = __ballot_sync(0xffffffffu, x < t1 && x < keep && !stay);
      const unsigned mv_m = __ballot_sync(0xffffffffu, x >= keep && stay);
      if (pass) {
        if ((out_m >> lane) & 1u) outs[no + __popc(out_m & lower)] = x;
        if ((mv_m >> lane) & 1u) mvs[nm + __popc(mv_m & lower)] = x;
      }
      tie += __popc(eqs);
      no += __popc(out_m);
      nm += __popc(mv_m);
    }
    if (pass == 0) {
      n_out = no;
      n_mv = nm;
      if (lane == 0) {
        part[1][warp] = n_out;
        part[2][warp] = n_mv;
      }
      __syncthreads();
      for (int k = 0; k < warp; ++k) {
        out_base += part[1][k];
        mv_base += part[2][k];
      }
    } else if (tid == kSelThreads - 1) {
      counts[item] = nm;               // = no: both are keep minus the kept slots < keep
    }
  }
}

// A warp moves kMoveRows rows at a time: their slots and pages are looked up by as many
// lanes at once, then the 16-byte pieces of all of them (head_vecs of K and of V each) are
// loaded four to a lane before the first is stored.
constexpr int kMoveWarps = 8, kMoveRows = 8;

__global__ void __launch_bounds__(kMoveWarps * 32)
    evict_move_kernel(const __grid_constant__ EvictArgs a, const int* __restrict__ counts,
                      const int* __restrict__ lists, int room, int head_vecs, int blocks_per_item) {
  grid_dependency_wait();
  const int item = blockIdx.x / blocks_per_item, blk = blockIdx.x - item * blocks_per_item;
  const int seq = item / a.c.kv_heads, h = item - seq * a.c.kv_heads;
  const int lane = threadIdx.x & 31;
  const int n = counts[item];
  const int* outs = lists + (size_t)item * 2 * room;
  const int* mvs = outs + room;
  const int pieces = 2 * head_vecs;                            // of a row; kMoveRows * pieces is a multiple of 128
  uint4* kp = reinterpret_cast<uint4*>(a.k_pages);
  uint4* vp = reinterpret_cast<uint4*>(a.v_pages);
  for (int i0 = (blk * kMoveWarps + (threadIdx.x >> 5)) * kMoveRows; i0 < n;
       i0 += blocks_per_item * kMoveWarps * kMoveRows) {
    int rt = -1, rf = -1;
    if (lane < kMoveRows && i0 + lane < n) {
      const int to = outs[i0 + lane], from = mvs[i0 + lane];
      rt = cache_row(a.c, seq, to, a.err);
      rf = cache_row(a.c, seq, from, a.err);
      const size_t at = (size_t)item * a.cap;
      a.weights[at + to] = a.weights[at + from];
      a.positions[at + to] = a.positions[at + from];
    }
    for (int x0 = lane; x0 < kMoveRows * pieces; x0 += 128) {
      uint4 d[4];
      uint4* to[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int x = x0 + 32 * u, r = x / pieces, c = x - r * pieces;
        const int from_row = __shfl_sync(0xffffffffu, rf, r), to_row = __shfl_sync(0xffffffffu, rt, r);
        uint4* pool = c < head_vecs ? kp : vp;
        const int cc = c < head_vecs ? c : c - head_vecs;
        to[u] = nullptr;
        if (from_row >= 0 && to_row >= 0) {
          d[u] = pool[((size_t)from_row * a.c.kv_heads + h) * head_vecs + cc];
          to[u] = pool + ((size_t)to_row * a.c.kv_heads + h) * head_vecs + cc;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (to[u]) *to[u] = d[u];
    }
  }
}

}  // namespace

int launch_paged_append(const AppendArgs& a, int row_bytes, cudaStream_t s) {
  if (a.n_rows == 0) return SFM_OK;
  const int row_vecs = row_bytes / 16;
  // about two 16-byte pieces of K and of V per thread, whole rows per CTA
  int rows = 2 * kAppendThreads / row_vecs;
  rows = rows < 1 ? 1 : rows > 16 ? 16 : rows;
  ProfScope ps(SFM_PROF_APPEND, s);
  paged_append_kernel<<<(unsigned)((a.n_rows + rows - 1) / rows), kAppendThreads, 0, s>>>(a, row_vecs, rows);
  return record_cuda(cudaGetLastError());
}

// Rows moved per (sequence, key head): at most the slots past `keep`, and at most `keep`.
static int evict_room(int max_tokens, int keep) {
  const int past = max_tokens - keep;
  return past <= 0 ? 0 : past < keep ? past : keep;
}

size_t paged_evict_workspace(int n_seq, int max_tokens, int kv_heads, int keep) {
  const size_t items = (size_t)n_seq * kv_heads;
  const size_t b = (items + items * 2 * evict_room(max_tokens, keep)) * sizeof(int);
  return (b + 15) / 16 * 16;
}

int launch_paged_evict(const EvictArgs& a, int row_bytes_head, void* workspace, cudaStream_t s) {
  const int room = evict_room(a.c.max_tokens, a.keep);
  if (room == 0) return SFM_OK;      // no sequence can be longer than keep
  const int items = a.c.n_seq * a.c.kv_heads;
  int* counts = (int*)workspace;
  int* lists = counts + items;
  ProfScope ps(SFM_PROF_APPEND, s);
  const int held = a.c.max_tokens < kHeldRanks ? a.c.max_tokens : kHeldRanks;
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kHeldRanks * (int)sizeof(unsigned));
  if (e != cudaSuccess) return record_cuda(e);
  evict_select_kernel<<<(unsigned)items, kSelThreads, held * sizeof(unsigned), s>>>(a, counts, lists, room, held);
  int rc = record_cuda(cudaGetLastError());
  if (rc) return rc;
  // kMoveRows rows per warp, and no more CTAs than fill the device several times over
  int blocks = (room + kMoveRows * kMoveWarps - 1) / (kMoveRows * kMoveWarps);
  const int most = (148 * 32 + items - 1) / items;
  if (blocks > most) blocks = most;
  return record_cuda(launch_dependent(evict_move_kernel, (unsigned)(items * blocks), kMoveWarps * 32, 0, s, a,
                                      (const int*)counts, (const int*)lists, room, row_bytes_head / 16, blocks));
}

}  // namespace sfm
