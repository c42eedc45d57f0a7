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
// the moves run in any order.  Two kernels (one where few rows can move: select moves them):
//   select  one CTA, or a cluster of 2 to 8, per (sequence, key head): the keep-th
//           largest rank by radix selection (digits of 11, 11 and 10 bits, a histogram
//           each), then the lists of evicted slots < keep and kept slots >= keep in slot
//           order.  The CTAs of a cluster take a run of slots each and read one another's
//           histograms and counts.
//   move    a warp per 8 moved rows (K and V rows of one head, weight, position)
//
// Measured (bf16): append of 8 x ~1,150 rows of 24 heads 38.7 us, 5.9 TB/s (0.89 of a copy's
// rate).  Eviction of 16 sequences x 8 heads from 30,500-36,000 to 30,000 slots 110 us: select 31 us,
// bound by its instructions (62 % issue); moves 70 us, bound by memory at 256 bytes a piece;
// of 4 x 1,200 to 924: 14 us, latency.  (Select alone with few moves, one sequence of 57,600:
// 24 heads 31 us.)
#include <limits.h>

#include "paged.cuh"
#include "sm100.cuh"

namespace sfm {

namespace {

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const __grid_constant__ AppendArgs a, int row_vecs, int rows_per_cta) {
  grid_dependency_wait();
  const int r0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.n_rows - r0);
  auto place = [&](int r, int* seq, int* i) -> bool {   // row -> sequence and index in it
    if (!a.row_starts) {
      *seq = r;
      *i = 0;
      return true;
    }
    int lo = 0, hi = a.c.n_seq;      // the last s with row_starts[s] <= r
    if (r < load_late(a.row_starts) || r >= load_late(a.row_starts + hi)) return false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (load_late(a.row_starts + mid) <= r) lo = mid;
      else hi = mid;
    }
    *seq = lo;
    *i = r - load_late(a.row_starts + lo);
    return true;
  };
  auto slot_of = [&](int seq, int i) -> int {           // -1: outside the table (recorded)
    const long long t = (long long)load_late(a.c.lengths + seq) + i;
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
    if (t < 0 || cache_row(a.c, seq, t, nullptr) < 0) continue;    // the row was dropped (and recorded) above
    const size_t at = ((size_t)seq * hk + h) * a.cap + t;
    if (a.positions) a.positions[at] = (a.pos0 ? load_late(a.pos0 + seq) : load_late(a.c.lengths + seq)) + i;
    if (a.weights) a.weights[at] = 0.f;
  }
}

// ---- eviction ---------------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBatch = 8;       // loads in flight per thread
constexpr int kHeldRanks = 48 * 1024;   // ranks in shared memory: 192 KB
constexpr int kSms = 148;

// Rank of a token as an unsigned number, larger = kept first: NaN below every number,
// -0 equal to +0, protected tokens above all.
__device__ __forceinline__ unsigned rank_of(float w, int pos, int first, bool recent, int recent_from) {
  if (pos < first || (recent && pos >= recent_from)) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const unsigned b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp moves kMoveRows rows at a time: their slots and pages are looked up by as many
// lanes at once, then the 16-byte pieces of all of them (head_vecs of K and of V each) are
// loaded four to a lane before the first is stored.
constexpr int kMoveWarps = 8, kMoveRows = 8;

// Warp `warp` of `warps` moves its share of an item's n rows.
__device__ __forceinline__ void move_rows(const EvictArgs& a, int item, const int* outs, const int* mvs, int n,
                                          int warp, int warps, int head_vecs) {
  const int seq = item / a.c.kv_heads, h = item - seq * a.c.kv_heads;
  const int lane = threadIdx.x & 31;
  const int pieces = 2 * head_vecs;                            // of a row; kMoveRows * pieces is a multiple of 128
  uint4* kp = reinterpret_cast<uint4*>(a.k_pages);
  uint4* vp = reinterpret_cast<uint4*>(a.v_pages);
  for (int i0 = warp * kMoveRows; i0 < n; i0 += warps * kMoveRows) {
    int rt = -1, rf = -1;
    if (lane < kMoveRows && i0 + lane < n) {
      const int to = outs[i0 + lane], from = mvs[i0 + lane];
      const size_t at = (size_t)item * a.cap;
      const float w = a.weights[at + from];
      const int pos = a.positions[at + from];
      rt = cache_row(a.c, seq, to, a.err);
      rf = cache_row(a.c, seq, from, a.err);
      if (rt >= 0 && rf >= 0) {                                // with a bad page on either side nothing moves
        a.weights[at + to] = w;
        a.positions[at + to] = pos;
      }
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

// slots of each CTA of a cluster, whole warps of them
__host__ __device__ inline int select_run(int n, int parts) { return ((n + parts - 1) / parts + 31) & ~31; }

struct __align__(8) SelectShared {
  unsigned hist[3][kBins];      // one for each digit: none is cleared while another CTA reads it
  int part[3][kSelWarps];
  int total[4];                 // of this CTA: newest position, ties, evicted, moved
  unsigned digit;
  int above;
};

// All threads of the cluster (or of the CTA that is alone); what they wrote to shared memory is seen.
__device__ __forceinline__ void cluster_barrier(int parts) {
  __syncwarp();                                                // (after loops of unequal length)
  if (parts == 1) __syncthreads();
  else sm100::cluster_sync();
}
// A word of shared memory at the place of `p` in CTA `rank` of the cluster.
__device__ __forceinline__ unsigned peer_word(const void* p, int rank) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(sm100::mapa_shared(sm100::smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 peer_words(const void* p, int rank) {          // 8 bytes
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(sm100::mapa_shared(sm100::smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}

// Ranks and lists.  lists: per (sequence, key head) `room` evicted slots then `room` moved slots;
// counts: one each.  The ranks are made once and kept in shared memory (`held` of them at most; a
// longer run of slots makes them again in each of its passes).  Bound by instructions: a CTA passes
// over its slots five times, so those passes over shared memory are kept short.
template <bool HOLD>
__device__ __forceinline__ void evict_select(const EvictArgs& a, int* counts, int* lists,
                                             int room, int item, int part_id, int parts, int from, int n,
                                             int fused_vecs, SelectShared& sh) {
  extern __shared__ unsigned ranks[];
  auto& part = sh.part;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this CTA's slots: from, ... from + n - 1 (none, at the end of a short sequence)
  const int keep = a.keep - from;
  const float* w = a.weights + (size_t)item * a.cap + from;
  const int* pos = a.positions + (size_t)item * a.cap + from;
  for (int b = tid; b < 3 * kBins; b += kSelThreads) sh.hist[0][b] = 0;
  // newest position
  int mx = INT_MIN;
  for (int t0 = tid; t0 < n; t0 += kBatch * kSelThreads) {
    int p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) p[u] = t0 + u * kSelThreads < n ? load_late(pos + t0 + u * kSelThreads) : INT_MIN;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) mx = max(mx, p[u]);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) part[0][warp] = mx;
  __syncthreads();
  mx = __reduce_max_sync(0xffffffffu, part[0][lane]);
  if (parts > 1) {
    if (tid == 0) sh.total[0] = mx;
    cluster_barrier(parts);
    mx = __reduce_max_sync(0xffffffffu, lane < parts ? (int)peer_word(&sh.total[0], lane) : INT_MIN);
  }
  const int recent_from = (int)max((long long)INT_MIN, (long long)mx - a.n_recent + 1);   // (n_recent > 0)
  auto make_rank = [&](int t) { return rank_of(load_late(w + t), load_late(pos + t), a.n_first, a.n_recent > 0, recent_from); };
  auto rank = [&](int t) { return HOLD ? ranks[t] : make_rank(t); };
  // the keep-th largest rank, digit by digit: `want` of the ranks that match the
  // prefix found so far are still to be taken.  The first digit is counted as the
  // ranks are made.
  unsigned prefix = 0, mask = 0;
  int want = a.keep;
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const unsigned bins = d == 2 ? 1024u : 2048u;
    unsigned* hist = sh.hist[d];
    if (d == 0) {
      for (int t0 = tid; t0 < n; t0 += kBatch * kSelThreads) {
        float wv[kBatch];
        int pv[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = min(t0 + u * kSelThreads, n - 1);      // (a slot past the end: not used below)
          wv[u] = load_late(w + t);
          pv[u] = load_late(pos + t);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int t = t0 + u * kSelThreads;
          const unsigned r = rank_of(wv[u], pv[u], a.n_first, a.n_recent > 0, recent_from);
          if (HOLD && t < n) ranks[t] = r;
          if (t < n) atomicAdd(&hist[r >> 21], 1u);
        }
      }
    } else {
#pragma unroll 8
      for (int t = tid; t < n; t += kSelThreads) {
        const unsigned r = rank(t);
        if ((r & mask) == prefix) atomicAdd(&hist[(r >> shift) & (bins - 1)], 1u);
      }
    }
    cluster_barrier(parts);
    // bins from the top: thread i holds bins (2047 - 2 i), (2046 - 2 i)
    const int b0 = kBins - 2 - 2 * tid;
    int c0 = 0, c1 = 0;
    if (parts == 1) {
      c0 = (int)hist[b0 + 1];
      c1 = (int)hist[b0];
    } else {
#pragma unroll 8
      for (int r = 0; r < parts; ++r) {
        const uint2 c = peer_words(&hist[b0], r);
        c0 += (int)c.y;
        c1 += (int)c.x;
      }
    }
    int inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) part[0][warp] = inc;
    __syncthreads();
    const int before = warp_sum(lane < warp ? part[0][lane] : 0);
    const int exc = before + inc - c0 - c1;
    if (exc < want && want <= exc + c0) {
      sh.digit = b0 + 1;
      sh.above = exc;
    } else if (exc + c0 < want && want <= exc + c0 + c1) {
      sh.digit = b0;
      sh.above = exc + c0;
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= (bins - 1) << shift;
    want -= sh.above;
    __syncthreads();
  }
  // Ranks above `prefix` stay, and of those equal to it the first `want` by slot.  Each warp
  // walks a contiguous run of slots, first counting: what it will list follows from the
  // ties before it.
  const int per = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int t0 = min(n, warp * per), t1 = min(n, t0 + per);
  const int mid = min(max(keep, t0), t1);                      // the run's slots < keep end here
  int tie_lo = 0, tie_hi = 0, n_out = 0, n_mv = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < mid; t += 32) {
    const unsigned r = rank(t);
    tie_lo += r == prefix;
    n_out += r < prefix;
  }
#pragma unroll 4
  for (int t = mid + lane; t < t1; t += 32) {
    const unsigned r = rank(t);
    tie_hi += r == prefix;
    n_mv += r > prefix;
  }
  tie_lo = warp_sum(tie_lo);
  tie_hi = warp_sum(tie_hi);
  n_out = warp_sum(n_out);
  n_mv = warp_sum(n_mv);
  if (lane == 0) part[0][warp] = tie_lo + tie_hi;
  __syncthreads();
  int tie_base = warp_sum(lane < warp ? part[0][lane] : 0);
  if (parts > 1) {                                             // and the CTAs before
    const int all = warp_sum(part[0][lane]);
    if (tid == 0) sh.total[1] = all;
    cluster_barrier(parts);
    tie_base += warp_sum(lane < part_id ? (int)peer_word(&sh.total[1], lane) : 0);
  }
  const int left = max(0, want - tie_base);                    // ties of this run that stay
  n_out += max(0, tie_lo - left);
  n_mv += min(tie_hi, max(0, left - tie_lo));
  if (lane == 0) {
    part[1][warp] = n_out;
    part[2][warp] = n_mv;
  }
  __syncthreads();
  int no = warp_sum(lane < warp ? part[1][lane] : 0), nm = warp_sum(lane < warp ? part[2][lane] : 0);
  if (parts > 1) {
    const int all_o = warp_sum(part[1][lane]), all_m = warp_sum(part[2][lane]);
    if (tid == 0) {
      sh.total[2] = all_o;
      sh.total[3] = all_m;
    }
    cluster_barrier(parts);
    no += warp_sum(lane < part_id ? (int)peer_word(&sh.total[2], lane) : 0);
    nm += warp_sum(lane < part_id ? (int)peer_word(&sh.total[3], lane) : 0);
  }
  int* outs = fused_vecs ? reinterpret_cast<int*>(sh.hist) : lists + (size_t)item * 2 * room;
  int* mvs = outs + room;
  const unsigned lower = (1u << lane) - 1u;
  int tie = tie_base;
  auto walk = [&](int begin, int to, bool behind, int* list, int at) {
    for (int t = begin; t < to; t += 32 * kBatch) {
      unsigned rv[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int x = t + 32 * u + lane;
        rv[u] = x < to ? rank(x) : 0u;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int x = t + 32 * u + lane;
        bool stay = rv[u] > prefix;
        if (tie_lo + tie_hi > 0) {                             // warp-uniform: most runs have none
          const bool eq = x < to && rv[u] == prefix;
          const unsigned eqs = __ballot_sync(0xffffffffu, eq);
          stay = stay || (eq && tie + __popc(eqs & lower) < want);
          tie += __popc(eqs);
        }
        const bool take = x < to && stay == behind;
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (take) list[at + __popc(m & lower)] = from + x;
        at += __popc(m);
      }
    }
    return at;
  };
  walk(t0, mid, false, outs, no);
  nm = walk(mid, t1, true, mvs, nm);
  if (fused_vecs) {                                            // a CTA that is alone, and few rows
    __syncthreads();
    move_rows(a, item, outs, mvs, warp_sum(part[2][lane]), warp, kSelWarps, fused_vecs);
    return;
  }
  // as many slots were evicted before `keep` as are kept behind it
  if (part_id == parts - 1 && warp == kSelWarps - 1 && lane == 0) counts[item] = nm;
  if (parts > 1) cluster_barrier(parts);                       // nobody leaves while its words are read
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictArgs a, int* counts,
                        int* lists, int room, int held, int parts, int fused_vecs) {
  __shared__ SelectShared sh;
  grid_dependency_wait();
  const int item = blockIdx.x / parts, part_id = blockIdx.x - item * parts;
  const int n = cache_len(a.c, item / a.c.kv_heads, a.err);
  if (n <= a.keep) {                                           // the same for the whole cluster
    if (threadIdx.x == 0 && part_id == 0 && !fused_vecs) counts[item] = 0;
    return;
  }
  const int run = select_run(n, parts), from = min(n, part_id * run), mine = min(n - from, run);
  if (run <= held) evict_select<true>(a, counts, lists, room, item, part_id, parts, from, mine, fused_vecs, sh);
  else evict_select<false>(a, counts, lists, room, item, part_id, parts, from, mine, fused_vecs, sh);
}

__global__ void __launch_bounds__(kMoveWarps * 32)
    evict_move_kernel(const __grid_constant__ EvictArgs a, const int* counts,
                      const int* lists, int room, int head_vecs, int blocks_per_item) {
  grid_dependency_wait();
  const int item = blockIdx.x / blocks_per_item, blk = blockIdx.x - item * blocks_per_item;
  const int* outs = lists + (size_t)item * 2 * room;
  move_rows(a, item, outs, outs + room, counts[item], blk * kMoveWarps + (threadIdx.x >> 5),
            blocks_per_item * kMoveWarps, head_vecs);
}

}  // namespace

int launch_paged_append(const AppendArgs& a, int row_bytes, cudaStream_t s) {
  if (a.n_rows == 0) return SFM_OK;
  const int row_vecs = row_bytes / 16;
  // about two 16-byte pieces of K and of V per thread, whole rows per CTA
  int rows = 2 * kAppendThreads / row_vecs;
  rows = rows < 1 ? 1 : rows > 16 ? 16 : rows;
  ProfScope ps(SFM_PROF_APPEND, s);
  return record_cuda(launch_dependent(paged_append_kernel, (unsigned)((a.n_rows + rows - 1) / rows), kAppendThreads, 0,
                                      s, a, row_vecs, rows));
}

// Rows moved per (sequence, key head): at most the slots past `keep`, and at most `keep`.
static int evict_room(int max_tokens, int keep) {
  const int past = max_tokens - keep;
  return past <= 0 ? 0 : past < keep ? past : keep;
}

// CTAs per item: a slot costs one CTA 0.6 ns, a cluster of 2, 4 or 8 costs 3.6, 6.3 and some 9 us
// for its barriers and histograms, and clusters fill about 128 SMs: two or four where a CTA has
// more than 12K slots (8 heads of 30,000: 27.8 us alone, 23.7, 22.6, and with eight 23.7; of
// 8,000: 14.6, 17.9, 19.6, 22.2), and as many as hold the ranks (24 heads of 57,600 in passes
// over global memory 101 us, held by four 30.8).
static int evict_parts(long long items, int max_tokens) {
  int parts = 1;
  while (parts < 4 && items * parts * 2 <= 128 && max_tokens / parts > 12 * 1024) parts *= 2;
  while (parts < 8 && select_run(max_tokens, parts) > kHeldRanks) parts *= 2;
  return parts;
}
// So few rows that the CTA that ranks an item moves them too: its lists stay in shared memory, and
// neither a workspace nor a second launch is needed.  The host's time is 14.8 -> 9.9 us; on the
// device, all rows moved, 8 items of 100 to 50: 11.8 -> 10.3 us, 32 of 1,200 to 924: 14.2 -> 15.8,
// 8 of 1,024 to 512: 13.1 -> 17.8 (one SM moves what all could), but 128 of them 20.3 -> 18.4; 384
// (several waves) 48 -> 53 with few moves.
constexpr int kFusedRows = 512, kFusedRowsFew = 320;
static bool evict_fused(long long items, int max_tokens, int keep) {
  const int rows = items > kSms ? 0 : items >= 64 ? kFusedRows : kFusedRowsFew;
  return evict_room(max_tokens, keep) <= rows && evict_parts(items, max_tokens) == 1;
}

size_t paged_evict_workspace(int n_seq, int max_tokens, int kv_heads, int keep) {
  const size_t items = (size_t)n_seq * kv_heads;
  if (evict_fused((long long)items, max_tokens, keep)) return 0;
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
  const int parts = evict_parts(items, a.c.max_tokens);
  const bool fused = evict_fused(items, a.c.max_tokens, a.keep);
  const int run = select_run(a.c.max_tokens, parts), held = run < kHeldRanks ? run : kHeldRanks;
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kHeldRanks * (int)sizeof(unsigned));
  if (e != cudaSuccess) return record_cuda(e);
  int rc = record_cuda(launch_dependent_clusters(evict_select_kernel, parts, (unsigned)(items * parts), kSelThreads,
                                                 held * sizeof(unsigned), s, a, counts, lists, room, held, parts,
                                                 fused ? row_bytes_head / 16 : 0));
  if (rc || fused) return rc;
  // kMoveRows rows per warp, and no more CTAs than fill the device several times over
  int blocks = (room + kMoveRows * kMoveWarps - 1) / (kMoveRows * kMoveWarps);
  const int most = (kSms * 32 + items - 1) / items;
  if (blocks > most) blocks = most;
  return record_cuda(launch_dependent(evict_move_kernel, (unsigned)(items * blocks), kMoveWarps * 32, 0, s, a,
                                      (const int*)counts, (const int*)lists, room, row_bytes_head / 16, blocks));
}

}  // namespace sfm
