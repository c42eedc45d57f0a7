// Attention of one new token per sequence over the paged K/V cache.
//
//   s_t = q . k_t / sqrt(D);  s = cap tanh(s / cap);  s -= slope_h |q_pos - pos_t|
//   O = sum_t softmax(s)_t v_t over the sequence's slots;  weights[t] += sum of the
//   softmax over the query heads that share the key head.
//
// Bound by reading K and V once: with G query heads per key head every 2-byte element
// takes part in 2 G operations, far below the tensor cores' ratio but above the CUDA
// cores' for G >= 4, so bf16 uses mma.sync m16n8k16 (a tcgen05 tile would be 128 rows
// high for G rows of work, and its round trips through TMEM add latency that the copy
// rate does not leave).  Both products are transposed so that the tile's long side is
// the matrix's M: S^T = K Q^T (16 tokens x 8 heads), O^T = V^T P^T (16 dims x 8 heads);
// P^T gets from the accumulator to the operand layout through movmatrix, in registers.
// P is used as a bf16 pair hi + lo (two products, 2^-15 of p left out): its rounding to one
// bf16 would be as large as the output's own, and the tensor cores wait for memory anyway.
//
// Work split: the sequences' 64-token tiles, all laid end to end, are cut into `slots`
// equal runs (lengths are read on the device, so ragged batches stay balanced and a
// captured graph follows the lengths); CTA (slot, head) walks its run.  The heads of
// one slot are neighbours in the grid: they read neighbouring 256-byte pieces of the
// same rows at about the same time.  A CTA's four warps take 16 tokens of each tile,
// each with its own ring of cp.async stages (no barrier until a sequence ends).  A
// sequence inside one run is finished there; otherwise its fp32 partials are joined by
// a second kernel, in slot order, so results do not depend on timing.
//
// Small batches of short sequences, where two launches cost more than the work, run as one
// kernel without a workspace: a cluster of up to 8 CTAs per (sequence, head group) cuts the
// sequence's tiles evenly, and joins (and adds weights) over distributed shared memory.
//
// Measured (bf16): one sequence of 57,600 tokens, 24 key heads, bias: 118 us, 6.0 TB/s, 0.91 of
// a copy's rate; 16 sequences of 500 to 12,000 tokens, 8 key heads of 3 query heads: 60 us,
// 5.7 TB/s, 62 us with a cap, 73 us with the cap and weights (the pass that adds them waits for
// its scores to come from L2, and for the sums).  2 sequences of 300 tokens, in clusters: 6.2 us,
// latency.  fp32, 8 sequences of 900 to 4,000, 2 key heads of 4, D 64: 11.4 us.
#include <math.h>

#include "paged.cuh"
#include "sm100.cuh"

namespace sfm {

using sm100::ex2_approx;
using sm100::smem_u32;

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kWarpTok = 16, kTile = kWarps * kWarpTok;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;     // a running max is moved once a score passes it by 2^8
constexpr float kHiPart = -0x1.fffffep-1f;   // -(1 - 2^-24)
constexpr int kSms = 148;

// What the kernels share about the split of one call.
struct Split {
  int slots;            // runs of tiles
  int hgroups;          // head groups: key heads x tiles of query heads
  int gt;               // query-head tiles per key head
  int hpt;              // query heads per tile
  float* part;          // [slots][hgroups][2][hpt][D]
  float* ml;            // [slots][hgroups][2][hpt][2]: running max (log2), sum
  float* lse;           // [n_seq][H] (log2; with weights, of sequences finished by one CTA: see leave_sum)
  float* scores;        // [n_seq][H][pitch] (log2, without the bias; with weights)
  int pitch;            // max_tokens
  int joins;            // CTAs of the finishing kernel that join, before those that add weights
  int parts;            // CTAs of a (sequence, head group)'s cluster, 0: runs of tiles and a join
  int held;             // with weights: scores of a head that a CTA of a cluster holds
};

// This CTA's share of the tiles, and the first of them.
struct Share {
  int hg, slot, part;   // head group; run, or CTA of the cluster
  int n_tiles;
};

// Number of tiles of all sequences, by one warp.
__device__ int total_tiles(const PagedCache& c, int lane, int* err) {
  int sum = 0;
  for (int s = lane; s < c.n_seq; s += 32) sum += (cache_len(c, s, err) + kTile - 1) / kTile;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The sequence that holds tile b of all (b < total) and that tile's index in it, by one warp.
__device__ void find_tile(const PagedCache& c, int b, int lane, int* seq, int* tile) {
  int base = 0;
  for (int s0 = 0; s0 < c.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const int nt = s < c.n_seq ? (cache_len(c, s, nullptr) + kTile - 1) / kTile : 0;
    int inc = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + inc > b);
    if (past) {
      const int l = __ffs(past) - 1;
      *seq = s0 + l;
      *tile = b - base - __shfl_sync(0xffffffffu, inc - nt, l);
      return;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  *seq = c.n_seq;     // not reached for b < total
  *tile = 0;
}

// A walk over tiles in order: sequence, tile in it, its length.
struct Walk {
  int seq, tile, len;
  __device__ __forceinline__ void next(const PagedCache& c) {
    ++tile;
    if (tile * kTile < len) return;
    tile = 0;
    do {
      ++seq;
      len = seq < c.n_seq ? cache_len(c, seq, nullptr) : 0;
    } while (len == 0 && seq < c.n_seq);
  }
};

template <bool CLUSTER>
__device__ __forceinline__ Share take_share(const DecodeArgs& a, const Split& sp, int lane, Walk* w) {
  Share s;
  if (CLUSTER) {
    const int item = blockIdx.x / sp.parts;
    s.part = blockIdx.x - item * sp.parts;
    w->seq = item / sp.hgroups;
    s.hg = item - w->seq * sp.hgroups;
    s.slot = 0;
    w->len = cache_len(a.c, w->seq, a.err);
    const int nt = (w->len + kTile - 1) / kTile, chunk = (nt + sp.parts - 1) / sp.parts;
    w->tile = min(nt, s.part * chunk);
    s.n_tiles = min(nt - w->tile, chunk);
    return s;
  }
  s.hg = blockIdx.x % sp.hgroups;
  s.slot = blockIdx.x / sp.hgroups;
  s.part = 0;
  const int total = total_tiles(a.c, lane, a.err);
  const int chunk = (total + sp.slots - 1) / sp.slots;
  const int b0 = s.slot * chunk;
  s.n_tiles = min(total, b0 + chunk) - b0;
  if (s.n_tiles > 0) {
    find_tile(a.c, b0, lane, &w->seq, &w->tile);
    w->len = cache_len(a.c, w->seq, nullptr);
  }
  return s;
}

// All threads of the cluster (or of the CTA that is alone); what they wrote to shared memory is seen.
__device__ __forceinline__ void cluster_barrier(int parts) {
  __syncwarp();                                                // (after loops of unequal length)
  if (parts == 1) __syncthreads();
  else sm100::cluster_sync();
}
// The float at the place of `p` in CTA `rank` of the cluster.
__device__ __forceinline__ float peer_float(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];"
               : "=f"(v)
               : "r"(sm100::mapa_shared(smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}

// One score in log2 units, without the bias.
template <bool CAP>
__device__ __forceinline__ float scaled_score(float dot, float scale, float cap, float inv_cap) {
  float s = dot * scale;
  if (CAP) s = cap * tanhf(s * inv_cap);
  return s * kLog2e;
}

// The bias.  A score with its bias is one number only where maxima are looked for: far from the
// query it is as large as slope x distance (41,000 for 1/2 x 57,600: 2^-8 apart in fp32), and its
// rounding would be the weights' error.  A weight takes score, bias and maximum apart, the product
// unrounded: 2^(s + fma(-slope, distance, -m)), the sum small wherever the weight is not.  The
// distance is taken in whole numbers first: a slope times an absolute position would lose what
// tells neighbours apart.
__device__ __forceinline__ float distance(int q_pos, int pos) { return fabsf((float)((long long)q_pos - pos)); }
__device__ __forceinline__ float with_bias(float s, float slope2, float dist) { return fmaf(-slope2, dist, s); }
__device__ __forceinline__ float weight_of(float s, float slope2, float dist, float m) {
  return ex2_approx(s + fmaf(-slope2, dist, -m));
}
__device__ __forceinline__ int query_position(const DecodeArgs& a, int seq, int len) {
  return a.q_positions ? load_late(a.q_positions + seq) : len - 1;
}

// The least and the largest distance of a sequence's slots, looked for by all threads of a CTA.  red:
// a free place of shared memory for 2 floats of each warp.  (Static shared memory would leave no room
// for a second CTA.)
struct Reach {
  float near, far;
  __device__ float at(float slope2) const { return slope2 < 0.f ? far : near; }
};
template <int THREADS>
__device__ Reach find_reach(const DecodeArgs& a, int seq, int hk, int n, float* red) {
  if (!a.positions) return {0.f, (float)(n - 1)};
  const int* ps = a.positions + ((size_t)seq * a.c.kv_heads + hk) * a.cap;
  const int q_pos = query_position(a, seq, n), lane = threadIdx.x & 31;
  float near = INFINITY, far = 0.f;
#pragma unroll 8
  for (int t = threadIdx.x; t < n; t += THREADS) {
    const float d = distance(q_pos, load_late(ps + t));
    near = fminf(near, d);
    far = fmaxf(far, d);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    near = fminf(near, __shfl_xor_sync(0xffffffffu, near, o));
    far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, o));
  }
  if (lane == 0) {
    red[threadIdx.x >> 5] = near;
    red[THREADS / 32 + (threadIdx.x >> 5)] = far;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    near = fminf(near, red[w]);
    far = fmaxf(far, red[THREADS / 32 + w]);
  }
  __syncthreads();                                             // the place is free again
  return {near, far};
}
// What the finishing kernel needs of a head of a sequence that one CTA finished: the maximum m and
// the sum, two numbers with a bias, as it may be far larger than the logarithm of the sum.  The sum
// is left behind the head's scores.  A sequence that fills its table has no place there: its
// log-sum-exp is left as one number, relative to the bias at its nearest slot (the farthest of a
// negative slope), next to which it is small, and both kernels look for that distance (some 6 us in
// each; 300 sequences of 2,000 tokens, all full: 546 -> 603 us).
__device__ __forceinline__ bool sum_behind(const Split& sp, int len) { return len < sp.pitch; }
template <bool BIAS>
__device__ __forceinline__ void leave_sum(const DecodeArgs& a, const Split& sp, int seq, int h, int len,
                                          const Reach& reach, float m, float sum) {
  const size_t row = (size_t)seq * a.heads + h;
  if (BIAS && sum_behind(sp, len)) {
    sp.lse[row] = sum == 0.f ? -INFINITY : m;
    sp.scores[row * sp.pitch + len] = sum;
    return;
  }
  const float slope2 = BIAS ? load_late(a.slopes + h) * kLog2e : 0.f;
  sp.lse[row] = fmaf(slope2, reach.at(slope2), m) + log2f(sum);
}

// The cluster's end: part_o [nh][D] and part_ml [nh][2] (max (log2), sum) hold this CTA's share of
// heads h0, ...; its scores of `count` slots from tok0 on, if weights are wanted, are
// scores[head * held + slot - tok0].
constexpr int kMaxParts = 8, kMaxTileHeads = 16;
constexpr int kHeldTiles = 2;                                   // tiles a CTA of a cluster has at most, with weights
template <typename T, int D>
__device__ __forceinline__ void cluster_finish(const DecodeArgs& a, const Split& sp, int seq, int len, int part, int h0,
                                               int nh, const float* part_o, float* part_ml, const float* scores,
                                               int tok0, int count) {
  // (behind the partials, where the rings were: static shared memory would leave no room for a
  // second CTA on the SM)
  float (*share)[kMaxParts] = reinterpret_cast<float (*)[kMaxParts]>(part_ml + 2 * kMaxTileHeads);
  float* top = part_ml + (2 + kMaxParts) * kMaxTileHeads;      // of each head: maximum (-inf: no visible slot),
  float* inv = top + kMaxTileHeads;                            // 1 / sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster_barrier(sp.parts);
  for (int hh = warp; hh < nh; hh += kWarps) {
    const bool in = lane < sp.parts;
    const float m = in ? peer_float(part_ml + 2 * hh, lane) : -INFINITY;
    const float l = in ? peer_float(part_ml + 2 * hh + 1, lane) : 0.f;
    float mx = m;
#pragma unroll
    for (int o = kMaxParts / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mb = mx == -INFINITY ? 0.f : mx, f = ex2_approx(m - mb);
    float sum = f * l;
#pragma unroll
    for (int o = kMaxParts / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool have = sum > 0.f || sum != sum;
    if (in) share[hh][lane] = l == 0.f ? -1.f : f / sum;       // (-1: no visible slot, maybe nothing written)
    if (lane == 0) {
      top[hh] = have ? mb : -INFINITY;
      inv[hh] = 1.f / sum;
    }
  }
  __syncthreads();
  for (int x = part * kThreads + threadIdx.x; x < nh * D; x += sp.parts * kThreads) {
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) {
      const float f = r < sp.parts ? share[x / D][r] : -1.f;
      if (!(f < 0.f)) o = fmaf(f, peer_float(part_o + x, r), o);   // (a share of 0 hides no infinity or NaN)
    }
    reinterpret_cast<T*>(a.o)[((size_t)seq * a.heads + h0) * D + x] = (T)o;
  }
  if (scores) {
    const size_t at = ((size_t)seq * a.c.kv_heads + h0 / (a.heads / a.c.kv_heads)) * a.cap + tok0;
    float* w = a.weights + at;
    const int q_pos = query_position(a, seq, len);
    for (int t = threadIdx.x; t < count; t += kThreads) {
      const float dist = a.slopes ? distance(q_pos, a.positions ? load_late(a.positions + at + t) : tok0 + t) : 0.f;
      float add = 0.f;
      for (int hh = 0; hh < nh; ++hh) {
        const float slope2 = a.slopes ? load_late(a.slopes + h0 + hh) * kLog2e : 0.f;
        if (top[hh] != -INFINITY) add += weight_of(scores[hh * sp.held + t], slope2, dist, top[hh]) * inv[hh];
      }
      w[t] += add;
    }
  }
  if (sp.parts > 1) cluster_barrier(sp.parts);                 // nobody leaves while its memory is read
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a run holds of a sequence: earlier runs have tiles before, later ones tiles behind.  A run
// has two places for partials: of the sequence that starts before it, and of the one that ends after.
struct Segment {
  bool starts_before, ends_after;
  __device__ bool partial() const { return starts_before || ends_after; }
  __device__ int index() const { return starts_before ? 0 : 1; }
};

// ------------------------------------------------------------------ bf16, D = 128

constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kWarpTok * 256;                 // K and V rows of 16 tokens
constexpr int kOPitch = 132;                                    // floats per head row of the merge buffer
constexpr int kOffMerge = kWarps * kStages * kStageBytes;       // 96 KB of rings, then
constexpr int kOffMl = kOffMerge + kWarps * 8 * kOPitch * 4;    // O^T of each warp, its max and sum
constexpr int kSmemBf16 = kOffMl + kWarps * 8 * 2 * 4;          // 115,456 bytes: two CTAs per SM

template <int NT, bool CAP, bool BIAS, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_bf16_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ Split sp) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  grid_dependency_wait();
  grid_dependency_trigger();                                  // the finishing kernel may be set up
  Walk ld;                                                    // of the loads
  const Share share = take_share<CLUSTER>(a, sp, lane, &ld);
  const int n_tiles = share.n_tiles;
  if (!CLUSTER && n_tiles <= 0) return;
  const int hg = share.hg, slot = share.slot;
  const int hk = hg / sp.gt;                                  // key head
  const int G = a.heads / a.c.kv_heads;
  const int g0 = (hg - hk * sp.gt) * (8 * NT);                // first query head of the group here
  const int nh = min(8 * NT, G - g0);                         // query heads of this tile
  const int h0 = hk * G + g0;
  const int tok0 = ld.tile * kTile, own_seq = ld.seq, own_len = ld.len;   // CLUSTER: its only sequence, first slot
  Walk cw = ld;                                               // of the arithmetic
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (kStages * kStageBytes);
  const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(a.k_pages) + (size_t)hk * 128;
  const __nv_bfloat16* vp = reinterpret_cast<const __nv_bfloat16*>(a.v_pages) + (size_t)hk * 128;
  const size_t row_elems = (size_t)a.c.kv_heads * 128;

  // pool row of this lane's token (lanes 0..15) of the next tile to load; -1: none
  auto lookup = [&](const Walk& w) -> int {
    const int t = w.tile * kTile + warp * kWarpTok + (lane & 15);
    return lane < 16 && t < w.len ? cache_row(a.c, w.seq, t, a.err) : -1;
  };
  // a tile's 16 K rows and 16 V rows: lane = 16-byte piece (lane & 15) of rows (lane >> 4) + 2 i;
  // pieces are stored at piece ^ (row & 7): no bank conflicts for ldmatrix, either way round
  auto issue = [&](int stage, int row) {
    const uint32_t dst = ring + (uint32_t)stage * kStageBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = 2 * i + (lane >> 4);
      const int row_i = __shfl_sync(0xffffffffu, row, rr);
      const size_t off = (size_t)max(row_i, 0) * row_elems + (lane & 15) * 8;
      const uint32_t d = dst + (uint32_t)(rr * 256 + (((lane & 15) ^ (rr & 7)) << 4));
      cp_async16(d, kp + off, row_i >= 0);
      cp_async16(d + kWarpTok * 256, vp + off, row_i >= 0);
    }
  };

  unsigned masks[kStages] = {};                               // which of the 16 tokens count
  int next_row = lookup(ld);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    masks[i] = 0;
    if (i < n_tiles) {
      masks[i] = __ballot_sync(0xffffffffu, next_row >= 0) & 0xffffu;
      issue(i, next_row);
      if (i + 1 < n_tiles) {
        ld.next(a.c);
        next_row = lookup(ld);
      }
    }
    cp_commit();
  }

  uint32_t qf[8][NT][2];                                      // Q^T operand of the current sequence
  float acc[8][NT][4];                                        // O^T: dims 16 i + g (+8), heads 2 t4 (+1)
  float m[NT][2], l[NT][2], slope[NT][2];
  bool fresh = true;
  const float scale = 0.08838834764831845f;                   // 1 / sqrt(128)
  const float inv_cap = CAP ? 1.f / a.softcap : 0.f;
  int q_pos = 0;
  const bool keep_scores = a.weights != nullptr;
  float* const own_scores = reinterpret_cast<float*>(smem + kSmemBf16);   // CLUSTER: [heads of the tile][held]
  float* const part_o = reinterpret_cast<float*>(smem);       // (where the rings were)
  float* const part_ml = part_o + 8 * NT * 128;
  const int pitch = CLUSTER ? sp.held : sp.pitch;
  float* score_rows = nullptr;                                // of head 2 t4 of the tile
  bool seg_start = false;

  for (int it = 0; it < n_tiles; ++it) {
    if (fresh) {
      fresh = false;
      seg_start = cw.tile != 0;                               // an earlier run has its first tiles
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + ((size_t)cw.seq * a.heads + h0) * 64;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool have = nt * 8 + g < nh;                    // heads past the group: zeros
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qf[ks][nt][0] = have ? load_late(q + (nt * 8 + g) * 64 + ks * 8 + t4) : 0u;
          qf[ks][nt][1] = have ? load_late(q + (nt * 8 + g) * 64 + ks * 8 + t4 + 4) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
          const int hh = nt * 8 + 2 * t4 + e;
          slope[nt][e] = BIAS && hh < nh ? load_late(a.slopes + h0 + hh) * kLog2e : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
      }
      if (BIAS) q_pos = query_position(a, cw.seq, cw.len);
      if (keep_scores)
        score_rows = CLUSTER ? own_scores + 2 * t4 * pitch - tok0
                             : sp.scores + ((size_t)cw.seq * a.heads + h0 + 2 * t4) * pitch;
    }
    // keep the ring full: the tile kStages - 1 ahead goes where the last one was consumed
    if (it + kStages - 1 < n_tiles) {
      masks[kStages - 1] = __ballot_sync(0xffffffffu, next_row >= 0) & 0xffffu;
      issue((it + kStages - 1) % kStages, next_row);
      if (it + kStages < n_tiles) {
        ld.next(a.c);
        next_row = lookup(ld);
      }
    }
    cp_commit();
    cp_wait<kStages - 1>();
    __syncwarp();

    const uint32_t ks_base = ring + (uint32_t)(it % kStages) * kStageBytes;
    const uint32_t vs_base = ks_base + kWarpTok * 256;
    const int tok = cw.tile * kTile + warp * kWarpTok + g;    // this thread's tokens: tok, tok + 8
    const unsigned mk = masks[0];
    if (mk || keep_scores) {                                  // (-inf is a score: bad pages)
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
      {
        const int r = lane & 15;                              // K rows as the A operand
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t ka[4];
          ldsm4(ka, ks_base + (uint32_t)(r * 256 + (((2 * ks + (lane >> 4)) ^ (r & 7)) << 4)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], ka, qf[ks][nt][0], qf[ks][nt][1]);
        }
      }
      const bool in0 = (mk >> g) & 1u, in1 = (mk >> (g + 8)) & 1u;
      float d0 = 0.f, d1 = 0.f;
      if (BIAS) {
        int p0 = tok, p1 = tok + 8;
        if (a.positions) {
          const int* ps = a.positions + ((size_t)cw.seq * a.c.kv_heads + hk) * a.cap;
          p0 = in0 ? load_late(ps + tok) : 0;
          p1 = in1 ? load_late(ps + tok + 8) : 0;
        }
        d0 = distance(q_pos, p0);
        d1 = distance(q_pos, p1);
      }
      auto biased = [&](int nt, int e) {
        return BIAS ? with_bias(s[nt][e], slope[nt][e & 1], e < 2 ? d0 : d1) : s[nt][e];
      };
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = e < 2 ? in0 : in1;
          s[nt][e] = in ? scaled_score<CAP>(s[nt][e], scale, a.softcap, inv_cap) : -INFINITY;
          grow |= biased(nt, e) > m[nt][e & 1] + kGrow;       // also from m = -inf
        }
      if (keep_scores) {
        // raw scores for the pass that accumulates weights: 8 consecutive tokens per head
        float* sc = score_rows + tok;
        const bool w0 = tok < cw.len, w1 = tok + 8 < cw.len;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hh = nt * 8 + 2 * t4;
          if (hh < nh) {
            if (w0) sc[0] = s[nt][0];
            if (w1) sc[8] = s[nt][2];
          }
          if (hh + 1 < nh) {
            if (w0) sc[pitch] = s[nt][1];
            if (w1) sc[pitch + 8] = s[nt][3];
          }
          sc += 8 * (size_t)pitch;
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(fmaxf(biased(nt, e), biased(nt, e + 2)), m[nt][e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // nothing seen yet: the accumulators are zeros
            const float al = m[nt][e] == -INFINITY ? 0.f : ex2_approx(m[nt][e] - mx);
            m[nt][e] = mx;
            l[nt][e] *= al;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i][nt][e] *= al;
              acc[i][nt][e + 2] *= al;
            }
          }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mb = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
          p[e] = BIAS ? weight_of(s[nt][e], slope[nt][e & 1], e < 2 ? d0 : d1, mb) : ex2_approx(s[nt][e] - mb);
          l[nt][e & 1] += p[e];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // hi by truncation and lo = p - hi (1 - 2^-24): both positive wherever p is, so that
          // an infinite V element stays infinite (0 x inf, or inf - inf, would not)
          const uint32_t hi = __byte_perm(__float_as_uint(p[2 * e]), __float_as_uint(p[2 * e + 1]), 0x7632);
          const float r0 = fmaf(__uint_as_float(hi << 16), kHiPart, p[2 * e]);
          const float r1 = fmaf(__uint_as_float(hi & 0xffff0000u), kHiPart, p[2 * e + 1]);
          ph[nt][e] = transpose8x8(hi);
          pl[nt][e] = transpose8x8(sm100::pack_bf16x2(r0, r1));
        }
      }
      {
        const int r = (lane & 7) + ((lane >> 4) << 3);        // V rows as the transposed A operand
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t va[4];
          ldsm4_t(va, vs_base + (uint32_t)(r * 256 + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) << 4)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(acc[i][nt], va, ph[nt][0], ph[nt][1]);
            mma16816(acc[i][nt], va, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
    __syncwarp();                                             // the stage may be refilled
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) masks[i] = masks[i + 1];
    const int seq = cw.seq, seq_len = cw.len;
    const bool seq_done = (cw.tile + 1) * kTile >= cw.len;
    if (it + 1 < n_tiles) cw.next(a.c);
    if ((CLUSTER || !seq_done) && it + 1 < n_tiles) continue;

    // ---- the sequence, or the run, ends here: merge the four warps
    fresh = true;
    Segment sg{seg_start, !seq_done};
    float* obuf = reinterpret_cast<float*>(smem + kOffMerge);
    float* mlbuf = reinterpret_cast<float*>(smem + kOffMl);
    Reach reach{0.f, 0.f};
    if (BIAS && !CLUSTER && sp.lse && !sg.partial() && !sum_behind(sp, seq_len))
      reach = find_reach<kThreads>(a, seq, hk, seq_len, mlbuf);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (g == 0) {
          mlbuf[(warp * 8 + 2 * t4 + e) * 2] = m[nt][e];
          mlbuf[(warp * 8 + 2 * t4 + e) * 2 + 1] = v;
        }
      }
      float* ob = obuf + warp * 8 * kOPitch;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ob[(2 * t4 + (e & 1)) * kOPitch + 16 * i + g + (e >> 1) * 8] = acc[i][nt][e];
      __syncthreads();
      const int d = threadIdx.x;
      for (int hh = 0; hh < 8 && nt * 8 + hh < nh; ++hh) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, mlbuf[(w * 8 + hh) * 2]);
        const float mb = mm == -INFINITY ? 0.f : mm;
        float sum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2_approx(mlbuf[(w * 8 + hh) * 2] - mb);
          sum = fmaf(f, mlbuf[(w * 8 + hh) * 2 + 1], sum);
          o = fmaf(f, obuf[(w * 8 + hh) * kOPitch + d], o);
        }
        const int ht = nt * 8 + hh;                           // head of the tile
        if (CLUSTER) {
          part_o[ht * 128 + d] = o;
          if (d == 0) {
            part_ml[2 * ht] = mm;
            part_ml[2 * ht + 1] = sum;
          }
        } else if (sg.partial()) {
          const size_t at = (((size_t)slot * sp.hgroups + hg) * 2 + sg.index()) * sp.hpt + ht;
          sp.part[at * 128 + d] = o;
          if (d == 0) {
            sp.ml[at * 2] = mm;
            sp.ml[at * 2 + 1] = sum;
          }
        } else {
          reinterpret_cast<__nv_bfloat16*>(a.o)[((size_t)seq * a.heads + h0 + ht) * 128 + d] =
              __float2bfloat16(sum > 0.f || sum != sum ? o / sum : 0.f);
          if (sp.lse && d == 0) leave_sum<BIAS>(a, sp, seq, h0 + ht, seq_len, reach, mb, sum);
        }
      }
      __syncthreads();
    }
  }
  cp_wait<0>();
  if (CLUSTER) {
    if (n_tiles <= 0 && threadIdx.x < nh) {
      part_ml[2 * threadIdx.x] = -INFINITY;
      part_ml[2 * threadIdx.x + 1] = 0.f;
    }
    cluster_finish<__nv_bfloat16, 128>(a, sp, own_seq, own_len, share.part, h0, nh, part_o, part_ml,
                                       keep_scores ? own_scores : nullptr, tok0, min(own_len - tok0, n_tiles * kTile));
  }
}

// ------------------------------------------------------------------ fp32, D = 32 DV

// CUDA cores.  A warp takes 16 tokens (8 for D = 128) at a time, in steps of 4, 8 lanes to a
// token: lane j of the eight holds the 16-byte pieces j + 8 i of the row, so a load covers whole
// 128-byte lines.  Rows come through a ring of cp.async stages, in which each lane finds the
// pieces that it fetched itself (no exchange, no bank conflicts).  The 8 lanes' sums of all
// (head, step) scores are reduced and scattered in one go: with 4 heads and 4 steps 14 shuffles
// leave each lane two scores, whose cap, bias and exponential are then done once and not by 8
// lanes (with the deeper ring: 21 -> 11.4 us at the size above).  GT query heads per CTA (a
// larger group reads its keys again, from L2).
template <int DV>
struct F32Ring {
  static constexpr int kSteps = DV == 4 ? 2 : 4, kTok = 4 * kSteps, kSub = kWarpTok / kTok;
  static constexpr int kHalf = kTok * DV * 128;                // bytes of a stage's K (or V)
  static constexpr int kDepth = DV == 3 ? 2 : 3;               // 24 KB a warp (DV = 1: 12)
  static constexpr int kBytes = kDepth * 2 * kHalf;
};
template <int DV, int GT>
constexpr int f32_smem() {                                     // rings, Q, O and (max, sum) of each warp
  return kWarps * F32Ring<DV>::kBytes + GT * DV * 128 + kWarps * GT * (DV * 128 + 8);
}

template <int DV, int GT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_fp32_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ Split sp) {
  using Ring = F32Ring<DV>;
  constexpr int D = 32 * DV, STEPS = Ring::kSteps, TOK = Ring::kTok, DEPTH = Ring::kDepth;
  constexpr int NV = GT * STEPS;                               // scores of a step group, v = head * STEPS + step
  constexpr int NO = NV >= 8 ? NV / 8 : 1;                     // of them a lane's own: v0, ... of one head,
  constexpr int DUP = NV >= 8 ? 1 : 8 / NV;                    // held by that many lanes
  constexpr int LPH = 8 / GT;                                  // lanes (of 8) of a head
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* qs = reinterpret_cast<float4*>(smem + kWarps * Ring::kBytes);    // [GT][D / 4]
  float* obuf = reinterpret_cast<float*>(qs + GT * (D / 4));               // [kWarps][GT][D]
  float* mlbuf = obuf + kWarps * GT * D;                                   // [kWarps][GT][2]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane & 7, grp = lane >> 3;
  grid_dependency_wait();
  grid_dependency_trigger();                                  // the finishing kernel may be set up
  Walk ld;                                                    // of the loads
  const Share share = take_share<CLUSTER>(a, sp, lane, &ld);
  if (!CLUSTER && share.n_tiles <= 0) return;
  const int hg = share.hg, slot = share.slot;
  const int hk = hg / sp.gt;
  const int G = a.heads / a.c.kv_heads;
  const int g0 = (hg - hk * sp.gt) * GT;
  const int nh = min(GT, G - g0);
  const int h0 = hk * G + g0;
  const int tok0 = ld.tile * kTile, own_seq = ld.seq, own_len = ld.len;   // CLUSTER: its only sequence, first slot
  Walk cw = ld;                                               // of the arithmetic
  const bool keep_scores = a.weights != nullptr;
  float* const own_scores = mlbuf + kWarps * GT * 2;          // CLUSTER: [GT][held]
  float* const part_o = reinterpret_cast<float*>(smem);       // (where the rings were)
  float* const part_ml = part_o + GT * D;
  const size_t row_vecs = (size_t)a.c.kv_heads * (D / 4);
  const float4* kp = reinterpret_cast<const float4*>(a.k_pages) + (size_t)hk * (D / 4) + j;
  const float4* vp = reinterpret_cast<const float4*>(a.v_pages) + (size_t)hk * (D / 4) + j;
  uint8_t* ring = smem + warp * Ring::kBytes + lane * 16;     // this lane's pieces
  const float scale = rsqrtf((float)D);
  const bool cap = a.softcap > 0.f;
  const float inv_cap = cap ? 1.f / a.softcap : 0.f;

  // pool row of this lane's token (lanes 0..15) of a tile; -1: none
  auto lookup = [&](const Walk& w) -> int {
    const int t = w.tile * kTile + warp * kWarpTok + lane;
    return lane < kWarpTok && t < w.len ? cache_row(a.c, w.seq, t, a.err) : -1;
  };
  const int n_its = share.n_tiles * Ring::kSub;
  unsigned masks[DEPTH] = {};                                 // which of a stage's tokens count
  int pos[DEPTH][NO];                                         // and the positions of the lane's own
  const int v0 = j * NV / 8, my_head = v0 / STEPS, my_step = v0 % STEPS;
  int next_row = lookup(ld), to_issue = 0;
  auto issue = [&](unsigned* mask, int* at) {
    const int sub = to_issue % Ring::kSub;
#pragma unroll
    for (int e = 0; e < NO; ++e) {
      at[e] = ld.tile * kTile + warp * kWarpTok + sub * TOK + (my_step + e) * 4 + grp;
      if (a.positions && at[e] < ld.len)
        at[e] = load_late(a.positions + ((size_t)ld.seq * a.c.kv_heads + hk) * a.cap + at[e]);
    }
    const uint32_t dst = smem_u32(ring) + (uint32_t)(to_issue % DEPTH) * (2 * Ring::kHalf);
    *mask = (__ballot_sync(0xffffffffu, next_row >= 0) >> (sub * TOK)) & ((1u << TOK) - 1u);
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const int row = __shfl_sync(0xffffffffu, next_row, sub * TOK + st * 4 + grp);
      const size_t off = (size_t)max(row, 0) * row_vecs;
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        const uint32_t d = dst + (uint32_t)((st * DV + i) * 512);
        cp_async16(d, kp + off + 8 * i, row >= 0);
        cp_async16(d + Ring::kHalf, vp + off + 8 * i, row >= 0);
      }
    }
    ++to_issue;
    if (to_issue % Ring::kSub == 0 && to_issue < n_its) {
      ld.next(a.c);
      next_row = lookup(ld);
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) {
    if (to_issue < n_its) issue(&masks[i], pos[i]);
    cp_commit();
  }

  float4 acc[GT][DV];
  float m = -INFINITY, l = 0.f, slope = 0.f;                  // of my_head
  bool fresh = true, seg_start = false;
  int q_pos = 0;
  for (int it = 0; it < n_its; ++it) {
    if (fresh) {
      fresh = false;
      seg_start = cw.tile != 0;
      for (int x = threadIdx.x; x < GT * (D / 4); x += kThreads) {
        const int hh = x / (D / 4), c = x - hh * (D / 4);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (hh < nh) f = load_late(reinterpret_cast<const float4*>(a.q) + ((size_t)cw.seq * a.heads + h0 + hh) * (D / 4) + c);
        qs[x] = f;
      }
      m = -INFINITY;
      l = 0.f;
      slope = a.slopes && my_head < nh ? load_late(a.slopes + h0 + my_head) * kLog2e : 0.f;
#pragma unroll
      for (int hh = 0; hh < GT; ++hh)
#pragma unroll
        for (int i = 0; i < DV; ++i) acc[hh][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      q_pos = query_position(a, cw.seq, cw.len);
      __syncthreads();
    }
    const int sub = it % Ring::kSub;
    const int base = cw.tile * kTile + warp * kWarpTok + sub * TOK;
    if (to_issue < n_its) issue(&masks[DEPTH - 1], pos[DEPTH - 1]);
    cp_commit();
    cp_wait<DEPTH - 1>();
    const unsigned mk = masks[0];
    if (mk || keep_scores) {                                   // (-inf is a score: bad pages)
      const float4* kst = reinterpret_cast<const float4*>(ring + (it % DEPTH) * (2 * Ring::kHalf));
      const float4* vst = kst + Ring::kHalf / 16;
      float s[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) s[v] = 0.f;
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        float4 kf[STEPS];
#pragma unroll
        for (int st = 0; st < STEPS; ++st) kf[st] = kst[(st * DV + i) * 32];
#pragma unroll
        for (int hh = 0; hh < GT; ++hh) {
          const float4 qv = qs[hh * (D / 4) + j + 8 * i];
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            float x = s[hh * STEPS + st];
            x = fmaf(qv.x, kf[st].x, x);
            x = fmaf(qv.y, kf[st].y, x);
            x = fmaf(qv.z, kf[st].z, x);
            s[hh * STEPS + st] = fmaf(qv.w, kf[st].w, x);
          }
        }
      }
      // the sums over the 8 lanes; lane j ends with those of v0 = j NV / 8 (+ 1)
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const int o = 4 >> b, n = NV >> (b + 1);
        const bool up = (j & o) != 0;
        if (n == 0) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float got = __shfl_xor_sync(0xffffffffu, up ? s[i] : s[i + n], o);
          s[i] = (up ? s[i + n] : s[i]) + got;
        }
      }
      bool grow = false;
      float dist[NO];
#pragma unroll
      for (int e = 0; e < NO; ++e) {
        const int x = (my_step + e) * 4 + grp;                 // token of the stage
        dist[e] = distance(q_pos, pos[0][e]);
        if (!((mk >> x) & 1u)) s[e] = -INFINITY;
        else if (cap) s[e] = scaled_score<true>(s[e], scale, a.softcap, inv_cap);
        else s[e] = scaled_score<false>(s[e], scale, 0.f, 0.f);
        grow |= with_bias(s[e], slope, dist[e]) > m + kGrow;   // also from m = -inf
        if (keep_scores && my_head < nh && base + x < cw.len) {
          if (CLUSTER) own_scores[my_head * sp.held + base + x - tok0] = s[e];
          else sp.scores[((size_t)cw.seq * a.heads + h0 + my_head) * sp.pitch + base + x] = s[e];
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
        float mx = m;
#pragma unroll
        for (int e = 0; e < NO; ++e) mx = fmaxf(mx, with_bias(s[e], slope, dist[e]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
          if (o < LPH || o >= 8) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float al = m == -INFINITY ? 0.f : ex2_approx(m - mx);
        m = mx;
        l *= al;
#pragma unroll
        for (int hh = 0; hh < GT; ++hh) {
          const float f = __shfl_sync(0xffffffffu, al, hh * LPH);
#pragma unroll
          for (int i = 0; i < DV; ++i) {
            acc[hh][i].x *= f;
            acc[hh][i].y *= f;
            acc[hh][i].z *= f;
            acc[hh][i].w *= f;
          }
        }
      }
      const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int e = 0; e < NO; ++e) {
        s[e] = weight_of(s[e], slope, dist[e], mb);
        l += s[e];
      }
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        float4 vf[DV];
#pragma unroll
        for (int i = 0; i < DV; ++i) vf[i] = vst[(st * DV + i) * 32];
#pragma unroll
        for (int hh = 0; hh < GT; ++hh) {
          const int v = hh * STEPS + st;
          const float p = __shfl_sync(0xffffffffu, s[v % NO], grp * 8 + v * 8 / NV);
#pragma unroll
          for (int i = 0; i < DV; ++i) {
            acc[hh][i].x = fmaf(p, vf[i].x, acc[hh][i].x);
            acc[hh][i].y = fmaf(p, vf[i].y, acc[hh][i].y);
            acc[hh][i].z = fmaf(p, vf[i].z, acc[hh][i].z);
            acc[hh][i].w = fmaf(p, vf[i].w, acc[hh][i].w);
          }
        }
      }
    }
    __syncwarp();                                              // the stage may be refilled
#pragma unroll
    for (int i = 0; i + 1 < DEPTH; ++i) {
      masks[i] = masks[i + 1];
#pragma unroll
      for (int e = 0; e < NO; ++e) pos[i][e] = pos[i + 1][e];
    }
    if (sub + 1 < Ring::kSub) continue;
    const int seq = cw.seq, seq_len = cw.len;
    const bool seq_done = (cw.tile + 1) * kTile >= cw.len;
    if (it + 1 < n_its) cw.next(a.c);
    if ((CLUSTER || !seq_done) && it + 1 < n_its) continue;

    // ---- the sequence, or the run, ends here: the warp's four groups, then the four warps
    fresh = true;
    Segment sg{seg_start, !seq_done};
    Reach reach{0.f, 0.f};
    if (!CLUSTER && a.slopes && sp.lse && !sg.partial() && !sum_behind(sp, seq_len))
      reach = find_reach<kThreads>(a, seq, hk, seq_len, mlbuf);
    float sum = l * (1.f / DUP);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o < LPH || o >= 8) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (grp == 0 && j % LPH == 0) {
      mlbuf[(warp * GT + my_head) * 2] = m;
      mlbuf[(warp * GT + my_head) * 2 + 1] = sum;
    }
#pragma unroll
    for (int hh = 0; hh < GT; ++hh)
#pragma unroll
      for (int i = 0; i < DV; ++i) {
        float v[4] = {acc[hh][i].x, acc[hh][i].y, acc[hh][i].z, acc[hh][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += __shfl_xor_sync(0xffffffffu, v[e], 8);
          v[e] += __shfl_xor_sync(0xffffffffu, v[e], 16);
        }
        if (grp == 0)
          *reinterpret_cast<float4*>(obuf + (warp * GT + hh) * D + (j + 8 * i) * 4) = make_float4(v[0], v[1], v[2], v[3]);
      }
    __syncthreads();
    for (int x = threadIdx.x; x < nh * D; x += kThreads) {
      const int hh = x / D, d = x - hh * D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, mlbuf[(w * GT + hh) * 2]);
      const float mb = mm == -INFINITY ? 0.f : mm;
      float sum = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(mlbuf[(w * GT + hh) * 2] - mb);
        sum = fmaf(f, mlbuf[(w * GT + hh) * 2 + 1], sum);
        o = fmaf(f, obuf[(w * GT + hh) * D + d], o);
      }
      if (CLUSTER) {
        part_o[x] = o;
        if (d == 0) {
          part_ml[2 * hh] = mm;
          part_ml[2 * hh + 1] = sum;
        }
      } else if (sg.partial()) {
        const size_t at = (((size_t)slot * sp.hgroups + hg) * 2 + sg.index()) * sp.hpt + hh;
        sp.part[at * D + d] = o;
        if (d == 0) {
          sp.ml[at * 2] = mm;
          sp.ml[at * 2 + 1] = sum;
        }
      } else {
        reinterpret_cast<float*>(a.o)[((size_t)seq * a.heads + h0 + hh) * D + d] =
            sum > 0.f || sum != sum ? o / sum : 0.f;
        if (sp.lse && d == 0) {
          if (a.slopes) leave_sum<true>(a, sp, seq, h0 + hh, seq_len, reach, mb, sum);
          else leave_sum<false>(a, sp, seq, h0 + hh, seq_len, reach, mb, sum);
        }
      }
    }
    __syncthreads();
  }
  cp_wait<0>();
  if (CLUSTER) {
    if (n_its <= 0 && threadIdx.x < nh) {
      part_ml[2 * threadIdx.x] = -INFINITY;
      part_ml[2 * threadIdx.x + 1] = 0.f;
    }
    cluster_finish<float, D>(a, sp, own_seq, own_len, share.part, h0, nh, part_o, part_ml,
                             keep_scores ? own_scores : nullptr, tok0, min(own_len - tok0, share.n_tiles * kTile));
  }
}

// ------------------------------------------------------------------ join

// Where a sequence's partials are: runs s0 .. s1 (one run: it was finished there), empty if
// it has no tiles.
struct Parts {
  int nt, s0, s1;
};

__device__ Parts find_parts(const PagedCache& c, const Split& sp, int seq, int lane) {
  int total = 0, start = 0;
  for (int s = lane; s < c.n_seq; s += 32) {
    const int nt = (cache_len(c, s, nullptr) + kTile - 1) / kTile;
    total += nt;
    start += s < seq ? nt : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    start += __shfl_xor_sync(0xffffffffu, start, o);
  }
  Parts p;
  p.nt = (cache_len(c, seq, nullptr) + kTile - 1) / kTile;
  if (p.nt == 0) {
    p.s0 = p.s1 = 0;
    return p;
  }
  const int chunk = (total + sp.slots - 1) / sp.slots;
  p.s0 = start / chunk;
  p.s1 = (start + p.nt - 1) / chunk;
  return p;
}

// index of the partial of query head h in run s: the run that holds tile 0 of the sequence
// wrote its second place, the later ones their first
__device__ __forceinline__ size_t part_at(const Split& sp, int G, int h, int s, int s0) {
  const int hk = h / G, gi = h - hk * G;
  return (((size_t)s * sp.hgroups + hk * sp.gt + gi / sp.hpt) * 2 + (s == s0 ? 1 : 0)) * sp.hpt + gi % sp.hpt;
}

// max (log2) and sum of a head's partials, by one warp
__device__ void join_ml(const Split& sp, int G, int h, const Parts& p, int lane, float* m, float* l) {
  float mx = -INFINITY, sum = 0.f;
  for (int s = p.s0 + lane; s <= p.s1; s += 32) mx = fmaxf(mx, sp.ml[part_at(sp, G, h, s, p.s0) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mb = mx == -INFINITY ? 0.f : mx;
  for (int s = p.s0 + lane; s <= p.s1; s += 32) {
    const float2 v = *reinterpret_cast<const float2*>(sp.ml + part_at(sp, G, h, s, p.s0) * 2);
    sum = fmaf(ex2_approx(v.x - mb), v.y, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  *m = mb;
  *l = sum;
}

constexpr int kFinThreads = 256, kAccTok = 1024;
constexpr int kTokThread = kAccTok / kFinThreads, kHeadsOnce = 4, kSumsOnce = 32;

// The finishing kernel.  Its first CTAs join, one per (sequence, query head): a sequence
// finished by one CTA is left alone, an empty one gets zeros; the partials are summed in a
// fixed order (float4 column x run, runs strided over the CTA, then over its groups).  The
// others add weights, one per (sequence, key head, kAccTok slots): weights += sum over the
// key head's query heads of 2^(score + bias - m) / l.  Only the part that does not depend on the
// attention kernel runs before the wait for it.  (80 registers; 64 spill and are 2 to 15 % slower
// with weights, 124, as the compiler would have them with a bias, 6 %, a kernel of 47 for the joins
// alone 2 to 5 % where few sequences are joined.)
template <typename T, bool BIAS>
__global__ void __launch_bounds__(kFinThreads, 3)
    paged_finish_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ Split sp, int blocks_per_item) {
  __shared__ float4 buf[kFinThreads];
  __shared__ float4 sh[kSumsOnce];                             // maximum (-inf: no visible slot), 1 / sum, slope, Reach
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.heads / a.c.kv_heads;
  if ((int)blockIdx.x < sp.joins) {
    const int seq = blockIdx.x / a.heads, h = blockIdx.x - seq * a.heads, D = a.c.head_dim;
    const Parts p = find_parts(a.c, sp, seq, lane);
    grid_dependency_wait();
    T* out = reinterpret_cast<T*>(a.o) + ((size_t)seq * a.heads + h) * D;
    if (p.nt == 0) {
      if (tid < D) out[tid] = (T)0.f;
      return;
    }
    if (p.s0 == p.s1) return;
    float mb, sum;
    join_ml(sp, G, h, p, lane, &mb, &sum);                     // every warp the same
    const int cols = D / 4, groups = kFinThreads / cols;       // 8, 16, 24 or 32 columns
    const int c = tid % cols, g = tid / cols;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g < groups) {
#pragma unroll 4
      for (int s = p.s0 + g; s <= p.s1; s += groups) {
        const size_t at = part_at(sp, G, h, s, p.s0);
        const float f = ex2_approx(sp.ml[at * 2] - mb);
        const float4 v = *reinterpret_cast<const float4*>(sp.part + at * D + 4 * c);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
    }
    buf[tid] = acc;
    __syncthreads();
    if (tid < D) {
      float o = 0.f;
      const int used = min(groups, p.s1 - p.s0 + 1);
      for (int i = 0; i < used; ++i) o += reinterpret_cast<const float*>(buf + i * cols)[tid];
      out[tid] = (T)(sum > 0.f || sum != sum ? o / sum : 0.f);
    }
    return;
  }
  const int b = blockIdx.x - sp.joins;
  const int item = b / blocks_per_item, blk = b - item * blocks_per_item;
  const int seq = item / a.c.kv_heads, hk = item - seq * a.c.kv_heads;
  const int n = cache_len(a.c, seq, nullptr);
  const int t1 = min(n, (blk + 1) * kAccTok);
  if (blk * kAccTok >= t1) {
    grid_dependency_wait();
    return;
  }
  const Parts p = find_parts(a.c, sp, seq, lane);
  float* w = a.weights + (size_t)item * a.cap;
  float add[kTokThread];                                       // the slots' weights so far
  float dist[kTokThread];
  const int q_pos = BIAS ? query_position(a, seq, n) : 0;
#pragma unroll
  for (int i = 0; i < kTokThread; ++i) {
    const int t = blk * kAccTok + i * kFinThreads + tid;
    add[i] = t < t1 ? w[t] : 0.f;
    dist[i] = BIAS ? distance(q_pos, t < t1 && a.positions ? load_late(a.positions + (size_t)item * a.cap + t) : t) : 0.f;
  }
  Reach reach{0.f, 0.f};
  if (BIAS && p.s0 == p.s1 && !sum_behind(sp, n)) reach = find_reach<kFinThreads>(a, seq, hk, n, reinterpret_cast<float*>(buf));
  grid_dependency_wait();
  const float* sc = sp.scores + ((size_t)seq * a.heads + hk * G) * sp.pitch + blk * kAccTok + tid;
  float step[kTokThread];
#pragma unroll
  for (int i = 0; i < kTokThread; ++i) step[i] = 0.f;
  for (int g0 = 0; g0 < G; g0 += kHeadsOnce) {
    // the scores of a few heads are on their way while the log-sum-exps of up to kSumsOnce are
    // made, a warp each
    float s[kHeadsOnce][kTokThread];
#pragma unroll
    for (int x = 0; x < kHeadsOnce; ++x)
#pragma unroll
      for (int i = 0; i < kTokThread; ++i) {
        const int t = blk * kAccTok + i * kFinThreads + tid;
        s[x][i] = g0 + x < G && t < t1 ? __ldcg(sc + (size_t)(g0 + x) * sp.pitch + i * kFinThreads) : -INFINITY;
      }
    if (g0 % kSumsOnce == 0) {
      if (g0) __syncthreads();
      for (int x = warp; x < kSumsOnce && g0 + x < G; x += kFinThreads / 32) {
        const int h = hk * G + g0 + x;
        const float slope2 = BIAS ? load_late(a.slopes + h) * kLog2e : 0.f;
        float m, l = 1.f;
        if (p.s0 == p.s1) {                                    // the attention kernel left it whole
          m = __ldcg(sp.lse + (size_t)seq * a.heads + h);
          if (BIAS && sum_behind(sp, n)) l = __ldcg(sp.scores + ((size_t)seq * a.heads + h) * sp.pitch + n);
        } else {
          join_ml(sp, G, h, p, lane, &m, &l);
          if (l == 0.f) m = -INFINITY;
        }
        if (lane == 0) sh[x] = make_float4(m, 1.f / l, slope2, reach.at(slope2));
      }
      __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < kHeadsOnce; ++x) {
      if (g0 + x >= G) continue;
      const float4 f = sh[g0 % kSumsOnce + x];
      if (f.x == -INFINITY) continue;                          // no visible slot (every page bad)
#pragma unroll
      for (int i = 0; i < kTokThread; ++i)
        step[i] += (BIAS ? weight_of(s[x][i], f.z, dist[i] - f.w, f.x) : ex2_approx(s[x][i] - f.x)) * f.y;
    }
  }
#pragma unroll
  for (int i = 0; i < kTokThread; ++i) {
    const int t = blk * kAccTok + i * kFinThreads + tid;
    if (t < t1) w[t] = add[i] + step[i];
  }
}

struct Plan {
  Split sp;
  size_t bytes;
};

// Query heads of a CTA: bf16 in tiles of 8 (one mma column block) or 16; fp32 up to 4.
int heads_per_tile(int G, int dtype) {
  if (dtype == SFM_DTYPE_BF16) return G <= 8 ? 8 : 16;
  return G >= 4 ? 4 : G >= 2 ? 2 : 1;
}

Plan make_plan(int n_seq, int max_tokens, int heads, int kv_heads, int head_dim, int dtype, bool weights,
               void* ws) {
  Plan p{};
  const int G = heads / kv_heads;
  Split& sp = p.sp;
  sp.hpt = heads_per_tile(G, dtype);
  sp.gt = (G + sp.hpt - 1) / sp.hpt;
  sp.hgroups = kv_heads * sp.gt;
  const int ctas = kSms * 2;                                   // one wave: two per SM, by shared memory
  sp.slots = ctas / sp.hgroups < 1 ? 1 : ctas / sp.hgroups;
  // Clusters, if they fit the device at once (those of 8 fill two thirds of it; with weights the
  // scores they hold leave room for one CTA on an SM), no CTA has more than 3 tiles (2 with 16
  // heads or with weights), and, with weights, nobody else adds to its slots.  2 sequences of 300:
  // 7.3 -> 6.2 us, and 15.9 -> 11.0 us of the host's time; 3 of 1,300, 24 heads, 3 tiles a CTA:
  // 10.1 -> 8.9 us, with weights and 6 tiles 10.2 -> 12.4; 192 heads of 12 in 288 CTAs: 17.6 -> 28.3.
  const int max_tiles = (max_tokens + kTile - 1) / kTile;
  const long long items = (long long)n_seq * sp.hgroups;
  const int most = weights ? 96 : 192, tiles = weights ? kHeldTiles : sp.hpt == 16 ? 2 : 3;
  int parts = 1;
  while (parts < kMaxParts && parts < max_tiles && items * parts * 2 <= most) parts *= 2;
  if (items * parts <= most && max_tiles <= tiles * parts && !(weights && sp.gt > 1)) {
    sp.parts = parts;
    sp.held = weights ? (max_tiles + parts - 1) / parts * kTile : 0;
    return p;
  }
  char* at = (char*)ws;
  auto take = [&](size_t floats) {
    float* r = (float*)at;
    const size_t b = (floats * sizeof(float) + 15) / 16 * 16;
    at += b;
    p.bytes += b;
    return r;
  };
  const size_t partials = (size_t)sp.slots * sp.hgroups * 2 * sp.hpt;
  sp.part = take(partials * head_dim);
  sp.ml = take(partials * 2);
  if (weights) {
    sp.lse = take((size_t)n_seq * heads);
    sp.scores = take((size_t)n_seq * heads * max_tokens);
  }
  sp.pitch = max_tokens;
  sp.joins = n_seq * heads;
  return p;
}

// The limit on shared memory belongs to the kernel, not to the call: every call sets the most that
// any call needs, so that one host thread's launch cannot meet a lower limit of another's.
template <typename K>
cudaError_t launch_attn(K kernel, int smem, const DecodeArgs& a, const Split& sp, cudaStream_t s) {
  const int head_row = sp.hpt * (int)sizeof(float);            // (hpt: fixed by the kernel)
  const int bytes = smem + head_row * sp.held, limit = smem + head_row * kHeldTiles * kTile;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
  if (e != cudaSuccess) return e;
  if (!sp.parts) return launch_dependent(kernel, (unsigned)(sp.slots * sp.hgroups), kThreads, bytes, s, a, sp);
  return launch_dependent_clusters(kernel, sp.parts, (unsigned)(a.c.n_seq * sp.hgroups * sp.parts), kThreads, bytes, s,
                                   a, sp);
}

template <int NT, bool CLUSTER>
cudaError_t launch_bf16(const DecodeArgs& a, const Split& sp, cudaStream_t s) {
  const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  auto kernel = cap && bias ? paged_attn_bf16_kernel<NT, true, true, CLUSTER>
                : cap       ? paged_attn_bf16_kernel<NT, true, false, CLUSTER>
                : bias      ? paged_attn_bf16_kernel<NT, false, true, CLUSTER>
                            : paged_attn_bf16_kernel<NT, false, false, CLUSTER>;
  return launch_attn(kernel, kSmemBf16, a, sp, s);
}

template <int DV, bool CLUSTER>
cudaError_t launch_fp32(const DecodeArgs& a, const Split& sp, cudaStream_t s) {
  if (sp.hpt == 4) return launch_attn(paged_attn_fp32_kernel<DV, 4, CLUSTER>, f32_smem<DV, 4>(), a, sp, s);
  if (sp.hpt == 2) return launch_attn(paged_attn_fp32_kernel<DV, 2, CLUSTER>, f32_smem<DV, 2>(), a, sp, s);
  return launch_attn(paged_attn_fp32_kernel<DV, 1, CLUSTER>, f32_smem<DV, 1>(), a, sp, s);
}

template <bool CLUSTER>
cudaError_t launch_any(const DecodeArgs& a, const Split& sp, int dtype, cudaStream_t s) {
  if (dtype == SFM_DTYPE_BF16)
    return sp.hpt == 8 ? launch_bf16<1, CLUSTER>(a, sp, s) : launch_bf16<2, CLUSTER>(a, sp, s);
  switch (a.c.head_dim / 32) {
    case 1: return launch_fp32<1, CLUSTER>(a, sp, s);
    case 2: return launch_fp32<2, CLUSTER>(a, sp, s);
    case 3: return launch_fp32<3, CLUSTER>(a, sp, s);
    default: return launch_fp32<4, CLUSTER>(a, sp, s);
  }
}

}  // namespace

size_t paged_attention_workspace(int n_seq, int max_tokens, int heads, int kv_heads, int head_dim, int dtype,
                                 bool weights) {
  return make_plan(n_seq, max_tokens, heads, kv_heads, head_dim, dtype, weights, nullptr).bytes;
}

int launch_paged_attention(const DecodeArgs& a, int dtype, void* workspace, cudaStream_t s) {
  const Split sp = make_plan(a.c.n_seq, a.c.max_tokens, a.heads, a.c.kv_heads, a.c.head_dim, dtype,
                             a.weights != nullptr, workspace).sp;
  {
    ProfScope ps(SFM_PROF_ATTN, s);
    const int rc = record_cuda(sp.parts ? launch_any<true>(a, sp, dtype, s) : launch_any<false>(a, sp, dtype, s));
    if (rc || sp.parts) return rc;
  }
  ProfScope ps(SFM_PROF_ATTN_MERGE, s);
  const int per_item = (a.c.max_tokens + kAccTok - 1) / kAccTok;
  const unsigned fin = (unsigned)(sp.joins + (a.weights ? a.c.n_seq * a.c.kv_heads * per_item : 0));
  const bool bias = a.weights && a.slopes;                     // (the joins do not look at it)
  auto kernel = dtype == SFM_DTYPE_BF16
                    ? (bias ? paged_finish_kernel<__nv_bfloat16, true> : paged_finish_kernel<__nv_bfloat16, false>)
                    : (bias ? paged_finish_kernel<float, true> : paged_finish_kernel<float, false>);
  return record_cuda(launch_dependent(kernel, fin, kFinThreads, 0, s, a, sp, per_item));
}

}  // namespace sfm
