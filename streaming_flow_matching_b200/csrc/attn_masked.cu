// Attention under per-query key ranges: packed documents, prefixes, causality and any
// other mask that leaves each query one interval of keys, with capped scores and a
// distance bias:
//   s_ij = q_i . k_j / sqrt(D);  s = cap tanh(s / cap);  s -= slope_h |pos_i - j|
//   O_i = sum_j softmax(s_i)_j v_j over j in [lo_i, hi_i);  an empty range gives zeros.
// Groups of query heads share a key head.
//
// bf16 (D = 128) runs on the tensor cores (tcgen05), bound by them and by the softmax
// beside them.  One CTA = two 128-row query tiles over the same key tiles: two heads of
// one group at the same rows (both tiles then have the same ranges and no key tile is
// loaded for the sake of one of them), and for an odd group's last head 256 of its rows.
// 384 threads:
//   warp 0      TMA producer: the Q tiles once, K tiles (128 keys) in a 3-stage ring, V
//               tiles in a 2-stage ring (128-byte swizzle)
//   warp 1      TMEM allocator; one lane issues S_t = Q_t K_j^T and O_t += P_t V_j (P from
//               TMEM), alternating the tiles
//   warps 4-11  softmax, thread = query row: a look at the largest product, then P against
//               the running max, which moves only when a score passes it by 2^8
//   warps 2-3   make V safe: a masked key has weight 0, and 0 x inf or 0 x NaN would
//               still reach rows that may not see it.  In key tiles that some row does not
//               see whole it scans V and replaces non-finite elements by 0; if it found
//               any, the rows that do see them get them added back at the end (a row's sum
//               with a non-finite term is that term, whatever its weight).
// The CTA's key tiles are those that the union of its rows' ranges touches (a reduction
// over the rows' bounds at the start; nothing outside is loaded); a tile inside every
// row's range is not masked.  The last query blocks go first in the grid: under a causal
// mask they have the most keys; within a block the key heads go round first, so that CTAs
// of equal work are neighbours (8,192 packed, 3 heads a group: 192 -> 186 us; the pairs'
// CTAs of one key head side by side: 204).
// Few query rows over many keys: the key tiles are cut into splits whose fp32 partials a
// second kernel joins.
//
// Measured (bf16): a block's 256 rows over 128 keys take ~1.9 us in the steady state, 1.3
// PFLOP/s, the softmax as long as the products beside it; set-up and output of a block 6 to 9
// us.  8,192 packed causal queries of 24 heads, cap 50: 187 us (166 without the cap); 8,000 with
// prefixes and a bias: 422 us (393 without); 48 queries over 2,148 keys: 17 us.
//
// fp32 runs on the CUDA cores in 32 x 64 tiles: 1,000 queries over 1,400 keys, 4 heads, D 64, in
// documents 26 us; 1,000 over 6,000, 24 heads 1.24 ms, 29.7 TFLOP/s.
#include <limits.h>
#include <math.h>

#include "attn_masked.cuh"
#include "dependent.cuh"
#include "sm100.cuh"

namespace sfm {

using namespace sm100;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ bounds

// Query i of document d (starts[d] <= pos < starts[d + 1]): keys from starts[d] up to the
// document's end, or (causal) up to max(pos + 1, starts[d] + prefix[d]).
__global__ void __launch_bounds__(256) attention_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  grid_dependency_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n_q) return;
  const int pos = a.n_kv - a.n_q + i;
  int lo = 0, hi = 0;
  int d = 0, start = 0, end = a.n_kv;
  bool in = true;
  if (a.doc_starts) {
    in = pos >= load_late(a.doc_starts) && pos < load_late(a.doc_starts + a.n_docs);
    int x = 0, y = a.n_docs;                       // the last d with starts[d] <= pos
    while (in && y - x > 1) {
      const int mid = (x + y) >> 1;
      if (load_late(a.doc_starts + mid) <= pos) x = mid;
      else y = mid;
    }
    d = x;
    if (in) {
      start = max(0, load_late(a.doc_starts + d));
      end = min(a.n_kv, load_late(a.doc_starts + d + 1));
    }
  }
  if (in) {
    lo = start;
    hi = end;
    if (a.causal) {
      const long long pre = (long long)start + (a.prefixes ? max(0, load_late(a.prefixes + d)) : 0);
      hi = (int)min((long long)end, max((long long)pos + 1, pre));
    }
  }
  a.key_lo[i] = lo;
  a.key_hi[i] = hi;
}

// ------------------------------------------------------------------ bf16, tcgen05

constexpr int BQ = 128, QT = 2, BKV = 128, D = 128;
constexpr int THREADS = 384;
constexpr int KST = 3, VST = 2;
constexpr int HALF = 128 * 64 * 2;
constexpr int TILE = 2 * HALF;
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + QT * TILE;
constexpr int OFF_V = OFF_K + KST * TILE;
constexpr int OFF_BAR = OFF_V + VST * TILE;
constexpr int SMEM = OFF_BAR + 512 + 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMaxKeySplits = 32;                               // a lane each in the join
constexpr int kSms = 148;

struct TcArgs {
  MaskedArgs m;
  int halves;          // 128-row blocks in a row block of the grid: 2 where an odd head takes both
  int units;           // CTAs of a key head and row block: the pairs of heads, block by block, an odd head
  int qblocks;         // row blocks
  int n_splits;
  float* o_part;       // [split][n_q][H][D]
  float* lse_part;     // [split][n_q][H] (log2, relative to the row's bias at bias_origin)
  int* err;
  unsigned long long wait_ns;
  int fault;
};

// the key range of query row i, empty as [0, 0)
__device__ __forceinline__ void row_range(const MaskedArgs& m, int i, int* lo, int* hi) {
  int a = m.key_lo ? max(0, load_late(m.key_lo + i)) : 0;
  int b = m.key_hi ? min(m.n_kv, load_late(m.key_hi + i)) : m.n_kv;
  if (a >= b) a = b = 0;
  *lo = a;
  *hi = b;
}

// The distance of the key whose bias is the largest in a row's range: the nearest's, or with a
// negative slope the farthest's.  A row's scores may be taken relative to the bias there: where all
// its keys are far (slope 1/2, 57,600 keys away: 41,000 in log2 units, 2^-8 apart in fp32) they would
// round away what tells the keys apart.
__device__ __forceinline__ int bias_origin(int pos, int lo, int hi, float slope) {
  if (slope < 0.f) return max(abs(pos - lo), abs(pos - (hi - 1)));
  return pos < lo ? lo - pos : pos >= hi ? pos - (hi - 1) : 0;
}

// columns [lo, hi) of up to 32 as a bit mask
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  if (lo >= hi) return 0u;
  return (0xffffffffu << lo) & (0xffffffffu >> (32 - hi));
}

__device__ __forceinline__ bool nonfinite16(uint32_t w) {   // either half's exponent all ones
  return (((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0u;
}

// tanh(x) = 1 - 2 / (2^(2 log2(e) x) + 1), and near 0, where that difference would lose what
// a large cap multiplies, x - x^3 / 3 + 2 x^5 / 15 (the next term is 17 x^7 / 315)
__device__ __forceinline__ float tanh_ex2(float x) {
  const float e = ex2_approx(x * (2.f * kLog2e));
  const float y = x * x;
  return fabsf(x) < 0.06f ? x * fmaf(y, fmaf(y, 2.f / 15.f, -1.f / 3.f), 1.f) : 1.f - __fdividef(2.f, e + 1.f);
}

// pairs of fp32 in one instruction
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void get(float* lo, float* hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

// tanh(y) = y P(y^2) on |y| <= 0.7, P a cubic fitted (by reweighted least squares) for the least
// maximum of the relative error, 6.7e-6: a score of 50 moves by 5e-4 in log2 units, where P's
// rounding to bf16 is worth 6e-3.  (One degree more, on 0.8: 2 % slower.)
constexpr float kTanhRange = 0.7f;
__device__ constexpr float kTanhC[4] = {0.999993311f, -0.332890456f, 0.128642044f, -0.037290386f};

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// what turns a row's raw products x into log2 scores
struct ScoreMap {
  float sc;         // scale log2(e), or scale / cap
  float cap2;       // cap log2(e)
  float slope2;     // slope log2(e)
  float x_lim;      // |x| up to which the polynomial serves: 0.7 cap / scale
};

template <bool CAP, bool BIAS>
__device__ __forceinline__ float score2(const ScoreMap& sm, float x, float fq, float col) {
  float z = x * sm.sc;
  if (CAP) z = sm.cap2 * tanh_ex2(z);
  if (BIAS) z = fmaf(-sm.slope2, fabsf(fq - col), z);
  return z;
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(THREADS, 1)
    attn_masked_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TcArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_ok = v_full + VST;      // V landed and safe to multiply
  uint64_t* v_empty = v_ok + VST;
  uint64_t* s_full = v_empty + VST;   // [QT]
  uint64_t* p_full = s_full + QT;     // [QT]
  uint64_t* o_done = p_full + QT;     // [QT]
  uint64_t* drain = o_done + QT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* dirty = reinterpret_cast<volatile int*>(tmem_slot + 2);   // non-finite V was replaced
  int* red = reinterpret_cast<int*>(tmem_slot + 4);                       // [4][8]

  const MaskedArgs& m_ = args.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rem = blockIdx.x;
  const int hk = rem % m_.kv_heads;
  rem /= m_.kv_heads;
  const int unit = rem % args.units;
  rem /= args.units;
  const int split = rem % args.n_splits;
  const int qb = args.qblocks - 1 - rem / args.n_splits;
  const int G = m_.heads / m_.kv_heads;
  const bool paired = unit < G / 2 * args.halves;
  const int h_a = hk * G + (paired ? unit / args.halves * 2 : G - 1);       // head of tile A
  const int dh = paired ? 1 : 0;                               // tile B: head h_a + dh,
  const int dr = paired ? 0 : BQ;                              //         rows + dr
  const int row0 = (qb * args.halves + (paired ? unit % args.halves : 0)) * BQ;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < KST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_ok[i], 2);
      mbar_init(&v_empty[i], 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(drain, 1);
    *abort = 0;
    *dirty = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  // only CTA-local set-up so far: the kernel before (which may have made the ranges, q, k, v) is
  // waited for here
  grid_dependency_wait();
  // the Q tiles do not wait for the ranges (the barrier's own initialising thread loads them)
  const bool loads = !(args.fault & SFM_FAULT_ATTN_NO_LOADS);
  if (threadIdx.x == 0) {
    if (loads) {
      mbar_arrive_expect_tx(q_full, QT * TILE);
      for (int t = 0; t < QT; ++t) {
        tma_load_3d(base + OFF_Q + t * TILE, &map_q, q_full, 0, h_a + t * dh, row0 + t * dr);
        tma_load_3d(base + OFF_Q + t * TILE + HALF, &map_q, q_full, 64, h_a + t * dh, row0 + t * dr);
      }
    }
    tma_prefetch(&map_k);
    tma_prefetch(&map_v);
  }
  // the rows' key ranges: this thread's row (softmax warps), and over the CTA's rows the
  // union and the intersection
  const int st = (warp - 4) >> 2;                              // tile of a softmax warp
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;
  int my_lo = 0, my_hi = m_.n_kv;
  bool live = false;                                           // the row exists
  if (warp >= 4) {
    const int i = row0 + st * dr + r;
    int u_lo = INT_MAX, u_hi = 0, n_lo = 0, n_hi = INT_MAX;
    if (i < m_.n_q) {                                          // rows past the end see all, write nothing
      live = true;
      row_range(m_, i, &my_lo, &my_hi);
      if (my_hi > my_lo) {                                     // an empty row's products are not used
        u_lo = n_lo = my_lo;
        u_hi = n_hi = my_hi;
      }
    }
    u_lo = __reduce_min_sync(0xffffffffu, u_lo);
    u_hi = __reduce_max_sync(0xffffffffu, u_hi);
    n_lo = __reduce_max_sync(0xffffffffu, n_lo);
    n_hi = __reduce_min_sync(0xffffffffu, n_hi);
    if (lane == 0) {
      red[0 * 8 + warp - 4] = u_lo;
      red[1 * 8 + warp - 4] = u_hi;
      red[2 * 8 + warp - 4] = n_lo;
      red[3 * 8 + warp - 4] = n_hi;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // key tiles that some row of each query tile sees, and keys that all its rows see
  int see0[QT], see1[QT], full_lo[QT], full_hi[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    int lo = INT_MAX, hi = 0;
    full_lo[t] = 0;
    full_hi[t] = INT_MAX;
#pragma unroll
    for (int w = 4 * t; w < 4 * t + 4; ++w) {
      lo = min(lo, red[w]);
      hi = max(hi, red[8 + w]);
      full_lo[t] = max(full_lo[t], red[16 + w]);
      full_hi[t] = min(full_hi[t], red[24 + w]);
    }
    see0[t] = lo < hi ? lo / BKV : INT_MAX;
    see1[t] = lo < hi ? (hi + BKV - 1) / BKV : 0;
  }
  const int u1 = max(see1[0], see1[1]);
  const int u0 = min(min(see0[0], see0[1]), u1);
  const int tps = (u1 - u0 + args.n_splits - 1) / args.n_splits;
  const int t0 = min(u1, u0 + split * tps);
  const int T = min(u1, t0 + tps) - t0;
  // The order of the key tiles.  With a bias the nearest keys go first -- from the last
  // row's own tile back, then on from there -- as their scores are the largest: the running
  // max then hardly moves, where in ascending order it would in every tile of a steep head.
  int near = 0;
  if (BIAS && T > 0) {
    const int pos = m_.n_kv - m_.n_q + min(row0 + dr + BQ, m_.n_q) - 1;
    near = min(max(pos / BKV - t0, 0), T - 1);
  }
  auto tile_at = [&](int i) { return !BIAS ? t0 + i : t0 + (i <= near ? near - i : i); };
  // some row of query tile t sees the key tile
  auto sees = [&](int t, int k) { return k >= see0[t] && k < see1[t]; };
  // a key tile (the j-th in order) that the query tiles which see anything of it see whole
  auto whole = [&](int j) {
    const int k = tile_at(j);
    bool w = true;
#pragma unroll
    for (int t = 0; t < QT; ++t) w = w && (!sees(t, k) || (k * BKV >= full_lo[t] && (k + 1) * BKV <= full_hi[t]));
    return w;
  };

  if (warp == 0) {
    if (lane == 0 && T == 0 && loads) mbar_drain(q_full, 0, args.wait_ns);   // nothing else waits for Q
    if (lane == 0 && T > 0 && loads) {
      // ---------------- TMA producer ----------------
      int kp[KST], vp[VST];
      for (int i = 0; i < KST; ++i) kp[i] = -1;
      for (int i = 0; i < VST; ++i) vp[i] = -1;
      bool ok = true;
      auto load_k = [&](int i) -> bool {
        const int s = i % KST;
        const uint32_t par = (uint32_t)((i / KST) & 1);
        if (!mbar_wait(&k_empty[s], par ^ 1u, abort, args.err, 0x401, args.wait_ns)) return false;
        mbar_arrive_expect_tx(&k_full[s], TILE);
        tma_load_3d(base + OFF_K + s * TILE, &map_k, &k_full[s], 0, hk, tile_at(i) * BKV);
        tma_load_3d(base + OFF_K + s * TILE + HALF, &map_k, &k_full[s], 64, hk, tile_at(i) * BKV);
        kp[s] = (int)par;
        return true;
      };
      auto load_v = [&](int i) -> bool {
        const int s = i % VST;
        const uint32_t par = (uint32_t)((i / VST) & 1);
        if (!mbar_wait(&v_empty[s], par ^ 1u, abort, args.err, 0x402, args.wait_ns)) return false;
        mbar_arrive_expect_tx(&v_full[s], TILE);
        tma_load_3d(base + OFF_V + s * TILE, &map_v, &v_full[s], 0, hk, tile_at(i) * BKV);
        tma_load_3d(base + OFF_V + s * TILE + HALF, &map_v, &v_full[s], 64, hk, tile_at(i) * BKV);
        vp[s] = (int)par;
        return true;
      };
      ok = load_k(0);
      if (ok && T > 1) ok = load_k(1);
      for (int j = 0; j < T && ok; ++j) {
        ok = load_v(j);
        if (ok && j + 2 < T) ok = load_k(j + 2);
      }
      if (!ok) {   // unwinding: let issued loads land before the CTA exits
        mbar_drain(q_full, 0, args.wait_ns);
        for (int i = 0; i < KST; ++i)
          if (kp[i] >= 0) mbar_drain(&k_full[i], (uint32_t)kp[i], args.wait_ns);
        for (int i = 0; i < VST; ++i)
          if (vp[i] >= 0) mbar_drain(&v_full[i], (uint32_t)vp[i], args.wait_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && T > 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc_s = idesc_bf16(BQ, BKV, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(BQ, D, false, true);
      bool ok = mbar_wait(q_full, 0, abort, args.err, 0x403, args.wait_ns), issued = false;
      int gt[QT] = {0, 0};                                     // S products issued for each query tile
      bool pv[QT] = {false, false};                            // the tile has had a P V
      auto issue_s = [&](int t, int ks) -> bool {              // S_t = Q_t K^T from K stage ks
        // S_t overwrites P_t: wait until its P V has completed
        if (pv[t] && !mbar_wait(&o_done[t], (uint32_t)((gt[t] - 1) & 1), abort, args.err, 0x40B, args.wait_ns))
          return false;
        tc_fence_after();
        const uint32_t qa = base + OFF_Q + t * TILE, ka = base + OFF_K + ks * TILE;
        const uint32_t d = tmem + (uint32_t)(t * 256);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t sub = (uint32_t)(kk >> 2) * HALF;
          const uint64_t da = sw128_desc(qa + sub, 16, 1024) + (uint64_t)(2 * (kk & 3));
          const uint64_t db = sw128_desc(ka + sub, 16, 1024) + (uint64_t)(2 * (kk & 3));
          umma_bf16(d, da, db, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[t]);
        ++gt[t];
        issued = true;
        return true;
      };
      if (ok && (ok = mbar_wait(&k_full[0], 0, abort, args.err, 0x404, args.wait_ns))) {
        const int k0 = tile_at(0);
#pragma unroll
        for (int t = 0; t < QT; ++t)
          if (sees(t, k0)) issue_s(t, 0);
        umma_commit(&k_empty[0]);
      }
      // per key tile j: P_A V, S_A(j+1), P_B V, S_B(j+1) -- tile A never waits on tile B, so
      // the two softmax warpgroups run half a period apart; a query tile skips the key tiles
      // that it sees nothing of
      for (int j = 0; j < T && ok; ++j) {
        const int vs = j % VST;
        const bool more = j + 1 < T;
        const int ks = (j + 1) % KST;
        const int k0 = tile_at(j), k1 = tile_at(j + 1);
        const uint32_t vpar = (uint32_t)((j / VST) & 1);
        if (!mbar_wait(&v_full[vs], vpar, abort, args.err, 0x406, args.wait_ns) ||
            !mbar_wait(&v_ok[vs], vpar, abort, args.err, 0x40C, args.wait_ns)) {
          ok = false;
          break;
        }
        const uint32_t va = base + OFF_V + vs * TILE;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          if (ok && sees(t, k0)) {
            ok = mbar_wait(&p_full[t], (uint32_t)((gt[t] - 1) & 1), abort, args.err, 0x405, args.wait_ns);
            if (ok) {
              tc_fence_after();
              const uint32_t pa = tmem + (uint32_t)(t * 256);
              const uint32_t d = tmem + (uint32_t)(t * 256 + 128);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint64_t db = sw128_desc(va + (uint32_t)kk * 2048u, HALF, 1024);
                umma_bf16_tmem_a(d, pa + (uint32_t)(kk * 8), db, idesc_o, (pv[t] || kk > 0) ? 1u : 0u);
              }
              umma_commit(&o_done[t]);
              pv[t] = true;
            }
          }
          if (ok && more && t == QT - 1) umma_commit(&v_empty[vs]);   // (nothing waits for the last)
          if (ok && more) {
            if (t == 0)
              ok = mbar_wait(&k_full[ks], (uint32_t)(((j + 1) / KST) & 1), abort, args.err, 0x404, args.wait_ns);
            if (ok && sees(t, k1)) ok = issue_s(t, ks);
            if (ok && t == QT - 1) umma_commit(&k_empty[ks]);
          }
        }
      }
      if (!ok && issued) {
        umma_commit(drain);
        mbar_drain(drain, 0, args.wait_ns);
      }
    }
  } else if (warp < 4) {
    // ---------------- V made safe: a half of each tile per warp ----------------
    for (int j = 0; j < T; ++j) {
      const int vs = j % VST;
      if (!__all_sync(0xffffffffu, mbar_wait(&v_full[vs], (uint32_t)((j / VST) & 1), abort, args.err, 0x409, args.wait_ns)))
        break;
      if (!whole(j)) {
        uint4* p = reinterpret_cast<uint4*>(smem + OFF_V + vs * TILE + (warp - 2) * HALF);
        bool found = false;
#pragma unroll 8
        for (int i = lane; i < HALF / 16; i += 32) {
          uint4 x = p[i];
          if (nonfinite16(x.x) | nonfinite16(x.y) | nonfinite16(x.z) | nonfinite16(x.w)) {
            uint32_t* w = &x.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xffff0000u;
              if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0x0000ffffu;
            }
            p[i] = x;
            found = true;
          }
        }
        if (__any_sync(0xffffffffu, found)) {
          if (lane == 0) *dirty = 1;
          fence_proxy_async_smem();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_ok[vs]);
    }
  } else if (warp >= 4) {
    // ---------------- softmax + output (thread = query row of tile st) ----------------
    const int t = st;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t col_s = (uint32_t)(t * 256), col_o = col_s + 128;
    const int h = h_a + t * dh;
    const int row_t = row0 + t * dr;                           // first row of the tile
    const int my_see0 = t ? see0[1] : see0[0], my_see1 = t ? see1[1] : see1[0];
    const int w_lo = __reduce_max_sync(0xffffffffu, my_lo), w_hi = __reduce_min_sync(0xffffffffu, my_hi);
    // what any row of the warp sees (an empty row, or one past the end: nothing)
    const int any_lo = __reduce_min_sync(0xffffffffu, live && my_hi > my_lo ? my_lo : INT_MAX);
    const int any_hi = __reduce_max_sync(0xffffffffu, live ? my_hi : 0);
    ScoreMap sm;
    const float scale = 0.08838834764831845f;                  // 1 / sqrt(128)
    sm.sc = CAP ? scale / m_.softcap : scale * kLog2e;
    sm.cap2 = m_.softcap * kLog2e;
    sm.slope2 = BIAS ? load_late(m_.slopes + h) * kLog2e : 0.f;
    sm.x_lim = CAP ? kTanhRange * m_.softcap / scale : 0.f;
    F2 poly[4];                                                // kTanhC in terms of x, times cap log2(e)
    if (CAP) {
      const float y2 = sm.sc * sm.sc;
      float f = sm.cap2 * sm.sc;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        poly[i] = F2(kTanhC[i] * f, kTanhC[i] * f);
        f *= y2;
      }
    }
    const F2 sc2(sm.sc, sm.sc);
    const int my_pos = m_.n_kv - m_.n_q + row_t + r;
    const int w_pos0 = my_pos - lane, w_pos1 = w_pos0 + 31;    // positions of the warp's rows
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int seen = 0;                                              // key tiles of this query tile so far
    for (int j = 0; j < T && ok; ++j) {
      if (!(tile_at(j) >= my_see0 && tile_at(j) < my_see1)) continue;
      const int key0 = tile_at(j) * BKV;
      const bool masked = !(key0 >= w_lo && key0 + BKV <= w_hi);
      const bool nothing = key0 >= any_hi || key0 + BKV <= any_lo;
      const int lo = my_lo - key0, hi = my_hi - key0;
      const float fq = (float)(my_pos - key0);
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[t], (uint32_t)(seen & 1), abort, args.err, 0x407, args.wait_ns))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (nothing) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(tmem + lane_base + col_s + c * 16, pk);
      } else {
        // The row's max may stay where it is while no score passes it by 2^8: first a bound
        // from the largest product (magnitude, with a cap) and the largest bias of the tile,
        // and only if that does not settle it the scores' own maximum.
        float top = CAP ? 0.f : -INFINITY;
        {
          uint32_t u[2][32];
          tmem_ld32(tmem + lane_base + col_s, u[0]);
          tmem_wait_ld(u[0]);
          float m4[4] = {top, top, top, top};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c + 1 < 4) tmem_ld32(tmem + lane_base + col_s + (c + 1) * 32, u[(c + 1) & 1]);
            const float* sv = reinterpret_cast<const float*>(u[c & 1]);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              m4[(i >> 1) & 3] = CAP ? fmax3(m4[(i >> 1) & 3], fabsf(sv[i]), fabsf(sv[i + 1]))
                                     : fmax3(m4[(i >> 1) & 3], sv[i], sv[i + 1]);
            if (c + 1 < 4) tmem_wait_ld(u[(c + 1) & 1]);
          }
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        float bound = CAP ? sm.cap2 * fminf(top * sm.sc, 1.f) : top * sm.sc;
        if (BIAS) {
          const float d0 = fabsf(fq), d1 = fabsf(fq - (float)(BKV - 1));
          const bool inside = fq >= 0.f && fq <= (float)(BKV - 1);
          bound -= sm.slope2 * (sm.slope2 < 0.f ? fmaxf(d0, d1) : inside ? 0.f : fminf(d0, d1));
        }
        if (__any_sync(0xffffffffu, !(bound <= m + kRescaleLog2))) {
          float mx = -INFINITY;                                // of the visible scores
          // With nothing masked and no bias the bound is itself the largest score, or (cap) as
          // far above it that no score is lost under 2^-126 while it is small.
          if (!BIAS && !masked && __all_sync(0xffffffffu, !CAP || bound <= 40.f)) {
            mx = bound;
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t w[32];
              tmem_ld32(tmem + lane_base + col_s + c * 32, w);
              tmem_wait_ld(w);
              const float* sv = reinterpret_cast<const float*>(w);
              const uint32_t bits = range_bits(lo - c * 32, hi - c * 32);
              const float fc = fq - (float)(c * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                // without a bias the score rises with the product: the largest product does
                const float z = BIAS ? score2<CAP, BIAS>(sm, sv[i], fc, (float)i) : sv[i];
                if ((bits >> i) & 1u) mx = fmaxf(mx, z);
              }
            }
            if (!BIAS) mx = score2<CAP, BIAS>(sm, mx, 0.f, 0.f);
          }
          if (__any_sync(0xffffffffu, mx > m + kRescaleLog2)) {   // also from m = -inf
            const float m_new = fmaxf(m, mx);
            const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);   // O, l are 0 then
            l *= alpha;
            m = m_new;
            if (seen > 0) {
              // O_t's previous P V has completed (S_t(j) was issued after it): rescale it
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_base + col_o + c * 32, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st32(tmem + lane_base + col_o + c * 32, o);
              }
            }
          }
        }
        // P = 2^(z - m) of the 128 columns, written over S as packed bf16 as it is made (the
        // 16 columns a chunk of 32 becomes have been read); masked columns give 0.
        // FAST: the bias linear in the column, as where the warp's rows lie on one side of the
        // keys (|slope fq| kept below 2^14: the sum then rounds at 2^-10 at most), and the cap
        // by its polynomial; else the general forms.
        const float side = key0 + BKV - 1 <= w_pos0 ? 1.f : key0 >= w_pos1 ? -1.f : 0.f;
        bool fast = true;
        if (BIAS) fast = side != 0.f && __all_sync(0xffffffffu, fabsf(sm.slope2 * fq) < 16384.f);
        if (CAP) fast = fast && __all_sync(0xffffffffu, top <= sm.x_lim);
        // The common form is unrolled over all 128 columns, the others (and all with a bias) over
        // 64: unrolled further they do not fit the instruction cache once the warps of a tile are
        // in different forms (a row short of its neighbours then cost its block 1 us a tile, 3 us
        // capped).
        auto make_p = [&](auto is_masked, auto is_fast) {
          constexpr bool MASKED = decltype(is_masked)::value, FAST = decltype(is_fast)::value;
          constexpr int ROUNDS = MASKED || BIAS ? 2 : 1, CHUNKS = 4 / ROUNDS, COLS = 32 * CHUNKS;
          F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
          const float neg_m = m == -INFINITY ? 0.f : -m;
          const float tilt = sm.slope2 * side;                 // z gains tilt (col - fq)
          const F2 step4(4.f * tilt, 4.f * tilt);
          uint32_t u[2][32];
          tmem_ld32(tmem + lane_base + col_s, u[0]);
          tmem_wait_ld(u[0]);
#pragma unroll 1
          for (int round = 0; round < ROUNDS; ++round) {
            const float fr = fq - (float)(COLS * round);
            const float t0 = BIAS && FAST ? fmaf(-tilt, fr, neg_m) : neg_m;
            const uint32_t src = tmem + lane_base + col_s + (uint32_t)(COLS * round);
            const uint32_t dst = tmem + lane_base + col_s + (uint32_t)(COLS / 2 * round);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
              // (CHUNKS is even: the next round's first chunk goes where this one's did)
              const bool next = c + 1 < CHUNKS || round + 1 < ROUNDS;
              if (next) tmem_ld32(src + (c + 1) * 32, u[(c + 1) & 1]);
              const float* sv = reinterpret_cast<const float*>(u[c & 1]);
              const uint32_t bits = MASKED ? range_bits(lo - COLS * round - c * 32, hi - COLS * round - c * 32) : 0u;
              uint32_t pk[16];
              F2 ramp[2];
              if (BIAS && FAST && !CAP) {
                const float c0 = (float)(c * 32);
                ramp[0] = F2(fmaf(tilt, c0, t0), fmaf(tilt, c0 + 1.f, t0));
                ramp[1] = F2(fmaf(tilt, c0 + 2.f, t0), fmaf(tilt, c0 + 3.f, t0));
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                F2 t(t0, t0);
                if (BIAS && FAST && !CAP) {
                  // two chains of pairs, 4 columns a step, begun anew every 32 columns: half the
                  // instructions of a product per column, and at most 8 roundings (8,000 queries
                  // with prefixes: 445 -> 419 us; with a cap beside it the registers run short)
                  t = ramp[i & 1];
                  ramp[i & 1] = add2(t, step4);
                } else if (BIAS) {
                  const float c0 = (float)(c * 32 + 2 * i), c1 = c0 + 1.f;
                  t = FAST ? F2(fmaf(tilt, c0, t0), fmaf(tilt, c1, t0))
                           : F2(fmaf(-sm.slope2, fabsf(fr - c0), t0), fmaf(-sm.slope2, fabsf(fr - c1), t0));
                }
                const float x0 = sv[2 * i], x1 = sv[2 * i + 1];
                const F2 x(x0, x1);
                F2 z;
                if (!CAP) {
                  z = fma2(x, sc2, t);
                } else if (FAST) {
                  const F2 y2 = mul2(x, x);
                  F2 w = poly[3];
#pragma unroll
                  for (int k = 2; k >= 0; --k) w = fma2(w, y2, poly[k]);
                  z = fma2(x, w, t);
                } else {
                  z = fma2(F2(sm.cap2, sm.cap2), F2(tanh_ex2(x0 * sm.sc), tanh_ex2(x1 * sm.sc)), t);
                }
                float p0, p1;
                z.get(&p0, &p1);
                if (MASKED) {
                  if (!((bits >> (2 * i)) & 1u)) p0 = -INFINITY;
                  if (!((bits >> (2 * i + 1)) & 1u)) p1 = -INFINITY;
                }
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                sum[i & 1] = add2(sum[i & 1], F2(p0, p1));
                pk[i] = pack_bf16x2(p0, p1);
              }
              if (next) tmem_wait_ld(u[(c + 1) & 1]);
              tmem_st16(dst + c * 16, pk);
            }
          }
          float a0, a1;
          add2(sum[0], sum[1]).get(&a0, &a1);
          l += a0 + a1;
        };
        if (fast && !masked) make_p(No{}, Yes{});
        else if (fast) make_p(Yes{}, Yes{});
        else if (CAP || BIAS) make_p(Yes{}, No{});
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
      ++seen;
    }
    // ---- output ----
    if (ok && seen > 0) {
      if (!__all_sync(0xffffffffu, mbar_wait(&o_done[t], (uint32_t)((seen - 1) & 1), abort, args.err, 0x40A, args.wait_ns))) ok = false;
      tc_fence_after();
    }
    const int q_rows = min(BQ, m_.n_q - row_t) - quarter * 32;  // of this warp; may be <= 0
    const size_t ld = (size_t)m_.heads * D;
    const bool have = ok && seen > 0 && (l > 0.f || l != l);
    const float inv = have ? 1.f / l : 0.f;
    const bool parts = args.n_splits > 1;
    if (ok && seen > 0) {
      // The warp's 32 normalised rows go through shared memory, 256 bytes of each at a time (a
      // whole bf16 row, or half of a partial's), so that whole lines are written.  The place
      // is the tile's own Q: its last S was issued before the P V that o_done signalled.  (The
      // other tile may still be at work on its own Q and on the K and V stages.)  16-byte
      // piece q of row i is at q ^ (i & 7): no bank conflicts either way.
      uint4* stage = reinterpret_cast<uint4*>(smem + OFF_Q + t * TILE) + (warp & 3) * (32 * 16);
      const bool fix = *dirty != 0;
      const size_t row_bytes = ld * (parts ? 4 : 2);
      char* out = (parts ? reinterpret_cast<char*>(args.o_part + (size_t)split * m_.n_q * ld)
                         : reinterpret_cast<char*>(m_.o)) +
                  (size_t)(row_t + quarter * 32) * row_bytes + (size_t)h * D * (parts ? 4 : 2) + (lane & 15) * 16;
      // the non-finite elements of V that row rr of the warp sees in columns [c, c + 4), in the
      // tiles they were taken out of: the row's sum is then theirs, whatever their weights
      auto add_back = [&](int rr, int c, float4* f) {
        const int lo = __shfl_sync(0xffffffffu, my_lo, rr), hi = __shfl_sync(0xffffffffu, my_hi, rr);
        for (int j = 0; j < T; ++j) {
          if (whole(j)) continue;
          const int k0 = tile_at(j) * BKV, k1 = min(hi, k0 + BKV);
          for (int k = max(lo, k0); k < k1; ++k) {
            const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(m_.v) +
                                                            ((size_t)k * m_.kv_heads + hk) * D + c);
            if (nonfinite16(x.x) || nonfinite16(x.y)) {
              const float v0 = __uint_as_float(x.x << 16), v1 = __uint_as_float(x.x & 0xffff0000u);
              const float v2 = __uint_as_float(x.y << 16), v3 = __uint_as_float(x.y & 0xffff0000u);
              if (!isfinite(v0)) f->x += v0;
              if (!isfinite(v1)) f->y += v1;
              if (!isfinite(v2)) f->z += v2;
              if (!isfinite(v3)) f->w += v3;
            }
          }
        }
      };
#pragma unroll 1
      for (int round = 0; round < (parts ? 2 : 1); ++round) {
        const int cols = parts ? 64 : 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 32 >= cols) break;                           // warp-uniform
          uint32_t u[32];
          tmem_ld32(tmem + lane_base + col_o + round * 64 + c * 32, u);
          tmem_wait_ld(u);
          float* f = reinterpret_cast<float*>(u);
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = have ? f[i] * inv : 0.f;
          if (parts) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              stage[lane * 16 + ((c * 8 + q) ^ (lane & 7))] = make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              stage[lane * 16 + ((c * 4 + q) ^ (lane & 7))] =
                  make_uint4(pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                             pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7]));
          }
        }
        __syncwarp();
        if (!fix) {
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            const int rr = 2 * i + (lane >> 4);
            if (rr < q_rows)
              *reinterpret_cast<uint4*>(out + rr * row_bytes) = stage[rr * 16 + ((lane & 15) ^ (rr & 7))];
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 16; ++i) {
            const int rr = 2 * i + (lane >> 4);
            const uint4 x = stage[rr * 16 + ((lane & 15) ^ (rr & 7))];
            float4 f = *reinterpret_cast<const float4*>(&x);
            if (parts) {
              add_back(rr, round * 64 + (lane & 15) * 4, &f);
              if (rr < q_rows) *reinterpret_cast<float4*>(out + rr * row_bytes) = f;
              continue;
            }
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              const uint32_t wa = e ? x.z : x.x, wb = e ? x.w : x.y;
              f = make_float4(__uint_as_float(wa << 16), __uint_as_float(wa & 0xffff0000u),
                              __uint_as_float(wb << 16), __uint_as_float(wb & 0xffff0000u));
              add_back(rr, (lane & 15) * 8 + e * 4, &f);
              if (rr < q_rows)
                *reinterpret_cast<uint2*>(out + rr * row_bytes + e * 8) =
                    make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
            }
          }
        }
        out += 256;
        __syncwarp();
      }
    } else if (lane < q_rows) {
      // No row of the tile sees a key (its Q may still be landing: no place to stage), or
      // unwinding after a timed-out wait: zeros, written directly.
      const size_t at = (size_t)(row_t + r) * ld + (size_t)h * D;
      uint4* d = parts ? reinterpret_cast<uint4*>(args.o_part + (size_t)split * m_.n_q * ld + at)
                       : reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(m_.o) + at);
      for (int q = 0; q < D / (parts ? 4 : 8); ++q) d[q] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (lane < q_rows && parts) {
      // relative to the bias at its origin: m alone may be so large that the sum would round away
      const float top = BIAS ? fmaf(sm.slope2, (float)bias_origin(my_pos, my_lo, my_hi, sm.slope2), m) : m;
      args.lse_part[((size_t)split * m_.n_q + row_t + r) * m_.heads + h] = have ? top + log2f(l) : -INFINITY;
    }
  }

  tc_fence_before();
  __syncwarp();                                                // the roles' single lanes are back
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the splits of a (row, head): one warp each, 4 dims per lane (lanes past the head's
// dims idle).  A row no split of which saw a key gets zeros.
template <typename T>
__global__ void __launch_bounds__(256)
    masked_join_kernel(const float* o_part, const float* lse_part,
                       T* o, long long rows_heads, int dim, int n_splits) {
  grid_dependency_wait();
  const long long gw = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= rows_heads) return;
  // lane s holds split s's log-sum-exp (at most 32 splits)
  const float mine = lane < n_splits ? lse_part[lane * rows_heads + gw] : -INFINITY;
  float mx = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  const bool bad = __any_sync(0xffffffffu, mine != mine);      // some split's sum was not a number
  const float mine_w = mine == -INFINITY ? 0.f : exp2f(mine - mx);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < n_splits; ++s) {
    const float w = __shfl_sync(0xffffffffu, mine_w, s);
    const bool none = __shfl_sync(0xffffffffu, mine == -INFINITY ? 1 : 0, s);
    if (none || lane * 4 >= dim) continue;                     // the split saw no key of this row
    const float4 p = reinterpret_cast<const float4*>(o_part + (s * rows_heads + gw) * dim)[lane];
    sum += w;
    acc.x = fmaf(w, p.x, acc.x);
    acc.y = fmaf(w, p.y, acc.y);
    acc.z = fmaf(w, p.z, acc.z);
    acc.w = fmaf(w, p.w, acc.w);
  }
  if (lane * 4 >= dim) return;
  const float inv = bad ? NAN : sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  if constexpr (sizeof(T) == 2)
    reinterpret_cast<uint2*>(o + gw * dim)[lane] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  else
    reinterpret_cast<float4*>(o + gw * dim)[lane] = acc;
}

template <typename T>
int launch_join(const float* o_part, const float* lse_part, void* o, long long rows_heads, int dim, int n_splits,
                cudaStream_t s) {
  ProfScope ps(SFM_PROF_ATTN_MERGE, s);
  return record_cuda(launch_dependent(masked_join_kernel<T>, (unsigned)((rows_heads * 32 + 255) / 256), 256, 0, s,
                                      o_part, lse_part, (T*)o, rows_heads, dim, n_splits));
}

// ------------------------------------------------------------------ fp32, CUDA cores

constexpr int FM = 32, FN = 64, FTHREADS = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
// tanh to about 4e-7 of its value without a branch: as tanh_ex2, the series up to x^9 (the next
// term is 1382 x^11 / 155925, 6e-8 of x at 0.3)
__device__ __forceinline__ float tanh_f32(float x) {
  const float y = x * x;
  float p = fmaf(y, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(p, y, 2.f / 15.f);
  p = fmaf(p, y, -1.f / 3.f);
  const float big = 1.f - __fdividef(2.f, ex2_approx(x * (2.f * kLog2e)) + 1.f);
  return fabsf(x) < 0.3f ? fmaf(x * y, p, x) : big;
}

__device__ __forceinline__ void ld_pairs(const void* src, F2 (&d)[2]) {      // 16 bytes of shared memory
  const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(src);
  d[0].v = x.x;
  d[1].v = x.y;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DV>
constexpr int f32_smem() {
  return ((FM + 2 * FN) * (32 * DV + 4) + FM * (FN + 4)) * 4;
}

// 32 query rows x 64 keys per step and key splits (64 rows without splits left half the SMs
// without work at 1,000 queries of four heads: 68 us); thread (ty, tx) of 8 x 16 holds 4 rows x
// 4 scores (keys tx + 16 k) and 4 rows x 2 DV outputs, as pairs of fp32 (even and odd dims of a
// score; neighbouring dims of an output).  K and V come by asynchronous copies, each while the
// other is at work; a tile alone on its SM takes 3.4 us (5 with loads in pairs through registers),
// bound then by latency, and among others by shared memory: a product of 2 x 2 fp32 per 16 bytes
// read is half of what the FMA pipes could take.  Masked scores are skipped by weight 0 and
// masked V rows by staging zeros for keys that no row of the tile sees; a key that only
// some rows see and that holds a non-finite value is left out row by row.
// n_splits > 1: the tiles of the rows' union are cut into that many runs, each writing a
// normalised partial and its log-sum-exp.
template <int DV>
__global__ void __launch_bounds__(FTHREADS)
    attn_masked_f32_kernel(const __grid_constant__ MaskedArgs a, int n_splits, float* o_part,
                           float* lse_part) {
  grid_dependency_wait();
  constexpr int DD = 32 * DV, P = DD + 4, SP = FN + 4;
  extern __shared__ __align__(16) float fsm[];
  float* qs = fsm;
  float* ks = qs + FM * P;
  float* vs = ks + FN * P;
  float* ps = vs + FN * P;
  __shared__ int red[2][FTHREADS / 32];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int h = blockIdx.x % a.heads;
  const int split = blockIdx.x / a.heads % n_splits;
  const int qblocks = (a.n_q + FM - 1) / FM;
  const int qb = qblocks - 1 - blockIdx.x / a.heads / n_splits;
  const int row0 = qb * FM;
  const int hk = h / (a.heads / a.kv_heads);
  const size_t ldq = (size_t)a.heads * DD, ldk = (size_t)a.kv_heads * DD;
  const float* q = reinterpret_cast<const float*>(a.q) + (size_t)h * DD;
  const float* k = reinterpret_cast<const float*>(a.k) + (size_t)hk * DD;
  const float* v = reinterpret_cast<const float*>(a.v) + (size_t)hk * DD;
  int lo[4], hi[4];
  int u_lo = INT_MAX, u_hi = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = hi[i] = 0;
    const int row = row0 + ty * 4 + i;
    if (row < a.n_q) row_range(a, row, &lo[i], &hi[i]);
    if (hi[i] > lo[i]) {
      u_lo = min(u_lo, lo[i]);
      u_hi = max(u_hi, hi[i]);
    }
  }
  u_lo = __reduce_min_sync(0xffffffffu, u_lo);
  u_hi = __reduce_max_sync(0xffffffffu, u_hi);
  if ((tid & 31) == 0) {
    red[0][tid >> 5] = u_lo;
    red[1][tid >> 5] = u_hi;
  }
  for (int x = tid; x < FM * (DD / 4); x += FTHREADS) {
    const int rr = x / (DD / 4), c = x - rr * (DD / 4);
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + rr < a.n_q) f = *reinterpret_cast<const float4*>(q + (size_t)(row0 + rr) * ldq + 4 * c);
    *reinterpret_cast<float4*>(qs + rr * P + 4 * c) = f;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < FTHREADS / 32; ++w) {
    u_lo = min(u_lo, red[0][w]);
    u_hi = max(u_hi, red[1][w]);
  }
  const float scale = rsqrtf((float)DD);
  const bool cap = a.softcap > 0.f;
  const float inv_cap = cap ? 1.f / a.softcap : 0.f;
  const float slope = a.slopes ? load_late(a.slopes + h) : 0.f;
  int origin[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) origin[i] = bias_origin(a.n_kv - a.n_q + row0 + ty * 4 + i, lo[i], hi[i], slope);
  float m[4], l[4];
  F2 o[4][DV];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) o[i][e] = F2(0.f, 0.f);
  }
  const int tile0 = u_lo < u_hi ? u_lo / FN : 0, tiles = u_lo < u_hi ? (u_hi + FN - 1) / FN - tile0 : 0;
  const int run = (tiles + n_splits - 1) / n_splits;
  const int k_begin = (tile0 + min(tiles, split * run)) * FN, k_end = (tile0 + min(tiles, (split + 1) * run)) * FN;
  // a tile of K or V on its way to shared memory, zeros for keys that no row sees
  auto fetch = [&](float* dst, const float* src, int k0) {
    if (k0 < k_end) {
#pragma unroll 4
      for (int x = tid; x < FN * (DD / 4); x += FTHREADS) {
        const int rr = x / (DD / 4), c = x - rr * (DD / 4);
        const bool in = k0 + rr >= u_lo && k0 + rr < u_hi;
        cp_async16(smem_u32(dst + rr * P + 4 * c), src + (size_t)(in ? k0 + rr : u_lo) * ldk + 4 * c, in);
      }
    }
    cp_commit();
  };
  // K of the next tile comes while this one's softmax and V are at work, V during the next scores
  fetch(ks, k, k_begin);
  fetch(vs, v, k_begin);
  for (int k0 = k_begin; k0 < k_end; k0 += FN) {
    cp_wait<1>();
    __syncthreads();
    F2 s2[4][4];                                               // even and odd dims' sums
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) s2[i][c] = F2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < DD; d += 4) {
      F2 qa[4][2], kb[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) ld_pairs(qs + (ty * 4 + i) * P + d, qa[i]);
#pragma unroll
      for (int c = 0; c < 4; ++c) ld_pairs(ks + (tx + 16 * c) * P + d, kb[c]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s2[i][c] = fma2(qa[i][1], kb[c][1], fma2(qa[i][0], kb[c][0], s2[i][c]));
    }
    __syncthreads();
    fetch(ks, k, k0 + FN);
    // scores; a row's max is moved only once a score passes it by 2^8
    float s[4][4];
    bool grow = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = a.n_kv - a.n_q + row0 + ty * 4 + i;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = k0 + tx + 16 * c;
        float z0, z;
        s2[i][c].get(&z0, &z);
        z = (z0 + z) * scale;
        if (cap) z = a.softcap * tanh_f32(z * inv_cap);
        z = fmaf(-slope, (float)(abs(pos - key) - origin[i]), z) * kLog2e;
        s[i][c] = key >= lo[i] && key < hi[i] ? z : -INFINITY;
        grow |= s[i][c] > m[i] + kRescaleLog2;                 // also from m = -inf
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = fmaxf(mx, m[i]);
        const float al = m[i] == -INFINITY ? 0.f : ex2_approx(m[i] - mx);
        m[i] = mx;
        l[i] *= al;
#pragma unroll
        for (int e = 0; e < DV; ++e) o[i][e] = mul2(o[i][e], F2(al, al));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mb = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = ex2_approx(s[i][c] - mb);
        l[i] += p;                                             // of this thread's columns
        ps[(ty * 4 + i) * SP + tx + 16 * c] = p;
      }
    }
    cp_wait<1>();
    float zero = 0.f;                                          // NaN with a non-finite V element here
#pragma unroll 4
    for (int x = tid; x < FN * (DD / 4); x += FTHREADS) {      // (the pieces that this thread fetched)
      const float4 f = *reinterpret_cast<const float4*>(vs + x / (DD / 4) * P + x % (DD / 4) * 4);
      zero = fmaf(f.x, 0.f, fmaf(f.y, 0.f, fmaf(f.z, 0.f, fmaf(f.w, 0.f, zero))));
    }
    if (!__syncthreads_or(zero != 0.f)) {
#pragma unroll 4
      for (int kk = 0; kk < FN; kk += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(ps + (ty * 4 + i) * SP + kk);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          F2 vv[DV];
#pragma unroll
          for (int e = 0; e < DV; ++e) vv[e] = *reinterpret_cast<const F2*>(vs + (kk + x) * P + 2 * tx + 32 * e);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
#pragma unroll
            for (int e = 0; e < DV; ++e) o[i][e] = fma2(F2(w, w), vv[e], o[i][e]);
          }
        }
      }
    } else {
      for (int kk = 0; kk < FN; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (k0 + kk < lo[i] || k0 + kk >= hi[i]) continue;
          const float w = ps[(ty * 4 + i) * SP + kk];
          const F2 pw(w, w);
#pragma unroll
          for (int e = 0; e < DV; ++e)
            o[i][e] = fma2(pw, *reinterpret_cast<const F2*>(vs + kk * P + 2 * tx + 32 * e), o[i][e]);
        }
    }
    __syncthreads();
    fetch(vs, v, k0 + FN);
  }
  cp_wait<0>();
  float* out = (n_splits > 1 ? o_part + (size_t)split * a.n_q * ldq : reinterpret_cast<float*>(a.o)) + (size_t)h * DD;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + ty * 4 + i;
    float sum = l[i];
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (row >= a.n_q) continue;
    const bool have = sum > 0.f || sum != sum;
#pragma unroll
    for (int e = 0; e < DV; ++e) {
      float o0, o1;
      o[i][e].get(&o0, &o1);
      *reinterpret_cast<float2*>(out + (size_t)row * ldq + 2 * tx + 32 * e) =
          have ? make_float2(o0 / sum, o1 / sum) : make_float2(0.f, 0.f);
    }
    if (n_splits > 1 && tx == 0)
      lse_part[((size_t)split * a.n_q + row) * a.heads + h] = have ? m[i] + log2f(sum) : -INFINITY;
  }
}

template <int DV>
cudaError_t run_f32(const MaskedArgs& a, int n_splits, float* o_part, float* lse_part, cudaStream_t s) {
  constexpr int smem = f32_smem<DV>();
  const cudaError_t e =
      cudaFuncSetAttribute(attn_masked_f32_kernel<DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((a.n_q + FM - 1) / FM) * (unsigned)a.heads * (unsigned)n_splits;
  return launch_dependent(attn_masked_f32_kernel<DV>, grid, FTHREADS, smem, s, a, n_splits, o_part, lse_part);
}

// The grid over rows and heads (see TcArgs): an odd group's last head takes 256 rows at a time,
// its pairs 128, so their row blocks are twice as many where there is more than one.
struct Cover {
  int halves, units, qblocks;
};
Cover cover(int n_q, int heads, int kv_heads) {
  const int g = heads / kv_heads, blocks = (n_q + BQ - 1) / BQ;
  Cover c;
  c.halves = g % 2 && blocks > 1 ? 2 : 1;
  c.units = g / 2 * c.halves + g % 2;
  c.qblocks = (blocks + c.halves - 1) / c.halves;
  return c;
}

long long base_ctas(int n_q, int heads, int kv_heads) {
  const Cover c = cover(n_q, heads, kv_heads);
  return (long long)c.qblocks * c.units * kv_heads;
}

}  // namespace

// Key splits, as many as cost least: a split's key tiles of the longest possible range (2 us each,
// fp32 3.4) and, bf16, a CTA's set-up and output (7 us), in every wave of CTAs; the join (3.5 us,
// and 2.5 of its 4 us of the host's time) and the partials (written and read, 4 TB/s).  bf16 runs
// one CTA on an SM, so that splits also even out the last wave (924 queries over 57,600 keys, 24
// heads, 96 CTAs: 900 us alone, 785 in three splits when the rule was made, 665 to 670 since), if they
// gain a tenth by this count: the waves read K and V again (1,200 queries, 120 CTAs: 1,012 us alone,
// 1,088 in six); fp32 runs several that share it (seven at D 32, four at 64, three at 96, two at 128;
// the rule counts four), and splits only fill the first.
// Against "at least two tiles a split (fp32: four), at most 16, within one wave": 1 query over
// 2,148 keys, 1 head 12.9 -> 10.5 us, over 30,000 37 -> 25; 300 queries over themselves, 24 heads:
// no splits either way.
int masked_splits(int n_q, int n_kv, int heads, int kv_heads, int head_dim, int dtype) {
  const bool tc = dtype == SFM_DTYPE_BF16;
  const long long ctas = tc ? base_ctas(n_q, heads, kv_heads) : (long long)((n_q + FM - 1) / FM) * heads;
  const int tiles = tc ? (n_kv + BKV - 1) / BKV : (n_kv + FN - 1) / FN;
  const int most = tiles < kMaxKeySplits ? tiles : kMaxKeySplits;
  const double tile = tc ? 2.0 : 3.4, cta = tc ? 7.0 : 0.0, part = 8e-6 / 4.0 * (head_dim + 1.0) * n_q * heads;
  double best = 0.;
  long long best_waves = 0;
  int splits = 1;
  for (int s = 1; s <= most; ++s) {
    if (!tc && s > 1 && ctas * s > 4 * kSms) break;
    const long long waves = tc ? (ctas * s + kSms - 1) / kSms : 1;
    const double cost = waves * (tile * ((tiles + s - 1) / s) + cta) + (s > 1 ? 6. + part * s : 0.);
    if (s == 1 || cost < (waves > best_waves ? 0.9 : 1.) * best) {
      best = cost;
      best_waves = waves;
      splits = s;
    }
  }
  return splits;
}

size_t masked_workspace(int n_q, int n_kv, int heads, int kv_heads, int head_dim, int dtype) {
  const int sp = masked_splits(n_q, n_kv, heads, kv_heads, head_dim, dtype);
  if (sp == 1) return 0;
  const size_t b = (size_t)sp * n_q * heads * (head_dim + 1) * sizeof(float);
  return (b + 15) / 16 * 16;
}

int launch_attention_masked_tc(const MaskedArgs& a, const CUtensorMap& mq, const CUtensorMap& mk,
                               const CUtensorMap& mv, void* workspace, const Guard& gd, cudaStream_t s) {
  TcArgs t{};
  t.m = a;
  const Cover c = cover(a.n_q, a.heads, a.kv_heads);
  t.halves = c.halves;
  t.units = c.units;
  t.qblocks = c.qblocks;
  t.n_splits = masked_splits(a.n_q, a.n_kv, a.heads, a.kv_heads, D, SFM_DTYPE_BF16);
  const long long rows_heads = (long long)a.n_q * a.heads;
  if (t.n_splits > 1) {
    t.o_part = (float*)workspace;
    t.lse_part = t.o_part + (size_t)t.n_splits * rows_heads * D;
  }
  t.err = gd.err;
  t.wait_ns = gd.wait_ns;
  t.fault = gd.fault;
  const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  auto kernel = cap ? (bias ? attn_masked_tc_kernel<true, true> : attn_masked_tc_kernel<true, false>)
                    : (bias ? attn_masked_tc_kernel<false, true> : attn_masked_tc_kernel<false, false>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return record_cuda(e);
  int rc;
  {
    ProfScope ps(SFM_PROF_ATTN, s);
    rc = record_cuda(launch_dependent(kernel, (unsigned)(t.qblocks * t.units * a.kv_heads * t.n_splits), THREADS, SMEM, s, mq, mk,
                                      mv, t));
  }
  if (rc || t.n_splits == 1) return rc;
  return launch_join<__nv_bfloat16>(t.o_part, t.lse_part, a.o, rows_heads, D, t.n_splits, s);
}

int launch_attention_masked_f32(const MaskedArgs& a, void* workspace, cudaStream_t s) {
  const int n_splits = masked_splits(a.n_q, a.n_kv, a.heads, a.kv_heads, a.head_dim, SFM_DTYPE_FP32);
  const long long rows_heads = (long long)a.n_q * a.heads;
  float *o_part = nullptr, *lse_part = nullptr;
  if (n_splits > 1) {
    o_part = (float*)workspace;
    lse_part = o_part + (size_t)n_splits * rows_heads * a.head_dim;
  }
  int rc;
  {
    ProfScope ps(SFM_PROF_ATTN, s);
    cudaError_t e;
    switch (a.head_dim / 32) {
      case 1: e = run_f32<1>(a, n_splits, o_part, lse_part, s); break;
      case 2: e = run_f32<2>(a, n_splits, o_part, lse_part, s); break;
      case 3: e = run_f32<3>(a, n_splits, o_part, lse_part, s); break;
      default: e = run_f32<4>(a, n_splits, o_part, lse_part, s); break;
    }
    rc = record_cuda(e);
  }
  if (rc || n_splits == 1) return rc;
  return launch_join<float>(o_part, lse_part, a.o, rows_heads, a.head_dim, n_splits, s);
}

int launch_attention_bounds(const BoundsArgs& a, cudaStream_t s) {
  ProfScope ps(SFM_PROF_ROWOPS, s);
  return record_cuda(launch_dependent(attention_bounds_kernel, (unsigned)((a.n_q + 255) / 256), 256, 0, s, a));
}

}  // namespace sfm
