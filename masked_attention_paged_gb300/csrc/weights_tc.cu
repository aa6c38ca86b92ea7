// weights_tc.cu -- attention weight received by every cached token (tcgen05 +
// TMEM + TMA): the sums that an eviction policy ranks tokens by.
//
// For a chunk of queries whose softmax LSE is known,
//   acc[key] (+)= sum over the KV head's query heads and the chunk's rows that
//                 see the key of 2^(scale_log2 q.k - lse_log2).
// Scores are computed transposed, S^T = K Q^T: keys are the MMA's rows (TMEM
// lanes) and queries its columns, so a thread owns a key and its sum stays in one
// register, with no exchange between threads.  K is read once per query chunk
// list (a pair of 128-key tiles stays in shared memory while all queries pass),
// V not at all.  Bound: HBM for single tokens (64 KB of K per pair, 1.4 us of an
// SM's share); for long chunks the exponentials (one per query row and key, 1024
// cycles a step of 256 keys x 128 rows) and the products (1024 at the nominal rate,
// ~1300 with the operands, the TMA writes and the LSEs' reads sharing the
// shared-memory port).  Measured, 32 query and 8 KV heads, D = 128: 64 single
// tokens over up to 8192, 136 us for 0.84 GB, 90 % of the measured copy rate; a
// causal prompt of 4096 tokens 71.5 us, where the MMAs alone take 36 at the measured
// cuBLAS rate: a step takes its two warpgroups about 1900 cycles.
//
// A chunk is the G heads of up to 128 / G tokens, one 5-D TMA box of q whatever
// its strides: column r is token r / G, head r % G.  A key at position x is seen
// by tokens t >= x - start, so a causal tile is one comparison per column, and
// chunks before the pair's first key are left out.  An item is a (sequence, KV
// head, key pair), its steps are its chunks; every SM takes an equal run of all
// steps, an item's start and end counted as kItemCost of them (as in tree_tc.cu; the
// prompt took 78 us with 0, 71.4 with 3), and an item cut between SMs leaves partial sums that
// its last piece adds up in order: the result does not depend on the timing.
//
// Warps: 0-3 stream K, 4 issues the MMAs, 5 streams query chunks, 6 their LSEs;
// 8-11 and 12-15 own the two key tiles.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged_tile.cuh"
#include "runs.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;       // keys per tile
constexpr int kPair = 2 * kBM;
constexpr int kBN = 128;       // query rows per chunk, at most
constexpr int kBS = 16;
constexpr int kBoxBytes = kBM * 128;
constexpr int kThreads = 512;
constexpr int kLseRing = 2;  // as the score buffers
constexpr int kSegs = 4;  // segments the planner is ahead
constexpr int kItemCost = 3;  // what an item costs a CTA besides its steps, in steps
constexpr int kBarBytes = 1024;

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int KS = D == 64 ? 8 : 4;  // K tile stages
  static constexpr int QS = D == 64 ? 4 : 3;  // query chunk stages
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kOffK + KS * kTileBytes;
  static constexpr int kOffLse = kOffQ + QS * kTileBytes;  // [kLseRing][kBN] negated log2 LSEs, -inf: no weight
  static constexpr int kOffBar = kOffLse + kLseRing * kBN * 4;
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

// A run [c0, c1) of one item's chunks: what every warp role works through.  One
// warp plans them and hands them on in a small ring (as in tree_tc.cu).
struct Seg {
  int b;  // -1: the end
  int g, pair, c0, c1;
  int n, start, keys;  // of the sequence
  int slot;            // where its partial sums go; -1: the item is whole
  int run0, pieces, head;  // a cut item: its first run, its runs, whether it is that run's first segment
};

struct Bars {
  uint64_t k_full[8], k_empty[8];
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2][2], s_free[2][2];  // [key tile][step & 1]: scores and LSEs are there, have been read
  uint64_t piece_full, piece_go, drained;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg segs[kSegs];
  uint32_t tmem_base;
  int abort, last;
  int odd[kLseRing];  // the chunk has columns without weight (padding, or rows that see nothing)
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block outgrew its shared-memory slot");

struct WeightParams {
  int B, T, Hq, Hkv, G;
  int ct, cr;  // tokens and rows (ct * G) of a chunk
  int causal;
  float scale_log2;
  const float* lse;  // [B, Hq, T]
  int num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start_pos;
  const int32_t* q_lens;  // or null: T each
  float* acc;             // [num_blocks, Hkv, 16]
  float* part;            // [2 n][kPair]
  unsigned long long* count;  // [B, Hkv, pairs] pieces done (count_last)
  int pairs_max;
  uint32_t gen;
  uint32_t* status;
};

// One sequence's work: `pairs` key pairs, the first `full` of which all chunks
// see; pair p >= full starts at chunk first(p).
struct SeqWork {
  int start, n, keys, pairs, chunks, full, ct;
  int64_t units;  // per KV head: its pairs' steps and kItemCost each
  // At most chunks - 1: the pair's first key is one of the sequence's keys.
  __device__ int first(int p) const { return p < full ? 0 : (p * kPair - start) / ct; }
};

__device__ __forceinline__ SeqWork seq_work(const WeightParams& p, int b, bool report_bad) {
  SeqWork w = {};
  w.ct = p.ct;
  w.start = p.start_pos[b];
  int n = p.q_lens != nullptr ? p.q_lens[b] : p.T;
  n = max(0, min(n, p.T));
  if (w.start < 0 || n == 0) return w;
  if (static_cast<int64_t>(w.start) + n > static_cast<int64_t>(p.max_blocks) * kBS) {
    if (report_bad) report(p.status, kStatusBounds);
    return w;
  }
  w.n = n;
  w.keys = w.start + n;
  w.pairs = (w.keys + kPair - 1) / kPair;
  w.chunks = (n + p.ct - 1) / p.ct;
  w.full = p.causal ? min(w.pairs, w.start / kPair + 1) : w.pairs;
  w.units = static_cast<int64_t>(w.full) * w.chunks + static_cast<int64_t>(w.pairs) * kItemCost;
  if (kPair % p.ct == 0) {
    // first(x) = k x - ceil(start / ct): an arithmetic series
    const int64_t k = kPair / p.ct, m = w.pairs - w.full;
    w.units += m * (w.chunks + (w.start + p.ct - 1) / p.ct) - k * (m * (w.full + w.pairs - 1) / 2);
  } else {
    for (int x = w.full; x < w.pairs; ++x) w.units += w.chunks - w.first(x);
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ WeightParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  float* lse_ring = reinterpret_cast<float*>(smem + C::kOffLse);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 32) {
    for (int s = 0; s < 2; ++s) {
      for (int t = 0; t < 2; ++t) {
        mbar_init(&bars->s_full[t][s], 2);  // the MMAs and the LSEs' warp
        mbar_init(&bars->s_free[t][s], 4);
      }
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bars->k_full[s], 2);  // two producer warps a tile
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&bars->seg_full[s], 1);
      mbar_init(&bars->seg_empty[s], 15);  // 4 producers, the issuer, Q's and the LSEs' warps, 8 that sum
    }
    mbar_init(&bars->piece_full, 8);
    mbar_init(&bars->piece_go, 1);
    mbar_init(&bars->drained, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  wait_for_launch_ahead();
  // the planner's state: the call's runs, and the place of this CTA's first step
  Runs64 runs = {};
  int64_t pos = 0, lo = 0, hi = 0, item0 = 0;
  int plan_b = 0, plan_g = 0, plan_pair = 0, plan_c = 0;
  SeqWork work = {};
  if (warp == 7) {
    int64_t total = 0, mine0 = 0;
    for (int base = 0; base < p.B; base += 32) {
      const int64_t mine =
          base + lane < p.B ? seq_work(p, base + lane, blockIdx.x == 0).units * p.Hkv : 0;
      if (base == 0) mine0 = mine;
      total += mine;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
    runs = Runs64::make(total, gridDim.x);
    const int cta = static_cast<int>(blockIdx.x);
    if (cta < runs.n) lo = runs.lo(cta), hi = runs.lo(cta + 1);
    pos = lo;
    int64_t run = 0;
    for (int base = 0; base < p.B && lo < hi; base += 32) {
      const int64_t mine =
          base == 0 ? mine0 : (base + lane < p.B ? seq_work(p, base + lane, false).units * p.Hkv : 0);
      int64_t incl = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + incl > lo);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        plan_b = base + l;
        run += __shfl_sync(0xffffffffu, incl - mine, l);
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_q);
    }
    if (lo < hi) {
      work = seq_work(p, plan_b, false);
      plan_g = static_cast<int>(div_pos(lo - run, work.units));
      int64_t rem = lo - run - plan_g * work.units;  // unit within the (sequence, KV head)
      const int64_t most = kItemCost + work.chunks;
      if (rem < work.full * most) {
        plan_pair = static_cast<int>(div_pos(rem, most));
        rem -= plan_pair * most;
      } else {
        plan_pair = work.full;
        rem -= work.full * most;
        while (rem >= most - work.first(plan_pair)) rem -= most - work.first(plan_pair), ++plan_pair;
      }
      plan_c = work.first(plan_pair) + static_cast<int>(rem) - kItemCost;
      item0 = lo - rem;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // scores of tile t, buffer j & 1, at column (2 t + (j & 1)) * 128

  // segment i, for a whole warp; false at the end
  auto seg_get = [&](int i, Seg& s) {
    if (!__all_sync(0xffffffffu, mbar_wait(&bars->seg_full[i % kSegs], (i / kSegs) & 1, abort, p.status))) return false;
    s = bars->segs[i % kSegs];
    return s.b >= 0;
  };
  auto seg_taken = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->seg_empty[i % kSegs]);
  };

  if (warp < 4) {
    // ------------------------------------------------------------ K
    // warp w, lane i < 4: block 4 w + i of the pair's sixteen, its id read a
    // segment ahead; warps 0, 1 fill the first tile, 2, 3 the second
    Seg s;
    const int t = warp >> 1, place = warp * kWarpBlocks + lane;  // block of the pair
    bool want_next = false;  // a key of the sequence is in it
    auto block_id = [&](const Seg& x) {
      const int blk = x.pair * (kPair / kBS) + place;
      want_next = lane < kWarpBlocks && blk * kBS < x.keys;
      return want_next ? p.bt[static_cast<int64_t>(x.b) * p.bt_stride + blk] : -1;
    };
    int n = t;
    bool more = seg_get(0, s);
    int id_next = more ? block_id(s) : -1;
    for (int i = 0; more; ++i) {
      int id = id_next;
      const bool want = want_next;
      const int g = s.g;
      seg_taken(i);
      more = seg_get(i + 1, s);
      if (more) id_next = block_id(s);
      if (id < 0 || id >= p.num_blocks) {  // a table may hold any id, -1 too
        if (want) report(p.status, kStatusBounds);
        id = -1;
      }
      const int st = n % C::KS;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * (kBS * D * 2);
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->k_empty[st], ((n / C::KS) & 1) ^ 1, abort, p.status))) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], bytes);
      __syncwarp();
      load_block<D>(smem + C::kOffK + st * C::kTileBytes, place % kTileBlocks, &tm_k, &bars->k_full[st], id, p.Hkv, g);
      n += 2;
    }
    if (lane == 0 && *abort)  // let the copies in flight land
      for (int x = max(t, n - C::KS); x < n; x += 2) drain_wait(&bars->k_full[x % C::KS], (x / C::KS) & 1);
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp goes through the loop, with values that are alike in all
    // lanes (uniform registers, which the descriptors have to be in), and one lane
    // issues: with one lane in the loop an MMA took ~120 cycles to issue.
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort, p.status)) != 0;
    };
    const uint32_t tm = uni(tmem);
    const uint64_t k0 = sdesc_sw128(smem_u32(smem + C::kOffK), 16, PagedTile<D>::kGroup);
    const uint64_t q0 = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    int n = 0, j = 0;
    bool ok = true;
    Seg s;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const int c0 = uni(s.c0), c1 = uni(s.c1), rows = uni(s.n);
      for (int c = c0; ok && c < c1; ++c, ++j) {
        const int qs = j % C::QS;
        ok = wait(&bars->q_full[qs], j / C::QS);
        if (!ok) break;
        const int cols = min(p.ct, rows - c * p.ct) * p.G;
        const uint32_t idesc = idesc_bf16_f32(kBM, (cols + 15) / 16 * 16, false, false);
        const uint64_t qd = q0 + qs * (C::kTileBytes >> 4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // half a chunk apart, the two tiles' exponentials do not come at once
          const int st = (n + t) % C::KS;
          ok = ok && (c > c0 || wait(&bars->k_full[st], (n + t) / C::KS)) &&
               wait(&bars->s_free[t][j & 1], (j >> 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = k0 + st * (C::kTileBytes >> 4);
          const uint32_t to = tm + (2 * t + (j & 1)) * 128;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)  // 16 dims = 32 bytes of a 128-byte row
              umma_bf16_ss(to, kd + (kk >> 2) * (PagedTile<D>::kHalf >> 4) + (kk & 3) * 2,
                           qd + (kk >> 2) * (kBoxBytes >> 4) + (kk & 3) * 2, idesc, kk > 0 ? 1u : 0u);
            umma_commit(&bars->s_full[t][j & 1]);
            if (c + 1 == c1) umma_commit(&bars->k_empty[st]);
            if (t == 1) umma_commit(&bars->q_empty[qs]);
          }
          __syncwarp();
        }
      }
      n += 2;
    }
    if (elect_one()) {
      umma_commit(&bars->drained);
      drain_wait(&bars->drained, 0);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ query chunks
    if (lane == 0) {
      int j = 0;
      bool ok = true;
      const uint32_t bytes = static_cast<uint32_t>(p.cr) * D * 2;  // tokens past T arrive as zeros
      for (int i = 0; ok; ++i) {
        ok = mbar_wait(&bars->seg_full[i % kSegs], (i / kSegs) & 1, abort, p.status);
        if (!ok) break;
        const Seg s = bars->segs[i % kSegs];
        if (s.b < 0) break;
        mbar_arrive(&bars->seg_empty[i % kSegs]);
        for (int c = s.c0; c < s.c1; ++c, ++j) {
          const int qs = j % C::QS;
          ok = mbar_wait(&bars->q_empty[qs], ((j / C::QS) & 1) ^ 1, abort, p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars->q_full[qs], bytes);
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_5d(smem + C::kOffQ + qs * C::kTileBytes + x * kBoxBytes, &tm_q, &bars->q_full[qs], x * 64, 0,
                        c * p.ct, s.g, s.b);
        }
      }
      if (*abort)
        for (int x = max(0, j - C::QS); x < j; ++x) drain_wait(&bars->q_full[x % C::QS], (x / C::QS) & 1);
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------ their LSEs
    // negated, in log2 units; -inf where a column has no weight (past the
    // chunk, or a row that saw nothing).  Loaded a chunk ahead of the store.
    Seg s;
    int j = 0;
    bool ok = true;
    float v[4];
    int dt[4], dh[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) dt[x] = (lane + 32 * x) / p.G, dh[x] = (lane + 32 * x) % p.G;
    auto publish = [&](int jj) {
      const int sl = jj % kLseRing;
      for (int t = 0; t < 2; ++t)
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_free[t][sl], ((jj / kLseRing) & 1) ^ 1, abort, p.status)))
          return false;
      bool odd = false;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float l = v[x] == -INFINITY ? -INFINITY : v[x] * -1.4426950408889634f;
        odd |= l == -INFINITY;
        lse_ring[sl * kBN + lane + 32 * x] = l;
      }
      odd = __any_sync(0xffffffffu, odd);
      if (lane == 0) bars->odd[sl] = odd;
      __syncwarp();
      if (lane < 2) mbar_arrive(&bars->s_full[lane][sl]);
      return true;
    };
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const float* row = p.lse + (static_cast<int64_t>(s.b) * p.Hq + static_cast<int64_t>(s.g) * p.G) * p.T;
      for (int c = s.c0; ok && c < s.c1; ++c, ++j) {
        float next[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = c * p.ct + dt[x];
          next[x] = dt[x] < p.ct && t < s.n ? row[static_cast<int64_t>(dh[x]) * p.T + t] : -INFINITY;
        }
        if (j > 0) ok = publish(j - 1);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = next[x];
      }
    }
    if (ok && j > 0) publish(j - 1);
  } else if (warp == 7) {
    // ------------------------------------------------------------ planner
    for (int i = 0;; ++i) {
      Seg s = {};
      s.b = -1;
      if (pos < hi && plan_c == work.chunks) {  // the item is done: the next pair, KV head or sequence
        item0 = pos;
        if (++plan_pair == work.pairs) {
          plan_pair = 0;
          if (++plan_g == p.Hkv) {
            plan_g = 0;
            do work = seq_work(p, ++plan_b, false);
            while (work.units == 0);
          }
        }
        plan_c = work.first(plan_pair) - kItemCost;
      }
      const int f = pos < hi ? work.first(plan_pair) : 0;
      if (plan_c < f) {  // the item's own cost, or as much of it as falls into this run
        const int skip = static_cast<int>(min(static_cast<int64_t>(f - plan_c), hi - pos));
        pos += skip;
        plan_c += skip;
      }
      if (pos < hi) {
        s.b = plan_b, s.g = plan_g, s.pair = plan_pair;
        s.c0 = plan_c;
        s.c1 = static_cast<int>(min(static_cast<int64_t>(work.chunks), plan_c + (hi - pos)));
        s.n = work.n, s.start = work.start, s.keys = work.keys;
        s.slot = -1;
        if (s.c0 != f || s.c1 != work.chunks) {
          const int64_t step0 = item0 + kItemCost;
          s.slot = 2 * static_cast<int>(blockIdx.x) + (i == 0 ? 0 : 1);
          s.run0 = runs.of(step0);
          s.pieces = runs.of(step0 + work.chunks - f - 1) - s.run0 + 1;
          s.head = runs.lo(s.run0) >= item0;  // nothing of the item before lies in that run
        }
        pos += s.c1 - plan_c;
        plan_c = s.c1;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->seg_empty[i % kSegs], ((i / kSegs) & 1) ^ 1, abort, p.status)))
        break;
      if (lane == 0) {
        bars->segs[i % kSegs] = s;
        mbar_arrive(&bars->seg_full[i % kSegs]);
      }
      if (s.b < 0) break;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ sums
    const int t = (warp >> 2) & 1;  // key tile
    const int row = (warp & 3) * 32 + lane;
    const int tid = t * kBM + row;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Seg s;
    int j = 0, pieces = 0;
    bool ok = true;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const int key = s.pair * kPair + t * kBM + row;
      const bool there = key < s.keys;
      const int blk = there ? p.bt[static_cast<int64_t>(s.b) * p.bt_stride + key / kBS] : -1;
      // The key's sum belongs to this thread alone, so an add without a return
      // value has no order to depend on, and no read to wait for.  A token of
      // the chunk itself starts from nothing.
      auto put = [&](float got) {
        if (blk < 0 || blk >= p.num_blocks) return;
        float* at = p.acc + (static_cast<int64_t>(blk) * p.Hkv + s.g) * kBS + key % kBS;
        if (key < s.start)
          asm volatile("red.global.add.f32 [%0], %1;" ::"l"(at), "f"(got) : "memory");
        else
          *at = got;
      };
      // tokens that see the key: t >= tmin; the warp's last key is seen by the fewest
      const int tmin = p.causal ? key - s.start : 0;
      const int warp_tmin = __shfl_sync(0xffffffffu, tmin, 31);
      uint64_t sum[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) sum[x] = f2_pack(0.f, 0.f);
      const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
      for (int c = s.c0; c < s.c1; ++c, ++j) {
        const int sl = j % kLseRing;  // the score buffer as well
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[t][sl], (j / kLseRing) & 1, abort, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int t0 = c * p.ct;
        const int cols = min(p.ct, s.n - t0) * p.G;
        const float* nl = lse_ring + sl * kBN;
        const bool masked = bars->odd[sl] != 0 || warp_tmin > t0;
        const int rel = max(0, min(tmin - t0, p.ct)) * p.G;  // columns >= rel see the key
        const uint32_t col = tmem + lane_addr + (2 * t + sl) * 128;
        auto add32 = [&](const uint32_t (&sr)[32], int cc, auto masked_c) {
          constexpr bool MASKED = decltype(masked_c)::value;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(nl + cc + i);
            float x0, x1, x2, x3;
            f2_unpack(ffma2(f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), sc2, f2_pack(l4.x, l4.y)), x0,
                      x1);
            f2_unpack(ffma2(f2_pack(__uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3])), sc2, f2_pack(l4.z, l4.w)),
                      x2, x3);
            float w0 = fast_exp2(x0), w1 = fast_exp2(x1), w2 = fast_exp2(x2), w3 = fast_exp2(x3);
            if constexpr (MASKED) {
              // selected, not multiplied: whatever a column without weight holds stays out
              w0 = (cc + i >= rel && l4.x != -INFINITY) ? w0 : 0.f;
              w1 = (cc + i + 1 >= rel && l4.y != -INFINITY) ? w1 : 0.f;
              w2 = (cc + i + 2 >= rel && l4.z != -INFINITY) ? w2 : 0.f;
              w3 = (cc + i + 3 >= rel && l4.w != -INFINITY) ? w3 : 0.f;
            }
            sum[(i >> 1) & 3] = fadd2(sum[(i >> 1) & 3], f2_pack(w0, w1));
            sum[((i >> 1) + 1) & 3] = fadd2(sum[((i >> 1) + 1) & 3], f2_pack(w2, w3));
          }
        };
        if (!masked) {
          // a whole chunk (one with a column of padding is masked)
          uint32_t sa[32], sb[32];
          tmem_ld32(col, sa);
          tmem_wait_ld(sa);
#pragma unroll
          for (int cc = 0; cc < kBN; cc += 64) {  // the next 32 columns load while these are added
            tmem_ld32(col + cc + 32, sb);
            add32(sa, cc, std::false_type());
            tmem_wait_ld(sb);
            if (cc + 64 < kBN) tmem_ld32(col + cc + 64, sa);
            add32(sb, cc + 32, std::false_type());
            if (cc + 64 < kBN) tmem_wait_ld(sa);
          }
        } else {
#pragma unroll 1
          for (int cc = 0; cc < cols; cc += 32) {
            uint32_t sr[32];
            tmem_ld32(col + cc, sr);
            tmem_wait_ld(sr);
            add32(sr, cc, std::true_type());
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[t][sl]);
      }
      if (!ok) break;
      float a0, a1;
      f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), a0, a1);
      const float got = a0 + a1;
      if (s.slot < 0) {
        put(got);
        continue;
      }
      // a cut item: leave the piece; the last one adds them in order
      p.part[static_cast<int64_t>(s.slot) * kPair + tid] = got;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->piece_full);
      if (tid < 32 && !__all_sync(0xffffffffu, mbar_wait(&bars->piece_full, pieces & 1, abort, p.status))) {
        ok = false;
        break;
      }
      if (tid == 0) {
        __threadfence();
        bars->last = count_last(p.count + (static_cast<int64_t>(s.b) * p.Hkv + s.g) * p.pairs_max + s.pair, p.gen,
                                s.pieces);
        mbar_arrive(&bars->piece_go);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->piece_go, pieces & 1, abort, p.status))) {
        ok = false;
        break;
      }
      ++pieces;
      if (bars->last) {
        __threadfence();
        float all = 0.f;
#pragma unroll 4
        for (int x = 0; x < s.pieces; ++x) {
          const int sl = 2 * (s.run0 + x) + ((x == 0 && !s.head) ? 1 : 0);
          all += __ldcg(p.part + static_cast<int64_t>(sl) * kPair + tid);
        }
        put(all);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const WeightArgs& a, const WeightParams& p, cudaStream_t stream) {
  CUtensorMap mk, mq;
  if (!make_paged_map(&mk, a.cache.k, a.cache.num_blocks, a.cache.Hkv, D) ||
      !make_rows_map(&mq, a.q, a.cache.Hkv, p.ct))
    return cudaErrorInvalidValue;
  auto kern = attn_weights_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(static_cast<unsigned>(a.n_cta)), kThreads, Cfg<D>::kSmemBytes, stream, mk, mq, p);
}

size_t part_bytes(int n_cta) { return static_cast<size_t>(2) * n_cta * kPair * sizeof(float); }
int pairs_of(int max_blocks) {
  return static_cast<int>((static_cast<int64_t>(max_blocks) * kBS + kPair - 1) / kPair);
}

}  // namespace

// Partial sums of two cut items per CTA, then one 8-byte count per item.
size_t weights_partial_bytes(int64_t B, int64_t Hkv, int max_blocks, int n_cta) {
  const size_t counts = static_cast<size_t>(B) * Hkv * pairs_of(max_blocks) * sizeof(unsigned long long);
  return ((part_bytes(n_cta) + 255) & ~size_t(255)) + ((counts + 255) & ~size_t(255));
}

cudaError_t launch_attn_weights(const WeightArgs& a, cudaStream_t stream) {
  WeightParams p = {};
  p.B = static_cast<int>(a.B);
  p.T = static_cast<int>(a.T);
  p.Hq = static_cast<int>(a.Hq);
  p.Hkv = a.cache.Hkv;
  p.G = p.Hq / p.Hkv;
  p.causal = a.causal;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.ct = std::min(p.T, kBN / p.G);
  p.cr = p.ct * p.G;
  p.lse = a.lse;
  p.num_blocks = static_cast<int>(a.cache.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.start_pos = a.start_pos;
  p.q_lens = a.q_lens;
  p.acc = a.acc;
  p.part = static_cast<float*>(a.partials);
  p.count = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(a.partials) +
                                                  ((part_bytes(a.n_cta) + 255) & ~size_t(255)));
  p.pairs_max = pairs_of(a.max_blocks);
  p.gen = a.gen;
  p.status = a.status;
  if (a.cache.D == 64) return launch<64>(a, p, stream);
  if (a.cache.D == 128) return launch<128>(a, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace attn
