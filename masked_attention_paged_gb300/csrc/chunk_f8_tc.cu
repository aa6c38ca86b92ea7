// chunk_f8_tc.cu -- attention of many query rows over an e4m3 paged cache (tcgen05 +
// TMEM + TMA): paged_attn_f8 for more than 16 rows per KV head.
//
// A row tile is the G heads of tb = min(T, 128 / G) queries (row r: query r / G, head
// r % G); NT row tiles (NT = 1 if one holds all rows, else 2) share every 128-key tile.
//  * Scores: K codes are an operand as they lie in the cache (kind::f8f6f4; a block's
//    rows land in shared memory as the matrix descriptor wants them).  q is two e4m3
//    numbers, (hi + lo) 2^e: bf16 has eight significant bits and e4m3 four, so the two
//    are q exactly, down to 2^-19 of the row's largest element.  Two products at twice
//    the bf16 rate cost what one bf16 product does, and K needs no conversion.  The block
//    scales multiply the scores, in the softmax's one FMA.
//  * Values: P (bf16, in TMEM) needs its range, so V is made bf16: four warps turn codes
//    into code * scale, exact in bf16 since scales are powers of two.
// Every SM takes an equal run of the call's tiles (runs.cuh): an item (sequence, row
// group, KV head) is its key tiles, causal ones ending at its last row's, plus kItemCost
// for its start and end.  Items inside a run are written at once; one that is cut
// leaves partials (normalised rows and log2 LSE), which a second launch joins in
// order, so results do not depend on timing.
//
// Warps: 0 streams the codes, 1 issues the MMAs, 2 waits for it, 3 plans the segments, 4-7
// convert V, 8-11 and 12-15 softmax (thread r owns row r: TMEM lane r; it also splits
// its row of q).  With NT = 2 each warpgroup has a row tile.  With NT = 1 both have the same rows
// and take the key tiles in turn, each with a score buffer, an accumulator and a running max
// and sum of its own, joined by the LSE rule when an item ends.
//
// What bounds it: 2 x 1024 tokens behind 8192 (32 heads over 8, D = 128) take 190 us where the
// products alone would take 123.  A tile takes 3000 cycles a CTA: 2 x 1030 of products, which
// also read shared memory at 128 bytes a cycle, all that it gives (8 KB a step of 65 cycles), so
// that the TMA's and the converters' bytes come on top; and two waits of the issuer, 230
// each.  A row tile's value product waits for all of its softmax, some 1310 cycles, so the two
// tiles' chains have nothing to spare.  An item's start and end cost some 12000 cycles.  With one
// row tile the conversion sets the pace, 2700 cycles a tile (16 x 16 tokens behind 8192: 87 us; some
// 72 with none at all).
// Not kept, next to the 200 us of then: two issuers, one a row tile, 261 (both products end
// late), in strict turns 224; two threads a row, 64 keys each, 229; 64-key tiles 292; waits
// polled instead of parked 203; the converting loop unrolled twice 214, and rolled to one
// vector a step 231.  Next to 195: q split ahead of the epilogue before it 199; values and weights
// in fp16, half the converters' instructions, 197; items joined in place by the last of up to four
// CTAs 192, but 98 for the 16 x 16.
//
// Slots past the last key may hold NaN codes: their V rows go in as zeros (P is 0
// there, but 0 x NaN is not).  A token that some rows see and others do not may be
// NaN, too: such codes go in as zeros, and the epilogue gives them to the rows that
// see them.
#include <cuda.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "internal.h"
#include "paged_tile.cuh"
#include "runs.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kBS = 16;
constexpr float kRescaleMargin = 8.0f;
constexpr int kBarBytes = 4096;
constexpr int kSegs = 4;      // segments the planner is ahead
// What an item costs a CTA besides its tiles, in tiles: the split of q, the products of the first
// tile, the epilogue.  Two chunks of 1024 behind 8192 tokens: 189 us with 6 and with 8, 192 with
// 3, 194 with none; two of 64: 34, 35, 39, 44; one of 2048 behind 10 tokens: 67, 67, 74, 152; 4 of
// 300 behind 1000: 47, 48, 49, 57.
constexpr int kItemCost = 6;
constexpr int kScales = 8;    // tiles whose key scales are held: more than K's stages and the scores ahead of P
constexpr int kNotes = 8;     // segments whose notes of NaNs are held: more than the planner is ahead
constexpr int kSpread = 256;  // most queries of a row group: tokens that not all of its rows see

template <int D, int NT>
struct Cfg {
  static constexpr int kThreads = 512;
  static constexpr int kQBytes = kBM * D;         // hi or lo of a row tile
  static constexpr int kCodeBytes = kBN * D;      // a tile of codes
  static constexpr int kTileBytes = kBN * D * 2;  // a tile of V in bf16
  // 227 KB hold, at D = 128, two row tiles and 3 + 2 tiles of codes, or one and 4 + 3
  static constexpr int KS = D == 64 || NT == 1 ? 4 : 3;
  static constexpr int VC = D == 64 ? 4 : (NT == 1 ? 3 : 2);
  static constexpr int VS = D == 64 ? 4 : 2;
  static constexpr int kOffQ = 0;  // [NT][hi, lo]
  static constexpr int kOffK = kOffQ + NT * 2 * kQBytes;
  static constexpr int kOffC = kOffK + KS * kCodeBytes;
  static constexpr int kOffV = kOffC + VC * kCodeBytes;
  static constexpr int kOffXch = kOffV + VS * kTileBytes;  // NT = 1: [2][kBM] running max and sum
  static constexpr int kOffBar = kOffXch + (NT == 1 ? 2 * kBM * 8 : 0);
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(KS + 2 < kScales, "the ring of scales outlasts the stages");
  static constexpr uint32_t kColO = 256;  // O of warpgroup w at kColO + w * D; its scores at w * 128
  // 512 threads launched with 128 registers; 256 x 56 + 256 x 200 = 65536 (184: the
  // softmax of NT = 2 spills)
  static constexpr int kRegsCtl = 56, kRegsSoft = 200;
  // codes of a row: 128 bytes, 128-byte swizzle (D = 128), or 64 and 64
  static constexpr uint32_t kGroup = 8 * D;  // next 8 rows
  static __device__ __forceinline__ uint32_t code_off(int r, int c) {  // 16-byte chunk c of row r
    return static_cast<uint32_t>(r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
  }
  static __device__ __forceinline__ uint64_t code_desc(uint32_t addr) {
    const uint64_t d = sdesc_sw128(addr, 16, kGroup);
    return D == 128 ? d : (d & ~(7ull << 61)) | 4ull << 61;  // 64-byte swizzle
  }
};

// A run of one item's tiles [t0, t1).
struct Seg {
  int b;  // -1: the end
  int g, i0, t0, t1;
  int start, n;  // the sequence's first position and queries
  int kend;      // keys that the item's last row sees
  int slot;      // where its partial goes; -1: the item is whole
};

struct Bars {
  uint64_t k_full[4], k_empty[4], c_full[4], c_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2];  // [warpgroup]
  uint64_t q_raw[2], q_full[2];
  uint64_t sc_full[kScales];
  uint64_t xch_full[2];  // NT = 1: a warpgroup's running max and sum are in smem
  uint64_t o_free;       // NT = 1: both warpgroups have read both accumulators
  uint64_t conv[kNotes];  // a segment's V has been converted
  uint64_t drained;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg segs[kSegs];
  alignas(16) float ks[kScales][8];  // read four at a time
  uint32_t there[kScales];  // blocks of the tile whose id is good
  float vs[4][8];           // by V code stage; -1: no such block
  uint32_t bad[kNotes][4][kSpread / 32];  // tokens start + i0 + .. whose V holds a NaN, by converting warp
  float qmul[2][kBM];  // rows' factors
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block outgrew its shared-memory slot");

struct CutItem {
  int b, g, i0;
  int pieces;         // in CTAs c, c + 1, ...; 0: no item
  int first_is_head;  // it is the first segment of CTA c's run
};

struct ChunkParams {
  int B, T, Hq, Hkv, G;
  int tb, RT;  // queries and rows (tb * G) of a row tile
  int MP;      // row groups (of NT tiles) per KV head
  int causal;
  float scale_log2;
  const uint16_t* q;
  int64_t q_stride[3];
  const float* ks;
  const float* vs;
  const uint8_t* vq;
  int num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start;
  const int32_t* lens;
  void* out;
  int out_bf16;
  int64_t out_stride[3];
  float* lse;
  float* part_o;    // [2 n][D][pitch]: a column's rows side by side, as the TMEM lanes hold them
  float* part_lse;  // [2 n][pitch]
  int pitch;        // rows of a partial: 128 a row tile
  int ctas;         // n: CTAs of the main launch
  CutItem* cuts;    // [n] the item that starts in CTA c's run and goes on past it
  uint32_t* status;
};

// A sequence's queries: none if it is idle or does not fit its table.
__device__ __forceinline__ int seq_queries(const ChunkParams& p, int b, int& start, bool& past) {
  start = p.start[b];
  const int n = p.lens != nullptr ? min(max(p.lens[b], 0), p.T) : p.T;
  past = start >= 0 && static_cast<int64_t>(start) + n > static_cast<int64_t>(p.max_blocks) * kBS;
  return start < 0 || past ? 0 : n;
}
// Keys of the row group that begins at query i0, and its tiles (a group that sees nothing has
// none, and is no item: the second launch writes it).
__device__ __forceinline__ int group_keys(const ChunkParams& p, int start, int n, int i0, int rows) {
  return i0 >= n ? 0 : start + (p.causal ? min(i0 + rows, n) : n);
}
__device__ __forceinline__ int key_tiles(int kend) { return (kend + kBN - 1) / kBN; }
// Keys of a tile that its MMAs cover: a multiple of 16, at least 16.
__device__ __forceinline__ int tile_keys(int kend, int tile) {
  return min(kBN, max(16, (kend - tile * kBN + 15) / 16 * 16));
}

// D[tmem] (+)= A[smem] * B[smem], e4m3 in, f32 out
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// f32 accumulation (1 in [4,6)), both formats e4m3 (0), both K-major, N>>3 and M>>4
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Joins the pieces of the cut items: out = sum_c 2^(lse_c - M) out_c / sum_c 2^(lse_c - M).
// grid (CTAs of the main launch, groups of 32 rows), a warp per D / 8 columns, a lane per row.
// Two pieces at a time go to shared memory by asynchronous copies, 128 bytes of a column each
// as they were written, so that an SM has most of its share on its way at once (in registers
// four waves of CTAs: 18 us for 37 MB, 13 so); the rows leave through shared memory, too.  CTAs past
// the main launch's write the rows of groups that see nothing.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int CW = D / 8;
  __shared__ __align__(16) float buf[2][D][32];
  float(*tile)[D + 1] = reinterpret_cast<float(*)[D + 1]>(&buf[0][0][0]);  // [32], when the pieces have been read
  static_assert(32 * (D + 1) <= 2 * D * 32, "");
  let_next_launch_in();
  wait_for_launch_ahead();
  const int c0 = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (c0 >= p.ctas) {
    const int span = p.pitch / kBM * p.tb;
    const int64_t all = static_cast<int64_t>(p.B) * p.MP * p.Hq;
    for (int64_t x = (c0 - p.ctas) * gridDim.y + blockIdx.y; x < all; x += (gridDim.x - p.ctas) * gridDim.y) {
      const int h = static_cast<int>(x % p.Hq), j = static_cast<int>(x / p.Hq), b = j / p.MP;
      const int i0 = (j - b * p.MP) * span;
      int start;
      bool past;
      if (i0 < seq_queries(p, b, start, past)) continue;
      for (int i = i0 + warp; i < min(i0 + span, p.T); i += kMergeThreads / 32) {
        const int64_t ob = b * p.out_stride[0] + h * p.out_stride[1] + i * p.out_stride[2];
        for (int d = 2 * lane; d < D; d += 64) {
          if (p.out_bf16)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + ob + d) = 0u;
          else
            *reinterpret_cast<float2*>(static_cast<float*>(p.out) + ob + d) = make_float2(0.f, 0.f);
        }
        if (lane == 0 && p.lse != nullptr) p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = -INFINITY;
      }
    }
    return;
  }
  const CutItem it = p.cuts[c0];
  if (it.pieces == 0) return;
  const int sr = blockIdx.y * 32 + lane;  // row of the partials
  auto place = [&](int r, int& i, int& h) {  // its query and head
    const int row = r % kBM;
    i = it.i0 + r / kBM * p.tb + row / p.G;
    h = it.g * p.G + row % p.G;
    return row < p.RT && i < p.T;
  };
  int i, h;
  const bool mine = place(sr, i, h);
  auto slot = [&](int c) { return static_cast<int64_t>(2 * (c0 + c) + ((c == 0 && !it.first_is_head) ? 1 : 0)); };
  // in order, with a running max
  float M = -INFINITY, acc[CW], ws = 0.f;
#pragma unroll
  for (int x = 0; x < CW; ++x) acc[x] = 0.f;
#pragma unroll 1
  for (int c = 0; c < it.pieces; c += 2) {
    const int n = min(2, it.pieces - c);
    if (c > 0) __syncthreads();  // the pieces before have been read
    float l[2] = {-INFINITY, -INFINITY};
    for (int k = 0; k < n; ++k) {
      const float* src = p.part_o + slot(c + k) * D * p.pitch + blockIdx.y * 32;
#pragma unroll
      for (int u = threadIdx.x; u < D * 8; u += kMergeThreads)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&buf[k][u / 8][u % 8 * 4])),
                     "l"(src + static_cast<int64_t>(u / 8) * p.pitch + u % 8 * 4)
                     : "memory");
      if (mine) l[k] = p.part_lse[slot(c + k) * p.pitch + sr];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const float top = fmaxf(M, fmaxf(l[0], l[1]));  // (a NaN gets to the row by its weight)
    const float alpha = M == -INFINITY ? 1.f : fast_exp2(M - top);
    M = top;
    ws *= alpha;
#pragma unroll
    for (int x = 0; x < CW; ++x) acc[x] *= alpha;
    for (int k = 0; k < n; ++k) {
      const float w = l[k] == -INFINITY ? 0.f : fast_exp2(l[k] - M);
      ws += w;
      if (w != 0.f) {  // (rows that are not there hold anything)
#pragma unroll
        for (int x = 0; x < CW; ++x) acc[x] = fmaf(w, buf[k][warp * CW + x][lane], acc[x]);
      }
    }
  }
  __syncthreads();  // (the tile takes the pieces' place)
  const bool any = !(ws == 0.f);  // a NaN is something
  const float inv = any ? 1.f / ws : 0.f;
#pragma unroll
  for (int x = 0; x < CW; ++x) tile[lane][warp * CW + x] = any ? acc[x] * inv : 0.f;
  if (warp == 0 && mine && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(it.b) * p.Hq + h) * p.T + i] =
        any ? (M + __log2f(ws)) * 0.6931471805599453f : -INFINITY;
  __syncthreads();
  const int r = threadIdx.x / 8, d = threadIdx.x % 8 * CW;
  if (!place(blockIdx.y * 32 + r, i, h)) return;
  const int64_t ob = it.b * p.out_stride[0] + h * p.out_stride[1] + i * p.out_stride[2] + d;
  const float* x = &tile[r][d];
  if (p.out_bf16) {
#pragma unroll
    for (int k = 0; k < CW; k += 4)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ob + k) =
          make_uint2(pack_bf16x2(x[k], x[k + 1]), pack_bf16x2(x[k + 2], x[k + 3]));
  } else {
#pragma unroll
    for (int k = 0; k < CW; k += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ob + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    paged_chunk_f8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ChunkParams p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  const int span = NT * p.tb;  // queries of a row group

  if (threadIdx.x == 32) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_raw[t], 1);
      mbar_init(&bars->q_full[t], NT == 1 ? 8 : 4);
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 5);  // four softmax warps, and warp 2
      mbar_init(&bars->xch_full[t], 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->c_full[s], 1);
      mbar_init(&bars->c_empty[s], 4);
      mbar_init(&bars->v_full[s], 4);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int s = 0; s < kScales; ++s) mbar_init(&bars->sc_full[s], 1);
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&bars->seg_full[s], 1);
      mbar_init(&bars->seg_empty[s], 15);  // the producer, the issuer, warp 2, 4 converting and 8 softmax warps
    }
    for (int s = 0; s < kNotes; ++s) mbar_init(&bars->conv[s], 4);
    mbar_init(&bars->o_free, 8);
    mbar_init(&bars->drained, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  let_next_launch_in();
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  wait_for_launch_ahead();
  // the planner's state: the call's runs, and the place of this CTA's first tile.  A pair
  // is a (sequence, row group), Hkv items of the same length.
  Runs runs = {};
  int pos = 0, hi = 0, lo = 0;
  int plan_j = 0, plan_g = 0, plan_t = 0;
  auto pair = [&](int j, int& start, int& n, int& i0, bool& past) {  // its tiles
    const int b = j / p.MP;
    n = seq_queries(p, b, start, past);
    i0 = (j - b * p.MP) * span;
    return key_tiles(group_keys(p, start, n, i0, span));
  };
  if (warp == 3) {
    // (all counts are below 2^31: f8_chunk_fits)
    const int pairs = p.B * p.MP;
    int total = 0, mine0 = 0;
    auto units = [&](int j, bool first) {
      if (j >= pairs) return 0;
      int start, n, i0;
      bool past;
      const int t = pair(j, start, n, i0, past);
      if (first && blockIdx.x == 0 && i0 == 0 && past) report(p.status, kStatusBounds);
      return t > 0 ? (kItemCost + t) * p.Hkv : 0;
    };
#pragma unroll 1
    for (int base = 0; base < pairs; base += 32) {
      const int mine = units(base + lane, true);
      if (base == 0) mine0 = mine;
      total += mine;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    const int c = static_cast<int>(blockIdx.x);
    runs = Runs::make(total, static_cast<int>(gridDim.x));
    if (c < runs.n) lo = runs.lo(c), hi = runs.lo(c + 1);
    pos = lo;
    int run = 0;
#pragma unroll 1
    for (int base = 0; base < pairs && lo < hi; base += 32) {
      const int mine = base == 0 ? mine0 : units(base + lane, false);
      int incl = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + incl > lo);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        const int local = lo - run - __shfl_sync(0xffffffffu, incl - mine, l);
        const int each = __shfl_sync(0xffffffffu, mine, l) / p.Hkv;
        plan_j = base + l;
        plan_g = local / each;
        plan_t = local - plan_g * each - kItemCost;
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      p.cuts[blockIdx.x].pieces = 0;  // unless an item starts here and goes on
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

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
  auto wait_all = [&](uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort, p.status)) != 0;
  };

  if (warp < 8) regs_dec<C::kRegsCtl>();
  if (warp == 0) {
    // ------------------------------------------------------------ K and V codes
    // Four tiles' blocks are looked up at a time, a lane each: ids a window ahead, scales
    // three tiles ahead, so that no tile waits for either.
    constexpr int kWindow = 32 / kTileBlocks;
    const int own = lane % kTileBlocks, wt = lane / kTileBlocks;  // the block of a tile, the tile of a window
    Seg s;
    int j = 0, k_issued = 0, c_issued = 0;
    bool ok = true;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const int32_t* bt_row = p.bt + static_cast<int64_t>(s.b) * p.bt_stride;
      const int blocks = (s.kend + kBS - 1) / kBS;
      auto block_id = [&](int tile0) {  // of the window that starts there; -1 past the segment
        const int tile = tile0 + wt, blk = tile * kTileBlocks + own;
        return tile < s.t1 && blk < blocks ? bt_row[blk] : INT_MIN;
      };
      float sck = -1.0f, scv = -1.0f;
      auto look = [&](int& id) {  // the id, checked, and its scales
        sck = scv = -1.0f;
        if (id >= 0 && id < p.num_blocks) {
          const int64_t at = static_cast<int64_t>(id) * p.Hkv + s.g;
          sck = p.ks[at];
          scv = p.vs[at];
        } else {
          if (id != INT_MIN) report(p.status, kStatusBounds);
          id = -1;
        }
      };
      int id_next = block_id(s.t0);
      look(id_next);
      int id = -1;
      float ks_id = -1.0f, vs_id = -1.0f;
      for (int tile = s.t0; tile < s.t1; ++tile, ++j) {
        const int w = (tile - s.t0) % kWindow;
        if (w == 0) {
          id = id_next, ks_id = sck, vs_id = scv;
          id_next = block_id(tile + kWindow);
        } else if (w == 1) {
          look(id_next);
        }
        const bool owns = wt == w;
        const uint32_t there = (__ballot_sync(0xffffffffu, id >= 0) >> (w * kTileBlocks)) & 0xffu;
        const uint32_t bytes = __popc(there) * (kBS * D);
        const int ks = j % C::KS, cs = j % C::VC;
        if (!wait_all(&bars->k_empty[ks], (j / C::KS) ^ 1)) {
          ok = false;
          break;
        }
        // (the tile that had this slot is kScales back: its weights are written)
        if (owns) bars->ks[j % kScales][own] = ks_id;
        if (lane == 0) bars->there[j % kScales] = there;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->sc_full[j % kScales]);
          mbar_arrive_expect_tx(&bars->k_full[ks], bytes);
        }
        __syncwarp();
        if (owns && id >= 0)
          tma_load_4d(smem + C::kOffK + ks * C::kCodeBytes + own * (kBS * D), &tm_k, &bars->k_full[ks], 0, 0, s.g, id);
        k_issued = j + 1;
        if (!wait_all(&bars->c_empty[cs], (j / C::VC) ^ 1)) {
          ok = false;
          break;
        }
        if (owns) bars->vs[cs][own] = vs_id;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&bars->c_full[cs], bytes);
        __syncwarp();
        if (owns && id >= 0)
          tma_load_4d(smem + C::kOffC + cs * C::kCodeBytes + own * (kBS * D), &tm_v, &bars->c_full[cs], 0, 0, s.g, id);
        c_issued = j + 1;
      }
    }
    if (lane == 0 && *abort) {  // let every copy in flight land before the CTA exits
      for (int x = max(0, k_issued - C::KS); x < k_issued; ++x) drain_wait(&bars->k_full[x % C::KS], (x / C::KS) & 1);
      for (int x = max(0, c_issued - C::VC); x < c_issued; ++x) drain_wait(&bars->c_full[x % C::VC], (x / C::VC) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp goes through the loop, with values that are alike in all lanes
    // (uniform registers, which the descriptors have to be in), and one lane issues.
    constexpr uint32_t idesc_o = idesc_bf16_f32(kBM, D, false, true);
    constexpr uint32_t half = PagedTile<D>::kHalf, group = PagedTile<D>::kGroup;
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uni(tmem);
    auto issue_s = [&](int w, int r, int keys, bool free) {  // S_w = Q K^T, ring tile r
      const uint32_t idesc_s = idesc_e4m3_f32(kBM, keys);
      const uint32_t qa = smem_u32(smem + C::kOffQ) + (NT == 2 ? w * 2 * C::kQBytes : 0);
      const uint64_t dq = C::code_desc(qa);
      const uint64_t dk = C::code_desc(smem_u32(smem + C::kOffK) + (r % C::KS) * C::kCodeBytes);
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < 2; ++x)  // hi, lo
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)  // 32 codes
            umma_e4m3_ss(tm + w * 128, dq + x * (C::kQBytes >> 4) + kk * 2, dk + kk * 2, idesc_s,
                         x + kk > 0 ? 1u : 0u);
        umma_commit(&bars->s_full[w]);
        if (free) umma_commit(&bars->k_empty[r % C::KS]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int w, int r, int keys, bool first, bool free) {  // O_w (+)= P_w V
      const uint64_t dv = sdesc_sw128(smem_u32(smem + C::kOffV) + (r % C::VS) * C::kTileBytes, half, group);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) {
          if (kk * 16 >= keys) break;
          umma_bf16_ts(tm + C::kColO + w * D, tm + w * 128 + kk * 8, dv + kk * (group >> 3), idesc_o,
                       (!first || kk > 0) ? 1u : 0u);
        }
        umma_commit(&bars->o_done[w]);
        if (free) umma_commit(&bars->v_empty[r % C::VS]);
      }
      __syncwarp();
    };
    auto wait_k = [&](int x) { return wait_all(&bars->k_full[x % C::KS], x / C::KS); };
    int j = 0;
    bool ok = true;
    Seg sg;
    for (int seg = 0; ok && seg_get(seg, sg); ++seg) {
      seg_taken(seg);
      const int t0 = uni(sg.t0), n = uni(sg.t1) - t0, kend = uni(sg.kend);
      auto keys = [&](int x) { return tile_keys(kend, t0 + x); };
      for (int t = 0; t < NT; ++t) ok = ok && wait_all(&bars->q_full[t], seg);
      if constexpr (NT == 1) {
        // tile j is warpgroup j & 1's; S runs two tiles ahead of PV
#pragma unroll 1
        for (int x = 0; ok && x < n + 2; ++x) {
          if (x >= 2) {  // P_(x - 2) V, before S_x takes its scores' place
            const int y = x - 2;
            // the accumulators of the segment before have been read
            if (y == 0 && seg > 0) ok = wait_all(&bars->o_free, seg - 1);
            ok = ok && wait_all(&bars->p_full[(j + y) & 1], (j + y) >> 1);
            if (!ok) break;
            tc_fence_after();
            issue_pv((j + y) & 1, j + y, keys(y), y < 2, true);
          } else if (x < n) {
            ok = wait_k(j + x);
            if (!ok) break;
            tc_fence_after();
          }
          if (x < n) issue_s((j + x) & 1, j + x, keys(x), true);
        }
        j += n;
      } else {
        // PV_A, S_A', PV_B, S_B': each tile's softmax runs under the other's MMAs
        ok = ok && wait_k(j);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, j, keys(0), false);
        issue_s(1, j, keys(0), true);
#pragma unroll 1
        for (int x = 0; ok && x < n; ++x, ++j) {
          const bool more = x + 1 < n;
#pragma unroll 1
          for (int w = 0; ok && w < 2; ++w) {
            ok = wait_all(&bars->p_full[w], j);
            if (!ok) break;
            tc_fence_after();
            issue_pv(w, j, keys(x), x == 0, w == 1);
            if (more) issue_s(w, j + 1, keys(x + 1), w == 1);
          }
        }
      }
    }
    // no MMA may be in flight when the TMEM is freed
    if (elect_one()) {
      umma_commit(&bars->drained);
      drain_wait(&bars->drained, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ the issuer's waits
    // For each tile, that its V is there and the K of the scores that the issuer goes on
    // with: one arrival more on p_full, so that the issuer has one wait (each takes it
    // over 200 cycles, ready or not) instead of three.
    Seg s;
    int j = 0;
    bool ok = true;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const int n = s.t1 - s.t0;
      for (int x = 0; ok && x < n; ++x, ++j) {
        constexpr int kAhead = NT == 1 ? 2 : 1;  // tiles that the scores are ahead
        const int k = j + kAhead;
        ok = wait_all(&bars->v_full[j % C::VS], j / C::VS) &&
             (x + kAhead >= n || wait_all(&bars->k_full[k % C::KS], k / C::KS));
        for (int w = 0; w < 2; ++w) {
          if (NT == 1 && w != (j & 1)) continue;
          const int phase = NT == 1 ? j >> 1 : j;  // the one before is over: this arrival is not its
          ok = ok && (phase == 0 || wait_all(&bars->p_full[w], phase - 1));
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars->p_full[w]);
        }
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ planner
    int start = 0, n = 0, i0 = 0, tiles = 0;
    bool past = false;
    if (pos < hi) tiles = pair(plan_j, start, n, i0, past);
    for (int i = 0;; ++i) {
      Seg s = {};
      s.b = -1;
      if (pos < hi && plan_t == tiles) {  // the item is done: the next KV head, or the next pair
        plan_t = -kItemCost;
        if (++plan_g == p.Hkv) {
          plan_g = 0;
          // (there is more to do, so an item follows)
          do tiles = pair(++plan_j, start, n, i0, past);
          while (tiles == 0 && plan_j + 1 < p.B * p.MP);
        }
      }
      if (plan_t < 0) {  // the item's own cost, or as much of it as falls into this run
        const int skip = min(-plan_t, hi - pos);
        pos += skip;
        plan_t += skip;
      }
      if (pos < hi) {
        s.b = plan_j / p.MP;
        s.g = plan_g;
        s.i0 = i0;
        s.t0 = plan_t;
        s.t1 = min(tiles, plan_t + (hi - pos));
        s.start = start;
        s.n = n;
        s.kend = group_keys(p, start, n, i0, span);
        const bool whole = s.t0 == 0 && s.t1 == tiles;
        s.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (i == 0 ? 0 : 1);
        if (!whole && s.t0 == 0 && lane == 0) {  // cut, and it starts here
          CutItem it;
          it.b = s.b, it.g = s.g, it.i0 = i0;
          it.pieces = runs.of(pos + tiles - 1) - static_cast<int>(blockIdx.x) + 1;
          it.first_is_head = i == 0;
          p.cuts[blockIdx.x] = it;
        }
        pos += s.t1 - plan_t;
        plan_t = s.t1;
      }
      if (!wait_all(&bars->seg_empty[i % kSegs], (i / kSegs) ^ 1)) break;
      if (lane == 0) {
        bars->segs[i % kSegs] = s;
        mbar_arrive(&bars->seg_full[i % kSegs]);
      }
      if (s.b < 0) break;
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ V to bf16
    // A lane takes a row's 16 codes at a time.  A quarter warp is four neighbouring
    // chunks of rows r and r ^ 5: loads and stores then meet no bank twice.
    constexpr int CH = D / 16;
    const int cw = warp - 4;
    const int r8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), c0 = lane & 3;
    Seg s;
    int j = 0;
    bool ok = true;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      // tokens from here on are not seen by all rows of the item
      const int first = p.causal ? s.start + s.i0 + 1 : 0x7fffffff;
      uint32_t* notes = bars->bad[i % kNotes][cw];
      if (lane < kSpread / 32) notes[lane] = 0u;
      __syncwarp();
      for (int tile = s.t0; tile < s.t1; ++tile, ++j) {
        const int cs = j % C::VC, vs = j % C::VS;
        if (!wait_all(&bars->c_full[cs], j / C::VC) || !wait_all(&bars->v_empty[vs], (j / C::VS) ^ 1)) {
          ok = false;
          break;
        }
        const uint8_t* src = smem + C::kOffC + cs * C::kCodeBytes;
        uint8_t* dst = smem + C::kOffV + vs * C::kTileBytes;
        const int left = s.kend - tile * kBN;      // keys there are
        const int keys = tile_keys(s.kend, tile);  // rows that the product reads
        const bool watch = tile * kBN + kBN > first;
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const int r = cw * 32 + x * 8 + r8;
          if (cw * 32 + x * 8 >= keys) break;
          const float sc = bars->vs[cs][r / kBS];  // -1: no such block
          const bool on = sc != -1.0f;
          const uint64_t sc2 = f2_pack(on ? sc : 0.0f, on ? sc : 0.0f);
          uint32_t u[CH / 4][4];
#pragma unroll
          for (int y = 0; y < CH / 4; ++y) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (on && r < left) w = *reinterpret_cast<const uint4*>(src + C::code_off(r, c0 + 4 * y));
            u[y][0] = w.x, u[y][1] = w.y, u[y][2] = w.z, u[y][3] = w.w;
          }
          const int token = tile * kBN + r;
          if (watch && token >= first - 1) {  // not all rows see it: NaNs go in as zeros
            uint32_t any = 0u;
#pragma unroll
            for (int y = 0; y < CH / 4; ++y)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t bad = nan_codes(u[y][k]);
                any |= bad;
                u[y][k] &= ~((bad >> 7) * 255u);
              }
            const int at = token - (first - 1);
            if (any != 0u && at < kSpread) atomicOr(&notes[at >> 5], 1u << (at & 31));
          }
#pragma unroll
          for (int y = 0; y < CH / 4; ++y) {
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float lo, hi;
              half2_f32(f8_half2(k & 1 ? u[y][k >> 1] >> 16 : u[y][k >> 1]), lo, hi);
              f2_unpack(fmul2(f2_pack(lo, hi), sc2), lo, hi);
              o[k] = pack_bf16x2(lo, hi);
            }
            const int c = 2 * (c0 + 4 * y);
            *reinterpret_cast<uint4*>(dst + swizzled_off(r, c, PagedTile<D>::kHalf, PagedTile<D>::kGroup)) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + swizzled_off(r, c + 1, PagedTile<D>::kHalf, PagedTile<D>::kGroup)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->v_full[vs]);
          mbar_arrive(&bars->c_empty[cs]);
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars->conv[i % kNotes]);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ softmax
    regs_inc<C::kRegsSoft>();
    const int wg = (warp >> 2) - 2;
    const int t = NT == 2 ? wg : 0;  // row tile
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = wg * 128, o_col = C::kColO + wg * D;
    float2* xch = reinterpret_cast<float2*>(smem + C::kOffXch);
    // PV of this warpgroup's tile number x (of all it has had) is done.  Asked only
    // about the latest one or the one before: the parity is never read a phase off.
    auto o_wait = [&](int x) { return mbar_wait(&bars->o_done[wg], x & 1, abort, p.status); };

    // The rows of q that this warp splits: its 32, or (NT = 1) half of them, the other
    // warpgroup's warp the rest.
    constexpr int kQRows = NT == 2 ? 32 : 16;
    const int q_row0 = NT == 2 ? 0 : wg * kQRows;
    // A row tile's queries, two boxes: rows' first halves to where hi will be, second
    // halves to lo's place.  Called when every S of the segment before is done; they land
    // while that one ends.
    const bool loads_q = quarter == 0 && lane == 0 && (NT == 2 || wg == 0);
    int q_loads = 0;
    auto load_q = [&](const Seg& n) {
      if (!loads_q) return;
      mbar_arrive_expect_tx(&bars->q_raw[t], static_cast<uint32_t>(p.RT) * 2u * D);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        tma_load_5d(smem + C::kOffQ + (2 * t + x) * C::kQBytes, &tm_q, &bars->q_raw[t], x * (D / 2), 0,
                    n.i0 + t * p.tb, n.g, n.b);
      ++q_loads;
    };

    Seg s;
    bool ok = true;
    int j = 0, n_mine = 0;  // tiles so far, and those that this warpgroup has had
    for (int seg = 0; ok && seg_get(seg, s); ++seg) {
      seg_taken(seg);
      if (seg == 0) load_q(s);
      const int qi = s.i0 + t * p.tb + row / p.G;     // the row's query
      const bool mine = row < p.RT && qi < p.T;       // the row exists
      const bool sees = row < p.RT && qi < s.n;       // and has keys
      const bool warp_on = __any_sync(0xffffffffu, mine);
      const int head = s.g * p.G + row % p.G;
      // (a row that sees nothing has zeros for q, and no limit that would hold up its warp:
      // its results are not used)
      const int row_lim = !sees ? 0x7fffffff : (p.causal ? s.start + qi + 1 : s.kend);

      // ---- q, from where load_q left it, as hi and lo: what a row's lanes (16 bytes each)
      // write is what they have read.  Rolled, four steps at a time: it runs once a segment,
      // and code that does costs its fetch.
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->q_raw[t], seg & 1, abort, p.status))) {
        ok = false;
        break;
      }
      if (warp_on) {
        constexpr int LPR = D / 8, RPI = 32 / LPR, NI = kQRows / RPI;  // lanes a row, rows a step, steps
        uint8_t* qs = smem + C::kOffQ + t * 2 * C::kQBytes;
        const int row0 = quarter * 32 + q_row0 + lane / LPR, c = lane % LPR;
        const uint32_t seen = __ballot_sync(0xffffffffu, sees);
#pragma unroll 1
        for (int it0 = 0; it0 < NI; it0 += 4) {
          uint32_t h[4][4], l[4][4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = row0 + (it0 + y) * RPI;
            uint4 w = *reinterpret_cast<const uint4*>(qs + c / (LPR / 2) * C::kQBytes + C::code_off(r, c % (LPR / 2)));
            // rows that see nothing may hold anything
            if (!((seen >> (r & 31)) & 1u)) w = make_uint4(0u, 0u, 0u, 0u);
            uint32_t top = bf16x2_max_abs(bf16x2_max_abs(w.x & 0x7fff7fffu, w.y), w.z);  // (a NaN is not the largest)
            top = bf16x2_max_abs(top, w.w);
#pragma unroll
            for (int m = 1; m < LPR; m *= 2) top = bf16x2_max_abs(top, __shfl_xor_sync(0xffffffffu, top, m));
            const float a = fmaxf(bf16lo_to_f32(top), bf16hi_to_f32(top));
            const int e = a > 0.0f && a < INFINITY ? f8_scale_exponent(a) : 0;
            // infinite scores make no distribution either
            const float inv = a < INFINITY ? pow2(-e) : NAN;
            const uint64_t inv2 = f2_pack(inv, inv);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x0, x1, y0, y1;
              f2_unpack(fmul2(f2_pack(bf16lo_to_f32(u[k]), bf16hi_to_f32(u[k])), inv2), x0, x1);
              h[y][k] = f8_codes(x0, x1);
              half2_f32(f8_half2(h[y][k]), y0, y1);
              l[y][k] = f8_codes(x0 - y0, x1 - y1);
            }
            if (c == 0) bars->qmul[t][r] = p.scale_log2 * pow2(e);
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t at = C::code_off(row0 + (it0 + y) * RPI, c / 2) + c % 2 * 8;
            *reinterpret_cast<uint2*>(qs + at) = make_uint2(h[y][0] | h[y][1] << 16, h[y][2] | h[y][3] << 16);
            *reinterpret_cast<uint2*>(qs + C::kQBytes + at) =
                make_uint2(l[y][0] | l[y][1] << 16, l[y][2] | l[y][3] << 16);
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_full[t]);
      if (NT == 1 && !__all_sync(0xffffffffu, mbar_wait(&bars->q_full[0], seg & 1, abort, p.status))) {
        ok = false;
        break;
      }
      const float mul = bars->qmul[t][row];  // log2 units of a score of q's codes with unscaled K codes

      const int mine_before = n_mine;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int tile = s.t0; ok && tile < s.t1; ++tile, ++j) {
        if (NT == 1 && (j & 1) != wg) continue;
        const int keys = tile_keys(s.kend, tile);
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->sc_full[j % kScales], (j / kScales) & 1, abort, p.status) &&
                                         mbar_wait(&bars->s_full[wg], n_mine & 1, abort, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (warp_on) {
          const uint32_t there = bars->there[j % kScales];
          const int lim = row_lim - tile * kBN;
          const bool masked = __any_sync(0xffffffffu, lim < kBN) || there != 0xffu;
          const float* ks = bars->ks[j % kScales];
          float alpha = 1.0f;
          bool raised = false;  // the reference max may have moved (alike in the warp)
          // it moves only when the step's exceeds it by the margin
          auto raise = [&](float mt) {
            raised = true;
            if (mt > m_run + kRescaleMargin || (m_run == -INFINITY && mt != -INFINITY)) {
              alpha = fast_exp2(m_run - mt);
              m_run = mt;
            }
          };
          // weights 2^(f s + neg) of 32 scores, f by block, and their sums
          auto weigh32 = [&](const uint32_t (&x)[32], uint32_t (&pw)[16], float f0, float f1, float neg,
                             uint64_t (&sum)[4]) {
            const uint64_t neg2 = f2_pack(neg, neg);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float f = i < 16 ? f0 : f1;
              float x0, x1;
              f2_unpack(ffma2(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), f2_pack(f, f), neg2), x0,
                        x1);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              pw[i >> 1] = pack_bf16x2(p0, p1);
              sum[(i >> 1) & 3] = fadd2(sum[(i >> 1) & 3], f2_pack(p0, p1));
            }
          };
          // scores in log2 units, -inf where the row may not look
          auto scale32 = [&](uint32_t (&x)[32], int c, float f0, float f1) {
            const int lim0 = (there >> (2 * c)) & 1u ? lim - c * 32 : 0;
            const int lim1 = (there >> (2 * c + 1)) & 1u ? lim - c * 32 : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = i < (i < 16 ? lim0 : lim1) ? __float_as_uint(__uint_as_float(x[i]) * (i < 16 ? f0 : f1))
                                                : 0xff800000u;
          };
          auto max32 = [&](const uint32_t (&x)[32], float (&mx)[4]) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx[(i >> 1) & 3] = fmax3(mx[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          };
          uint64_t sum[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = f2_pack(0.f, 0.f);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          bool done = false;
          // Bound by this chain's latency: scores go to registers, half of them ahead of the
          // others, and are weighed against the reference max at hand, without a max
          // pass, unless some row's sum says its scores outgrew it.
          if (!masked && __all_sync(0xffffffffu, m_run != -INFINITY)) {
            uint32_t sr[4][32], pw[4][16];
            tmem_ld32(tmem + lane_addr + s_col, sr[0]);
            tmem_ld32(tmem + lane_addr + s_col + 32, sr[1]);
            tmem_wait_ld(sr[0]);
            tmem_wait_ld(sr[1]);
            tmem_ld32(tmem + lane_addr + s_col + 64, sr[2]);
            tmem_ld32(tmem + lane_addr + s_col + 96, sr[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c == 2) {
                tmem_wait_ld(sr[2]);
                tmem_wait_ld(sr[3]);
              }
              weigh32(sr[c], pw[c], mul * ks[2 * c], mul * ks[2 * c + 1], -m_run, sum);
            }
            float a0, a1;
            f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), a0, a1);
            // What the margin lets through (above it some weight is past the margin, so that the passes
            // below do move the max): the accumulators hold values up to 2^92.  False for a NaN.
            static_assert(kRescaleMargin == 8.0f, "2^kRescaleMargin below");
            done = __all_sync(0xffffffffu, a0 + a1 <= kBN * 256.0f);
            if (done) {
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_st16(tmem + lane_addr + s_col + c * 16, pw[c]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] = f2_pack(0.f, 0.f);
            }
          }
          if (!done) {
            // Two rolled passes over the scores in TMEM, 32 at a time (code that runs once costs
            // its fetch).  The second writes P over scores that it has read.
            const int nc = (keys + 31) / 32;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              const float f0 = mul * ks[2 * c], f1 = mul * ks[2 * c + 1];
              uint32_t x[32];
              tmem_ld32(tmem + lane_addr + s_col + c * 32, x);
              tmem_wait_ld(x);
              scale32(x, c, f0, f1);
              max32(x, mx);
            }
            raise(fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])));
            const float neg = m_run == -INFINITY ? 0.0f : -m_run;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              const float f0 = mul * ks[2 * c], f1 = mul * ks[2 * c + 1];
              uint32_t x[32], pw[16];
              tmem_ld32(tmem + lane_addr + s_col + c * 32, x);
              tmem_wait_ld(x);
              if (masked) {
                scale32(x, c, f0, f1);
                weigh32(x, pw, 1.0f, 1.0f, neg, sum);
              } else {
                weigh32(x, pw, f0, f1, neg, sum);
              }
              tmem_st16(tmem + lane_addr + s_col + c * 16, pw);
            }
          }
          if (raised && n_mine > mine_before && __any_sync(0xffffffffu, alpha != 1.0f)) {
            if (!__all_sync(0xffffffffu, o_wait(n_mine - 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tmem + lane_addr + o_col + c * 32, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tmem + lane_addr + o_col + c * 32, o);
            }
          }
          tmem_wait_st();
          float a0, a1;
          f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), a0, a1);
          l_run = l_run * alpha + (a0 + a1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[wg]);
        ++n_mine;
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      // NT = 1: both warpgroups' states joined; warpgroup w writes half w of the output
      // columns.  f0, f1: what accumulators 0 and 1 weigh.
      float f0 = 1.0f, f1 = 1.0f;
      if constexpr (NT == 1) {
        // the other warpgroup has read the segment before's
        if (seg > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->o_free, (seg - 1) & 1, abort, p.status))) {
          ok = false;
          break;
        }
        xch[wg * kBM + row] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->xch_full[wg]);
        const int others = j - n_mine;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&bars->xch_full[wg ^ 1], seg & 1, abort, p.status) &&
                            (n_mine == 0 || mbar_wait(&bars->o_done[wg], (n_mine - 1) & 1, abort, p.status)) &&
                            (others == 0 || mbar_wait(&bars->o_done[wg ^ 1], (others - 1) & 1, abort, p.status)))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float2 a = xch[row], b = xch[kBM + row];
        const float M = fmaxf(a.x, b.x);
        // a state without tiles (or keys) has max -inf and sum 0: weight 0
        f0 = a.x == -INFINITY && !(a.y != 0.0f) ? 0.0f : fast_exp2(a.x - M);
        f1 = b.x == -INFINITY && !(b.y != 0.0f) ? 0.0f : fast_exp2(b.x - M);
        m_run = M;
        l_run = f0 * a.y + f1 * b.y;
        if (s.t1 - s.t0 == 1) {  // one tile: the other accumulator holds an older segment's
          if ((j & 1) == 0)
            f0 = 0.0f;
          else
            f1 = 0.0f;
        }
      } else {
        if (!__all_sync(0xffffffffu, o_wait(n_mine - 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      {
        Seg ahead;
        if (seg_get(seg + 1, ahead)) load_q(ahead);
      }
      // tokens from i0 on that this row sees and whose V holds a NaN (none of an earlier part's)
      const bool straddles = p.causal && s.t1 * kBN > s.start + s.i0 + 1;
      bool fix = false;
      if (straddles) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->conv[seg % kNotes], (seg / kNotes) & 1, abort, p.status))) {
          ok = false;
          break;
        }
        uint32_t any = 0u;
#pragma unroll
        for (int x = 0; x < 4 * kSpread / 32; ++x) any |= bars->bad[seg % kNotes][0][x];
        fix = any != 0u;  // alike in the whole warp
      }
      const bool empty = !sees || l_run == 0.0f;
      const bool whole = s.slot < 0;
      const float inv = empty ? 0.0f : 1.0f / l_run;
      const float lse2 = empty ? -INFINITY : m_run + __log2f(l_run);
      const int64_t obase = s.b * p.out_stride[0] + head * p.out_stride[1] + qi * p.out_stride[2];
      if (warp_on) {
        // 32 columns at a time, rolled (it runs once a segment: its code's fetch counts)
#pragma unroll 1
        for (int c = NT == 1 ? wg * (D / 2) : 0; c < (NT == 1 ? (wg + 1) * (D / 2) : D); c += 32) {
          uint32_t o[32];
          if constexpr (NT == 2) {
            tmem_ld32(tmem + lane_addr + o_col + c, o);
            tmem_wait_ld(o);
          } else {
            uint32_t o1[32];
            tmem_ld32(tmem + lane_addr + C::kColO + c, o);
            tmem_ld32(tmem + lane_addr + C::kColO + D + c, o1);
            tmem_wait_ld(o);
            tmem_wait_ld(o1);
            // an accumulator of weight 0 may hold anything
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint((f0 != 0.0f ? f0 * __uint_as_float(o[i]) : 0.0f) +
                                     (f1 != 0.0f ? f1 * __uint_as_float(o1[i]) : 0.0f));
          }
          if (mine) {
            if (fix) {
#pragma unroll 1
              for (int x = 0; x < kSpread; ++x) {
                const int token = s.start + s.i0 + x;
                uint32_t word = 0u;
                for (int w = 0; w < 4; ++w) word |= bars->bad[seg % kNotes][w][x >> 5];
                if (!((word >> (x & 31)) & 1u) || token >= row_lim || !sees) continue;
                const int id = p.bt[static_cast<int64_t>(s.b) * p.bt_stride + token / kBS];
                if (id < 0 || id >= p.num_blocks) continue;
                const uint8_t* v =
                    p.vq + ((static_cast<int64_t>(id) * p.Hkv + s.g) * kBS + token % kBS) * static_cast<int64_t>(D) + c;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((v[i] & 0x7f) == 0x7f) o[i] = 0x7fc00000u;
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = empty ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
            if (!whole) {
              float* dst = p.part_o + (static_cast<int64_t>(s.slot) * D + c) * p.pitch + t * kBM + row;
#pragma unroll
              for (int i = 0; i < 32; ++i) dst[i * (NT * kBM)] = __uint_as_float(o[i]);
            } else if (p.out_bf16) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + obase + c);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])));
            } else {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + obase + c);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                     __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
            }
          }
          __syncwarp();
        }
        if (mine && (NT == 2 || wg == 0)) {
          if (!whole)
            p.part_lse[static_cast<int64_t>(s.slot) * p.pitch + t * kBM + row] = lse2;
          else if (p.lse != nullptr)
            p.lse[(static_cast<int64_t>(s.b) * p.Hq + head) * p.T + qi] = lse2 * 0.6931471805599453f;
        }
      }
      tc_fence_before();  // O is read: the next segment's PV may overwrite it
      if constexpr (NT == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free);
      }
    }
    if (q_loads > 0 && *abort) drain_wait(&bars->q_raw[t], (q_loads - 1) & 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int tile_queries(int64_t T, int64_t G) { return static_cast<int>(std::min(T, kBM / G)); }
// One row tile where it holds all rows (16 x 16 tokens of 4 heads behind 8192: 87 us, with two tiles
// 96; 16 x 32 behind 4000: 56, 64), else two (2 x 1024 behind 8192 189 us, 279 with one at a
// time; 16 x 40 behind 2000 50, 66).
int chunk_nt(int64_t T, int64_t G) { return T <= kBM / G ? 1 : 2; }
size_t part_rows(int64_t T, int64_t G, int n_cta) { return static_cast<size_t>(2) * n_cta * chunk_nt(T, G) * kBM; }
size_t part_bytes(int64_t T, int64_t G, int D, int n_cta) {
  return (part_rows(T, G, n_cta) * (D + 1) * sizeof(float) + 255) & ~size_t(255);
}

template <int D, int NT>
cudaError_t launch(const F8AttnArgs& a, const ChunkParams& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  CUtensorMap mq, mk, mv;
  if (!make_half_rows_map(&mq, a.q, a.cache.Hkv, p.tb, D) ||
      !make_code_map(&mk, a.cache.k, a.cache.num_blocks, a.cache.Hkv, D) ||
      !make_code_map(&mv, a.cache.v, a.cache.num_blocks, a.cache.Hkv, D))
    return cudaErrorInvalidValue;
  auto kern = paged_chunk_f8_kernel<D, NT>;
  {
    // the setmaxnreg split must fit in what the launch gives (a larger one waits forever)
    static const bool fits = [&] {
      cudaFuncAttributes fa;
      return cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
             256 * C::kRegsCtl + 256 * C::kRegsSoft <= fa.numRegs * C::kThreads;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
  }
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_early(kern, dim3(static_cast<unsigned>(a.n_cta)), C::kThreads, C::kSmemBytes, stream, mq, mk, mv, p);
  if (e != cudaSuccess) return e;
  // groups of 32 rows up to the last that any row tile uses
  // (and, for groups that see nothing, a few CTAs more)
  const int64_t heads = static_cast<int64_t>(p.B) * p.MP * p.Hq;
  const dim3 grid(static_cast<unsigned>(a.n_cta + std::min<int64_t>(a.n_cta, (heads + 31) / 32)),
                  static_cast<unsigned>(((NT - 1) * kBM + p.RT + 31) / 32));
  return launch_early(chunk_merge_kernel<D>, grid, kMergeThreads, 0, stream, p);
}

}  // namespace

size_t f8_chunk_partial_bytes(int64_t T, int64_t G, int D, int n_cta) {
  return part_bytes(T, G, D, n_cta) + ((n_cta * sizeof(CutItem) + 255) & ~size_t(255));
}

bool f8_chunk_fits(int64_t B, int64_t Hkv, int64_t T, int64_t G, int64_t max_blocks) {
  const int64_t span = chunk_nt(T, G) * tile_queries(T, G);
  const int64_t units = (max_blocks * kBS + kBN - 1) / kBN + 1 + kItemCost;
  return B * Hkv * ((T + span - 1) / span) <= 0x7fffffff / units;
}

cudaError_t launch_chunk_f8(const F8AttnArgs& a, cudaStream_t stream) {
  ChunkParams p = {};
  p.B = static_cast<int>(a.B);
  p.T = static_cast<int>(a.T);
  p.Hq = static_cast<int>(a.Hq);
  p.Hkv = a.cache.Hkv;
  p.G = p.Hq / p.Hkv;
  const int nt = chunk_nt(p.T, p.G);
  p.tb = tile_queries(p.T, p.G);
  p.RT = p.tb * p.G;
  p.MP = (p.T + nt * p.tb - 1) / (nt * p.tb);
  p.causal = a.causal;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.q = static_cast<const uint16_t*>(a.q.data);
  for (int i = 0; i < 3; ++i) p.q_stride[i] = a.q.stride[i], p.out_stride[i] = a.out.stride[i];
  p.ks = a.cache.k_scale;
  p.vs = a.cache.v_scale;
  p.vq = a.cache.v;
  p.num_blocks = static_cast<int>(a.cache.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.start = a.start_pos;
  p.lens = a.lens;
  p.out = a.out.data;
  p.out_bf16 = a.out.dtype == ATTN_BF16;
  p.lse = a.lse;
  p.pitch = nt * kBM;
  p.ctas = a.n_cta;
  p.part_o = static_cast<float*>(a.partials);
  p.part_lse = p.part_o + part_rows(p.T, p.G, a.n_cta) * a.cache.D;
  p.cuts = reinterpret_cast<CutItem*>(static_cast<uint8_t*>(a.partials) + part_bytes(p.T, p.G, a.cache.D, a.n_cta));
  p.status = a.status;
  if (a.cache.D == 64) return nt == 1 ? launch<64, 1>(a, p, stream) : launch<64, 2>(a, p, stream);
  return nt == 1 ? launch<128, 1>(a, p, stream) : launch<128, 2>(a, p, stream);
}

}  // namespace attn
