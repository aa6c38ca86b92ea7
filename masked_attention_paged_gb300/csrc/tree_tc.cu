// tree_tc.cu -- attention of a tree of drafted tokens over a paged KV cache
// (tcgen05 + TMEM + TMA), with the drafts' append in the same launch.
//
// Sequence b holds ctx tokens in its cache and T drafts; draft t attends to the
// whole context and, among the drafts, to itself and its ancestors:
//   s_j = scale q.k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j e^{s_j}.
//
// Few query rows read a long cache, so K and V are read once for all drafts and
// query heads of a KV head that fit NT row tiles.  A row tile is the G heads of tb = min(T,
// 128 / G) drafts (row r: draft r / G, head r % G), one 5-D TMA box of q whatever
// its strides; NT row tiles share every K/V tile (NT = 1 if one holds all drafts,
// else 2).  What bounds it is HBM (a 128-key tile of K and V at D = 128 is 64 KB,
// 1.4 us of an SM's share), until rows pass 256 a KV head and the tensor cores and
// exponentials do.  Measured (merge and path acceptance included; Hkv = 8, D = 128):
//   64 sequences x 25 drafts, G = 4, up to 8192 tokens   269 us, 1.66 GB, 91 % of
//                                                        the measured copy rate
//   16 x 27, G = 4, up to 4096 tokens                    56 us (28 us of bytes): 17
//        tiles a CTA; the rest is each segment's start and end and the merge
//   1 x 64, G = 8, 131063 tokens                         225 us (144 us of MMAs):
//        the chain of a row tile: scores arrive, 2300 cycles of softmax, 1650 for
//        the products of both row tiles
//   1 x 8, G = 2, D = 64, 700 tokens                     18 us, three launches'
//        latency: a tile passes through in 8 us, the drafts' in 11
//
// Every SM takes an equal run of the call's K/V tiles: an item (sequence, KV
// head, group of row tiles) is its context tiles followed by its draft tiles (whose
// masks are built meanwhile), the items are laid end to end, and each CTA takes an
// equal run (runs.cuh) of tiles and of kItemCost for each item: its start and end
// cost about 4 us, so equal runs of tiles alone left the CTAs with three short
// segments 11 us behind those with one (16 x 27: 62 us, with 3 counted 59.5, with 2
// 60.3, with 4 60.1).
// An item inside one run is written at once; one that is cut leaves partials
// (normalised rows and log2 LSE; at most two per CTA), which a second launch
// merges in order, so results do not depend on the timing.  That launch spreads
// the rows over the whole GPU: left to the piece that finished last, the merge of
// 108 rows took as long as the attention (16 x 27 drafts, 118 us against ~60).
//
// Warps: 0-1 stream K and 2-3 V (TMA: context tiles through the block table, draft
// tiles from k_new / v_new, or from the cache's blocks when they are there
// already, shifted by the context's last partial block), 4 issues the MMAs, 6-7
// build the ancestor masks, clean the drafts' V and append K and V from shared
// memory, 8-11 and 12-15 the softmax (thread r owns row r: TMEM lane r).  With NT =
// 2 each warpgroup has a row tile.  With NT = 1 both have the same rows and take
// the K/V tiles in turn, each with a score buffer, an output accumulator and a
// running max and sum of its own, joined by the LSE rule when an item ends: one
// warpgroup alone took 2.1 us a tile, more than the tile's bytes.  P goes over its
// S as bf16 (relative rounding 2^-8; row sums are taken in fp32 before it).
//
// V rows past the context's end and rows of absent drafts are zeroed: P is 0
// there, but 0 x NaN is not.  A draft's own V may hold infinities or NaN that
// only its descendants may see: such elements enter the tile as zeros, and the
// epilogue adds p x v for the rows that do attend to them.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged_tile.cuh"
#include "runs.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kBS = 16;
constexpr int kBoxBytes = kBM * 128;
constexpr float kRescaleMargin = 8.0f;
constexpr int kBarBytes = 1024;
constexpr int kSegs = 4;   // segments the planner is ahead
constexpr int kItemCost = 3;  // what an item costs a CTA besides its tiles, in tiles
constexpr int kSide = 48;  // draft keys that have a place of their own in shared memory (NT = 1)
constexpr uint32_t kAbsent = 0x7fc0a5a5u;  // a partial's LSE for the row of an absent draft (a NaN of its own)

template <int D, int NT>
struct Cfg {
  static constexpr int kThreads = 512;
  static constexpr int kMaxT = NT == 1 ? 128 : kTreeMaxDrafts;
  static constexpr int kWords = kMaxT / 32;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBM * D * 2;
  // D = 128: K runs a tile further ahead than V (its S is issued earlier), and
  // 227 KB hold Q and five tiles (NT = 1) or four
  static constexpr int KS = D == 64 ? 4 : (NT == 1 ? 3 : 2);
  static constexpr int VS = D == 64 ? 4 : 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + NT * kTileBytes;
  static constexpr int kOffV = kOffK + KS * kTileBytes;
  static constexpr int kOffAnc = kOffV + VS * kTileBytes;  // [2][kMaxT][kWords] ancestor bits
  static constexpr int kOffPar = kOffAnc + 2 * kMaxT * kWords * 4;  // [kMaxT] parents
  static constexpr int kOffRow = kOffPar + kMaxT * 4;      // [kMaxT] cache rows of the drafts
  // NT = 1: [2][kBM] running max and sum; K and V of up to kSide draft keys
  static constexpr int kOffXch = kOffRow + kMaxT * 8;
  static constexpr int kSideBytes = kSide * D * 2;
  static constexpr int kOffSide = (kOffXch + (NT == 1 ? 2 * kBM * 8 : 0) + 1023) / 1024 * 1024;
  static constexpr int kOffBar = kOffSide + (NT == 1 ? 2 * kSideBytes : 0);
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static constexpr uint32_t kColO = 256;  // O of warpgroup w at kColO + w * D; its scores at w * 128
  // 512 threads launched with 128 registers; 256 x 72 + 256 x 184 = 65536
  static constexpr int kRegsCtl = 72, kRegsSoft = 184;
};

// A run of one item's tiles [t0, t1): what every warp role works through.  One
// warp plans them and hands them on in a small ring: with the arithmetic inlined
// in each role the kernel was 136 KB of code, more than the instruction cache.
struct Seg {
  int b;  // -1: the end
  int g, m, t0, t1, nct, ctx;  // nct: the item's context tiles; the drafts' follow
  int slot;   // where its partial goes; -1: the item is whole
  int there;  // the sequence is present (not idle, and fits its table)
};

struct Bars {
  uint64_t q_full[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2];  // [warpgroup]
  uint64_t xch_full[2];  // NT = 1: a warpgroup's running max and sum are in smem
  uint64_t o_free;       // NT = 1: both warpgroups have read both accumulators
  uint64_t draft_in[4];  // a draft tile's K and V have landed in K stage ks (and the tile's V stage)
  uint64_t mask_full[2], mask_empty[2];
  uint64_t side_in, side_ready, side_free;  // drafts in their own place: landed, clean, read
  uint64_t drained;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg segs[kSegs];
  uint32_t bad[2][8];  // drafts whose V holds a non-finite element
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block outgrew its shared-memory slot");

struct TreeParams {
  int B, T, Hq, Hkv, G;
  int tb, RT;  // drafts and rows (tb * G) of a row tile
  int MP;      // groups of NT row tiles per KV head
  int shares;  // of the CTAs, one for each such group (or 1: a share takes all groups)
  int ntd;     // draft tiles
  int side;    // the drafts (one tile, at most kSide keys) have a place of their own, not ring stages
  int new_box; // rows of a k_new / v_new box: T up to a multiple of 16, or 128
  float scale_log2;
  int scale_positive;
  const uint16_t* q;
  int64_t q_stride[3];
  const uint16_t* k_new;  // null: the drafts are in the cache
  const uint16_t* v_new;
  int64_t kn_stride[3], vn_stride[3];
  uint16_t* kc;
  uint16_t* vc;
  int num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* parents;
  int64_t par_stride;
  void* out;
  int out_bf16;
  int64_t out_stride[3];
  float* lse;
  float* part_o;    // [2 n][D][pitch]: a column's rows side by side, as the TMEM lanes hold them
  float* part_lse;  // [2 n][pitch]
  int pitch;        // rows of a partial: 128 a row tile
  struct CutItem* cuts;  // [n] the item that starts in CTA c's run and goes on past it
  uint32_t* status;
};

// pieces == 0: no item of the kind.  A CTA's first segment uses partial slot 2c, a
// later one (only its last can be cut) slot 2c + 1.
struct CutItem {
  int b, g, node0;
  int pieces;         // in CTAs c, c + 1, ...
  int first_is_head;  // it is the first segment of CTA c's run
};

// A sequence that does not fit its table, or is idle, has no context and no drafts.
__device__ __forceinline__ int seq_ctx(const TreeParams& p, int b, bool& ok) {
  const int c = p.ctx_lens[b];
  ok = c >= 0 && static_cast<int64_t>(c) + p.T <= static_cast<int64_t>(p.max_blocks) * kBS;
  return ok ? c : 0;
}
__device__ __forceinline__ int seq_tiles(const TreeParams& p, int b, int& ctx, bool& ok) {
  ctx = seq_ctx(p, b, ok);
  return (ctx + kBN - 1) / kBN + p.ntd;
}

// The drafts' first key in their tiles: a block's start when they come from the cache.
__device__ __forceinline__ int draft_off(const TreeParams& p, int ctx) { return p.k_new != nullptr ? 0 : ctx % kBS; }
// Keys of a tile that its MMAs cover: a multiple of 16, at least 16.
__device__ __forceinline__ int tile_keys(const TreeParams& p, int tile, int nct, int ctx) {
  const int left = tile >= nct ? p.T + draft_off(p, ctx) - (tile - nct) * kBN : ctx - tile * kBN;
  return min(kBN, max(16, (left + 15) / 16 * 16));
}

// Layout of tile `tile`: fresh drafts arrive as 64-column boxes of rows, cached
// rows block by block.
struct Layout {
  uint32_t half, group;  // bytes to the next 64 columns, to the next 8 rows
};
template <int D>
__device__ __forceinline__ Layout tile_layout(const TreeParams& p, bool draft) {
  if (draft && p.k_new != nullptr) return {static_cast<uint32_t>(p.side ? kSide * 128 : kBoxBytes), 1024u};
  return {PagedTile<D>::kHalf, PagedTile<D>::kGroup};
}

// bf16 pair with its non-finite elements cleared; `any` reports them
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool& any) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u, any = true;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu, any = true;
  return w;
}

// the cache row of slot `slot` of (b, g), or -1 for a bad block id (reported)
__device__ __forceinline__ int64_t cache_row(const TreeParams& p, int b, int g, int slot) {
  const int blk = p.bt[static_cast<int64_t>(b) * p.bt_stride + slot / kBS];
  if (blk < 0 || blk >= p.num_blocks) {
    report(p.status, kStatusBounds);
    return -1;
  }
  return (static_cast<int64_t>(blk) * p.Hkv + g) * kBS + slot % kBS;
}

template <int D>
__device__ __forceinline__ const uint16_t* draft_row(const TreeParams& p, bool is_v, int b, int g, int j, int ctx) {
  if (p.k_new != nullptr)
    return is_v ? p.v_new + b * p.vn_stride[0] + g * p.vn_stride[1] + j * p.vn_stride[2]
                : p.k_new + b * p.kn_stride[0] + g * p.kn_stride[1] + j * p.kn_stride[2];
  const int64_t row = cache_row(p, b, g, ctx + j);
  return row < 0 ? nullptr : (is_v ? p.vc : p.kc) + row * D;
}

// The merge: out = sum_c 2^(lse_c - M) out_c / sum_c 2^(lse_c - M) over a cut
// item's pieces.  grid (CTAs of the main launch, groups of 32 rows), a warp per D /
// 16 columns, a lane per row: partials are read as they were written, 128 bytes a
// warp, and the rows leave through shared memory.
constexpr int kMergeThreads = 512;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int CW = D / 16;
  __shared__ float tile[32][D + 1];
  let_next_launch_in();
  wait_for_launch_ahead();
  const int c0 = blockIdx.x;
  const CutItem it = p.cuts[c0];
  if (it.pieces == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sr = blockIdx.y * 32 + lane;  // row of the partials
  // its draft and head
  auto place = [&](int r, int& t, int& h) {
    const int row = r % kBM;
    t = it.node0 + r / kBM * p.tb + row / p.G;
    h = it.g * p.G + row % p.G;
    return row < p.RT && t < p.T;
  };
  int t, h;
  const bool mine = place(sr, t, h);
  auto slot = [&](int c) { return static_cast<int64_t>(2 * (c0 + c) + ((c == 0 && !it.first_is_head) ? 1 : 0)); };
  float M = -INFINITY;
  bool any = false, absent = false;  // a NaN counts as something: it has to reach the row
#pragma unroll 8
  for (int c = 0; c < it.pieces; ++c) {
    const float l = mine ? p.part_lse[slot(c) * p.pitch + sr] : -INFINITY;
    absent |= __float_as_uint(l) == kAbsent;
    any |= l != -INFINITY;
    M = fmaxf(M, l);
  }
  float acc[CW], ws = 0.f;
#pragma unroll
  for (int i = 0; i < CW; ++i) acc[i] = 0.f;
  const bool empty = absent || !any;
#pragma unroll 32 / CW
  for (int c = 0; c < it.pieces; ++c) {
    const float l = mine ? p.part_lse[slot(c) * p.pitch + sr] : -INFINITY;
    const float* o = p.part_o + (slot(c) * D + warp * CW) * p.pitch + sr;
    const bool use = l != -INFINITY;  // a piece that saw nothing holds zeros
    const float w = use ? fast_exp2(l - M) : 0.f;
    ws += w;
#pragma unroll
    for (int i = 0; i < CW; ++i) acc[i] = fmaf(w, use ? o[static_cast<int64_t>(i) * p.pitch] : 0.f, acc[i]);
  }
  const float inv = empty ? 0.f : 1.f / ws;
#pragma unroll
  for (int i = 0; i < CW; ++i) tile[lane][warp * CW + i] = empty ? 0.f : acc[i] * inv;
  if (warp == 0 && mine && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(it.b) * p.Hq + h) * p.T + t] =
        empty ? -INFINITY : (M + __log2f(ws)) * 0.6931471805599453f;
  __syncthreads();
  const int r = threadIdx.x / 16, d = threadIdx.x % 16 * CW;
  if (!place(blockIdx.y * 32 + r, t, h)) return;
  const int64_t ob = it.b * p.out_stride[0] + h * p.out_stride[1] + t * p.out_stride[2] + d;
  const float* x = &tile[r][d];
  if (p.out_bf16) {
#pragma unroll
    for (int i = 0; i < CW; i += 4)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ob + i) =
          make_uint2(pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < CW; i += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + ob + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    paged_tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                         const __grid_constant__ CUtensorMap tm_vn, const __grid_constant__ TreeParams p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  uint32_t* anc = reinterpret_cast<uint32_t*>(smem + C::kOffAnc);
  int32_t* par = reinterpret_cast<int32_t*>(smem + C::kOffPar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;

  if (threadIdx.x == 32) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->xch_full[t], 4);
      mbar_init(&bars->mask_full[t], 1);
      mbar_init(&bars->mask_empty[t], 8);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->k_full[s], 2);  // two producer warps each
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 2);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->draft_in[s], 4);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&bars->seg_full[s], 1);
      mbar_init(&bars->seg_empty[s], 15);  // 4 producers, the issuer, 2 drafts' and 8 softmax warps
    }
    mbar_init(&bars->o_free, 8);
    mbar_init(&bars->drained, 1);
    mbar_init(&bars->side_in, 1);
    mbar_init(&bars->side_ready, 1);
    mbar_init(&bars->side_free, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  let_next_launch_in();
  if (warp == 4) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  // query rows past a row tile's box: zeros, once
#pragma unroll 1
  for (int x = threadIdx.x; x < NT * C::kBoxes * (kBM - p.RT) * 8; x += C::kThreads) {
    const int box = x / ((kBM - p.RT) * 8), y = x % ((kBM - p.RT) * 8);
    *reinterpret_cast<uint4*>(smem + C::kOffQ + box * kBoxBytes + p.RT * 128 + y * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  wait_for_launch_ahead();
  // the planner's state: the call's runs, and the place of this CTA's first tile
  Runs runs = {};
  int pos = 0, hi = 0, lo = 0, share = 0;
  int plan_b = 0, plan_item = 0, plan_t = 0;
  if (warp == 5) {
    // (all counts are below 2^31: tree_units_fit)
    const int items = p.shares > 1 ? p.Hkv : p.Hkv * p.MP;  // of a sequence, in this CTA's share
    int total = 0, mine0 = 0;
    auto seq_items = [&](int b, bool first) {
      if (b >= p.B) return 0;
      int ctx;
      bool ok;
      const int n = (kItemCost + seq_tiles(p, b, ctx, ok)) * items;
      if (first && blockIdx.x == 0 && !ok && p.ctx_lens[b] >= 0) report(p.status, kStatusBounds);
      return n;
    };
#pragma unroll 1
    for (int base = 0; base < p.B; base += 32) {
      const int mine = seq_items(base + lane, true);
      if (base == 0) mine0 = mine;
      total += mine;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    const int per = gridDim.x / p.shares, c = static_cast<int>(blockIdx.x) % per;
    share = static_cast<int>(blockIdx.x) / per;
    runs = Runs::make(total, per);
    if (share < p.shares && c < runs.n) lo = runs.lo(c), hi = runs.lo(c + 1);
    pos = lo;
    int run = 0;
#pragma unroll 1
    for (int base = 0; base < p.B && lo < hi; base += 32) {
      const int mine = base == 0 ? mine0 : seq_items(base + lane, false);
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
        const int units = __shfl_sync(0xffffffffu, mine, l) / items;
        plan_b = base + l;
        plan_item = local / units;
        plan_t = local - plan_item * units - kItemCost;
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

  if (warp < 8) regs_dec<C::kRegsCtl>();
  if (warp < 4) {
    // ------------------------------------------------------------ K/V tiles
    // warps 0, 1 the halves of K, 2, 3 of V; lane i < 4 owns block 4 (warp & 1) + i
    // of a tile, its id read a tile ahead.  A draft tile's data go to the drafts'
    // warps first (draft_in, all four producers' arrivals), which hand the stages on.
    const bool is_v = warp >= 2;
    const int S = is_v ? C::VS : C::KS;  // this operand's stages
    const void* map = is_v ? static_cast<const void*>(&tm_v) : &tm_k;
    const void* map_new = is_v ? static_cast<const void*>(&tm_vn) : &tm_kn;
    uint64_t* full = is_v ? bars->v_full : bars->k_full;
    uint64_t* empty = is_v ? bars->v_empty : bars->k_empty;
    uint8_t* base = smem + (is_v ? C::kOffV : C::kOffK);
    const int place = (warp & 1) * kWarpBlocks + lane;
    Seg s;
    int j = 0, issued = 0, st = 0, ks = 0;  // st, ks: tile j's stage, and its K stage
    uint32_t ph = 1u;                       // parity of the stage's last release
    bool ok = true;
    for (int i = 0; ok && seg_get(i, s); ++i) {
      seg_taken(i);
      const int t_end = p.side ? min(s.t1, s.nct) : s.t1;  // drafts with their own place take no stage
      const int32_t* bt_row = p.bt + static_cast<int64_t>(s.b) * p.bt_stride;
      auto block_id = [&](int tile, bool& want) {
        want = false;
        if (tile >= t_end || lane >= kWarpBlocks) return -1;
        int blk, end;  // the block, and where the tile's kind of blocks ends
        if (tile >= s.nct) {
          if (p.k_new != nullptr || !s.there) return -1;
          blk = s.ctx / kBS + (tile - s.nct) * kTileBlocks + place;
          end = (s.ctx + p.T + kBS - 1) / kBS;
        } else {
          blk = tile * kTileBlocks + place;
          end = (s.ctx + kBS - 1) / kBS;
        }
        want = blk < end;
        return want ? bt_row[blk] : -1;
      };
      bool want_next;
      int id_next = block_id(s.t0, want_next);
      for (int tile = s.t0; tile < t_end; ++tile, ++j) {
        int id = id_next;
        const bool want = want_next;
        id_next = block_id(tile + 1, want_next);
        if (id < 0 || id >= p.num_blocks) {
          // a table may hold any id here, -1 too; a draft's is the drafts' warps' to
          // report, who know whether the draft is there
          if (want && tile < s.nct) report(p.status, kStatusBounds);
          id = -1;
        }
        uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * (kBS * D * 2);
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ph, abort, p.status))) {
          ok = false;
          break;
        }
        const bool draft = tile >= s.nct;
        // one box of k_new (v_new) per 64 columns, by the operand's first warp
        const bool fresh = draft && p.k_new != nullptr && (warp & 1) == 0;
        if (fresh) bytes = static_cast<uint32_t>(p.new_box) * D * 2;
        uint64_t* bar = draft ? &bars->draft_in[ks] : &full[st];
        uint8_t* dst = base + st * C::kTileBytes;
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (fresh) {
          if (lane < C::kBoxes) tma_load_5d(dst + lane * kBoxBytes, map_new, bar, lane * 64, 0,
                                             (tile - s.nct) * kBN, s.g, s.b);
        } else {
          load_block<D>(dst, place, map, bar, id, p.Hkv, s.g);
        }
        issued = j + 1;
        if (++st == S) st = 0, ph ^= 1u;
        if (++ks == C::KS) ks = 0;
      }
    }
    if (lane == 0 && *abort) {
      // let every copy in flight land before the CTA exits (a wait on a barrier
      // without copies, as a draft tile's that nobody took over, runs out or passes)
      for (int x = max(0, issued - S); x < issued; ++x) drain_wait(&full[x % S], (x / S) & 1);
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp goes through the loop, with values that are alike in all
    // lanes (uniform registers, which the descriptors have to be in), and one lane
    // issues: a lane alone in the loop took over 100 cycles an MMA.
    constexpr uint32_t idesc_o = idesc_bf16_f32(kBM, D, false, true);
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uni(tmem);
    // w: the warpgroup whose scores and accumulator these are; ka, va: the tile; free:
    // told (if not null) when the tile's stage has been read.  A descriptor's start
    // address counts 16 bytes in its low bits.
    auto issue_s = [&](int w, uint32_t ka, int keys, Layout l, uint64_t* free) {  // S_w = Q K^T
      const uint32_t idesc_s = idesc_bf16_f32(kBM, keys, false, false);
      const uint64_t dq = sdesc_sw128(smem_u32(smem + C::kOffQ) + (NT == 2 ? w * C::kTileBytes : 0), 16, 1024);
      const uint64_t dk = sdesc_sw128(ka, 16, l.group);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // 16 dims = 32 bytes of a 128-byte row
          umma_bf16_ss(tm + w * 128, dq + (kk >> 2) * (kBoxBytes >> 4) + (kk & 3) * 2,
                       dk + (kk >> 2) * (l.half >> 4) + (kk & 3) * 2, idesc_s, kk > 0 ? 1u : 0u);
        umma_commit(&bars->s_full[w]);
        if (free != nullptr) umma_commit(free);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int w, uint32_t va, int keys, Layout l, bool first, uint64_t* free) {  // O_w (+)= P_w V
      const uint64_t dv = sdesc_sw128(va, l.half, l.group);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) {
          if (kk * 16 >= keys) break;
          umma_bf16_ts(tm + C::kColO + w * D, tm + w * 128 + kk * 8, dv + kk * (l.group >> 3), idesc_o,
                       (!first || kk > 0) ? 1u : 0u);
        }
        umma_commit(&bars->o_done[w]);
        if (free != nullptr) umma_commit(free);
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort, p.status)) != 0;
    };
    auto k_at = [&](int r) { return smem_u32(smem + C::kOffK + (r % C::KS) * C::kTileBytes); };
    auto v_at = [&](int r) { return smem_u32(smem + C::kOffV + (r % C::VS) * C::kTileBytes); };
    int r = 0, round = 0;  // ring tiles, and drafts in their own place, so far
    int j = 0;
    bool ok = true;
    Seg sg;
    for (int seg = 0; ok && seg_get(seg, sg); ++seg) {
      seg_taken(seg);
      const int t0 = uni(sg.t0), t1 = uni(sg.t1), nct = uni(sg.nct), ctx = uni(sg.ctx);
      const int n = t1 - t0;
      auto keys = [&](int x) { return tile_keys(p, t0 + x, nct, ctx); };
      auto lay = [&](int x) { return tile_layout<D>(p, t0 + x >= nct); };
      for (int t = 0; t < NT; ++t) ok = ok && wait(&bars->q_full[t], seg);
      if constexpr (NT == 1) {
        // tile j is warpgroup j & 1's; S runs two tiles ahead of PV.  x: tile of the
        // segment (r + x: its ring tile); the drafts, last, may lie aside.
        auto aside = [&](int x) { return p.side && t0 + x >= nct; };
        auto scores = [&](int x) {
          const bool a = aside(x);
          if (!wait(a ? &bars->side_ready : &bars->k_full[(r + x) % C::KS], a ? round : (r + x) / C::KS)) return false;
          tc_fence_after();
          issue_s((j + x) & 1, a ? smem_u32(smem + C::kOffSide) : k_at(r + x), keys(x), lay(x),
                  a ? nullptr : &bars->k_empty[(r + x) % C::KS]);
          return true;
        };
#pragma unroll 1
        for (int x = 0; ok && x < n + 2; ++x) {
          if (x >= 2) {  // P_(x - 2) V, before S_x takes its scores' place
            const int y = x - 2;
            const bool a = aside(y);
            // the accumulators of the segment before have been read
            if (y == 0 && seg > 0) ok = wait(&bars->o_free, seg - 1);
            ok = ok && wait(&bars->p_full[(j + y) & 1], (j + y) >> 1) &&
                 (a || wait(&bars->v_full[(r + y) % C::VS], (r + y) / C::VS));
            if (!ok) break;
            tc_fence_after();
            issue_pv((j + y) & 1, a ? smem_u32(smem + C::kOffSide + C::kSideBytes) : v_at(r + y), keys(y), lay(y),
                     y < 2, a ? &bars->side_free : &bars->v_empty[(r + y) % C::VS]);
          }
          if (x < n) ok = scores(x);
        }
        if (!ok) break;
        j += n;
        const bool had = p.side && t1 > nct;
        r += had ? n - 1 : n;
        round += had;
      } else {
        auto wait_k = [&](int x) { return wait(&bars->k_full[x % C::KS], x / C::KS); };
        auto wait_v = [&](int x) { return wait(&bars->v_full[x % C::VS], x / C::VS); };
        // PV_A, S_A', PV_B, S_B': each tile's softmax runs under the other's MMAs
#pragma unroll 1
        for (int x = -1; ok && x < n; ++x) {
#pragma unroll 1
          for (int w = 0; ok && w < 2; ++w) {
            if (x >= 0) {
              ok = wait(&bars->p_full[w], j) && (w > 0 || wait_v(j));
              if (!ok) break;
              tc_fence_after();
              issue_pv(w, v_at(j), keys(x), lay(x), x == 0, w == 1 ? &bars->v_empty[j % C::VS] : nullptr);
            }
            if (x + 1 < n) {
              const int jn = x < 0 ? j : j + 1;
              ok = w > 0 || wait_k(jn);
              if (!ok) break;
              tc_fence_after();
              issue_s(w, k_at(jn), keys(x + 1), lay(x + 1), w == 1 ? &bars->k_empty[jn % C::KS] : nullptr);
            }
          }
          if (x >= 0) ++j;
        }
      }
    }
    // no MMA may be in flight when the TMEM is freed
    if (elect_one()) {
      umma_commit(&bars->drained);
      drain_wait(&bars->drained, 0);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ planner
    int ctx = 0, tiles = 0;
    bool there = false;
    if (pos < hi) tiles = seq_tiles(p, plan_b, ctx, there);
    for (int i = 0;; ++i) {
      Seg s = {};
      s.b = -1;
      if (pos < hi && plan_t == tiles) {  // the item is done: the next one, or the next sequence
        plan_t = -kItemCost;
        if (++plan_item == (p.shares > 1 ? p.Hkv : p.Hkv * p.MP)) {
          plan_item = 0;
          tiles = seq_tiles(p, ++plan_b, ctx, there);
        }
      }
      if (plan_t < 0) {  // the item's own cost, or as much of it as falls into this run
        const int skip = min(-plan_t, hi - pos);
        pos += skip;
        plan_t += skip;
      }
      if (pos < hi) {
        s.b = plan_b;
        s.g = p.shares > 1 ? plan_item : plan_item / p.MP;
        s.m = p.shares > 1 ? share : plan_item % p.MP;
        s.t0 = plan_t;
        s.t1 = min(tiles, plan_t + (hi - pos));
        s.nct = tiles - p.ntd;
        s.ctx = ctx;
        s.there = there;
        const bool whole = s.t0 == 0 && s.t1 == tiles;
        s.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (i == 0 ? 0 : 1);
        if (!whole && s.t0 == 0 && lane == 0) {  // cut, and it starts here
          CutItem it;
          it.b = s.b, it.g = s.g, it.node0 = s.m * NT * p.tb;
          it.pieces = runs.of(pos + tiles - 1) - static_cast<int>(blockIdx.x % (gridDim.x / p.shares)) + 1;
          it.first_is_head = i == 0;
          p.cuts[blockIdx.x] = it;
        }
        pos += s.t1 - plan_t;
        plan_t = s.t1;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->seg_empty[i % kSegs], ((i / kSegs) & 1) ^ 1, abort, p.status)))
        break;
      if (lane == 0) {
        bars->segs[i % kSegs] = s;
        mbar_arrive(&bars->seg_full[i % kSegs]);
      }
      if (s.b < 0) break;
    }
  } else if (warp == 6 || warp == 7) {
    // ------------------------------------------------------------ drafts
    constexpr int CH = D / 8;  // 16-byte chunks per row
    constexpr int NL = 64;
    const int lt = threadIdx.x - 192;
    Seg s;
    int64_t* dst_row = reinterpret_cast<int64_t*>(smem + C::kOffRow);
    int j0 = 0, round = 0;
    uint32_t in = 0u;  // bit ks: parity of the next draft tile in K stage ks
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = seg_get(i, s);
      ok = !named_bar_or(1, NL, !ok);  // the two warps go the same way
      if (!ok) break;
      seg_taken(i);
      if (s.t1 > s.nct) {
        const int mb = round & 1;
        uint32_t* am = anc + mb * C::kMaxT * C::kWords;
        // parents and block ids set out first, and are put down after the waits
        int up_of[C::kMaxT / NL], blk_of[C::kMaxT / NL];
        const bool append = s.there && p.k_new != nullptr && s.m == 0;
        const bool placed = append || p.k_new == nullptr;  // the drafts' blocks are written, or read
#pragma unroll
        for (int x = 0; x < C::kMaxT / NL; ++x) {
          const int t = lt + x * NL;
          up_of[x] = s.there && t < p.T ? p.parents[s.b * p.par_stride + t] : -2;
          blk_of[x] =
              placed && s.there && t < p.T ? p.bt[static_cast<int64_t>(s.b) * p.bt_stride + (s.ctx + t) / kBS] : -1;
        }
        // the masks of two segments before may still be in use
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->mask_empty[mb], ((round >> 1) & 1) ^ 1, abort, p.status));
        ok = !named_bar_or(1, NL, !ok);
        if (!ok) break;
        const int off = draft_off(p, s.ctx);
        uint8_t* k_side = smem + C::kOffSide;
        uint8_t* v_side = k_side + C::kSideBytes;
        if (NT == 1 && p.side) {
          // into their own place, once the drafts before have been read
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->side_free, (round & 1) ^ 1, abort, p.status));
          ok = !named_bar_or(1, NL, !ok);
          if (!ok) break;
          if (warp == 6) {
            int id = -1;  // lane i: block i of the cached drafts
            const int blk = s.ctx / kBS + lane;
            if (p.k_new == nullptr && s.there && lane < kSide / kBS && blk < (s.ctx + p.T + kBS - 1) / kBS) {
              id = p.bt[static_cast<int64_t>(s.b) * p.bt_stride + blk];
              if (id < 0 || id >= p.num_blocks) id = -1;  // reported below, if a draft of it is there
            }
            const int blocks = __popc(__ballot_sync(0xffffffffu, id >= 0));
            if (lane == 0)
              mbar_arrive_expect_tx(&bars->side_in, 2u * (p.k_new != nullptr ? p.new_box : blocks * kBS) * D * 2);
            __syncwarp();
            if (p.k_new != nullptr) {
              if (lane < 2 * C::kBoxes) {
                const int x = lane % C::kBoxes;
                tma_load_5d((lane < C::kBoxes ? k_side : v_side) + x * kSide * 128,
                            lane < C::kBoxes ? &tm_kn : &tm_vn, &bars->side_in, x * 64, 0, 0, s.g, s.b);
              }
            } else {
              load_block<D>(k_side, lane, &tm_k, &bars->side_in, id, p.Hkv, s.g);
              load_block<D>(v_side, lane, &tm_v, &bars->side_in, id, p.Hkv, s.g);
            }
          }
        }
        // Ancestors by doubling: node t holds the set of those up to, not with, the
        // node to_go[t]; it takes that node's set and where it stands, until a root
        // (-1) or an absent node (-2) is met.  Nodes go on at their own pace: a place is
        // read before the set that leads to it and written after, so a set is never
        // smaller than its place says.  (A walk up took 46 us for chains of 100.)
        volatile int32_t* to_go = par;
        volatile uint32_t* set = am;
#pragma unroll
        for (int x = 0; x < C::kMaxT / NL; ++x) {
          const int t = lt + x * NL;
          if (t >= p.T) break;
          const bool bad = up_of[x] >= t;  // parents come before children
          if (bad) report(p.status, kStatusBounds);
          to_go[t] = bad || up_of[x] < -1 ? -2 : up_of[x];
#pragma unroll
          for (int w = 0; w < C::kWords; ++w) set[t * C::kWords + w] = w == (t >> 5) ? 1u << (t & 31) : 0u;
          dst_row[t] = blk_of[x];
        }
        if (lt < 8) bars->bad[mb][lt] = 0u;
        named_bar_sync(1, NL);
#pragma unroll 1
        for (int t = lt; t < p.T; t += NL) {
          int up = to_go[t];
#pragma unroll 1
          while (up >= 0) {  // up falls with every turn
            const int next = to_go[up];
            __threadfence_block();
#pragma unroll
            for (int w = 0; w < C::kWords; ++w) {
              const uint32_t theirs = set[up * C::kWords + w];
              set[t * C::kWords + w] = set[t * C::kWords + w] | theirs;
            }
            __threadfence_block();
            to_go[t] = up = next;
          }
          if (up == -2) {  // absent: whoever stands on it, or meets what it met, is too
#pragma unroll
            for (int w = 0; w < C::kWords; ++w) set[t * C::kWords + w] = 0u;
          }
          // present: where it is to be cached
          const int64_t blk = dst_row[t];
          int64_t at = -1;
          if (up == -1 && placed) {
            if (blk < 0 || blk >= p.num_blocks)
              report(p.status, kStatusBounds);
            else if (append)
              at = (blk * p.Hkv + s.g) * kBS + (s.ctx + t) % kBS;
          }
          dst_row[t] = at;
        }
        named_bar_sync(1, NL);
#pragma unroll 1
        for (int tile = max(s.t0, s.nct); ok && tile < s.t1; ++tile) {
          const int j = j0 + tile - s.t0;
          const int ks = j % C::KS, vs = j % C::VS;
          const bool side = NT == 1 && p.side;
          ok = __all_sync(0xffffffffu, side ? mbar_wait(&bars->side_in, round & 1, abort, p.status)
                                            : mbar_wait(&bars->draft_in[ks], (in >> ks) & 1u, abort, p.status));
          if (!side) in ^= 1u << ks;
          ok = !named_bar_or(1, NL, !ok);
          if (!ok) break;
          const uint8_t* kt = side ? k_side : smem + C::kOffK + ks * C::kTileBytes;
          uint8_t* vt = side ? v_side : smem + C::kOffV + vs * C::kTileBytes;
          const int rows = tile_keys(p, tile, s.nct, s.ctx);
          const Layout lay = tile_layout<D>(p, true);
#pragma unroll 1
          for (int x = lt; x < rows * CH; x += NL) {
            const int r = x / CH, ch = x % CH, node = (tile - s.nct) * kBN + r - off;
            const uint32_t at = swizzled_off(r, ch, lay.half, lay.group);
            uint4* vp = reinterpret_cast<uint4*>(vt + at);
            // present: its own bit is set
            if (node < 0 || node >= p.T || !((am[node * C::kWords + (node >> 5)] >> (node & 31)) & 1u)) {
              *vp = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            uint4 vw = *vp;
            const int64_t row = dst_row[node];
            if (row >= 0) {
              *reinterpret_cast<uint4*>(p.kc + row * D + ch * 8) = *reinterpret_cast<const uint4*>(kt + at);
              *reinterpret_cast<uint4*>(p.vc + row * D + ch * 8) = vw;
            }
            bool bad = false;
            vw.x = finite_pair(vw.x, bad), vw.y = finite_pair(vw.y, bad);
            vw.z = finite_pair(vw.z, bad), vw.w = finite_pair(vw.w, bad);
            if (bad) {
              *vp = vw;
              atomicOr(&bars->bad[mb][node >> 5], 1u << (node & 31));
            }
          }
          fence_proxy_async_smem();
          named_bar_sync(1, NL);
          if (lt == 0 && side) mbar_arrive(&bars->side_ready);
          if (lt == 0 && !side) {
            for (int x = 0; x < 2; ++x) {  // for both producers of each
              mbar_arrive(&bars->k_full[ks]);
              mbar_arrive(&bars->v_full[vs]);
            }
          }
        }
        if (ok && lt == 0) mbar_arrive(&bars->mask_full[mb]);
        ++round;
      }
      j0 += s.t1 - s.t0;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ softmax
    regs_inc<C::kRegsSoft>();
    const int wg = (warp >> 2) - 2;
    const int t = NT == 2 ? wg : 0;  // row tile
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tid = threadIdx.x - 256;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = wg * 128, o_col = C::kColO + wg * D;
    constexpr int CH = D / 8;

    // this row tile's queries: every S of the segment before is done by then
    auto load_q = [&](const Seg& s) {
      if (quarter != 0 || lane != 0) return;  // NT = 1: called by one warpgroup only
      mbar_arrive_expect_tx(&bars->q_full[t], static_cast<uint32_t>(p.RT) * D * 2);
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x)
        tma_load_5d(smem + C::kOffQ + t * C::kTileBytes + x * kBoxBytes, &tm_q, &bars->q_full[t], x * 64, 0,
                    (s.m * NT + t) * p.tb, s.g, s.b);
    };

    // PV of this warpgroup's tile number x (of all it has had) is done.  Asked only
    // about the latest one or the one before: S of the tile after x, seen by then,
    // follows the PV before x, so the parity is never read a phase early; and the
    // phase after needs this warp's next P, so never a phase late.
    auto o_wait = [&](int x) { return mbar_wait(&bars->o_done[wg], x & 1, abort, p.status); };
    float2* xch = reinterpret_cast<float2*>(smem + C::kOffXch);

    Seg s;
    bool ok = true;
    int j = 0, jr = 0, round = 0;  // tiles, ring tiles, segments with drafts so far
    int n_mine = 0;                // tiles this warpgroup has had
    for (int seg = 0; ok && seg_get(seg, s); ++seg) {
      seg_taken(seg);
      if (seg == 0 && (NT == 2 || wg == 0)) load_q(s);
      const int node = (s.m * NT + t) * p.tb + row / p.G;
      const bool mine = row < p.RT && node < p.T;               // the row exists
      const bool warp_on = __any_sync(0xffffffffu, mine);
      const int head = s.g * p.G + row % p.G;
      const bool has_draft = s.t1 > s.nct;
      const int mb = round & 1;
      const uint32_t* am = anc + mb * C::kMaxT * C::kWords + (mine ? node : 0) * C::kWords;
      const int off = draft_off(p, s.ctx);
      const int mine_before = n_mine;
      bool masks = false;  // this warp has waited for the segment's masks
      float m_run = -INFINITY, l_run = 0.0f;
      for (int tile = s.t0; tile < s.t1; ++tile, ++j, jr += !(p.side && tile > s.nct)) {
        if (NT == 1 && (j & 1) != wg) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[wg], n_mine & 1, abort, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (tile == s.t1 - 1) {  // every S of this segment is done: the next one's queries
          Seg ahead;
          if (seg_get(seg + 1, ahead)) load_q(ahead);
        }
        if (tile >= s.nct && !masks) {
          masks = true;
          if (!__all_sync(0xffffffffu, mbar_wait(&bars->mask_full[mb], (round >> 1) & 1, abort, p.status))) {
            ok = false;
            break;
          }
        }
        // which of the tile's keys [32 x, +32) this row may see, a bit each
        const int lim = s.ctx - tile * kBN;  // of a context tile
        bool masked = !p.scale_positive;
        auto see = [&](int x) -> uint32_t {
          if (tile < s.nct) {
            const int left = lim - x * 32;
            return left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u);
          }
          if (!mine) return 0u;
          // bits [32 x - off, +32) of the tile's drafts
          const int w = (tile - s.nct) * 4 + x - (off > 0 ? 1 : 0);
          const uint32_t lo = w >= 0 && w < C::kWords ? am[w] : 0u;
          if (off == 0) return lo;
          return __funnelshift_r(lo, w + 1 < C::kWords ? am[w + 1] : 0u, 32 - off);
        };
        if (tile >= s.nct) {
          masked = true;
        } else {
          if (lim < kBN) {
            masked = true;
            // V rows past the context: whatever the slots hold, or nothing loaded
            const int vs = jr % C::VS;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->v_full[vs], (jr / C::VS) & 1, abort, p.status))) {
              ok = false;
              break;
            }
            uint8_t* vt = smem + C::kOffV + vs * C::kTileBytes;
#pragma unroll 1
            for (int x = tid & 127; x < (tile_keys(p, tile, s.nct, s.ctx) - lim) * CH; x += 128)
              *reinterpret_cast<uint4*>(vt + swizzled_off(lim + x / CH, x % CH, PagedTile<D>::kHalf,
                                                          PagedTile<D>::kGroup)) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
        }
        if (warp_on) {
          float alpha = 1.0f, rs;
          // the reference max moves only when the tile's exceeds it by the margin
          auto raise = [&](float mt) {
            if (mt > m_run + kRescaleMargin || (m_run == -INFINITY && mt != -INFINITY)) {
              alpha = fast_exp2(m_run - mt);
              m_run = mt;
            }
          };
          // weights 2^(mul s + neg) of 32 scores: P to TMEM, and their sums
          auto weigh32 = [&](const uint32_t (&x)[32], int c, float mul, float neg, uint64_t (&sum)[4]) {
            const uint64_t mul2 = f2_pack(mul, mul), neg2 = f2_pack(neg, neg);
            uint32_t pw[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0, x1;
              f2_unpack(ffma2(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), mul2, neg2), x0, x1);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              pw[i >> 1] = pack_bf16x2(p0, p1);
              sum[(i >> 1) & 3] = fadd2(sum[(i >> 1) & 3], f2_pack(p0, p1));
            }
            tmem_st16(tmem + lane_addr + s_col + c * 16, pw);
          };
          // scores in log2 units, -inf where the row may not look
          auto mask32 = [&](uint32_t (&x)[32], uint32_t w) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = ((w >> i) & 1u) ? __float_as_uint(__uint_as_float(x[i]) * p.scale_log2) : 0xff800000u;
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
          if constexpr (NT == 1) {
            // Bound by HBM, with time to spare: two rolled passes over the scores in
            // TMEM, 32 at a time.  (Code that runs once costs its fetch: unrolled
            // over the 128 scores, a first tile took 2.3 us and this warp's code
            // displaced the producers'.)  The second pass writes P over scores that
            // it has read: chunk c's 16 columns end before chunk c + 1's begin.  Chunks
            // past the tile's keys have no scores, and no P that the MMAs read.
            const int nc = masked ? (tile_keys(p, tile, s.nct, s.ctx) + 31) / 32 : 4;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              uint32_t x[32];
              tmem_ld32(tmem + lane_addr + s_col + c * 32, x);
              tmem_wait_ld(x);
              if (masked) mask32(x, see(c));
              max32(x, mx);
            }
            const float mul = masked ? 1.0f : p.scale_log2;  // > 0
            raise(fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * mul);
            const float neg = m_run == -INFINITY ? 0.0f : -m_run;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              uint32_t x[32];
              tmem_ld32(tmem + lane_addr + s_col + c * 32, x);
              tmem_wait_ld(x);
              if (masked) mask32(x, see(c));
              weigh32(x, c, mul, neg, sum);
            }
          } else {
            // Bound by this chain's latency: scores go to registers, the first 32 ahead of
            // the others, and are weighed against the reference max at hand, without a
            // max pass; if some row's sum says its scores outgrew it (128 weights of 2^8,
            // the margin of a max pass, so that P V keeps the same room; or NaN), once more
            // with one.
            uint32_t sr[4][32];
            tmem_ld32(tmem + lane_addr + s_col, sr[0]);
            const bool fast = !masked && __all_sync(0xffffffffu, m_run != -INFINITY);
            tmem_wait_ld(sr[0]);
#pragma unroll
            for (int c = 1; c < 4; ++c) tmem_ld32(tmem + lane_addr + s_col + c * 32, sr[c]);
            bool done = false;
            if (fast) {
              weigh32(sr[0], 0, p.scale_log2, -m_run, sum);
#pragma unroll
              for (int c = 1; c < 4; ++c) tmem_wait_ld(sr[c]);
#pragma unroll
              for (int c = 1; c < 4; ++c) weigh32(sr[c], c, p.scale_log2, -m_run, sum);
              float a0, a1;
              f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), a0, a1);
              done = __all_sync(0xffffffffu, a0 + a1 <= kBN * 256.0f);  // 2^kRescaleMargin
              if (!done) {
                tmem_wait_st();
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = f2_pack(0.f, 0.f);
              }
            } else {
#pragma unroll
              for (int c = 1; c < 4; ++c) tmem_wait_ld(sr[c]);
            }
            if (!done) {
              float mul = p.scale_log2;
              if (masked) {
                mul = 1.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) mask32(sr[c], see(c));
              }
#pragma unroll
              for (int c = 0; c < 4; ++c) max32(sr[c], mx);
              raise(fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * mul);
              const float neg = m_run == -INFINITY ? 0.0f : -m_run;
#pragma unroll
              for (int c = 0; c < 4; ++c) weigh32(sr[c], c, mul, neg, sum);
            }
          }
          float a0, a1;
          f2_unpack(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), a0, a1);
          rs = a0 + a1;
          l_run = l_run * alpha + rs;
          if (n_mine > mine_before && __any_sync(0xffffffffu, alpha != 1.0f)) {
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
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[wg]);
        ++n_mine;
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      // NT = 1: both warpgroups' states joined; warpgroup w writes half w of the
      // output columns.  f0, f1: what accumulators 0 and 1 weigh.
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
        // (its own accumulator, and the other's: that warpgroup's last tile)
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
      const bool whole = s.slot < 0;
      // drafts this row sees whose V is not finite, and whether the row's own draft is absent
      bool absent = false;
      uint32_t fix_any = 0u;
      if (has_draft && !masks &&
          !__all_sync(0xffffffffu, mbar_wait(&bars->mask_full[mb], (round >> 1) & 1, abort, p.status))) {
        ok = false;  // this warpgroup had no draft tile, and has not seen the masks
        break;
      }
      if (has_draft && mine) {
        uint32_t own = 0u;
#pragma unroll
        for (int x = 0; x < C::kWords; ++x) {
          own |= am[x];
          fix_any |= am[x] & bars->bad[mb][x];
        }
        absent = own == 0u;
      }
      const bool empty = absent || l_run == 0.0f;
      const float inv = empty ? 0.0f : 1.0f / l_run;
      const float lse2 = empty ? -INFINITY : m_run + __log2f(l_run);
      const int64_t prow = static_cast<int64_t>(s.slot) * p.pitch + t * kBM + row;
      const int64_t obase = s.b * p.out_stride[0] + head * p.out_stride[1] + node * p.out_stride[2];
      if (warp_on) {
        // 16 columns at a time, rolled (it runs once a segment: its code's fetch counts)
#pragma unroll 1
        for (int c = NT == 1 ? wg * (D / 2) : 0; c < (NT == 1 ? (wg + 1) * (D / 2) : D); c += 16) {
          uint32_t o[16];
          if constexpr (NT == 2) {
            tmem_ld16_now(tmem + lane_addr + o_col + c, o);
          } else {
            uint32_t o1[16];
            tmem_ld16x2_now(tmem + lane_addr + C::kColO + c, o, tmem + lane_addr + C::kColO + D + c, o1);
            // an accumulator of weight 0 may hold anything
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint((f0 != 0.0f ? f0 * __uint_as_float(o[i]) : 0.0f) +
                                     (f1 != 0.0f ? f1 * __uint_as_float(o1[i]) : 0.0f));
          }
          if (mine) {
            if (fix_any != 0u) {
#pragma unroll 1
              for (int a = max(0, (s.t0 - s.nct) * kBN - off); a < min(p.T, (s.t1 - s.nct) * kBN - off); ++a) {
                if (!((am[a >> 5] & bars->bad[mb][a >> 5]) >> (a & 31) & 1u)) continue;
                const uint16_t* kr = draft_row<D>(p, false, s.b, s.g, a, s.ctx);
                const uint16_t* vr = draft_row<D>(p, true, s.b, s.g, a, s.ctx);
                const uint16_t* qr = p.q + s.b * p.q_stride[0] + head * p.q_stride[1] + node * p.q_stride[2];
                if (kr == nullptr || vr == nullptr) continue;
                float dot = 0.f;
#pragma unroll 1
                for (int d = 0; d < D; ++d)
                  dot = fmaf(__uint_as_float(static_cast<uint32_t>(qr[d]) << 16),
                             __uint_as_float(static_cast<uint32_t>(kr[d]) << 16), dot);
                const float w = fast_exp2(dot * p.scale_log2 - m_run);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float v = __uint_as_float(static_cast<uint32_t>(vr[c + i]) << 16);
                  if (!isfinite(v)) o[i] = __float_as_uint(fmaf(w, v, __uint_as_float(o[i])));
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = empty ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
            if (!whole) {
              float* dst = p.part_o + (static_cast<int64_t>(s.slot) * D + c) * p.pitch + t * kBM + row;
#pragma unroll
              for (int i = 0; i < 16; ++i) dst[i * (NT * kBM)] = __uint_as_float(o[i]);
            } else if (p.out_bf16) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + obase + c);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                dst[i] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5])),
                                    pack_bf16x2(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])));
            } else {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + obase + c);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                     __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
            }
          }
          __syncwarp();
        }
        if (mine && (NT == 2 || wg == 0)) {
          if (!whole)
            p.part_lse[prow] = absent ? __uint_as_float(kAbsent) : lse2;
          else if (p.lse != nullptr)
            p.lse[(static_cast<int64_t>(s.b) * p.Hq + head) * p.T + node] = lse2 * 0.6931471805599453f;
        }
      }
      tc_fence_before();  // O is read: the next segment's PV may overwrite it
      if constexpr (NT == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free);
      }
      if (has_draft) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->mask_empty[mb]);
        ++round;
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

// Row tiles: tb drafts each, one or two to a CTA
int tile_drafts(int64_t T, int64_t G) { return static_cast<int>(std::min(T, kBM / G)); }
int tree_nt(int64_t T, int64_t G) { return T <= kBM / G ? 1 : 2; }

template <int D, int NT>
cudaError_t launch(const TreeArgs& a, TreeParams& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  CUtensorMap mq, mk, mv, mkn, mvn;
  if (!make_rows_map(&mq, a.q, a.cache.Hkv, p.tb) ||
      !make_paged_map(&mk, a.cache.k, a.cache.num_blocks, a.cache.Hkv, D) ||
      !make_paged_map(&mv, a.cache.v, a.cache.num_blocks, a.cache.Hkv, D))
    return cudaErrorInvalidValue;
  mkn = mk, mvn = mv;  // not read without k_new
  if (p.k_new != nullptr && (!make_rows_map(&mkn, a.k_new, a.cache.Hkv, p.new_box) ||
                             !make_rows_map(&mvn, a.v_new, a.cache.Hkv, p.new_box)))
    return cudaErrorInvalidValue;
  auto kern = paged_tree_tc_kernel<D, NT>;
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
  const dim3 ctas(static_cast<unsigned>(a.n_cta));
  e = launch_early(kern, ctas, C::kThreads, C::kSmemBytes, stream, mq, mk, mv, mkn, mvn, p);
  if (e != cudaSuccess) return e;
  // groups of 32 rows up to the last that any row tile uses
  const dim3 grid(static_cast<unsigned>(a.n_cta), static_cast<unsigned>(((NT - 1) * kBM + p.RT + 31) / 32));
  return launch_early(tree_merge_kernel<D>, grid, kMergeThreads, 0, stream, p);
}

}  // namespace

// Partials of two cut items per CTA (their rows), and a CutItem per CTA.
size_t tree_partial_bytes(int64_t T, int64_t G, int D, int n_cta) {
  if (T == 0 || G == 0 || G > kBM) return 0;
  const size_t rows = static_cast<size_t>(2) * n_cta * tree_nt(T, G) * kBM;
  const size_t parts = (rows * (D + 1) * sizeof(float) + 255) & ~size_t(255);
  return parts + ((n_cta * sizeof(CutItem) + 255) & ~size_t(255));
}

bool tree_units_fit(int64_t B, int64_t Hkv, int64_t T, int64_t G, int64_t max_blocks) {
  if (T == 0) return true;
  const int64_t rows = tree_nt(T, G) * tile_drafts(T, G);
  const int64_t units = (max_blocks * kBS + kBN - 1) / kBN + (T + kBS - 1 + kBN - 1) / kBN + kItemCost;
  return B * Hkv * ((T + rows - 1) / rows) <= 0x7fffffff / units;
}

cudaError_t launch_paged_tree(const TreeArgs& a, cudaStream_t stream) {
  TreeParams p = {};
  p.B = static_cast<int>(a.B);
  p.T = static_cast<int>(a.T);
  p.Hq = static_cast<int>(a.Hq);
  p.Hkv = a.cache.Hkv;
  p.G = p.Hq / p.Hkv;
  const int nt = tree_nt(p.T, p.G);
  p.tb = tile_drafts(p.T, p.G);
  p.RT = p.tb * p.G;
  p.MP = (p.T + nt * p.tb - 1) / (nt * p.tb);
  // Each row group to a share of the CTAs of its own: they come to a K/V tile at the
  // same time, and all but one of them find it in L2.  With one share for all, its
  // groups came to it half a run apart (1 x 64 drafts, G = 8, 131063 tokens: 1.08 GB
  // read for 0.54).  At most 8 shares leave 3 % of 152 CTAs idle.
  p.shares = p.MP <= std::min(8, a.n_cta) ? p.MP : 1;
  p.new_box = std::min(kBN, (p.T + 15) / 16 * 16);
  p.side = nt == 1 && p.T + (a.k_new.data != nullptr ? 0 : kBS - 1) <= kSide;
  p.ntd = a.k_new.data != nullptr ? (p.T + kBN - 1) / kBN : (p.T + kBS - 1 + kBN - 1) / kBN;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.scale_positive = p.scale_log2 > 0.0f;
  p.q = static_cast<const uint16_t*>(a.q.data);
  p.k_new = static_cast<const uint16_t*>(a.k_new.data);
  p.v_new = static_cast<const uint16_t*>(a.v_new.data);
  for (int i = 0; i < 3; ++i) {
    p.q_stride[i] = a.q.stride[i];
    p.kn_stride[i] = a.k_new.stride[i];
    p.vn_stride[i] = a.v_new.stride[i];
    p.out_stride[i] = a.out.stride[i];
  }
  p.kc = static_cast<uint16_t*>(a.cache.k);
  p.vc = static_cast<uint16_t*>(a.cache.v);
  p.num_blocks = static_cast<int>(a.cache.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctx_lens = a.ctx_lens;
  p.parents = a.parents;
  p.par_stride = a.par_stride;
  p.out = a.out.data;
  p.out_bf16 = a.out.dtype == ATTN_BF16;
  p.lse = a.lse;
  p.pitch = nt * kBM;
  const size_t rows = static_cast<size_t>(2) * a.n_cta * p.pitch;
  p.part_o = static_cast<float*>(a.partials);
  p.part_lse = p.part_o + rows * a.cache.D;
  const size_t parts = (rows * (a.cache.D + 1) * sizeof(float) + 255) & ~size_t(255);
  p.cuts = reinterpret_cast<CutItem*>(static_cast<uint8_t*>(a.partials) + parts);
  p.status = a.status;
  if (a.cache.D == 64) return nt == 1 ? launch<64, 1>(a, p, stream) : launch<64, 2>(a, p, stream);
  if (a.cache.D == 128) return nt == 1 ? launch<128, 1>(a, p, stream) : launch<128, 2>(a, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace attn
