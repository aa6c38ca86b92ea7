// attn_f8.cu -- attention of few query rows (at most 16 per KV head: decode steps and
// short drafts) over an e4m3 paged cache (paged_attn_f8).
//
// A warp takes a block (16 tokens of one KV head) at a time, with no conversion of K:
//  * q is split into two e4m3 numbers, q = (hi + lo) 2^e, with 2^e the power of two that
//    brings the row's largest element to 448 or below.  bf16 has eight significant
//    bits and e4m3 four, so hi + lo is q exactly, down to 2^-19 of the largest
//    element.  hi and lo of eight rows are the 16 rows of one m16n8k32 product with
//    the codes as they lie in the cache; adding a lane's two accumulators is the score,
//    and the block's scale multiplies it.  (fp16 throughout, K converted like V, took 151
//    us where this took 140.)
//  * the values go in transposed, O^T = V^T W^T (m16n8k16, fp16): a row's weights
//    are, register for register, their score fragment, and codes become fp16 exactly,
//    two an instruction.  The block's value scale multiplies the products.
// Softmax is online with a lazy running max (log2 units, it moves when a block exceeds
// it by kLazy).  Weights are taken times 2^kLift, so that fp16 has room above for what kLazy lets
// through (2^15 at most) and loses a weight only below 2^-32 of the largest: the sum keeps
// those in 32 bits, and a long tail beside a few large weights would otherwise count there
// and be missing from the values.
//
// What bounds it is HBM, so nothing may stop the stream of blocks.  All blocks of the
// call, item (sequence, KV head) after item, are laid end to end, and every warp takes an
// equal run of them, kStages ahead in a ring of its own, across the items' borders.  No
// warp waits for another: an item inside a run is written at once, one that is cut
// leaves partials (normalised rows and log2 LSE; at most two a warp), which a second
// launch joins in order, so results do not depend on timing.  (CTAs of 1024 tokens of an
// item, joined by the last to come, spent 4 us each on their start and end.)
// 64 sequences of up to 8192 tokens (32 heads over 8, D = 128) take 132 us, 0.81 GB at 91 % of
// what a copy does; one of 700 (D = 64) 10 us (13 to 14 as eager calls on other inputs each
// time), two launches of dependent loads.  With 9 to 16 rows a KV head the registers of two row
// groups leave eight warps an SM, too few to hide latency: 233 us for the 64 sequences with 16 rows,
// where the bytes are 137.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "internal.h"
#include "runs.cuh"

namespace attn {
namespace {

constexpr int kBS = 16;
constexpr int kMostWarps = 12;  // of an SM
constexpr int kFewWarps = 4;    // of a CTA of a small call
constexpr float kLazy = 8.0f;
constexpr float kLift = 7.0f;  // kLift + kLazy < 16, fp16's range
constexpr float kUnlift = 1.0f / 128.0f;
static_assert(kLift + kLazy <= 15.0f && kUnlift * (1 << static_cast<int>(kLift)) == 1.0f, "");

struct F8MmaParams {
  CUtensorMap kmap, vmap;  // D = 128: codes [num_blocks, Hkv, 16, 128], box = one (block, head)
  const uint8_t* kq;
  const uint8_t* vq;
  const float* ks;
  const float* vs;
  int64_t num_blocks;
  int Hkv, Hq, G, T;
  const uint16_t* q;
  int64_t q_stride[3];
  int B;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start;
  const int32_t* lens;
  int causal;
  float scale_log2;
  void* out;
  int out_bf16;
  int64_t out_stride[3];
  float* lse;
  int warps;        // of the launch
  int side;         // heads side by side: warps that take the same run, a head each
  float* part_o;    // [2 warps][8 NR][D]: a warp's first segment, and a later one
  float* part_lse;  // [2 warps][8 NR], log2 units
  Runs64* runs;     // for the second launch: the runs, and where an item's blocks begin in them (times
  int64_t* first;   // two, plus one if that is a warp's first segment), [B][Hkv / side]
  uint32_t* status;
};

// D (16 x 8, f32) += A (16 x 32, e4m3) B (32 x 8, e4m3)
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D (16 x 8, f32) = A (16 x 16, f16) B (16 x 8, f16)
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <uint32_t SEL>
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "n"(SEL));
  return d;
}
// Token of position n (0..15) of a block in the order the fragments use: with the
// 128-byte swizzle, fragment loads of K and of V then meet no bank twice.
__device__ __forceinline__ int tok_of(int n) { return n ^ ((n & 1) << 2); }
// A sequence's queries: n of them (0: idle, or past its table), from position `start` on.
__device__ __forceinline__ int queries(const F8MmaParams& p, int b, int& start, bool& past) {
  start = p.start[b];
  const int n = p.lens != nullptr ? min(max(p.lens[b], 0), p.T) : p.T;
  past = start >= 0 && static_cast<int64_t>(start) + n > static_cast<int64_t>(p.max_blocks) * kBS;
  return start < 0 || past ? 0 : n;
}

// An item's blocks: those with a key that some row sees.
__device__ __forceinline__ int seq_blocks(const F8MmaParams& p, int b, int& start, int& n, bool& past) {
  n = queries(p, b, start, past);
  return n == 0 ? 0 : (start + n - 1) / kBS + 1;
}
// The sum of f(b) over the sequences, for a whole warp (64 bits: tables may be wide).
template <typename F>
__device__ __forceinline__ int64_t sum_over(int lane, int B, F f) {
  int64_t s = 0;
  for (int b = lane; b < B; b += 32) s += f(b);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}
// The first sequence after b that has blocks (B: none), for a whole warp.
__device__ __forceinline__ int next_seq(const F8MmaParams& p, int lane, int b, int& n_blocks) {
  for (int base = b + 1; base < p.B; base += 32) {
    int start, n, k = 0;
    bool past;
    if (base + lane < p.B) k = seq_blocks(p, base + lane, start, n, past);
    const uint32_t some = __ballot_sync(0xffffffffu, k > 0);
    if (some != 0u) {
      const int l = __ffs(static_cast<int>(some)) - 1;
      n_blocks = __shfl_sync(0xffffffffu, k, l);
      return base + l;
    }
  }
  n_blocks = 0;
  return p.B;
}
// Runs of at least kLeast blocks: a shorter one is all start and end (8: 14.0 us for one
// sequence of 700 tokens and D = 64 where 2 take 10.1).
constexpr int kLeast = 2;
// Heads side by side: their rows of a block lie together in memory, and are read at about the
// same time (64 sequences of 8192: 133 us; 135 with 8 heads or 2).
constexpr int kSide = 4;
__device__ __forceinline__ Runs64 runs_of(int64_t total, int warps) {
  return Runs64::make(total, static_cast<int>(min(static_cast<int64_t>(warps), (total + kLeast - 1) / kLeast)));
}

// Eight (D = 64) or sixteen dims of a row, scaled.
template <int E>
__device__ __forceinline__ void write_dims(void* out, int out_bf16, int64_t at, const float (&x)[E]) {
  if (out_bf16) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < E / 8; ++i)
      dst[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                          pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

template <int D, int NR>
struct MmaCfg {
  // Warps of an SM, by registers: 64 sequences of 8192 tokens with 4 rows take 133 us on twelve
  // (168 registers), 150 on sixteen and 149 on eight; with 16 rows 231 on eight and 286 on twelve,
  // which spill (with q's fragments in shared memory instead 221, but 4 of 2000 27 instead of 23);
  // 64 of 4096 with 16 rows and D = 64 96 on eight, 84 on twelve.
  static constexpr int kSmWarps = D == 128 && NR == 2 ? 8 : 12;
  // Twelve are one CTA where the call can fill the GPU, so that it is placed on an SM as a whole.
  // (Of three CTAs of four, one or two were placed while a launch ahead of them still held shared
  // memory, and the third after they were done: 188 us.)  Eight are two CTAs, whose warps do not
  // run in step (257 us as one).  Calls with less for each SM spread it in CTAs of four (one
  // sequence of 500 tokens and 16 rows 15 us, 20 in large ones).
  static constexpr int kWarps = kSmWarps == 8 ? 4 : 12;
  // More blocks in flight make the stream slower: the 133 us with three are 136 with four (134 with
  // two; with each head on its own 195 with five); with 16 rows 236 with six, 234 with four.
  static constexpr int kStages = NR == 1 ? 3 : 4;
  static constexpr int kCodeBytes = kBS * D;  // one (block, head) of K or V
  static constexpr int smem(int warps) { return 1024 + warps * kStages * (2 * kCodeBytes + 16); }
};

template <int D, int NR>
__global__ void __launch_bounds__(MmaCfg<D, NR>::kWarps * 32, MmaCfg<D, NR>::kSmWarps / MmaCfg<D, NR>::kWarps)
    paged_attn_f8_mma_kernel(const __grid_constant__ F8MmaParams p) {
  using C = MmaCfg<D, NR>;
  constexpr int kStages = C::kStages, kCodeBytes = C::kCodeBytes;
  constexpr int kRows = 8 * NR;
  constexpr int kSteps = D / 32;  // of the score product
  constexpr int kTiles = D / 16;  // of the output's dims
  extern __shared__ uint8_t smem_raw[];
  uint8_t* codes = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // [warp][stage][K, V]
  const int warps = blockDim.x >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(codes + warps * kStages * 2 * kCodeBytes);
  float2* scales = reinterpret_cast<float2*>(bars + warps * kStages);  // [warp][stage] K's and V's; x = -inf: no block
  __shared__ int abort_flag[C::kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* wcodes = codes + warp * kStages * 2 * kCodeBytes;
  uint64_t* wbar = bars + warp * kStages;
  float2* wscale = scales + warp * kStages;
  int* abort = &abort_flag[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&wbar[s], 1);
    *abort = 0;
    if constexpr (D == 128) {
      tma_prefetch_desc(&p.kmap);
      tma_prefetch_desc(&p.vmap);
    }
  }
  fence_mbar_init();
  let_next_launch_in();
  __syncwarp();
  wait_for_launch_ahead();

  // ---- this warp's run, and where it begins
  const int me = blockIdx.x * warps + warp;
  auto blocks_of = [&](int b) {
    int start, n;
    bool past;
    return seq_blocks(p, b, start, n, past);
  };
  const int run_of_warp = me / p.side, off = me - run_of_warp * p.side;
  const int Hgr = p.Hkv / p.side;  // groups of heads
  const int64_t total = Hgr * sum_over(lane, p.B, [&](int b) {
    int start, n;
    bool past;
    const int k = seq_blocks(p, b, start, n, past);
    if (past && me == 0) report(p.status, kStatusBounds);
    return k;
  });
  const Runs64 runs = runs_of(total, p.warps / p.side);
  if (run_of_warp >= runs.n) return;
  const int64_t lo = runs.lo(run_of_warp);
  const int64_t hi = runs.lo(run_of_warp + 1);
  if (me == 0 && lane == 0) *p.runs = runs;
  int left = static_cast<int>(hi - lo);  // blocks to take (a run of 2^31 would be 2^35 tokens)
  int b = 0, grp = 0, blk = 0;                        // the next one
  {
    int64_t run = 0;
    for (int base = 0;; base += 32) {
      const int64_t mine = base + lane < p.B ? static_cast<int64_t>(blocks_of(base + lane)) * Hgr : 0;
      int64_t incl = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + incl > lo);
      if (past != 0u) {
        const int l = __ffs(static_cast<int>(past)) - 1;
        const int64_t local = lo - run - __shfl_sync(0xffffffffu, incl - mine, l);
        const int each = static_cast<int>(__shfl_sync(0xffffffffu, mine, l) / Hgr);
        b = base + l;
        grp = static_cast<int>(div_pos(local, static_cast<int64_t>(each)));
        blk = static_cast<int>(local - static_cast<int64_t>(grp) * each);
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }

  // ---- the stream: blocks are asked for kStages ahead, lane i looking up number i of a
  // window of 32 in an item
  int ib = b, ig = grp, iblk = blk, inum = blocks_of(b), ileft = left;  // the next to be asked for
  int win = 0, wlen = 0, wat = 0;  // the window's first block, its length, and the place in it
  int my_id = -1;
  float my_ks = 0.f, my_vs = 0.f;
  int stage_in = 0;
  auto issue = [&]() {  // for the whole warp
    if (ileft == 0) return;
    if (wat == wlen) {
      if (iblk == inum) {  // the next item
        iblk = 0;
        if (++ig == Hgr) {
          ig = 0;
          ib = next_seq(p, lane, ib, inum);  // (there is more to take, so one follows)
        }
      }
      win = iblk;
      wlen = min(32, min(inum - iblk, ileft));
      wat = 0;
      my_id = -1;
      if (lane < wlen) {
        my_id = p.bt[ib * p.bt_stride + win + lane];
        if (my_id < 0 || my_id >= p.num_blocks) {
          report(p.status, kStatusBounds);
          my_id = -1;
        } else {
          my_ks = p.ks[static_cast<int64_t>(my_id) * p.Hkv + ig * p.side + off];
          my_vs = p.vs[static_cast<int64_t>(my_id) * p.Hkv + ig * p.side + off];
        }
      }
    }
    if (lane == wat) {
      uint64_t* bar = &wbar[stage_in];
      uint8_t* dst = wcodes + stage_in * 2 * kCodeBytes;
      if (my_id < 0) {  // bad id: the phase completes without data; the block is left out
        wscale[stage_in] = make_float2(-INFINITY, 0.f);
        mbar_arrive(bar);
      } else {
        wscale[stage_in] = make_float2(my_ks, my_vs * kUnlift);  // (exact, down to the subnormal numbers too)
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, 2 * kCodeBytes);
        if constexpr (D == 128) {
          tma_load_4d(dst, &p.kmap, bar, 0, 0, ig * p.side + off, my_id);
          tma_load_4d(dst + kCodeBytes, &p.vmap, bar, 0, 0, ig * p.side + off, my_id);
        } else {
          const int64_t at = (static_cast<int64_t>(my_id) * p.Hkv + ig * p.side + off) * kCodeBytes;
          bulk_load(dst, p.kq + at, kCodeBytes, bar);
          bulk_load(dst + kCodeBytes, p.vq + at, kCodeBytes, bar);
        }
      }
    }
    __syncwarp();
    ++wat, ++iblk, --ileft;
    if (++stage_in == kStages) stage_in = 0;
  };
  for (int s = 0; s < kStages; ++s) issue();

  const int T[4] = {tok_of(2 * t), tok_of(2 * t + 1), 8 + tok_of(2 * t), 8 + tok_of(2 * t + 1)};
  const int krow = tok_of(g);
  const int R = p.T * p.G;  // rows of the KV head: query r / G, head r % G
  bool ok = true;
  int s = 0;
  uint32_t ph = 0;
  for (int seg = 0; ok && left > 0; ++seg) {
    const int gkv = grp * p.side + off;
    int start, n;
    bool past;
    const int nblk = seq_blocks(p, b, start, n, past);
    const int blk0 = blk, count = min(left, nblk - blk);
    if (blk0 == 0 && off == 0 && lane == 0) p.first[static_cast<int64_t>(b) * Hgr + grp] = 2 * (hi - left) + (seg == 0);
    // the keys that row r sees: [0, limit)
    auto limit = [&](int r) {
      const int i = r / p.G;
      return r >= R || i >= n ? 0 : (p.causal ? start + i + 1 : start + n);
    };
    const int kend = limit(n * p.G - 1);  // keys of the last row that sees any
    const int kfirst = limit(0);          // and of the first

    // ---- q as e4m3 A fragments, hi in rows 0..7, lo in rows 8..15.  The lane's dims are
    // 16 t .. 16 t + 15 (and, D = 128, 64 more on): the word w of a token's 16 codes there
    // meets q's word w, whatever order the product gives them.
    uint32_t qa[NR][kSteps][4];
    float mul[NR];  // scores in log2 units from products of q's codes with unscaled K codes
    int lim[NR];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = 8 * nr + g;
      lim[nr] = limit(r);
      float x[kSteps * 8], a = 0.f;
      const bool there = lim[nr] > 0;
      const uint16_t* row =
          p.q + b * p.q_stride[0] + (gkv * p.G + r % p.G) * p.q_stride[1] + r / p.G * p.q_stride[2];
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const uint4 w = there ? *reinterpret_cast<const uint4*>(row + 16 * t + 64 * (c / 2) + 8 * (c % 2))
                              : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[8 * c + 2 * k] = bf16lo_to_f32(u[k]);
          x[8 * c + 2 * k + 1] = bf16hi_to_f32(u[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kSteps * 8; ++k) {
        if (fabsf(x[k]) < INFINITY)
          a = fmaxf(a, fabsf(x[k]));
        else
          x[k] = NAN;  // infinite scores make no distribution either
      }
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const int e2 = a > 0.f ? f8_scale_exponent(a) : 0;
      const float inv = pow2(-e2);
      mul[nr] = p.scale_log2 * pow2(e2);
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // the word's four dims
          uint32_t hi = 0u, lo = 0u;
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float x0 = x[8 * c + 4 * k + e] * inv, x1 = x[8 * c + 4 * k + e + 1] * inv;
            const uint32_t h2 = f8_codes(x0, x1);
            float y0, y1;
            half2_f32(f8_half2(h2), y0, y1);
            hi |= h2 << (8 * e);
            lo |= f8_codes(x0 - y0, x1 - y1) << (8 * e);
          }
          qa[nr][c][2 * k] = hi;
          qa[nr][c][2 * k + 1] = lo;
        }
    }

    // O^T: tile j holds dims (D / 8) g + 2 j (rows g) and the next one (rows g + 8) of every
    // row; columns 2t, 2t + 1 are this lane's rows
    float o[NR][kTiles][4];
    float m_run[NR], l_part[NR];  // of row g: running max (log2) less kLift, this lane's sum
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      m_run[nr] = -INFINITY, l_part[nr] = 0.f;
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nr][j][e] = 0.f;
    }

    for (; blk < blk0 + count; ++blk, --left) {
      if (!__all_sync(0xffffffffu, mbar_wait(&wbar[s], ph, abort, p.status))) {
        ok = false;
        break;
      }
      const float2 two = wscale[s];
      const float ks = two.x, vs = two.y;
      if (ks != -INFINITY) {
        const uint8_t* kb = wcodes + s * 2 * kCodeBytes;
        const uint8_t* vb = kb + kCodeBytes;
        const int tok0 = blk * kBS;
        // ---- scores: n-tile j holds tokens 8 j + tok_of(n)
        uint32_t pb[NR][2];
        float sc[NR][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint8_t* rowp = kb + (8 * j + krow) * D;
          uint32_t w[kSteps][2];
          if constexpr (D == 128) {
            const uint4 k0 = *reinterpret_cast<const uint4*>(rowp + ((t ^ krow) << 4));
            const uint4 k1 = *reinterpret_cast<const uint4*>(rowp + (((t + 4) ^ krow) << 4));
            w[0][0] = k0.x, w[0][1] = k0.y, w[1][0] = k0.z, w[1][1] = k0.w;
            w[2][0] = k1.x, w[2][1] = k1.y, w[3][0] = k1.z, w[3][1] = k1.w;
          } else {
            const uint4 k0 = *reinterpret_cast<const uint4*>(rowp + (t << 4));
            w[0][0] = k0.x, w[0][1] = k0.y, w[1][0] = k0.z, w[1][1] = k0.w;
          }
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
              mma_e4m3(acc, qa[nr][c][0], qa[nr][c][1], qa[nr][c][2], qa[nr][c][3], w[c][0], w[c][1]);
            sc[nr][2 * j] = acc[0] + acc[2];
            sc[nr][2 * j + 1] = acc[1] + acc[3];
          }
        }
        // ---- softmax
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          const float f = mul[nr] * ks;
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[nr][k] = tok0 + T[k] < lim[nr] ? sc[nr][k] * f : -INFINITY;
          float bm = fmaxf(fmaxf(sc[nr][0], sc[nr][1]), fmaxf(sc[nr][2], sc[nr][3]));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
          // the reference max moves only by more than the margin
          const bool moves = bm > m_run[nr] + (kLift + kLazy);
          if (__any_sync(0xffffffffu, moves)) {
            const float alpha = moves ? fast_exp2(m_run[nr] - (bm - kLift)) : 1.f;  // 0 when m_run was -inf
            if (moves) m_run[nr] = bm - kLift;
            l_part[nr] *= alpha;
            const float f0 = __shfl_sync(0xffffffffu, alpha, 8 * t), f1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              o[nr][j][0] *= f0;
              o[nr][j][1] *= f1;
              o[nr][j][2] *= f0;
              o[nr][j][3] *= f1;
            }
          }
          const float ref = m_run[nr] == -INFINITY ? 0.f : m_run[nr];
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = fast_exp2(sc[nr][k] - ref);
          l_part[nr] += (w[0] + w[1]) + (w[2] + w[3]);
          pb[nr][0] = pack_half2(w[0], w[1]);
          pb[nr][1] = pack_half2(w[2], w[3]);
        }
        // ---- values: the lane's D / 8 dims of its four tokens
        constexpr int kWords = D / 32;
        uint32_t vw[4][kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + T[k] * D + ((g ^ (T[k] & 7)) << 4));
            vw[k][0] = x.x, vw[k][1] = x.y, vw[k][2] = x.z, vw[k][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vb + T[k] * D + g * 8);
            vw[k][0] = x.x, vw[k][1] = x.y;
          }
        }
        // Slots past the last key may hold NaN codes, and 0 x NaN is NaN.  So do tokens that
        // some rows see and others do not: their NaN codes go in as zeros and are
        // handed to the rows that see them.
        if (tok0 + kBS > kfirst) {
          uint32_t bad[4][kWords], any = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < kWords; ++c) {
              if (tok0 + T[k] >= kend) vw[k][c] = 0u;
              bad[k][c] = nan_codes(vw[k][c]);
              any |= bad[k][c];
            }
          if (__any_sync(0xffffffffu, any != 0u)) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int c = 0; c < kWords; ++c) vw[k][c] &= ~((bad[k][c] >> 7) * 255u);
            // which of the dims have a NaN that the row sees: a product of ones
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              uint32_t see[2];
#pragma unroll
              for (int k = 0; k < 2; ++k)
                see[k] = (tok0 + T[2 * k] < lim[nr] ? 0x3c00u : 0u) |
                         (tok0 + T[2 * k + 1] < lim[nr] ? 0x3c000000u : 0u);
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                uint32_t a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // rows g + 8 (e & 1): dim 2 j + (e & 1); tokens 2 (e >> 1), + 1
                  const int byte = 2 * j + (e & 1), k = 2 * (e >> 1);
                  a[e] = ((bad[k][byte / 4] >> (8 * (byte % 4) + 7)) & 1u ? 0x3c00u : 0u) |
                         ((bad[k + 1][byte / 4] >> (8 * (byte % 4) + 7)) & 1u ? 0x3c000000u : 0u);
                }
                float hit[4];
                mma_f16_zero(hit, a, see[0], see[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (hit[e] > 0.f) o[nr][j][e] = NAN;
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
          const uint32_t ab0 = prmt<0x5140u>(vw[0][c], vw[1][c]), ab1 = prmt<0x7362u>(vw[0][c], vw[1][c]);
          const uint32_t cd0 = prmt<0x5140u>(vw[2][c], vw[3][c]), cd1 = prmt<0x7362u>(vw[2][c], vw[3][c]);
          const uint32_t a0[4] = {f8_half2(ab0), f8_half2(ab0 >> 16), f8_half2(cd0), f8_half2(cd0 >> 16)};
          const uint32_t a1[4] = {f8_half2(ab1), f8_half2(ab1 >> 16), f8_half2(cd1), f8_half2(cd1 >> 16)};
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float x[4];
            mma_f16_zero(x, a0, pb[nr][0], pb[nr][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nr][2 * c][e] = fmaf(x[e], vs, o[nr][2 * c][e]);
            mma_f16_zero(x, a1, pb[nr][0], pb[nr][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nr][2 * c + 1][e] = fmaf(x[e], vs, o[nr][2 * c + 1][e]);
          }
        }
      }
      __syncwarp();
      if (++s == kStages) s = 0, ph ^= 1u;
      issue();  // into the stage that was just read
    }
    if (!ok) break;

    // ---- the segment's end: rows 2t and 2t + 1 of each group are this lane's, their states
    // rows g's
    const bool whole = blk0 == 0 && count == nblk;
    const int64_t slot = 2 * static_cast<int64_t>(me) + (seg > 0 ? 1 : 0);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float l = l_part[nr];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m_run[nr] + __log2f(l);
      const int r = 8 * nr + g;
      if (t == 0 && r < R) {
        if (!whole)
          p.part_lse[slot * kRows + r] = lse2;
        else if (p.lse != nullptr)
          p.lse[(static_cast<int64_t>(b) * p.Hq + gkv * p.G + r % p.G) * p.T + r / p.G] = lse2 * 0.6931471805599453f;
      }
#pragma unroll
      for (int hc = 0; hc < 2; ++hc) {
        const float f = __shfl_sync(0xffffffffu, inv, 8 * t + 4 * hc) * (1.0f / kUnlift);
        const int rr = 8 * nr + 2 * t + hc;
        float x[2 * kTiles];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          // (a row that sees nothing has weights of zero, but may have met a NaN)
          x[2 * j] = f == 0.f ? 0.f : o[nr][j][hc] * f;
          x[2 * j + 1] = f == 0.f ? 0.f : o[nr][j][2 + hc] * f;
        }
        if (rr >= R) continue;
        if (whole)
          write_dims(p.out, p.out_bf16,
                     b * p.out_stride[0] + (gkv * p.G + rr % p.G) * p.out_stride[1] + rr / p.G * p.out_stride[2] +
                         (D / 8) * g,
                     x);
        else
          write_dims(p.part_o, 0, (slot * kRows + rr) * D + (D / 8) * g, x);
      }
    }
    if (blk == nblk) {  // the next item
      blk = 0;
      if (++grp == Hgr) {
        grp = 0;
        int n_blocks;
        if (left > 0) b = next_seq(p, lane, b, n_blocks);
      }
    }
  }
  // after a wait that gave up: let the copies in flight land
  for (; left > ileft; --left) {
    drain_wait(&wbar[s], ph);
    if (++s == kStages) s = 0, ph ^= 1u;
  }
}

// Joins the pieces of the items that are cut between warps, and writes those that have no
// blocks.  Where an item's pieces are, the first launch has left (found again from all the
// sequences' lengths it took 1200 us of 8192 short sequences, 233 now in all).  An item's rows go
// to as many CTAs as fill the GPU, a CTA's warps share them.
constexpr int kMergeWarps = 16;  // at most
template <int D, int NR>
__global__ void __launch_bounds__(kMergeWarps * 32) f8_mma_merge_kernel(const __grid_constant__ F8MmaParams p) {
  constexpr int kRows = 8 * NR, E = D / 32;
  __shared__ float acc_of[kMergeWarps][D];
  __shared__ float2 sum_of[kMergeWarps];
  let_next_launch_in();
  wait_for_launch_ahead();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.Hkv, gkv = blockIdx.x - b * p.Hkv;
  const int R = p.T * p.G;
  const int rows = (R + gridDim.y - 1) / gridDim.y;  // of this CTA, `per` warps each
  const int per = static_cast<int>(blockDim.x >> 5) / rows;
  int start, queries;
  bool past;
  const int nblk = seq_blocks(p, b, start, queries, past);
  int w0 = 0, n = 0, head = 0;  // the pieces' runs: the first, their number; whether that is its run's first segment
  if (nblk > 0) {
    const Runs64 runs = *p.runs;
    const int64_t first = p.first[static_cast<int64_t>(b) * (p.Hkv / p.side) + gkv / p.side], u0 = first >> 1;
    if (u0 < 0 || u0 + nblk > runs.lo(runs.n)) return;  // (not written: a wait of the first launch gave up)
    w0 = runs.of(u0);
    n = runs.of(u0 + nblk - 1) - w0 + 1;
    head = static_cast<int>(first & 1);
    if (n == 1) return;  // written where it was computed
  }
  const int part = warp / per, sub = warp - part * per, row = blockIdx.y * rows + part;
  const bool on = part < rows && row < R;
  auto at_piece = [&](int i) {
    return (2 * (static_cast<int64_t>(w0 + i) * p.side + gkv % p.side) + (i == 0 && !head ? 1 : 0)) * kRows + row;
  };
  // this warp's pieces are sub, sub + per, ...: a lane per piece for their weights, then four
  // pieces' rows at a time
  float M = -INFINITY, ws = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int mine = on && n > sub ? (n - sub + per - 1) / per : 0;
  for (int q0 = 0; q0 < mine; q0 += 32) {
    const int here = min(32, mine - q0);
    const float l = lane < here ? p.part_lse[at_piece(sub + (q0 + lane) * per)] : -INFINITY;
    float top = fmaxf(l, M);  // (a NaN is not the largest: it gets to the row by its weight)
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float alpha = M == -INFINITY ? 1.f : fast_exp2(M - top);
    M = top;
    const float w = l == -INFINITY ? 0.f : fast_exp2(l - M);
    ws = ws * alpha + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll 1
    for (int k = 0; k < here; k += 4) {
      float x[4][E], f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f[u] = __shfl_sync(0xffffffffu, w, (k + u) & 31);  // (0 past the last)
        const float* o = p.part_o + at_piece(sub + (q0 + min(k + u, here - 1)) * per) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o);
          x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(o);
          x[u][0] = v.x, x[u][1] = v.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (k + u < here) acc[e] = fmaf(f[u], x[u][e], acc[e]);
    }
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, m);
  if (per > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc_of[warp][lane * E + e] = acc[e];
    if (lane == 0) sum_of[warp] = make_float2(M, ws);
    __syncthreads();
    if (sub != 0 || !on) return;
    float top = M;
    for (int k = 1; k < per; ++k) top = fmaxf(top, sum_of[warp + k].x);
    // (a warp without a max has weights of 0, or a NaN)
    auto factor = [&](float m) { return m == -INFINITY ? 1.f : fast_exp2(m - top); };
    const float own = factor(M);
    ws *= own;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= own;
    for (int k = 1; k < per; ++k) {
      const float2 s = sum_of[warp + k];
      const float f = factor(s.x);
      ws = fmaf(f, s.y, ws);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, acc_of[warp + k][lane * E + e], acc[e]);
    }
    M = top;
  }
  if (!on) return;
  const bool any = !(ws == 0.f);  // a NaN is something
  const int h = gkv * p.G + row % p.G, i = row / p.G;
  const float inv = any ? 1.f / ws : 0.f;
  const int64_t at = b * p.out_stride[0] + h * p.out_stride[1] + i * p.out_stride[2] + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = any ? acc[e] * inv : 0.f, y = any ? acc[e + 1] * inv : 0.f;
    if (p.out_bf16)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at + e) = pack_bf16x2(x, y);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at + e) = make_float2(x, y);
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] =
        any ? (M + __log2f(ws)) * 0.6931471805599453f : -INFINITY;
}

// Rows of a KV head; more go to chunk_f8_tc.cu, whose tile has 128.  Both sides with 16 rows
// (D = 128, 8 KV heads): 64 sequences of 8192 tokens 234 us here and 289 there, 64 of
// 4096 129 and 181, one of 20000 26 and 34, one of 500 14 and 21.
constexpr int64_t kMostRows = 16;
int rows_of(int64_t rows) { return rows <= 8 ? 8 : 16; }
// offsets and size of the workspace
struct Layout {
  size_t lse, runs, first, bytes;
};
static_assert(sizeof(Runs64) == 16, "its place in the workspace");
Layout layout(int64_t items, int64_t rows, int D, int n_cta) {
  const size_t n = static_cast<size_t>(2) * n_cta * kMostWarps * rows_of(rows);
  Layout l;
  l.lse = n * D * 4;
  l.runs = l.lse + n * 4;
  l.first = l.runs + 16;
  l.bytes = (l.first + items * 8 + 255) & ~size_t(255);
  return l;
}

template <int D, int NR>
cudaError_t launch_mma(const F8AttnArgs& a, F8MmaParams& p, cudaStream_t stream) {
  if (D == 128 && (!make_code_cache_map(&p.kmap, a.cache.k, a.cache.num_blocks, a.cache.Hkv) ||
                   !make_code_cache_map(&p.vmap, a.cache.v, a.cache.num_blocks, a.cache.Hkv)))
    return cudaErrorInvalidValue;
  auto kern = paged_attn_f8_mma_kernel<D, NR>;
  auto join = f8_mma_merge_kernel<D, NR>;
  using C = MmaCfg<D, NR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::kWarps));
  // an SM shares its memory out anew only when it is empty: where it has more than one CTA of this
  // launch, the second one asks for the same
  if constexpr (C::kSmWarps > C::kWarps)
    for (const void* k : {reinterpret_cast<const void*>(kern), reinterpret_cast<const void*>(join)})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  p.warps = a.n_cta * C::kSmWarps;
  // no more warps than the call could have runs for
  const int64_t runs = (a.B * (a.cache.Hkv / p.side) * static_cast<int64_t>(a.max_blocks) + kLeast - 1) / kLeast;
  const int64_t most = std::min<int64_t>(p.warps, runs * p.side);
  const int warps = most > kFewWarps * a.n_cta ? C::kWarps : kFewWarps;
  const dim3 grid(static_cast<unsigned>((most + warps - 1) / warps));
  e = launch_early(kern, grid, warps * 32, C::smem(warps), stream, p);
  if (e != cudaSuccess) return e;
  // The second launch: with few rows in all, sixteen warps for each (one sequence of 20000 tokens
  // and 16 rows: 25 us, 36 with eight); else CTAs of eight warps for an item, or half its rows,
  // that fit in one wave (64 sequences of 8192 tokens: 136 us, 140 with sixteen).
  const int64_t items = a.B * a.cache.Hkv, rows = a.T * p.G;
  const bool few = items * rows <= 2 * a.n_cta;
  const int join_warps = few ? 16 : 8;
  const int64_t shares = few ? rows
                             : std::min<int64_t>(rows, std::max<int64_t>((rows + join_warps - 1) / join_warps,
                                                                         4 * a.n_cta / items));
  const dim3 join_grid(static_cast<unsigned>(items), static_cast<unsigned>(shares));
  return launch_early(join, join_grid, join_warps * 32, 0, stream, p);
}

}  // namespace

size_t f8_attn_partial_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t T, int64_t max_blocks, int D, int n_cta) {
  const int64_t G = Hq / Hkv;
  return T * G > kMostRows ? f8_chunk_partial_bytes(T, G, D, n_cta) : layout(B * Hkv, T * G, D, n_cta).bytes;
}

bool f8_attn_fits(int64_t B, int64_t Hq, int64_t Hkv, int64_t T, int64_t max_blocks) {
  const int64_t G = Hq / Hkv;
  return T * G <= kMostRows ? B * Hkv <= 0x7fffffff : f8_chunk_fits(B, Hkv, T, G, max_blocks);  // (a CTA an item)
}

cudaError_t launch_paged_attn_f8(const F8AttnArgs& a, cudaStream_t stream) {
  const int G = static_cast<int>(a.Hq / a.cache.Hkv);
  if (a.T * G > kMostRows) return launch_chunk_f8(a, stream);
  F8MmaParams p = {};
  const Layout l = layout(a.B * a.cache.Hkv, a.T * G, a.cache.D, a.n_cta);
  p.kq = a.cache.k;
  p.vq = a.cache.v;
  p.ks = a.cache.k_scale;
  p.vs = a.cache.v_scale;
  p.num_blocks = a.cache.num_blocks;
  p.Hkv = a.cache.Hkv;
  p.Hq = static_cast<int>(a.Hq);
  p.G = G;
  p.T = static_cast<int>(a.T);
  p.q = static_cast<const uint16_t*>(a.q.data);
  for (int i = 0; i < 3; ++i) p.q_stride[i] = a.q.stride[i], p.out_stride[i] = a.out.stride[i];
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.start = a.start_pos;
  p.lens = a.lens;
  p.causal = a.causal;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.B = static_cast<int>(a.B);
  p.side = 1;
  while (p.side < kSide && p.Hkv % (2 * p.side) == 0) p.side *= 2;
  p.out = a.out.data;
  p.out_bf16 = a.out.dtype == ATTN_BF16;
  p.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(a.partials);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + l.lse);
  p.runs = reinterpret_cast<Runs64*>(ws + l.runs);
  p.first = reinterpret_cast<int64_t*>(ws + l.first);
  p.status = a.status;
  if (a.cache.D == 64)
    return rows_of(a.T * G) == 8 ? launch_mma<64, 1>(a, p, stream) : launch_mma<64, 2>(a, p, stream);
  return rows_of(a.T * G) == 8 ? launch_mma<128, 1>(a, p, stream) : launch_mma<128, 2>(a, p, stream);
}

}  // namespace attn
