// attn_f8.cu -- attention of few query rows (at most 16 per KV head: decode steps and
// short drafts) over an e4m3 paged cache (paged_attn_f8).
//
// A warp takes a block (16 tokens of one KV head) at a time, with no conversion of K:
//  * q is split into two e4m3 numbers, q = (hi + lo) 2^e, with 2^e the power of two that
//    brings the row's largest element to 448 or below.  bf16 has eight significant
//    bits and e4m3 four, so hi + lo is q exactly, down to 2^-19 of the largest
//    element.  hi and lo of eight rows are the 16 rows of one m16n8k32 product with
//    the codes as they lie in the cache; adding a lane's two accumulators is the score,
//    and the block's scale multiplies it.
//  * the values go in transposed, O^T = V^T W^T (m16n8k16, fp16): a head's weights
//    are, register for register, their score fragment, and codes become fp16 exactly,
//    two an instruction.  The block's value scale multiplies the products.
// A warp's blocks arrive in its own ring of kStages; softmax is online with a lazy
// running max (log2 units, it moves when a block exceeds it by kLazy).
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "f8.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kBS = 16;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr float kLazy = 8.0f;

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
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start;
  const int32_t* lens;
  int causal;
  float scale_log2;
  int split_tokens, n_split;
  void* out;
  int out_bf16;
  int64_t out_stride[3];
  float* lse;
  float* part_o;    // [(b, KV head, split)][8 NR][D]
  float* part_lse;  // [the same][8 NR], log2 units
  unsigned long long* count;  // [b, KV head]
  uint32_t gen;
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

template <int D>
__device__ __forceinline__ void write_row(const F8MmaParams& p, int b, int h, int i, int d, float x, float y) {
  const int64_t at = b * p.out_stride[0] + h * p.out_stride[1] + i * p.out_stride[2] + d;
  if (p.out_bf16)
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = pack_bf16x2(x, y);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(x, y);
}

// grid (splits, KV heads, sequences)
template <int D, int NR>
__global__ void __launch_bounds__(kWarps * 32, NR == 1 ? 4 : 3)
    paged_attn_f8_mma_kernel(const __grid_constant__ F8MmaParams p) {
  constexpr int kCodeBytes = kBS * D;  // one (block, head) of K or V
  constexpr int kRows = 8 * NR;
  constexpr int kSteps = D / 32;       // of the score product
  constexpr int kTiles = D / 16;       // of the output's dims
  constexpr int kRec = D + 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* codes = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // [warp][stage][K, V]
  uint64_t* bars = reinterpret_cast<uint64_t*>(codes + kWarps * kStages * 2 * kCodeBytes);
  float* comb = reinterpret_cast<float*>(codes);  // [warp][row][D + 2] at the end
  static_assert(kWarps * kRows * kRec * 4 <= kWarps * kStages * 2 * kCodeBytes, "records fit");
  __shared__ int abort_flag, s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* wcodes = codes + warp * kStages * 2 * kCodeBytes;
  uint64_t* wbar = bars + warp * kStages;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&wbar[s], 1);
    if (warp == 0) {
      abort_flag = 0;
      if constexpr (D == 128) {
        tma_prefetch_desc(&p.kmap);
        tma_prefetch_desc(&p.vmap);
      }
    }
  }
  fence_mbar_init();
  let_next_launch_in();
  __syncthreads();
  wait_for_launch_ahead();

  const int split = blockIdx.x, gkv = blockIdx.y, b = blockIdx.z;
  const int R = p.T * p.G;  // rows of the KV head: query r / G, head r % G
  int start;
  bool past;
  const int n = queries(p, b, start, past);
  if (past && threadIdx.x == 0 && split == 0) report(p.status, kStatusBounds);
  // the keys that row r sees: [0, limit)
  auto limit = [&](int r) {
    const int i = r / p.G;
    return r >= R || i >= n ? 0 : (p.causal ? start + i + 1 : start + n);
  };
  const int kend = n == 0 ? 0 : limit(n * p.G - 1);  // keys of the last row that sees any
  const int kfirst = limit(0);                        // and of the first
  auto write_empty = [&](int r) {
    const int h = gkv * p.G + r % p.G, i = r / p.G;
    for (int d = 2 * lane; d < D; d += 64) write_row<D>(p, b, h, i, d, 0.f, 0.f);
    if (lane == 0 && p.lse != nullptr) p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = -INFINITY;
  };
  const int t_begin = split * p.split_tokens;
  if (t_begin >= kend) {
    if (split == 0)  // no row sees anything
      for (int r = warp; r < R; r += kWarps) write_empty(r);
    return;
  }
  const int t_end = min(kend, t_begin + p.split_tokens);
  const int nblk = (t_end - t_begin + kBS - 1) / kBS;
  const int lb0 = t_begin / kBS;

  const int my_n = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;  // at most 32
  int my_blk = -1;
  float my_ks = 0.f, my_vs = 0.f;
  if (lane < my_n) {
    my_blk = p.bt[b * p.bt_stride + lb0 + warp + kWarps * lane];
    if (my_blk < 0 || my_blk >= p.num_blocks) {
      report(p.status, kStatusBounds);
      my_blk = -1;
    } else {
      my_ks = p.ks[static_cast<int64_t>(my_blk) * p.Hkv + gkv];
      my_vs = p.vs[static_cast<int64_t>(my_blk) * p.Hkv + gkv];
    }
  }
  auto issue = [&](int s, int blk) {
    if (blk < 0) {  // bad id: the phase completes without data; the block is left out
      mbar_arrive(&wbar[s]);
      return;
    }
    uint8_t* dst = wcodes + s * 2 * kCodeBytes;
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(&wbar[s], 2 * kCodeBytes);
    if constexpr (D == 128) {
      tma_load_4d(dst, &p.kmap, &wbar[s], 0, 0, gkv, blk);
      tma_load_4d(dst + kCodeBytes, &p.vmap, &wbar[s], 0, 0, gkv, blk);
    } else {
      const int64_t at = (static_cast<int64_t>(blk) * p.Hkv + gkv) * kCodeBytes;
      bulk_load(dst, p.kq + at, kCodeBytes, &wbar[s]);
      bulk_load(dst + kCodeBytes, p.vq + at, kCodeBytes, &wbar[s]);
    }
  };
  int issued = 0;
  for (; issued < kStages && issued < my_n; ++issued) {
    const int blk = __shfl_sync(0xffffffffu, my_blk, issued);
    if (lane == 0) issue(issued, blk);
  }

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
        p.q + b * p.q_stride[0] + (gkv * p.G + r % p.G) * p.q_stride[1] + static_cast<int64_t>(r / p.G) * p.q_stride[2];
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

  const int T[4] = {tok_of(2 * t), tok_of(2 * t + 1), 8 + tok_of(2 * t), 8 + tok_of(2 * t + 1)};
  const int krow = tok_of(g);
  // O^T: tile j holds dims (D / 8) g + 2 j (rows g) and the next one (rows g + 8) of every
  // row; columns 2t, 2t + 1 are this lane's rows
  float o[NR][kTiles][4];
  float m_run[NR], l_part[NR];  // of row g: running max (log2), this lane's sum
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    m_run[nr] = -INFINITY, l_part[nr] = 0.f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nr][j][e] = 0.f;
  }

  bool ok = true;
  int s = 0;
  uint32_t ph = 0;
  for (int i = 0; i < my_n; ++i) {
    const int blk = __shfl_sync(0xffffffffu, my_blk, i);
    const float ks = __shfl_sync(0xffffffffu, my_ks, i), vs = __shfl_sync(0xffffffffu, my_vs, i);
    if (!__all_sync(0xffffffffu, mbar_wait(&wbar[s], ph, &abort_flag, p.status))) {
      ok = false;
      break;
    }
    if (blk >= 0) {
      const uint8_t* kb = wcodes + s * 2 * kCodeBytes;
      const uint8_t* vb = kb + kCodeBytes;
      const int tok0 = (lb0 + warp + kWarps * i) * kBS;
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
        const bool moves = bm > m_run[nr] + kLazy;
        if (__any_sync(0xffffffffu, moves)) {
          const float alpha = moves ? fast_exp2(m_run[nr] - bm) : 1.f;  // 0 when m_run was -inf
          if (moves) m_run[nr] = bm;
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
              see[k] = (tok0 + T[2 * k] < lim[nr] ? 0x3c00u : 0u) | (tok0 + T[2 * k + 1] < lim[nr] ? 0x3c000000u : 0u);
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
    if (issued < my_n) {
      const int nb = __shfl_sync(0xffffffffu, my_blk, issued);
      if (lane == 0) issue(s, nb);
      ++issued;
    }
    if (++s == kStages) s = 0, ph ^= 1u;
  }
  if (!ok)  // let the copies in flight land
    for (int i = max(0, issued - kStages); i < issued; ++i) drain_wait(&wbar[i % kStages], (i / kStages) & 1);

  // ---- the warps' states, joined in shared memory
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    l_part[nr] += __shfl_xor_sync(0xffffffffu, l_part[nr], 1);
    l_part[nr] += __shfl_xor_sync(0xffffffffu, l_part[nr], 2);
  }
  __syncthreads();  // every warp's codes have been read
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    if (t == 0) {
      float* rec = comb + (warp * kRows + 8 * nr + g) * kRec + D;
      rec[0] = m_run[nr];
      rec[1] = l_part[nr];
    }
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) {
      float* rec = comb + (warp * kRows + 8 * nr + 2 * t + hc) * kRec + (D / 8) * g;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        rec[2 * j] = o[nr][j][hc];
        rec[2 * j + 1] = o[nr][j][2 + hc];
      }
    }
  }
  __syncthreads();
  const int ns = (kend + p.split_tokens - 1) / p.split_tokens;  // splits with keys
  const int64_t unit = static_cast<int64_t>(b) * p.Hkv + gkv;
  for (int r = warp; r < R; r += kWarps) {
    float M = -INFINITY, wgt[kWarps], l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, comb[(w * kRows + r) * kRec + D]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* rec = comb + (w * kRows + r) * kRec + D;
      // a warp that saw nothing has max -inf and sum 0; a NaN sum is something
      wgt[w] = rec[0] == -INFINITY ? (rec[1] == 0.f ? 0.f : 1.f) : fast_exp2(rec[0] - M);
      l = fmaf(wgt[w], rec[1], l);
    }
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    const float lse2 = empty ? -INFINITY : M + __log2f(l);
    const int h = gkv * p.G + r % p.G, i = r / p.G;
    const int64_t slot = (unit * p.n_split + split) * kRows + r;
    for (int d = 2 * lane; d < D; d += 64) {
      float x = 0.f, y = 0.f;
      if (!empty) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* rec = comb + (w * kRows + r) * kRec + d;
          if (wgt[w] == 0.f) continue;
          x = fmaf(wgt[w], rec[0], x);
          y = fmaf(wgt[w], rec[1], y);
        }
      }
      if (ns == 1)
        write_row<D>(p, b, h, i, d, x * inv, y * inv);
      else
        *reinterpret_cast<float2*>(p.part_o + slot * D + d) = make_float2(x * inv, y * inv);
    }
    if (lane == 0) {
      if (ns > 1)
        p.part_lse[slot] = lse2;
      else if (p.lse != nullptr)
        p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = lse2 * 0.6931471805599453f;
    }
  }
  if (ns == 1) return;

  // ---- the last split of the unit to come here joins them all, in order
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = count_last(p.count + unit, p.gen, ns);
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int r = warp; r < R; r += kWarps) {
    const int64_t first = unit * p.n_split * kRows + r;
    float M = -INFINITY;
    bool any = false;
    for (int k = lane; k < ns; k += 32) {
      const float l = __ldcg(p.part_lse + first + static_cast<int64_t>(k) * kRows);
      M = fmaxf(M, l);
      any |= l != -INFINITY;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    any = __any_sync(0xffffffffu, any);
    const int h = gkv * p.G + r % p.G, i = r / p.G;
    if (!any) {
      write_empty(r);
      continue;
    }
    float2 acc[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) acc[c] = make_float2(0.f, 0.f);
    float ws = 0.f;
#pragma unroll 4
    for (int k = 0; k < ns; ++k) {
      const int64_t at = first + static_cast<int64_t>(k) * kRows;
      const float l = __ldcg(p.part_lse + at);
      const float w = l == -INFINITY ? 0.f : fast_exp2(l - M);
      ws += w;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part_o + at * D + 2 * lane + 64 * c));
        acc[c].x = fmaf(w, x.x, acc[c].x);
        acc[c].y = fmaf(w, x.y, acc[c].y);
      }
    }
    const float inv = 1.f / ws;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) write_row<D>(p, b, h, i, 2 * lane + 64 * c, acc[c].x * inv, acc[c].y * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + i] = (M + __log2f(ws)) * 0.6931471805599453f;
  }
}

constexpr int64_t kMostRows = 16;  // of a KV head; more go to chunk_f8_tc.cu
int rows_of(int64_t rows) { return rows <= 8 ? 8 : 16; }
// tokens of a split
int split_tokens(int64_t units, int64_t max_blocks, int n_cta) {
  // half a split as long as the GPU has room for the CTAs, down to a block a warp
  int tokens = 1024;
  while (tokens > kWarps * kBS && units * ((max_blocks * kBS + tokens - 1) / tokens) < 4 * n_cta) tokens /= 2;
  return tokens;
}

struct Layout {
  int64_t units, n_split;
  int tokens;
  size_t o, lse, count, bytes;  // offsets and size of the workspace
};
Layout layout(int64_t B, int64_t Hq, int64_t Hkv, int64_t T, int64_t max_blocks, int D, int n_cta) {
  Layout l;
  l.units = B * Hkv;
  l.tokens = split_tokens(l.units, max_blocks, n_cta);
  l.n_split = std::max<int64_t>(1, (max_blocks * kBS + l.tokens - 1) / l.tokens);
  const size_t rows = static_cast<size_t>(l.units) * l.n_split * rows_of(T * (Hq / Hkv));
  l.o = 0;
  l.lse = rows * D * 4;
  l.count = (l.lse + rows * 4 + 255) & ~size_t(255);
  l.bytes = (l.count + l.units * 8 + 255) & ~size_t(255);
  return l;
}

template <int D, int NR>
cudaError_t launch_mma(const F8AttnArgs& a, F8MmaParams& p, const Layout& l, cudaStream_t stream) {
  if (D == 128 && (!make_code_cache_map(&p.kmap, a.cache.k, a.cache.num_blocks, a.cache.Hkv) ||
                   !make_code_cache_map(&p.vmap, a.cache.v, a.cache.num_blocks, a.cache.Hkv)))
    return cudaErrorInvalidValue;
  auto kern = paged_attn_f8_mma_kernel<D, NR>;
  constexpr int smem = 1024 + kWarps * kStages * (2 * kBS * D + 8);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(l.n_split), static_cast<unsigned>(a.cache.Hkv),
                  static_cast<unsigned>(a.B));
  return launch_early(kern, grid, kWarps * 32, smem, stream, p);
}

}  // namespace

size_t f8_attn_partial_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t T, int64_t max_blocks, int D, int n_cta) {
  const int64_t G = Hq / Hkv;
  return T * G > kMostRows ? f8_chunk_partial_bytes(T, G, D, n_cta) : layout(B, Hq, Hkv, T, max_blocks, D, n_cta).bytes;
}

bool f8_attn_fits(int64_t B, int64_t Hq, int64_t Hkv, int64_t T, int64_t max_blocks) {
  const int64_t G = Hq / Hkv;
  return T * G <= kMostRows || f8_chunk_fits(B, Hkv, T, G, max_blocks);
}

cudaError_t launch_paged_attn_f8(const F8AttnArgs& a, cudaStream_t stream) {
  const int G = static_cast<int>(a.Hq / a.cache.Hkv);
  if (a.T * G > kMostRows) return launch_chunk_f8(a, stream);
  F8MmaParams p = {};
  const Layout l = layout(a.B, a.Hq, a.cache.Hkv, a.T, a.max_blocks, a.cache.D, a.n_cta);
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
  p.split_tokens = l.tokens;
  p.n_split = static_cast<int>(l.n_split);
  p.out = a.out.data;
  p.out_bf16 = a.out.dtype == ATTN_BF16;
  p.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(a.partials);
  p.part_o = reinterpret_cast<float*>(ws + l.o);
  p.part_lse = reinterpret_cast<float*>(ws + l.lse);
  p.count = reinterpret_cast<unsigned long long*>(ws + l.count);
  p.gen = a.gen;
  p.status = a.status;
  if (a.cache.D == 64)
    return rows_of(a.T * G) == 8 ? launch_mma<64, 1>(a, p, l, stream) : launch_mma<64, 2>(a, p, l, stream);
  return rows_of(a.T * G) == 8 ? launch_mma<128, 1>(a, p, l, stream) : launch_mma<128, 2>(a, p, l, stream);
}

}  // namespace attn
