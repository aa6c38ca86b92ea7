// kv_edit.cu -- moves of whole K/V rows inside a paged cache.
//   kv_tree_accept   the accepted drafts' rows move up behind the context
//   kv_evict         the tokens worth keeping go to the blocks of another table
// Bit copies in 16-byte vectors; the work is the rows' bytes.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kBS = 16;  // tokens per cache block

struct AcceptParams {
  uint4* kc;
  uint4* vc;
  int64_t num_blocks;
  int Hkv, ch;  // ch: 16-byte chunks per row
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* path;
  int64_t path_stride;
  int max_path;
  const int32_t* n_accept;
  uint32_t* status;
};

// One CTA per (KV head, sequence).  The path is strictly increasing, so row i
// comes from a slot at or past i and the sources of rows >= i lie at or past
// i: a pass that reads its rows before it writes them leaves every later
// pass's sources as they were.  A pass is 8 vectors a thread (64 rows of K and
// V at D = 128: one pass for the usual path).
constexpr int kAcceptThreads = 256, kAcceptVecs = 8;
__global__ void __launch_bounds__(kAcceptThreads) kv_tree_accept_kernel(const AcceptParams p) {
  const int g = blockIdx.x, b = blockIdx.y;
  const int ctx = p.ctx_lens[b], n = p.n_accept[b];
  if (ctx < 0 || n <= 0) return;  // idle, or nothing accepted
  const int32_t* path = p.path + b * p.path_stride;
  const int64_t slots = static_cast<int64_t>(p.max_blocks) * kBS;
  bool bad = n > p.max_path;
  for (int i = threadIdx.x; !bad && i < n; i += kAcceptThreads)
    bad = path[i] < 0 || static_cast<int64_t>(ctx) + path[i] >= slots || (i > 0 && path[i] <= path[i - 1]);
  if (__syncthreads_or(bad)) {  // the sequence is left as it was
    if (threadIdx.x == 0 && g == 0) report(p.status, kStatusBounds);
    return;
  }
  const int32_t* bt = p.bt + b * p.bt_stride;
  auto row = [&](int slot) -> int64_t {  // first chunk of the slot's row, or -1
    const int blk = bt[slot / kBS];
    if (blk < 0 || blk >= p.num_blocks) {
      report(p.status, kStatusBounds);
      return -1;
    }
    return ((static_cast<int64_t>(blk) * p.Hkv + g) * kBS + slot % kBS) * p.ch;
  };
  const int vecs = n * 2 * p.ch;  // K and V chunks of a row side by side
  for (int x0 = 0; x0 < vecs; x0 += kAcceptThreads * kAcceptVecs) {
    uint4 w[kAcceptVecs];
    int64_t dst[kAcceptVecs];
#pragma unroll
    for (int u = 0; u < kAcceptVecs; ++u) {
      const int x = x0 + u * kAcceptThreads + threadIdx.x;
      dst[u] = -1;
      if (x >= vecs) continue;
      const int i = x / (2 * p.ch), c = x % (2 * p.ch);
      if (path[i] == i) continue;  // in place already
      const int64_t from = row(ctx + path[i]), to = row(ctx + i);
      if (from < 0 || to < 0) continue;
      w[u] = (c < p.ch ? p.kc : p.vc)[from + c % p.ch];
      dst[u] = to + c % p.ch;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kAcceptVecs; ++u) {
      const int x = x0 + u * kAcceptThreads + threadIdx.x;
      if (dst[u] >= 0) (x % (2 * p.ch) < p.ch ? p.kc : p.vc)[dst[u]] = w[u];
    }
    // No barrier here: the next pass reads only slots at or past its own rows.
  }
}

// ---------------------------------------------------------------------------
// kv_evict, first launch: which tokens stay.  One cluster per (KV head,
// sequence); its CTAs split the context into consecutive ranges.  A token's rank
// is its accumulated weight as an unsigned key (order-preserving bits; NaN below
// everything, protected tokens above).  The keep-th largest key is found by
// bisection on its bits, two at a time: 16 rounds of counting the keys at or
// above three thresholds, in registers (kKeys a thread; longer ranges are read
// again from L2 each round), one reduction and one cluster barrier a round.
// Ties at the threshold go to the lowest slots.  The cost is the rounds'
// latency, not the bytes: 4160 tokens about 5 us.
// ---------------------------------------------------------------------------
struct EvictParams {
  const uint4* kc;
  const uint4* vc;
  uint4* kd;  // the same tensors, as destinations
  uint4* vd;
  float* acc;  // [num_blocks, Hkv, 16]
  int64_t num_blocks;
  int Hkv, ch;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* dst;
  int64_t dst_stride;
  int dst_blocks;
  const int32_t* ctx_lens;
  int keep, sink, recent;
  int32_t* new_lens;
  int32_t* kept;  // [B, Hkv, keep]
  uint32_t* status;
};

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kKeys = 16;  // keys a thread holds
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t rank_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0: they tie
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// store to the word at the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ void peer_store(int* p, uint32_t rank, int v) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// grid (cluster size, Hkv, B), clusters along x
__global__ void __launch_bounds__(kSelThreads, 1) kv_evict_select_kernel(const EvictParams p, const int nc) {
  __shared__ int warp_cnt[kSelWarps][3];
  // every CTA's counts, pushed by their owners, alternating between rounds (a
  // cluster barrier separates a buffer's readers from its next writers)
  __shared__ int cta_cnt[2][kMaxCluster][3];
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z;
  const int rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hkv + g) * p.keep;
  const int len = p.ctx_lens[b];
  const int64_t slots = static_cast<int64_t>(p.max_blocks) * kBS;
  const int L = len < 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(len), slots));
  if (rank == 0 && threadIdx.x == 0 && g == 0) {
    if (len > slots) report(p.status, kStatusBounds);
    p.new_lens[b] = len < 0 ? len : min(L, p.keep);
  }
  if (L <= p.keep) {  // everything stays (the whole cluster leaves here)
    for (int i = rank * kSelThreads + threadIdx.x; i < p.keep; i += nc * kSelThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const int32_t* bt = p.bt + b * p.bt_stride;
  auto key_of = [&](int i) -> uint32_t {
    if (i < p.sink || i >= L - p.recent) return 0xffffffffu;
    const int blk = bt[i / kBS];
    if (blk < 0 || blk >= p.num_blocks) {
      report(p.status, kStatusBounds);
      return 0u;
    }
    return rank_key(p.acc[(static_cast<int64_t>(blk) * p.Hkv + g) * kBS + i % kBS]);
  };
  // this warp's tokens [w0, w1): a consecutive range of the cluster's warps, 32
  // aligned, element e of lane l at w0 + 32 e + l
  const int per = ((L + nc * kSelWarps - 1) / (nc * kSelWarps) + 31) / 32 * 32;
  const int w0 = min(L, (rank * kSelWarps + warp) * per), w1 = min(L, w0 + per);
  const int ne = (w1 - w0 + 31) / 32;
  const bool held = per <= 32 * kKeys;  // the same for the whole cluster
  uint32_t key[kKeys];
  if (held) {
    // all block ids, then all sums: two round trips to memory
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      const int i = w0 + 32 * e + lane;
      key[e] = i < w1 ? static_cast<uint32_t>(bt[i / kBS]) : 0u;
    }
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      const int i = w0 + 32 * e + lane;
      const bool there = i < w1 && key[e] < static_cast<uint64_t>(p.num_blocks);
      if (i < w1 && !there) report(p.status, kStatusBounds);
      const float x = there ? p.acc[(static_cast<int64_t>(key[e]) * p.Hkv + g) * kBS + i % kBS] : 0.f;
      key[e] = there ? rank_key(x) : 0u;
      if (i < w1 && (i < p.sink || i >= L - p.recent)) key[e] = 0xffffffffu;
    }
  }
  // largest threshold that at least `keep` keys reach (a filler key 0 is only
  // counted at threshold 0, which is never asked about)
  uint32_t thr = 0u;
  int above = 0;  // keys >= thr + (1 << shift) of the last round: after it, keys > thr
  for (int round = 0; round < 16; ++round) {
    const int shift = 30 - 2 * round;
    const uint32_t t1 = thr + (1u << shift), t2 = thr + (2u << shift), t3 = thr + (3u << shift);
    int c1 = 0, c2 = 0, c3 = 0;
    if (held) {
#pragma unroll
      for (int e = 0; e < kKeys; ++e) {
        if (e >= ne) break;
        c1 += key[e] >= t1, c2 += key[e] >= t2, c3 += key[e] >= t3;
      }
    } else {
      for (int e = 0; e < ne; ++e) {
        const int i = w0 + 32 * e + lane;
        const uint32_t k = i < w1 ? key_of(i) : 0u;
        c1 += k >= t1, c2 += k >= t2, c3 += k >= t3;
      }
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if (lane == 0) warp_cnt[warp][0] = c1, warp_cnt[warp][1] = c2, warp_cnt[warp][2] = c3;
    __syncthreads();
    if (threadIdx.x < 3 * nc) {
      const int c = threadIdx.x % 3;
      int s = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) s += warp_cnt[w][c];
      peer_store(&cta_cnt[round & 1][rank][c], threadIdx.x / 3, s);
    }
    cluster_sync();
    c1 = c2 = c3 = 0;
    for (int r = 0; r < nc; ++r) {
      c1 += cta_cnt[round & 1][r][0];
      c2 += cta_cnt[round & 1][r][1];
      c3 += cta_cnt[round & 1][r][2];
    }
    if (c3 >= p.keep)
      thr = t3;
    else if (c2 >= p.keep)
      thr = t2, above = c3;
    else if (c1 >= p.keep)
      thr = t1, above = c2;
    else
      above = c1;
  }
  // `above` keys are greater than thr; the first keep - above of those equal to it stay too
  const int need = p.keep - above;
  int gt = 0, eq = 0;
  auto key_at = [&](int e) -> uint32_t {
    const int i = w0 + 32 * e + lane;
    return i < w1 ? key_of(i) : 0u;
  };
  if (held) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      if (e >= ne) break;
      const bool in = w0 + 32 * e + lane < w1;
      gt += in && key[e] > thr, eq += in && key[e] == thr;
    }
  } else {
    for (int e = 0; e < ne; ++e) {
      const bool in = w0 + 32 * e + lane < w1;
      const uint32_t k = key_at(e);
      gt += in && k > thr, eq += in && k == thr;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
  __syncthreads();
  if (threadIdx.x < 2 * nc) {
    const int c = threadIdx.x & 1;
    int s = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) s += c ? warp_eq[w] : warp_gt[w];
    peer_store(&cta_cnt[0][rank][c], threadIdx.x >> 1, s);  // round 15 used buffer 1
  }
  cluster_sync();
  int gt0 = 0, eq0 = 0;  // before this warp's range
  if (lane < warp) gt0 = warp_gt[lane], eq0 = warp_eq[lane];
  if (lane < rank) gt0 += cta_cnt[0][lane][0], eq0 += cta_cnt[0][lane][1];
  gt0 = __reduce_add_sync(0xffffffffu, gt0);
  eq0 = __reduce_add_sync(0xffffffffu, eq0);
  const uint32_t below = (1u << lane) - 1u;
  auto place = [&](int e, uint32_t k) {
    const int i = w0 + 32 * e + lane;
    const bool in = i < w1;
    const uint32_t mg = __ballot_sync(0xffffffffu, in && k > thr), me = __ballot_sync(0xffffffffu, in && k == thr);
    const int e_rank = eq0 + __popc(me & below);
    if (in && (k > thr || (k == thr && e_rank < need))) kept[gt0 + __popc(mg & below) + min(e_rank, need)] = i;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  };
  if (held) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      if (e >= ne) break;
      place(e, key[e]);
    }
  } else {
    for (int e = 0; e < ne; ++e) place(e, key_at(e));
  }
}

// kv_evict, second launch: the kept rows and their weights to the other table's
// blocks.  grid (row groups, Hkv, B).  The rows' places come first, one thread a
// row (kept slot -> block -> row: three dependent loads, once), then the rows
// stream through registers, kCopyVecs 16-byte vectors a thread in flight.
constexpr int kCopyThreads = 256, kCopyVecs = 8, kCopyRows = 128;
template <int CH>  // 16-byte chunks per row
__global__ void __launch_bounds__(kCopyThreads) kv_evict_copy_kernel(const EvictParams p) {
  __shared__ int64_t from[kCopyRows], to[kCopyRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z;
  const int r0 = blockIdx.x * kCopyRows;
  const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hkv + g) * p.keep + r0;
  // the cache row of a slot, or -1
  auto place = [&](const int32_t* table, int blocks, int slot) -> int64_t {
    const int blk = slot / kBS < blocks ? table[slot / kBS] : -1;
    if (blk < 0 || blk >= p.num_blocks) {
      report(p.status, kStatusBounds);
      return -1;
    }
    return (static_cast<int64_t>(blk) * p.Hkv + g) * kBS + slot % kBS;
  };
  if (threadIdx.x < kCopyRows) {
    const int i = threadIdx.x;
    int64_t f = -1, d = -1;
    const int slot = r0 + i < p.keep ? kept[i] : -1;
    if (slot >= 0) {
      f = place(p.bt + b * p.bt_stride, p.max_blocks, slot);
      d = place(p.dst + b * p.dst_stride, p.dst_blocks, r0 + i);
    }
    if (f >= 0 && d >= 0)
      p.acc[d] = p.acc[f];
    else
      f = -1;
    from[i] = f;
    to[i] = d;
  }
  __syncthreads();
  constexpr int kRowsPerStep = kCopyThreads / CH;
  const int c = threadIdx.x % CH, i0 = threadIdx.x / CH;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const uint4* src = half ? p.vc : p.kc;
    uint4* dst = half ? p.vd : p.kd;
#pragma unroll 1
    for (int i = i0; i < kCopyRows; i += kRowsPerStep * kCopyVecs) {
      uint4 w[kCopyVecs];
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u) {
        const int r = i + u * kRowsPerStep;
        if (r < kCopyRows && from[r] >= 0) w[u] = src[from[r] * CH + c];
      }
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u) {
        const int r = i + u * kRowsPerStep;
        if (r < kCopyRows && from[r] >= 0) dst[to[r] * CH + c] = w[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t stream) {
  EvictParams p;
  p.kc = static_cast<const uint4*>(a.cache.k);
  p.vc = static_cast<const uint4*>(a.cache.v);
  p.kd = static_cast<uint4*>(a.cache.k);
  p.vd = static_cast<uint4*>(a.cache.v);
  p.acc = a.acc;
  p.num_blocks = a.cache.num_blocks;
  p.Hkv = a.cache.Hkv;
  p.ch = a.cache.D / 8;
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.dst = a.dst_table;
  p.dst_stride = a.dst_stride;
  p.dst_blocks = a.dst_blocks;
  p.ctx_lens = a.ctx_lens;
  p.keep = a.keep;
  p.sink = a.sink;
  p.recent = a.recent;
  p.new_lens = a.new_lens;
  p.kept = a.kept;
  p.status = a.status;
  // a CTA per kSelThreads * kKeys tokens of the longest possible context, up to a portable cluster
  const int64_t slots = static_cast<int64_t>(a.max_blocks) * kBS;
  int nc = 1;
  while (nc < kMaxCluster && static_cast<int64_t>(nc) * kSelThreads * kKeys < slots) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nc), static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(nc);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_select_kernel, p, nc);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((a.keep + kCopyRows - 1) / kCopyRows),
                     static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(kCopyThreads);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return p.ch == 16 ? cudaLaunchKernelEx(&cfg, kv_evict_copy_kernel<16>, p)
                    : cudaLaunchKernelEx(&cfg, kv_evict_copy_kernel<8>, p);
}

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  AcceptParams p;
  p.kc = static_cast<uint4*>(a.cache.k);
  p.vc = static_cast<uint4*>(a.cache.v);
  p.num_blocks = a.cache.num_blocks;
  p.Hkv = a.cache.Hkv;
  p.ch = a.cache.D / 8;
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctx_lens = a.ctx_lens;
  p.path = a.path;
  p.path_stride = a.path_stride;
  p.max_path = a.max_path;
  p.n_accept = a.n_accept;
  p.status = a.status;
  dim3 grid(static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  kv_tree_accept_kernel<<<grid, kAcceptThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
