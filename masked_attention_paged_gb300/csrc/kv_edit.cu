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
  let_next_launch_in();
  wait_for_launch_ahead();
  const int g = blockIdx.x, b = blockIdx.y;
  const int32_t* path = p.path + b * p.path_stride;
  const int ctx = p.ctx_lens[b], n = p.n_accept[b];
  // the path's start sets out with the lengths (and is in L1 from here on)
  const int mine = threadIdx.x < p.max_path ? path[threadIdx.x] : 0;
  const int before = threadIdx.x > 0 && threadIdx.x < p.max_path ? path[threadIdx.x - 1] : -1;
  if (ctx < 0 || n <= 0) return;  // idle, or nothing accepted
  const int64_t slots = static_cast<int64_t>(p.max_blocks) * kBS;
  bool bad = n > p.max_path;
  const auto wrong = [&](int at, int last) { return at <= last || static_cast<int64_t>(ctx) + at >= slots; };
  if (!bad && static_cast<int>(threadIdx.x) < n) bad = wrong(mine, before);  // the first entry against -1
  for (int i = threadIdx.x + kAcceptThreads; !bad && i < n; i += kAcceptThreads) bad = wrong(path[i], path[i - 1]);
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
// everything, protected tokens above).  The keep-th largest key is found eight
// bits at a time: a histogram of the keys that agree with the bits found so far
// in every CTA, added up into every CTA of the cluster, and the digit at which
// the count from above reaches `keep`.  Ties at the threshold go to the lowest
// slots.  Keys lie in shared memory and the loops over them stay rolled (a range
// longer than kKeys is read again from L2 in each pass): the cost is latency,
// of the passes and of fetching the code once, not the bytes.  It ends with the
// pass after which every key of the digit stays: the third, for distinct sums.  2 x 8
// contexts of 65521 tokens: 20 us (22 with all four passes, 45 with sixteen rounds of
// counting two bits at a time).  Past 65536 tokens, a cluster's keys, every walk reads
// again: the whole call for 1 x 8 contexts of 65536 tokens 22 us, of 65552 50, of
// 131072 86 (D = 64).
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
  bool vec_acc;  // acc begins on a 16-byte boundary
};

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kKeys = 8192;  // keys a CTA holds
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
// Not the .aligned forms: lanes may come here from different sides of a branch.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// the word at the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_word(const int* p, uint32_t rank) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  return addr;
}

// grid (cluster size, Hkv, B), clusters along x.  Two CTAs an SM (54 registers): left to
// itself the compiler took 40 and a spill, for three, and 64 x 4160 tokens took 341 us
// instead of 335.
__global__ void __launch_bounds__(kSelThreads, 2) kv_evict_select_kernel(const EvictParams p, const int nc) {
  __shared__ __align__(16) uint32_t keys[kKeys];
  __shared__ int hist[256];
  // the cluster's histogram, alternating between passes: a CTA clears one before
  // the cluster barrier after which its peers add to it
  __shared__ __align__(16) int total[2][256];
  __shared__ int warp_cnt[2][kSelWarps], cta_cnt[kMaxCluster][2];
  let_next_launch_in();
  wait_for_launch_ahead();
  const int g = blockIdx.y, b = blockIdx.z;
  const int rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hkv + g) * p.keep;
  const int len = p.ctx_lens[b];
  const int64_t slots = static_cast<int64_t>(p.max_blocks) * kBS;
  const int L = len < 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(len), slots));
  if (rank == 0 && threadIdx.x == 0 && g == 0 && len > slots) report(p.status, kStatusBounds);
  if (L <= p.keep) {  // everything stays (the whole cluster leaves here)
    for (int i = rank * kSelThreads + threadIdx.x; i < p.keep; i += nc * kSelThreads) kept[i] = i < L ? i : -1;
    return;
  }
  for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = total[0][i] = 0;
  cluster_arrive();
  const int32_t* bt = p.bt + b * p.bt_stride;
  const auto block_sums = [&](int blk) { return p.acc + (static_cast<int64_t>(blk) * p.Hkv + g) * kBS; };
  const auto known = [&](int blk) { return blk >= 0 && blk < p.num_blocks; };
  const auto protect = [&](int i) { return i < p.sink || i >= L - p.recent; };
  // this warp's tokens [w0, w1): a consecutive range of the cluster's warps
  const int per = ((L + nc * kSelWarps - 1) / (nc * kSelWarps) + 31) / 32 * 32;
  const int w0 = static_cast<int>(min(static_cast<int64_t>(L), static_cast<int64_t>(rank * kSelWarps + warp) * per));
  const int w1 = min(L, w0 + per);
  const bool held = per <= kKeys / kSelWarps;  // the same for the whole cluster
  uint32_t* mine = keys + warp * (kKeys / kSelWarps);
  if (held) {
    // four tokens of a block a lane and step: all block ids, then all sums
    constexpr int kSteps = kKeys / kSelWarps / 128;
    int blk[kSteps];
    float4 x[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int i = w0 + 128 * s + 4 * lane;
      blk[s] = i < w1 ? bt[i / kBS] : -1;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int i = w0 + 128 * s + 4 * lane;
      x[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!known(blk[s])) continue;
      const float* at = block_sums(blk[s]) + i % kBS;
      if (p.vec_acc)
        x[s] = *reinterpret_cast<const float4*>(at);
      else
        x[s] = make_float4(at[0], at[1], at[2], at[3]);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int i = w0 + 128 * s + 4 * lane;
      if (i >= w1) continue;
      uint32_t k[4] = {rank_key(x[s].x), rank_key(x[s].y), rank_key(x[s].z), rank_key(x[s].w)};
      if (!known(blk[s])) {
        report(p.status, kStatusBounds);
        k[0] = k[1] = k[2] = k[3] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (protect(i + c)) k[c] = 0xffffffffu;
      *reinterpret_cast<uint4*>(mine + 128 * s + 4 * lane) = make_uint4(k[0], k[1], k[2], k[3]);
    }
  }
  const auto key_at = [&](int i) -> uint32_t {  // i in [w0, w1)
    if (held) return mine[i - w0];
    if (protect(i)) return 0xffffffffu;
    const int blk = bt[i / kBS];
    if (!known(blk)) {
      report(p.status, kStatusBounds);
      return 0u;
    }
    return rank_key(block_sums(blk)[i % kBS]);
  };
  cluster_wait();  // every CTA's words are zero
  __syncwarp();
  uint32_t thr = 0u;  // the bits found so far
  int above = 0;      // keys whose found bits are greater
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    const int turn = (shift >> 3) & 1;
    int* sum = total[turn ^ 1];
#pragma unroll 4
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      const uint32_t k = i < w1 ? key_at(i) : 0u;
      const bool in = i < w1 && ((k ^ thr) >> shift >> 8) == 0u;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (m == 0u) continue;
      // the first lane counts for all that share its digit: equal and nearly
      // equal sums would queue at one word otherwise
      const int first = __ffs(static_cast<int>(m)) - 1, digit = static_cast<int>((k >> shift) & 255u);
      const int lead = __shfl_sync(0xffffffffu, digit, first);
      const bool same = in && digit == lead;
      const int n = __popc(__ballot_sync(0xffffffffu, same));
      if (in && (!same || lane == first)) atomicAdd(&hist[digit], same ? n : 1);
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      const int v = hist[threadIdx.x];
      hist[threadIdx.x] = 0;
      total[turn][threadIdx.x] = 0;
      if (v != 0)
        for (int r = 0; r < nc; ++r)
          asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(
                           peer_word(sum + threadIdx.x, static_cast<uint32_t>(r))),
                       "r"(v)
                       : "memory");
    }
    cluster_arrive();
    cluster_wait();
    // every warp alike: eight digits a lane, counted from the largest down
    const int4 lo = reinterpret_cast<const int4*>(sum)[2 * lane], hi = reinterpret_cast<const int4*>(sum)[2 * lane + 1];
    const int n[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int own = ((n[0] + n[1]) + (n[2] + n[3])) + ((n[4] + n[5]) + (n[6] + n[7]));
    int from = own;  // of this lane's digits and all greater ones
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_down_sync(0xffffffffu, from, d);
      if (lane + d < 32) from += up;
    }
    const int need = p.keep - above;
    // the lane that holds the digit: the largest that reaches `need`
    const int at = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, from >= need)));
    int past = from - own, digit = 7;
#pragma unroll
    for (int d = 7; d > 0; --d)
      if (digit == d && past + n[d] < need) past += n[d], digit = d - 1;
    int count = n[7];  // keys of that digit
#pragma unroll
    for (int d = 0; d < 7; ++d)
      if (digit == d) count = n[d];
    thr |= static_cast<uint32_t>(8 * at + __shfl_sync(0xffffffffu, digit, at)) << shift;
    above += __shfl_sync(0xffffffffu, past, at);
    if (__shfl_sync(0xffffffffu, count, at) == p.keep - above) {
      // All of them stay (with distinct sums, after three passes mostly): the greater
      // keys are those from thr on.  thr > 0: as many as `keep` keys reach it, of more.
      thr -= 1u;
      above = p.keep;
      break;  // the cluster's warps all alike
    }
  }
  // `above` keys are greater than thr; the first keep - above of those equal to it stay too
  const int need = p.keep - above;
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key_at(i);
    gt += k > thr, eq += k == thr;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) warp_cnt[0][warp] = gt, warp_cnt[1][warp] = eq;
  __syncthreads();
  if (threadIdx.x < 2 * nc) {
    const int c = threadIdx.x & 1;
    int s = 0;
    for (int w = 0; w < kSelWarps; ++w) s += warp_cnt[c][w];
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(
                     peer_word(&cta_cnt[rank][c], static_cast<uint32_t>(threadIdx.x >> 1))),
                 "r"(s)
                 : "memory");
  }
  cluster_arrive();
  cluster_wait();
  int gt0 = 0, eq0 = 0;  // before this warp's range
  if (lane < warp) gt0 = warp_cnt[0][lane], eq0 = warp_cnt[1][lane];
  if (lane < rank) gt0 += cta_cnt[lane][0], eq0 += cta_cnt[lane][1];
  gt0 = __reduce_add_sync(0xffffffffu, gt0);
  eq0 = __reduce_add_sync(0xffffffffu, eq0);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const bool in = i < w1;
    const uint32_t k = in ? key_at(i) : 0u;
    const uint32_t mg = __ballot_sync(0xffffffffu, in && k > thr), me = __ballot_sync(0xffffffffu, in && k == thr);
    const int e_rank = eq0 + __popc(me & below);
    if (in && (k > thr || (k == thr && e_rank < need))) kept[gt0 + __popc(mg & below) + min(e_rank, need)] = i;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  }
}

// kv_evict, second launch: the kept rows and their weights to the other table's
// blocks, and the new lengths: new_lens may be ctx_lens itself, which every cluster of
// the selection reads for itself and nothing here but the thread that writes.  grid (row groups, Hkv, B).  The rows' places come first, one thread a
// row (kept slot -> block -> row: three dependent loads, once), then the rows
// stream through registers, kCopyVecs 16-byte vectors a thread in flight.  64
// sequences x 8 heads, 4096 rows of D = 128 kept: 310 us for 2.15 GB, the measured
// copy rate; the whole call 334 us.
constexpr int kCopyThreads = 256, kCopyVecs = 8, kCopyRows = 128;
template <int CH>  // 16-byte chunks per row
__global__ void __launch_bounds__(kCopyThreads) kv_evict_copy_kernel(const EvictParams p) {
  __shared__ int64_t from[kCopyRows], to[kCopyRows];
  wait_for_launch_ahead();
  const int g = blockIdx.y, b = blockIdx.z;
  const int r0 = blockIdx.x * kCopyRows;
  const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hkv + g) * p.keep + r0;
  if (r0 == 0 && g == 0 && threadIdx.x == 0) {
    const int len = p.ctx_lens[b];
    const int64_t most = min(static_cast<int64_t>(p.max_blocks) * kBS, static_cast<int64_t>(p.keep));
    p.new_lens[b] = static_cast<int>(min(static_cast<int64_t>(len), most));  // an idle sequence's stays negative
  }
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
  p.vec_acc = reinterpret_cast<uintptr_t>(a.acc) % 16 == 0;
  // a CTA per kKeys tokens of the longest possible context, up to a portable cluster
  const int64_t slots = static_cast<int64_t>(a.max_blocks) * kBS;
  int nc = 1;
  while (nc < kMaxCluster && static_cast<int64_t>(nc) * kKeys < slots) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nc), static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(nc);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_select_kernel, p, nc);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.keep + kCopyRows - 1) / kCopyRows),
                  static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  const auto copy = p.ch == 16 ? kv_evict_copy_kernel<16> : kv_evict_copy_kernel<8>;
  return launch_early(copy, grid, kCopyThreads, 0, stream, p);
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
  const dim3 grid(static_cast<unsigned>(a.cache.Hkv), static_cast<unsigned>(a.B));
  return launch_early(kv_tree_accept_kernel, grid, kAcceptThreads, 0, stream, p);
}

}  // namespace attn
