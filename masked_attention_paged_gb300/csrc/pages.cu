// pages.cu -- blocks of a paged cache with owner counts: given back, given out, shared
// by forked sequences, and moved to the front of the pool.
//
// Which blocks are new is decided by one CTA (the lowest free ones, in row order: a
// prefix sum over the rows, and one over the free blocks); the bytes are then moved by
// as many CTAs as fill the GPU.  Deciding is latency: a pool of 16384 blocks is one
// pass of 16 loads a thread.
//
// Measured: 4100 blocks (4.3 GB read and written) moved to the front of a pool of 16384 in 680
// to 695 us, 91 to 93 % of what a copy does.  A step of a search, 64 rows given back, forked anew
// from 16 prompts in eight layers and reserved for, takes 20 us (24 of other contents each time),
// of which the bytes (8.4 MB read, 33.6 written) are 6: four launches and their decisions, each
// a chain of loads by one CTA.  One prompt and four rows take 11 us (13).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kBS = 16;         // tokens per block
constexpr int kThreads = 1024;  // of the deciding CTA
constexpr int kWarps = kThreads / 32;
constexpr int kPerLane = 16;    // counts a lane looks at in a pass
constexpr int kPass = kThreads * kPerLane;
// Bytes a CTA moves in a step: 4100 blocks of 16 x 32 KB take 680 us (8 KB: 707, 32 KB: 902), the
// step of 64 rows above 20.1 (21.3, 28.2).
constexpr int kPiece = 16384;
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = kPiece / 16 / kMoveThreads;

// Sums of v over the threads before this one, and over all of them.
__device__ __forceinline__ int sum_before(int v, int* warp_sum, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  __syncthreads();  // the sums of the call before have been read
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int w = warp_sum[lane];
  static_assert(kWarps == 32, "a lane per warp");
  int at = w;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, at, d);
    if (lane >= d) at += up;
  }
  total = __shfl_sync(0xffffffffu, at, 31);
  return incl - v + __shfl_sync(0xffffffffu, at - w, warp);
}

// One pass over the counts [base, base + kPass): a warp's 512 are consecutive, and
// mask[k] has a bit for each lane's k-th (id = first + 32 k + lane).
struct Pass {
  int first;
  uint32_t mask[kPerLane];
};
template <typename Pick>
__device__ __forceinline__ int look(const int32_t* refs, int n, int base, Pass& s, Pick pick) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  s.first = base + warp * 32 * kPerLane;
  int32_t r[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    const int id = s.first + 32 * k + lane;
    r[k] = id < n ? refs[id] : 0;
  }
  int count = 0;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    const int id = s.first + 32 * k + lane;
    s.mask[k] = __ballot_sync(0xffffffffu, id < n && pick(id, r[k]));
    count += __popc(s.mask[k]);
  }
  return count;  // of the warp
}
// put(rank, id) for the pass's picked ids, the warp's first being number `rank`
template <typename Put>
__device__ __forceinline__ void each(const Pass& s, int rank, Put put) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    if ((s.mask[k] >> lane) & 1u) put(rank + __popc(s.mask[k] & ((1u << lane) - 1u)), s.first + 32 * k + lane);
    rank += __popc(s.mask[k]);
  }
}

// list[0 .. min(want, free)): the lowest free blocks; returns how many.  s, mine: the
// first pass, looked at by look_free before it was known how many are wanted.
__device__ __forceinline__ int look_free(const int32_t* refs, int n, int base, Pass& s) {
  return look(refs, n, base, s, [](int, int32_t r) { return r == 0; });
}
__device__ int lowest_free(const int32_t* refs, int n, int want, int32_t* list, int* warp_sum, Pass& s, int mine) {
  int found = 0;
  for (int base = 0; base < n && found < want; base += kPass) {
    if (base > 0) mine = look_free(refs, n, base, s);
    int total;
    const int before = sum_before((threadIdx.x & 31) == 0 ? mine : 0, warp_sum, total);
    each(s, found + __shfl_sync(0xffffffffu, before, 0), [&](int rank, int id) {
      if (rank < want) list[rank] = id;
    });
    found += total;
  }
  return min(found, want);
}

// ---------------------------------------------------------------------------
// kv_free: a thread per table entry
// ---------------------------------------------------------------------------
struct FreeParams {
  int32_t* refs;
  int num_blocks;
  int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  int32_t* ctx_lens;
  const int32_t* done;
  uint32_t* status;
};
constexpr int kFreeThreads = 256;
__global__ void __launch_bounds__(kFreeThreads) kv_free_kernel(const FreeParams p) {
  let_next_launch_in();
  wait_for_launch_ahead();
  const int b = blockIdx.x;
  if (p.done != nullptr && p.done[b] == 0) return;
  int32_t* row = p.bt + b * p.bt_stride;
  if (blockIdx.y == 0 && threadIdx.x == 0) p.ctx_lens[b] = -1;
  for (int i = blockIdx.y * kFreeThreads + threadIdx.x; i < p.max_blocks; i += gridDim.y * kFreeThreads) {
    const int id = row[i];
    if (id < 0) continue;
    row[i] = -1;
    if (id >= p.num_blocks) {
      report(p.status, kStatusBounds);
      continue;
    }
    if (atomicSub(&p.refs[id], 1) <= 0) {  // nobody's: taken back
      atomicAdd(&p.refs[id], 1);
      report(p.status, kStatusBounds);
    }
  }
}

// ---------------------------------------------------------------------------
// kv_reserve: one CTA, a warp per row
// ---------------------------------------------------------------------------
struct ReserveParams {
  int32_t* refs;
  int num_blocks;
  int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* n_new;
  int rows;
  int32_t* count;  // [rows] workspace
  int32_t* list;   // [num_blocks] workspace
  uint32_t* status;
};
__global__ void __launch_bounds__(kThreads) kv_reserve_kernel(const ReserveParams p) {
  __shared__ int warp_sum[kWarps];
  let_next_launch_in();
  wait_for_launch_ahead();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Pass ahead;
  const int mine = look_free(p.refs, p.num_blocks, 0, ahead);
  // the columns of row b that the new tokens' slots are in
  auto columns = [&](int b, int& end) {
    const int64_t ctx = p.ctx_lens[b], n = p.n_new[b];
    end = 0;
    if (ctx < 0 || n <= 0) return 0;
    const int64_t last = (ctx + n + kBS - 1) / kBS;
    if (last > p.max_blocks) {
      if (lane == 0) report(p.status, kStatusBounds);
      return 0;
    }
    end = static_cast<int>(last);
    return static_cast<int>(ctx / kBS);
  };
  for (int b = warp; b < p.rows; b += kWarps) {
    int end, n = 0;
    for (int i = columns(b, end) + lane; i < end; i += 32) n += p.bt[b * p.bt_stride + i] < 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) p.count[b] = n;
  }
  __syncthreads();
  // the rows before each (past the blocks there are, any number will do)
  int want = 0;
  for (int base = 0; base < p.rows; base += kThreads) {
    const int b = base + threadIdx.x;
    const int n = b < p.rows ? p.count[b] : 0;
    int total;
    const int before = sum_before(min(n, p.num_blocks), warp_sum, total);
    if (b < p.rows) p.count[b] = min(want + before, p.num_blocks);
    want = min(want + total, p.num_blocks);
  }
  const int got = lowest_free(p.refs, p.num_blocks, want, p.list, warp_sum, ahead, mine);
  __syncthreads();
  for (int b = warp; b < p.rows; b += kWarps) {
    int end, rank = p.count[b];
    for (int i = columns(b, end) + lane; i - lane < end; i += 32) {
      int32_t* at = p.bt + b * p.bt_stride + i;
      const bool need = i < end && *at < 0;
      const uint32_t m = __ballot_sync(0xffffffffu, need);
      const int r = rank + __popc(m & ((1u << lane) - 1u));
      rank += __popc(m);
      if (!need) continue;
      if (r < got) {
        *at = p.list[r];
        p.refs[p.list[r]] = 1;
      } else {
        *at = -1;
        report(p.status, kStatusBounds);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// moves of whole blocks, in every tensor of the pool
// ---------------------------------------------------------------------------
template <int CAP>  // room for so many: the arguments of a launch are copied each time
struct PoolTensors {
  int n;
  uint8_t* data[CAP];
  int64_t bytes[CAP];
  int first[CAP + 1];  // pieces of a block in the tensors before
  uint8_t unit[CAP];   // 16, 4 or 1 bytes at a time: what base and block size allow
};

// A piece of a block to move: at most kPiece bytes.
struct Move {
  const uint8_t* src;
  uint8_t* dst;
  int len, unit;  // len 0: none
};
// piece r of block `from` to block `to`
template <int CAP>
__device__ __forceinline__ Move piece_of(const PoolTensors<CAP>& pt, int r, int64_t from, int64_t to) {
  int t = 0;
#pragma unroll
  for (int step = CAP / 2; step > 0; step /= 2)  // the last tensor that begins at or before r
    if (t + step < pt.n && pt.first[t + step] <= r) t += step;
  const int64_t bytes = pt.bytes[t], off = static_cast<int64_t>(r - pt.first[t]) * kPiece;
  Move m;
  m.src = pt.data[t] + from * bytes + off;
  m.dst = pt.data[t] + to * bytes + off;
  m.len = static_cast<int>(min(static_cast<int64_t>(kPiece), bytes - off));
  m.unit = pt.unit[t];
  return m;
}

// Moves get(w) for w = first, first + step, ... below n, the next one's place looked up
// (a chain of loads) while the bytes of this one are on their way.
template <typename Get>
__device__ __forceinline__ void move_all(int64_t first, int64_t n, int64_t step, Get get) {
  if (first >= n) return;
  Move m = get(first);
  for (int64_t w = first; w < n; w += step) {
    Move next;
    next.len = 0;
    if (m.len > 0 && m.unit == 16) {
      uint4 x[kMoveVecs];
      const int vecs = m.len / 16;
#pragma unroll
      for (int u = 0; u < kMoveVecs; ++u) {
        const int i = u * kMoveThreads + threadIdx.x;
        if (i < vecs) x[u] = __ldcs(reinterpret_cast<const uint4*>(m.src) + i);
      }
      if (w + step < n) next = get(w + step);
#pragma unroll
      for (int u = 0; u < kMoveVecs; ++u) {
        const int i = u * kMoveThreads + threadIdx.x;
        if (i < vecs) reinterpret_cast<uint4*>(m.dst)[i] = x[u];
      }
    } else {
      if (m.unit == 4) {
        for (int i = threadIdx.x; i < m.len / 4; i += kMoveThreads)
          reinterpret_cast<uint32_t*>(m.dst)[i] = reinterpret_cast<const uint32_t*>(m.src)[i];
      } else {
        for (int i = threadIdx.x; i < m.len; i += kMoveThreads) m.dst[i] = m.src[i];
      }
      if (w + step < n) next = get(w + step);
    }
    m = next;
  }
}
// w = q * d + r, both below 2^31 mostly
__device__ __forceinline__ int quotient(int64_t w, int d) {
  return w >> 31 == 0 ? static_cast<int>(static_cast<uint32_t>(w) / static_cast<uint32_t>(d)) : static_cast<int>(w / d);
}

// ---------------------------------------------------------------------------
// kv_fork: one CTA gives out the new blocks, then rows and copies
// ---------------------------------------------------------------------------
struct ForkParams {
  int32_t* refs;
  int num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* ctx_lens;
  int batch;
  const int32_t* src;
  int32_t* child;
  int64_t child_stride;
  int child_blocks;
  int32_t* child_lens;
  int children;
  int2* copies;   // [children] workspace: from a block to a new one; .y -1: none needed, -2: an idle child
  int32_t* list;  // [num_blocks] workspace
  uint32_t* status;
};
__global__ void __launch_bounds__(kThreads) kv_fork_plan_kernel(const ForkParams p) {
  __shared__ int warp_sum[kWarps];
  let_next_launch_in();
  wait_for_launch_ahead();
  Pass ahead;
  const int mine = look_free(p.refs, p.num_blocks, 0, ahead);
  // what child j needs: 1 a new block (and which one it copies), 0 none, -1 nothing (idle)
  auto needs = [&](int j, int& from, int& L) {
    const int s = p.src[j];
    from = L = -1;
    if (s < 0) return -1;
    if (s < p.batch) L = p.ctx_lens[s];
    if (s < p.batch && L < 0) return -1;
    const int last = (L - 1) / kBS;  // the block of the last token
    bool bad = s >= p.batch || (L > 0 && (last >= p.max_blocks || last >= p.child_blocks));
    if (!bad && L % kBS != 0) {
      from = p.bt[s * p.bt_stride + last];
      bad = from < 0 || from >= p.num_blocks;
    }
    if (bad) report(p.status, kStatusBounds);
    return bad ? -1 : (L % kBS != 0 ? 1 : 0);
  };
  int want = 0;
  for (int base = 0; base < p.children; base += kThreads) {
    const int j = base + threadIdx.x;
    int from = -1, L = -1;
    const int n = j < p.children ? needs(j, from, L) : -1;
    int total;
    const int before = sum_before(n > 0 ? 1 : 0, warp_sum, total);
    if (j < p.children) {
      p.copies[j] = make_int2(from, n > 0 ? want + before : (n == 0 ? -1 : -2));
      p.child_lens[j] = n < 0 ? -1 : L;
    }
    want += total;
  }
  const int got = lowest_free(p.refs, p.num_blocks, want, p.list, warp_sum, ahead, mine);
  __syncthreads();
  for (int j = threadIdx.x; j < p.children; j += kThreads) {
    const int rank = p.copies[j].y;
    if (rank < 0) continue;
    if (rank < got) {
      const int block = p.list[rank];
      p.refs[block] = 1;
      p.copies[j].y = block;
    } else {  // no block left
      p.copies[j].y = -2;
      p.child_lens[j] = -1;
      report(p.status, kStatusBounds);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kMoveThreads, 8)
    kv_fork_apply_kernel(const __grid_constant__ ForkParams p, const __grid_constant__ PoolTensors<CAP> pt,
                         const int rows) {
  let_next_launch_in();
  wait_for_launch_ahead();
  const int pieces = pt.first[pt.n];
  // `rows` CTAs write the children's rows, the others copy partial blocks
  if (blockIdx.x < rows) {
    for (int j = blockIdx.x; j < p.children; j += rows) {
      const int f = p.copies[j].y;
      const int full = f == -2 ? 0 : p.child_lens[j] / kBS;
      const int32_t* from = p.bt + (f == -2 ? 0 : p.src[j]) * p.bt_stride;
      for (int i = threadIdx.x; i < p.child_blocks; i += kMoveThreads) {
        int id = -1;
        if (i < full) {
          id = from[i];
          if (id < 0 || id >= p.num_blocks) {
            report(p.status, kStatusBounds);
            id = -1;
          } else {
            atomicAdd(&p.refs[id], 1);
          }
        } else if (i == full && f >= 0) {
          id = f;
        }
        p.child[j * p.child_stride + i] = id;
      }
    }
    return;
  }
  move_all(blockIdx.x - rows, static_cast<int64_t>(p.children) * pieces, gridDim.x - rows, [&](int64_t w) {
    const int j = quotient(w, pieces);
    const int2 c = p.copies[j];
    Move m;
    m.len = 0;
    if (c.y >= 0) m = piece_of(pt, static_cast<int>(w - static_cast<int64_t>(j) * pieces), c.x, c.y);
    return m;
  });
}

// ---------------------------------------------------------------------------
// kv_compact: one CTA pairs blocks and holes, then copies and table entries
// ---------------------------------------------------------------------------
struct CompactParams {
  int32_t* refs;
  int num_blocks;
  int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  int batch;
  int32_t* used;
  // workspace: how many move; number r goes from from[r] to to[r]; rank[id] = r
  int32_t* moves;
  int32_t* from;
  int32_t* to;
  int32_t* rank;
  uint32_t* status;
};
__global__ void __launch_bounds__(kThreads) kv_compact_plan_kernel(const CompactParams p) {
  __shared__ int warp_sum[kWarps];
  let_next_launch_in();
  wait_for_launch_ahead();
  const int n = p.num_blocks;
  const bool lead = (threadIdx.x & 31) == 0;
  int used = 0;
  Pass s;  // (a pool of one pass is looked at once)
  for (int base = 0; base < n; base += kPass) {
    const int mine = look(p.refs, n, base, s, [](int, int32_t r) { return r != 0; });
    int total;
    sum_before(lead ? mine : 0, warp_sum, total);
    used += total;
  }
  int holes = 0, moves = 0;
  for (int base = 0; base < n; base += kPass) {
    if (n > kPass) look(p.refs, n, base, s, [](int, int32_t r) { return r != 0; });
    Pass hole = s, move = s;  // free below `used`, in use from there on
    int count[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int below = min(max(used - (s.first + 32 * k), 0), 32);  // ids of the mask that are
      const uint32_t m = below == 32 ? ~0u : (1u << below) - 1u;
      hole.mask[k] = ~s.mask[k] & m;
      move.mask[k] = s.mask[k] & ~m;
      count[0] += __popc(hole.mask[k]);
      count[1] += __popc(move.mask[k]);
    }
    int total;  // both counts in one sum: at most 2^14 each
    const int before = sum_before(lead ? count[0] | count[1] << 16 : 0, warp_sum, total);
    const int mine = __shfl_sync(0xffffffffu, before, 0);
    each(hole, holes + (mine & 0xffff), [&](int r, int id) { p.to[r] = id; });
    each(move, moves + (mine >> 16), [&](int r, int id) {
      p.from[r] = id;
      p.rank[id] = r;
    });
    holes += total & 0xffff;
    moves += total >> 16;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < moves; r += kThreads) {
    const int a = p.from[r], b = p.to[r];
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    p.used[0] = used;
    p.moves[0] = moves;
  }
}

template <int CAP>
__global__ void __launch_bounds__(kMoveThreads, 8)
    kv_compact_apply_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ PoolTensors<CAP> pt,
                            const int rows) {
  let_next_launch_in();
  wait_for_launch_ahead();
  const int pieces = pt.first[pt.n];
  const int moves = p.moves[0];
  if (blockIdx.x < rows) {
    const int used = p.used[0];
    for (int b = blockIdx.x; b < p.batch; b += rows) {
      int32_t* row = p.bt + b * p.bt_stride;
      for (int i = threadIdx.x; i < p.max_blocks; i += kMoveThreads) {
        const int id = row[i];
        if (id < used) continue;  // stays, or no block
        const int r = id < p.num_blocks ? p.rank[id] : -1;
        // ranks of blocks that did not move are whatever the workspace held
        if (r >= 0 && r < moves && p.from[r] == id)
          row[i] = p.to[r];
        else
          report(p.status, kStatusBounds);
      }
    }
    return;
  }
  move_all(blockIdx.x - rows, static_cast<int64_t>(moves) * pieces, gridDim.x - rows, [&](int64_t w) {
    const int r = quotient(w, pieces);
    return piece_of(pt, static_cast<int>(w - static_cast<int64_t>(r) * pieces), p.from[r], p.to[r]);
  });
}

// the tensors' pieces; false if a block has more than 31 bits of them
template <int CAP>
bool lay_out(const PoolArgs& a, PoolTensors<CAP>& pt) {
  pt.n = a.n_tensors;
  int64_t at = 0;
  for (int t = 0; t < a.n_tensors; ++t) {
    pt.data[t] = static_cast<uint8_t*>(a.tensors[t].data);
    pt.bytes[t] = a.tensors[t].block_bytes;
    pt.first[t] = static_cast<int>(at);
    const uint64_t both = reinterpret_cast<uintptr_t>(pt.data[t]) | static_cast<uint64_t>(pt.bytes[t]);
    pt.unit[t] = both % 16 == 0 ? 16 : (both % 4 == 0 ? 4 : 1);
    at += (pt.bytes[t] + kPiece - 1) / kPiece;
    if (at > 0x7fffffff) return false;
  }
  pt.first[a.n_tensors] = static_cast<int>(at);
  return true;
}

// CTAs that move pieces: eight an SM at most, as many as there is work for
int move_ctas(int64_t items) {
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(items, 1), 8 * device_sm_count()));
}

template <int CAP>
cudaError_t fork(const PoolArgs& a, const ForkParams& p, cudaStream_t stream) {
  PoolTensors<CAP> pt;
  if (!lay_out(a, pt)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_early(kv_fork_plan_kernel, dim3(1), kThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  const int rows = std::min(p.children, device_sm_count());
  const int ctas = rows + move_ctas(static_cast<int64_t>(p.children) * pt.first[pt.n]);
  return launch_early(kv_fork_apply_kernel<CAP>, dim3(static_cast<unsigned>(ctas)), kMoveThreads, 0, stream, p, pt,
                      rows);
}

template <int CAP>
cudaError_t compact(const PoolArgs& a, const CompactParams& p, cudaStream_t stream) {
  PoolTensors<CAP> pt;
  if (!lay_out(a, pt)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_early(kv_compact_plan_kernel, dim3(1), kThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  const int rows = std::max(1, std::min(a.batch, device_sm_count()));
  const int ctas = rows + move_ctas(a.num_blocks / 2 * pt.first[pt.n]);  // at most half of the blocks move
  return launch_early(kv_compact_apply_kernel<CAP>, dim3(static_cast<unsigned>(ctas)), kMoveThreads, 0, stream, p, pt,
                      rows);
}

}  // namespace

// kv_reserve: a number a row and a list of blocks; kv_fork: two numbers; kv_compact: three lists
size_t pool_workspace_bytes(int64_t num_blocks, int64_t rows) {
  return ((3 * static_cast<size_t>(num_blocks) + 2 * rows + 64) * 4 + 255) & ~size_t(255);
}

cudaError_t launch_kv_free(const PoolArgs& a, const int32_t* done, cudaStream_t stream) {
  FreeParams p;
  p.refs = a.refs;
  p.num_blocks = static_cast<int>(a.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctx_lens = a.ctx_lens;
  p.done = done;
  p.status = a.status;
  const dim3 grid(static_cast<unsigned>(a.batch),
                  static_cast<unsigned>(std::min(64, (a.max_blocks + kFreeThreads - 1) / kFreeThreads)));
  return launch_early(kv_free_kernel, grid, kFreeThreads, 0, stream, p);
}

cudaError_t launch_kv_reserve(const PoolArgs& a, const int32_t* n_new, cudaStream_t stream) {
  ReserveParams p;
  p.refs = a.refs;
  p.num_blocks = static_cast<int>(a.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctx_lens = a.ctx_lens;
  p.n_new = n_new;
  p.rows = a.batch;
  p.list = static_cast<int32_t*>(a.scratch);
  p.count = p.list + a.num_blocks;
  p.status = a.status;
  return launch_early(kv_reserve_kernel, dim3(1), kThreads, 0, stream, p);
}

cudaError_t launch_kv_fork(const PoolArgs& a, const int32_t* src, int32_t* child_table, int64_t child_stride,
                           int child_blocks, int32_t* child_lens, int children, cudaStream_t stream) {
  ForkParams p;
  p.refs = a.refs;
  p.num_blocks = static_cast<int>(a.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ctx_lens = a.ctx_lens;
  p.batch = a.batch;
  p.src = src;
  p.child = child_table;
  p.child_stride = child_stride;
  p.child_blocks = child_blocks;
  p.child_lens = child_lens;
  p.children = children;
  p.copies = static_cast<int2*>(a.scratch);
  p.list = reinterpret_cast<int32_t*>(p.copies + children);
  p.status = a.status;
  // (a launch copies its arguments: room for 256 tensors is 0.3 us more of a small step's 11)
  return a.n_tensors <= 64 ? fork<64>(a, p, stream) : fork<kPoolMaxTensors>(a, p, stream);
}

cudaError_t launch_kv_compact(const PoolArgs& a, int32_t* used, cudaStream_t stream) {
  CompactParams p;
  p.refs = a.refs;
  p.num_blocks = static_cast<int>(a.num_blocks);
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.batch = a.batch;
  p.used = used;
  p.moves = static_cast<int32_t*>(a.scratch);
  p.from = p.moves + 64;
  p.to = p.from + a.num_blocks;
  p.rank = p.to + a.num_blocks;
  p.status = a.status;
  return a.n_tensors <= 64 ? compact<64>(a, p, stream) : compact<kPoolMaxTensors>(a, p, stream);
}

}  // namespace attn
