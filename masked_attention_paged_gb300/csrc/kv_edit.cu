// kv_edit.cu -- moves of whole K/V rows inside a paged cache.
//   kv_tree_accept   the accepted drafts' rows move up behind the context
// Bit copies in 16-byte vectors; the work is the rows' bytes.
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

}  // namespace

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
