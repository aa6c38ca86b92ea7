// verify.cu -- which drafts of a tree the target model keeps, and the token after
// them (draft_verify).
//
// A refusal turns the target's row p into max(r - (S / Q) q, 0), again and again for
// further siblings.  Since max(max(a, 0) - c, 0) = max(a - c, 0) for c >= 0, that is
// max(p - C q, 0) with one growing scalar C: nothing is stored per token, and each
// refusal that a sibling follows costs one sum over the row.
//
// One cluster per sequence.  Its CTAs go down the tree alike (a draft's test takes two
// numbers, gathered for all drafts at once), and share every sum over the vocabulary,
// a consecutive range each, a consecutive part of it per warp.  The next token is found
// in the CTA, the warp and the lane whose range the drawn number falls into.
//
// Tests and sums decide between whole numbers, so they carry twice a float's digits:
// p - C q as an unevaluated sum of two floats (the products' and differences' errors
// are exact by FMA), summed the same way, and in double above a lane.  Doubles
// throughout would bound the kernel: the SM does two a cycle, and a row of 131072
// needs five for each entry.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;    // of a cluster
constexpr int kMaxDrafts = kVerifyMaxDrafts;
constexpr int kUnroll = 8;

struct VerifyParams {
  const void* p;
  const void* q;  // or null
  int64_t ps0, ps1, qs0, qs1;
  const int32_t* tokens;
  int64_t tok_stride;
  const int32_t* parents;
  int64_t par_stride;
  const float* uniforms;
  int64_t uni_stride;
  int T, V;
  int replacement;
  int32_t* path;
  int32_t* n_accept;
  int32_t* next;
  uint32_t* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// every thread of every CTA of the cluster
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <bool BF16>
__device__ __forceinline__ float load(const void* row, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << 16);
  else
    return static_cast<const float*>(row)[i];
}
template <bool BF16>
__device__ __forceinline__ const void* row_at(const void* base, int64_t off) {
  return static_cast<const uint8_t*>(base) + off * (BF16 ? 2 : 4);
}

// hi + lo += x + y, |y| far below |x| (the error of hi + x is exact)
__device__ __forceinline__ void add_pair(float& hi, float& lo, float x, float y) {
  const float s = hi + x, b = s - hi;
  lo += ((hi - (s - b)) + (x - b)) + y;
  hi = s;
}

// What the walk asks of the whole cluster.
struct Ask {
  int node;
  double c;    // sum of max(p - c q, 0) over node's row, without its refused tokens if the drafts are certain
  int sum;     // a sum is needed (else: the last one serves)
  int done;    // the walk is over
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const VerifyParams p, const int nc) {
  __shared__ float px[kMaxDrafts], qx[kMaxDrafts], uni[kMaxDrafts];
  __shared__ int par[kMaxDrafts], tok[kMaxDrafts];
  __shared__ uint8_t refused[kMaxDrafts];  // of the node where the sequence stands
  __shared__ double warp_sum[kWarps], cta_sum[2][kMaxCtas];
  __shared__ Ask ask;
  let_next_launch_in();
  wait_for_launch_ahead();
  const int b = blockIdx.y, rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.T, V = p.V;
  const bool certain = p.q == nullptr;
  for (int t = threadIdx.x; t < T; t += kThreads) {
    int up = p.parents[b * p.par_stride + t];
    const int x = t > 0 ? p.tokens[b * p.tok_stride + t] : 0;
    bool bad = up >= t;
    if (!bad && up >= 0 && (x < 0 || x >= V)) bad = true;
    if (bad) {
      if (rank == 0) report(p.status, kStatusBounds);
      up = -2;
    }
    par[t] = up;
    tok[t] = x;
    uni[t] = p.uniforms[b * p.uni_stride + t];
    refused[t] = 0;
    if (up >= 0) {
      px[t] = fmaxf(load<BF16>(p.p, b * p.ps0 + up * p.ps1 + x), 0.f);  // 0 for a NaN
      qx[t] = certain ? 1.0f : fmaxf(load<BF16>(p.q, b * p.qs0 + up * p.qs1 + x), 0.f);
    }
  }
  __syncthreads();
  int32_t* path = p.path + static_cast<int64_t>(b) * T;
  if (par[0] != -1) {  // idle (the whole cluster alike)
    if (rank == 0) {
      for (int t = threadIdx.x; t < T; t += kThreads) path[t] = -1;
      if (threadIdx.x == 0) {
        p.n_accept[b] = 0;
        p.next[b] = -1;
      }
    }
    return;
  }

  // this warp's part of a row: [w0, w1)
  const int per = (((V + nc * kWarps - 1) / (nc * kWarps)) + 31) / 32 * 32;
  const int w0 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(rank * kWarps + warp) * per));
  const int w1 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(w0) + per));
  int turn = 0;
  // the sum that `ask` asks for, alike in every thread of the cluster; warp_sum and
  // cta_sum[turn] hold its parts afterwards
  auto row_sum = [&](int node, double c, bool without) -> double {
    const void* pr = row_at<BF16>(p.p, b * p.ps0 + node * p.ps1);
    float hi = 0.f, lo = 0.f;
    if (c == 0.0) {
      for (int v0 = w0 + lane; v0 < w1; v0 += 32 * kUnroll) {
        float x[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) x[k] = v0 + 32 * k < w1 ? load<BF16>(pr, v0 + 32 * k) : 0.f;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) add_pair(hi, lo, x[k] > 0.f ? x[k] : 0.f, 0.f);
      }
    } else {
      const void* qr = row_at<BF16>(p.q, b * p.qs0 + node * p.qs1);
      const float ch = static_cast<float>(c), cl = static_cast<float>(c - ch);
      for (int v0 = w0 + lane; v0 < w1; v0 += 32 * kUnroll) {
        float x[kUnroll], y[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const bool in = v0 + 32 * k < w1;
          x[k] = in ? load<BF16>(pr, v0 + 32 * k) : 0.f;
          y[k] = in ? fmaxf(load<BF16>(qr, v0 + 32 * k), 0.f) : 0.f;  // 0 for a NaN
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const float t = __fmul_rn(ch, y[k]), d = x[k] - t;
            // errors of the product and, where d > 0, of the difference
          const float e = ((x[k] - d) - t) - fmaf(cl, y[k], fmaf(ch, y[k], -t));
          const bool on = d + e > 0.f;
          add_pair(hi, lo, on ? d : 0.f, on ? e : 0.f);
        }
      }
    }
    double s = static_cast<double>(hi) + static_cast<double>(lo);
    if (without) {  // the refused tokens of this warp's part (each once)
      for (int t = node + 1 + lane; t < T; t += 32)
        if (refused[t] && tok[t] >= w0 && tok[t] < w1 && px[t] > 0.f) s -= px[t];
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) warp_sum[warp] = fmax(s, 0.0);
    __syncthreads();
    turn ^= 1;
    if (threadIdx.x < nc) {
      double all = 0.0;
      for (int w = 0; w < kWarps; ++w) all += warp_sum[w];
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(at)
                   : "r"(smem_u32(&cta_sum[turn][rank])), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(all) : "memory");
    }
    cluster_sync();
    double all = 0.0;
    for (int r = 0; r < nc; ++r) all += cta_sum[turn][r];
    return all;
  };

  // ---- the walk, in warp 0 of every CTA alike
  int node = 0, n = 1, t = 0;
  double c = 0.0, mass = 1.0, left = 1.0;
  bool known = true;   // mass is this row's at c
  bool summed = false; // the parts of the last sum are this node's at c
  for (;;) {
    if (warp == 0) {
      bool need = false;
      for (;;) {
        // the next child of `node` after t
        int found = -1;
        for (int base = (t + 1) & ~31; base < T; base += 32) {
          const int i = base + lane;
          const uint32_t m = __ballot_sync(0xffffffffu, i > t && i < T && par[i] == node);
          if (m != 0u) {
            found = base + __ffs(static_cast<int>(m)) - 1;
            break;
          }
        }
        if (found < 0) break;
        const int x = tok[found];
        if (certain || !p.replacement) {  // a token that was refused here is not tested again
          bool seen = false;
          for (int i = node + 1 + lane; i < found; i += 32) seen |= refused[i] && tok[i] == x;
          if (__any_sync(0xffffffffu, seen) || left <= 0.0) {
            t = found;
            continue;
          }
        }
        if (!known) {
          need = true;
          break;
        }
        const double u = uni[found], pv = px[found], qv = qx[found];
        bool yes;
        if (certain) {
          yes = u * mass < pv;
        } else {
          const double r = pv - c * qv;
          yes = u * qv * mass < (r > 0.0 ? r : 0.0) * left;
        }
        t = found;
        if (yes) {
          // (refused drafts of the node that is left are none of the new one's)
          for (int i = node + 1 + lane; i < T; i += 32) refused[i] = 0;
          __syncwarp();
          node = found;
          if (rank == 0 && lane == 0) path[n] = node;
          ++n;
          c = 0.0, mass = 1.0, left = 1.0;
          known = true, summed = false;
        } else {
          if (certain) {
            mass -= pv;
          } else {
            c += mass / left;
            if (!p.replacement) left -= qv;
            known = false;
          }
          if (lane == 0) refused[found] = 1;
          __syncwarp();
          summed = false;
        }
      }
      if (lane == 0) {
        ask.node = node;
        ask.c = c;
        ask.sum = !summed;
        ask.done = !need;
      }
    }
    __syncthreads();
    const Ask a = ask;
    if (a.sum) {
      const double s = row_sum(a.node, a.c, certain);
      if (!certain) mass = s;
      known = summed = true;
    }
    if (a.done) break;
    __syncthreads();  // ask has been read
  }
  // (only warp 0 kept n; every warp has the last ask)
  const int last = ask.node;
  double cc = ask.c;
  bool without = certain;
  double total = 0.0;
  for (int r = 0; r < nc; ++r) total += cta_sum[turn][r];
  if (!(total > 0.0) && (cc != 0.0 || without)) {  // nothing is left: from p itself
    cc = 0.0;
    without = false;
    total = row_sum(last, 0.0, false);
  }
  if (rank == 0) {
    if (warp == 0) {
      if (lane == 0) {
        path[0] = 0;
        p.n_accept[b] = n;
        if (!(total > 0.0)) {
          p.next[b] = -1;
          report(p.status, kStatusBounds);
        }
      }
      for (int i = n + lane; i < T; i += 32) path[i] = -1;
    }
  }
  if (!(total > 0.0)) return;

  // ---- the next token: which CTA, which warp, which lane
  const double goal = static_cast<double>(uni[0]) * total;
  double before = 0.0;
  int owner = -1, last_on = 0;
  double at_owner = 0.0, at_last = 0.0;
  for (int r = 0; r < nc; ++r) {
    const double s = cta_sum[turn][r];
    if (s > 0.0) last_on = r, at_last = before;
    if (owner < 0 && before + s > goal) owner = r, at_owner = before;
    before += s;
  }
  if (owner < 0) owner = last_on, at_owner = at_last;
  if (owner != rank) return;
  before = at_owner;
  int who = -1, last_warp = 0;
  for (int w = 0; w < kWarps; ++w) {
    const double s = warp_sum[w];
    if (s > 0.0) last_warp = w, at_last = before;
    if (who < 0 && before + s > goal) who = w, at_owner = before;
    before += s;
  }
  if (who < 0) who = last_warp, at_owner = at_last;
  if (who != warp) return;
  before = at_owner;
  const void* pr = row_at<BF16>(p.p, b * p.ps0 + last * p.ps1);
  const void* qr = cc != 0.0 ? row_at<BF16>(p.q, b * p.qs0 + last * p.qs1) : nullptr;
  auto weight = [&](int v) -> double {
    double w = load<BF16>(pr, v);
    if (qr != nullptr) w -= cc * static_cast<double>(fmaxf(load<BF16>(qr, v), 0.f));
    if (without)
      for (int i = last + 1; i < T; ++i)
        if (refused[i] && tok[i] == v) w = 0.0;
    return w > 0.0 ? w : 0.0;
  };
  const int each = (w1 - w0 + 31) / 32;
  const int v0 = min(w1, w0 + lane * each), v1 = min(w1, v0 + each);
  double mine = 0.0;
  for (int v = v0; v < v1; ++v) mine += weight(v);
  double incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const double up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, before + incl > goal);
  const uint32_t on = __ballot_sync(0xffffffffu, mine > 0.0);
  if (on == 0u) return;  // (a warp with a positive sum has a positive weight)
  const int pick = past != 0u ? __ffs(static_cast<int>(past)) - 1 : 31 - __clz(static_cast<int>(on));
  if (lane != pick) return;
  double sum = before + (incl - mine);
  int token = -1;
  for (int v = v0; v < v1; ++v) {
    const double w = weight(v);
    if (w > 0.0) token = v;
    sum += w;
    if (sum > goal) break;
  }
  p.next[b] = token;
}

template <bool BF16>
cudaError_t launch(const VerifyArgs& a, const VerifyParams& p, cudaStream_t stream) {
  auto kern = draft_verify_kernel<BF16>;
  // CTAs a sequence: as many as fill the GPU once, and no fewer than 1024 entries each
  int nc = 1;
  while (nc < kMaxCtas && 2 * nc * a.B <= 4 * device_sm_count() && static_cast<int64_t>(nc) * 2048 <= a.V) nc *= 2;
  if (nc > 8) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nc), static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(kThreads);
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
  return cudaLaunchKernelEx(&cfg, kern, p, nc);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t stream) {
  VerifyParams p;
  p.p = a.p.data;
  p.q = a.q.data;
  p.ps0 = a.p.stride[0];
  p.ps1 = a.p.stride[1];
  p.qs0 = a.q.stride[0];
  p.qs1 = a.q.stride[1];
  p.tokens = a.tokens;
  p.tok_stride = a.tok_stride;
  p.parents = a.parents;
  p.par_stride = a.par_stride;
  p.uniforms = a.uniforms;
  p.uni_stride = a.uni_stride;
  p.T = static_cast<int>(a.T);
  p.V = static_cast<int>(a.V);
  p.replacement = a.replacement;
  p.path = a.path;
  p.n_accept = a.n_accept;
  p.next = a.next;
  p.status = a.status;
  return a.p.dtype == ATTN_BF16 ? launch<true>(a, p, stream) : launch<false>(a, p, stream);
}

}  // namespace attn
