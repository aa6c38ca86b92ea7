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
// are exact by FMA), and sums and products of such pairs.  Doubles would bound the
// kernel: the SM does two a cycle, and a chain of them (a test, a quotient) took the
// walk 2 us at each refusal.
//
// What bounds it is latency, in the sequence with the most refusals: 64 x 25 drafts over
// 131072 tokens take 43 us, four row sums one after the other and the draw in the longest,
// where the bytes of all 100 sums are 15 us of HBM (116 us with doubles and CTAs of 512
// threads).  A lane asks for single entries, eight at a time, so once the other sequences are
// done an SM has 16 KB on its way (8 KB of two-byte entries), and HBM is 15 % busy.  16 x 27
// over 100003 tokens 21.5 us; 1 x 5 over 32000 6.6: a launch, two loads that depend on each
// other, and the draw.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;    // of a cluster
constexpr int kMaxDrafts = kVerifyMaxDrafts;
constexpr int kUnroll = 8;  // entries of a row that a lane has in flight

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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

// A number as an unevaluated sum of two floats, |y| far below |x|.
using Pair = float2;
// acc += x + y (the error of the first sum is exact)
__device__ __forceinline__ void add_to(Pair& acc, float x, float y) {
  const float s = acc.x + x, b = s - acc.x;
  acc.y += ((acc.x - (s - b)) + (x - b)) + y;
  acc.x = s;
}
__device__ __forceinline__ Pair tidy(Pair a) {
  const float s = a.x + a.y;
  return make_float2(s, a.y - (s - a.x));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  add_to(a, b.x, b.y);
  return tidy(a);
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int m) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, m), __shfl_xor_sync(0xffffffffu, a.y, m));
}
__device__ __forceinline__ Pair shfl_up(Pair a, int d) {
  return make_float2(__shfl_up_sync(0xffffffffu, a.x, d), __shfl_up_sync(0xffffffffu, a.y, d));
}
__device__ __forceinline__ Pair shfl(Pair a, int l) {
  return make_float2(__shfl_sync(0xffffffffu, a.x, l), __shfl_sync(0xffffffffu, a.y, l));
}
__device__ __forceinline__ bool greater(Pair a, Pair b) { return (a.x - b.x) + (a.y - b.y) > 0.f; }
__device__ __forceinline__ Pair of(float x) { return make_float2(x, 0.f); }
__device__ __forceinline__ Pair negative(Pair a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ Pair times(Pair a, Pair b) {
  const float h = __fmul_rn(a.x, b.x);
  return tidy(make_float2(h, fmaf(a.x, b.x, -h) + fmaf(a.x, b.y, a.y * b.x)));
}
__device__ __forceinline__ Pair over(Pair a, Pair b) {  // the quotient, and that of what it leaves
  const float h = __fdividef(a.x, b.x);
  const Pair rest = add(a, negative(times(b, of(h))));
  const float l = __fdividef(rest.x, b.x);
  const Pair rest2 = add(rest, negative(times(b, of(l))));
  Pair q = tidy(make_float2(h, l));
  q.y += __fdividef(rest2.x, b.x);
  return tidy(q);
}
// sums over the lanes up to this one
__device__ __forceinline__ Pair scan(Pair a, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Pair up = shfl_up(a, d);
    if (lane >= d) a = add(a, up);
  }
  return a;
}
// The lane in whose part of [before, ...) `goal` falls, `mine` being each lane's part: the first
// whose end is past it, else (by rounding) the last with a part at all.  before: that
// lane's start.
__device__ __forceinline__ int pick(Pair mine, Pair goal, Pair& before, int lane) {
  const Pair upto = add(before, scan(mine, lane));
  const uint32_t past = __ballot_sync(0xffffffffu, greater(upto, goal));
  const uint32_t on = __ballot_sync(0xffffffffu, mine.x > 0.f);
  const uint32_t among = past & on;
  const int l = among != 0u ? __ffs(static_cast<int>(among)) - 1 : (on != 0u ? 31 - __clz(static_cast<int>(on)) : 0);
  const Pair ahead = shfl_up(upto, 1);
  const Pair start = lane == 0 ? before : ahead;
  before = shfl(start, l);
  return l;
}
// p - c q > 0 as a pair (0 if not), c = ch + cl
__device__ __forceinline__ Pair residual(float x, float y, float ch, float cl) {
  const float t = __fmul_rn(ch, y), d = x - t;
  // errors of the product and, where d > 0, of the difference
  const float e = ((x - d) - t) - fmaf(cl, y, fmaf(ch, y, -t));
  return d + e > 0.f ? make_float2(d, e) : make_float2(0.f, 0.f);
}

// What the walk asks of the whole cluster.
struct Ask {
  int node;
  Pair c;      // sum of max(p - c q, 0) over node's row, without its refused tokens if the drafts are certain
  int sum;     // a sum is needed (else: the last one serves)
  int done;    // the walk is over
};

template <bool BF16>
// Four CTAs an SM: 64 sequences are 512.
__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(const VerifyParams p, const int nc) {
  __shared__ float px[kMaxDrafts], qx[kMaxDrafts], uni[kMaxDrafts];
  __shared__ int par[kMaxDrafts], tok[kMaxDrafts];
  __shared__ uint8_t refused[kMaxDrafts];  // of the node where the sequence stands
  __shared__ uint8_t first[kMaxDrafts];    // taken, if it is the first to be tested at its node: u q < p
  __shared__ Pair warp_sum[kWarps], cta_sum[2][kMaxCtas], found_start, found_goal;
  __shared__ Ask ask;
  __shared__ int found;     // the warp whose part the next token is in; -1: not this CTA's
  __shared__ bool remains;  // the last row's sum is positive (not in `found`, which warp 0 sets while others read this)
  let_next_launch_in();
  // The first sum stores into the other CTAs' shared memory, which they must have begun to
  // run for: the barrier's other half is there, behind the loads and the walk (1 x 5: 6.6 us; 7.0
  // with this half behind the loads).
  cluster_arrive();
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
      first[t] = fmaf(-uni[t], qx[t], px[t]) > 0.f;  // the sign is exact: one rounding
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
    cluster_wait();
    return;
  }
  bool started = false;  // alike in the whole cluster

  // this warp's part of a row: [w0, w1)
  const int per = (((V + nc * kWarps - 1) / (nc * kWarps)) + 31) / 32 * 32;
  const int w0 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(rank * kWarps + warp) * per));
  const int w1 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(w0) + per));
  int turn = 0;
  // the sum that `ask` asks for, in warp 0 of every CTA alike; warp_sum and
  // cta_sum[turn] hold its parts afterwards
  auto row_sum = [&](int node, Pair c, bool without) -> Pair {
    const void* pr = row_at<BF16>(p.p, b * p.ps0 + node * p.ps1);
    Pair acc = make_float2(0.f, 0.f);
    if (c.x == 0.f) {
      for (int v0 = w0 + lane; v0 < w1; v0 += 32 * kUnroll) {
        float x[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) x[k] = v0 + 32 * k < w1 ? load<BF16>(pr, v0 + 32 * k) : 0.f;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) add_to(acc, fmaxf(x[k], 0.f), 0.f);
      }
    } else {
      const void* qr = row_at<BF16>(p.q, b * p.qs0 + node * p.qs1);
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
          const Pair r = residual(x[k], y[k], c.x, c.y);
          add_to(acc, r.x, r.y);
        }
      }
    }
    if (without) {  // the refused tokens of this warp's part (each once)
      for (int t = node + 1 + lane; t < T; t += 32)
        if (refused[t] && tok[t] >= w0 && tok[t] < w1) add_to(acc, -px[t], 0.f);
    }
    acc = tidy(acc);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) acc = add(acc, shfl_xor(acc, m));
    if (lane == 0) warp_sum[warp] = acc.x > 0.f ? acc : make_float2(0.f, 0.f);
    if (!started) cluster_wait();  // every CTA has begun
    started = true;
    __syncthreads();
    turn ^= 1;
    const auto all_lanes = [&](Pair s) {  // of the first 16 lanes, the others hold 0
#pragma unroll
      for (int m = 8; m >= 1; m >>= 1) s = add(s, shfl_xor(s, m));
      return s;
    };
    const Pair none = make_float2(0.f, 0.f);
    if (warp == 0) {
      const Pair s = all_lanes(lane % 16 < kWarps ? warp_sum[lane % kWarps] : none);
      if (lane < nc) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at)
                     : "r"(smem_u32(&cta_sum[turn][rank])), "r"(lane));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(s.x), "f"(s.y) : "memory");
      }
    }
    cluster_arrive();
    cluster_wait();
    if (warp != 0) return none;
    return shfl(all_lanes(lane % 16 < nc ? cta_sum[turn][lane % 16] : none), 0);
  };
  static_assert(kWarps <= 16 && kMaxCtas == 16, "a lane per part");

  // ---- the walk, in warp 0 of every CTA alike
  int node = 0, n = 1, t = 0;
  // (p and q enter the tests times 2^60: products of small numbers stay normal)
  constexpr float kUp = 1152921504606846976.f;
  const Pair zero = of(0.f), one = of(1.f);
  Pair c = zero, mass = one, left = one, total = zero;
  bool known = true;   // mass is this row's at c
  bool fresh = true;   // nothing has been refused at the node
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
        if (!fresh && (certain || !p.replacement)) {  // a token that was refused here is not tested again
          bool seen = false;
          for (int i = node + 1 + lane; i < found; i += 32) seen |= refused[i] && tok[i] == x;
          if (__any_sync(0xffffffffu, seen) || !(left.x > 0.f)) {
            t = found;
            continue;
          }
        }
        if (!known) {
          need = true;
          break;
        }
        bool yes;
        if (fresh) {
          yes = first[found];
        } else if (certain) {
          yes = greater(of(px[found]), times(of(uni[found]), mass));
        } else {
          const float qv = qx[found] * kUp;
          const Pair r = tidy(residual(px[found] * kUp, qv, c.x, c.y));
          yes = greater(times(r, left), times(times(of(uni[found]), of(qv)), mass));
        }
        t = found;
        if (yes) {
          if (!fresh) {  // (refused drafts of the node that is left are none of the new one's)
            for (int i = node + 1 + lane; i < T; i += 32) refused[i] = 0;
            __syncwarp();
          }
          node = found;
          if (rank == 0 && lane == 0) path[n] = node;
          ++n;
          c = zero, mass = left = one;
          known = fresh = true;
          summed = false;
        } else {
          if (certain) {
            mass = add(mass, of(-px[found]));
          } else {
            c = fresh ? one : add(c, p.replacement ? mass : over(mass, left));
            if (!p.replacement) left = add(left, of(-qx[found]));
            known = false;
          }
          fresh = false;
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
      total = row_sum(a.node, a.c, certain);
      if (!certain) mass = total;
      known = summed = true;
    }
    if (a.done) break;
    __syncthreads();  // ask has been read
  }
  const int last = ask.node;
  // nothing is left of a row that something was taken from: the token comes from p itself
  bool whole = ask.c.x == 0.f && !certain;
  if (warp == 0 && lane == 0) remains = total.x > 0.f;
  __syncthreads();
  if (!remains && !whole) {  // (the cluster's CTAs alike)
    whole = true;
    total = row_sum(last, zero, false);
  }
  if (warp == 0) {
    if (rank == 0) {
      if (lane == 0) {
        path[0] = 0;
        p.n_accept[b] = n;
        if (!(total.x > 0.f)) {
          p.next[b] = -1;
          report(p.status, kStatusBounds);
        }
      }
      for (int i = n + lane; i < T; i += 32) path[i] = -1;
    }
    // ---- the next token: which CTA, which warp's part
    int who = -1;
    if (total.x > 0.f) {
      const Pair goal = times(of(uni[0]), total), none = make_float2(0.f, 0.f);
      Pair before = none;
      if (pick(lane < nc ? cta_sum[turn][lane] : none, goal, before, lane) == rank)
        who = pick(lane < kWarps ? warp_sum[lane] : none, goal, before, lane);
      found_start = before;
      found_goal = goal;
    }
    if (lane == 0) found = who;
  }
  __syncthreads();
  if (found < 0) return;
  // ---- in it: all warps take a piece of that part, then one warp the piece's entries
  const void* pr = row_at<BF16>(p.p, b * p.ps0 + last * p.ps1);
  const void* qr = row_at<BF16>(p.q, b * p.qs0 + last * p.qs1);
  const Pair cp = whole ? zero : ask.c;
  auto weight = [&](int v) -> Pair {
    const float x = load<BF16>(pr, v);
    if (!whole && certain) {
      for (int i = last + 1; i < T; ++i)
        if (refused[i] && tok[i] == v) return make_float2(0.f, 0.f);
    }
    if (cp.x == 0.f) return make_float2(fmaxf(x, 0.f), 0.f);
    return tidy(residual(x, fmaxf(load<BF16>(qr, v), 0.f), cp.x, cp.y));
  };
  const int part0 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(rank * kWarps + found) * per));
  const int part1 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(part0) + per));
  const int piece = ((part1 - part0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int v0 = min(part1, part0 + warp * piece), v1 = min(part1, v0 + piece);
  Pair acc = make_float2(0.f, 0.f);
  for (int v = v0 + lane; v < v1; v += 32) {
    const Pair w = weight(v);
    add_to(acc, w.x, w.y);
  }
  acc = tidy(acc);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) acc = add(acc, shfl_xor(acc, m));
  __syncthreads();  // the parts' sums have been read
  if (lane == 0) warp_sum[warp] = acc;
  __syncthreads();
  if (warp != 0) return;
  const Pair goal = found_goal;
  Pair before = found_start;
  const int w = pick(lane < kWarps ? warp_sum[lane] : make_float2(0.f, 0.f), goal, before, lane);
  const int e0 = min(part1, part0 + w * piece), e1 = min(part1, e0 + piece);
  int token = -1;
  for (int v = e0; v < e1; v += 32) {  // 32 entries at a time
    const Pair mine = v + lane < e1 ? weight(v + lane) : make_float2(0.f, 0.f);
    const Pair upto = add(before, scan(mine, lane));
    const uint32_t past = __ballot_sync(0xffffffffu, mine.x > 0.f && greater(upto, goal));
    const uint32_t on = __ballot_sync(0xffffffffu, mine.x > 0.f);
    if (past != 0u) {
      token = v + __ffs(static_cast<int>(past)) - 1;
      break;
    }
    if (on != 0u) token = v + 31 - __clz(static_cast<int>(on));
    before = shfl(upto, 31);
  }
  if (lane == 0) p.next[b] = token;
}

template <bool BF16>
cudaError_t launch(const VerifyArgs& a, const VerifyParams& p, cudaStream_t stream) {
  auto kern = draft_verify_kernel<BF16>;
  // CTAs a sequence: as many as the GPU holds at four an SM, and no fewer than 1024 entries each.
  // 64 x 25 drafts over 131072 tokens: 43.3 us on eight; 43.2 on 16, 65 on four, 102 on two; 1 x 5
  // over 32000 6.6 us, 7.0 with no fewer than 2048 entries.
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
