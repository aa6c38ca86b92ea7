// append_f8.cu -- new tokens into an e4m3 paged cache (kv_append_f8).
//
// One scale serves the 16 rows of a (block, KV head), so a row may enlarge it: the
// older rows' codes are then rounded again, to a scale that is a larger power of two,
// which moves their exponents and leaves their fractions alone (above the smallest
// codes).  e4m3 has exponents of its own, so a power of two costs no precision either.
//
// A warp takes the K or the V rows of one (block, KV head): 16 rows of D in eight-
// element vectors, all in registers, so the rows are read once, their largest element
// is a reduction over the warp's lanes, and codes leave eight bytes a lane.
//
// Latency bounds it: 16 sequences of 1024 new tokens (8 KV heads, D = 128) move 88 MB in 17.6 us,
// 74 % of what a copy does, with HBM 42 % and the issue slots 46 % busy (caches flushed).  A warp's
// work is one chain, from the position to the block's id, the rows, their largest element and
// the stores, and nothing of another block is on its way meanwhile.  So what counts is how many
// warps are on an SM: seven CTAs by 72 registers.  (Over the same 88 MB again and again, of which
// L2 keeps the stores: 15.2 us; without the bound, 161 registers, 18.2; eight CTAs spill, 15.5.)  One
// token each of 64 sequences is the launch and that chain, 3.4 us.
#include "common.cuh"
#include "f8.cuh"
#include "internal.h"

namespace attn {
namespace {

constexpr int kBS = 16;
constexpr int kWarps = 4;

struct F8AppendParams {
  uint8_t* codes[2];  // K, V
  float* scale[2];
  int64_t num_blocks;
  int Hkv;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start;
  const int32_t* lens;
  int T;
  const uint16_t* rows[2];
  int64_t stride[2][3];
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 7) kv_append_f8_kernel(const F8AppendParams p) {
  constexpr int kLanes = D / 8;          // lanes a row
  constexpr int kRows = 32 / kLanes;     // rows a step
  constexpr int kSteps = kBS / kRows;
  let_next_launch_in();
  wait_for_launch_ahead();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z;
  const int x = blockIdx.y * kWarps + warp;  // (KV head, K or V)
  const int g = x >> 1, is_v = x & 1;
  if (g >= p.Hkv) return;
  const int start = p.start[b];
  const int n = p.lens != nullptr ? min(max(p.lens[b], 0), p.T) : p.T;
  if (start < 0 || n == 0) return;
  if (static_cast<int64_t>(start) + n > static_cast<int64_t>(p.max_blocks) * kBS) {
    if (x == 0 && blockIdx.x == 0 && lane == 0) report(p.status, kStatusBounds);
    return;
  }
  const int lb = start / kBS + blockIdx.x;
  const int first = lb * kBS;
  if (first >= start + n) return;
  const int blk = p.bt[b * p.bt_stride + lb];  // (looked at after the rows have been asked for)
  const int s0 = max(start - first, 0), s1 = min(start + n - first, kBS);  // the block's new slots
  const int row = lane / kLanes, col = lane % kLanes * 8;
  const uint16_t* src = p.rows[is_v] + b * p.stride[is_v][0] + g * p.stride[is_v][1] + col;
  uint4 w[kSteps];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = i * kRows + row;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= s0 && slot < s1)
      w[i] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(first + slot - start) * p.stride[is_v][2]);
  }
  if (blk < 0 || blk >= p.num_blocks) {
    if (lane == 0) report(p.status, kStatusBounds);
    return;
  }
  const int64_t at = static_cast<int64_t>(blk) * p.Hkv + g;
  const float old = s0 > 0 ? p.scale[is_v][at] : 0.f;
  const auto finite_abs = [](float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.f; };  // 0 for a NaN
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) a = fmaxf(a, fmaxf(finite_abs(bf16lo_to_f32(u[k])), finite_abs(bf16hi_to_f32(u[k]))));
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  const float need = a > 0.f ? pow2(f8_scale_exponent(a)) : 0.f;
  const bool grows = !(old >= need);  // (a scale that was never written too)
  const float sc = grows ? need : old;
  const float inv = sc > 0.f ? 1.0f / sc : 1.0f;  // a power of two
  uint8_t* dst = p.codes[is_v] + at * kBS * D + col;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = i * kRows + row;
    uint2* out = reinterpret_cast<uint2*>(dst + slot * D);
    if (slot >= s0 && slot < s1) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = f8_codes(bf16lo_to_f32(u[k]) * inv, bf16hi_to_f32(u[k]) * inv);
      *out = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    } else if (slot < s0 && grows) {
      const uint2 was = *out;
      const float r = old * inv;  // (0 if the older rows are zeros, or infinities whose codes stood for 0)
      const uint32_t u[4] = {was.x & 0xffffu, was.x >> 16, was.y & 0xffffu, was.y >> 16};
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        half2_f32(f8_half2(u[k]), lo, hi);
        c[k] = f8_codes(lo * r, hi * r);
      }
      *out = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
  }
  if (lane == 0) p.scale[is_v][at] = sc;
}

}  // namespace

cudaError_t launch_kv_append_f8(const F8AppendArgs& a, cudaStream_t stream) {
  F8AppendParams p;
  p.codes[0] = a.cache.k;
  p.codes[1] = a.cache.v;
  p.scale[0] = a.cache.k_scale;
  p.scale[1] = a.cache.v_scale;
  p.num_blocks = a.cache.num_blocks;
  p.Hkv = a.cache.Hkv;
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.start = a.start_pos;
  p.lens = a.lens;
  p.T = static_cast<int>(a.T);
  p.rows[0] = static_cast<const uint16_t*>(a.k_new.data);
  p.rows[1] = static_cast<const uint16_t*>(a.v_new.data);
  for (int i = 0; i < 3; ++i) p.stride[0][i] = a.k_new.stride[i], p.stride[1][i] = a.v_new.stride[i];
  p.status = a.status;
  // blocks that T tokens touch at most
  const dim3 grid(static_cast<unsigned>((a.T + kBS - 2) / kBS + 1),
                  static_cast<unsigned>((2 * a.cache.Hkv + kWarps - 1) / kWarps), static_cast<unsigned>(a.B));
  return a.cache.D == 128 ? launch_early(kv_append_f8_kernel<128>, grid, kWarps * 32, 0, stream, p)
                          : launch_early(kv_append_f8_kernel<64>, grid, kWarps * 32, 0, stream, p);
}

}  // namespace attn
