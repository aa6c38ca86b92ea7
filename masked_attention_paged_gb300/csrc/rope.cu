// rope.cu -- rotary positions: rotate queries and keys by their tokens'
// positions, and write the rotated keys with their values into the paged cache
// in the same launch.
//
// Pair i of a row (dims 2i, 2i + 1 interleaved; i, i + n in the half layout,
// n = rotary_dim / 2) turns by the angle theta = position * f_i:
//   u = a cos theta - b sin theta,   v = a sin theta + b cos theta;
// dims from rotary_dim on are copied.  f_i comes as a 64-bit fraction of a
// turn, so position * f_i modulo one turn is one wrapping integer product,
// exact at any position (a float32 angle is off by 0.06 rad at a million);
// the nearest quarter turn is taken off in integers too, and what is left, at
// most an eighth of a turn, goes through sincospif with an absolute error below
// 2^-24 radians.
//
// The work is bytes: each row is read and written once.  A CTA takes a few
// tokens and a range of their heads; its threads first compute the tokens'
// sines and cosines into shared memory (one sincospif each: shared by all heads
// of a token), then move rows, 16 elements (two 16-byte vectors of bf16) a
// thread and step.  16 sequences x 1024 tokens (32 query and 8 KV heads, D =
// 128): 66 us for 403 MB, 6.1 TB/s, 90 % of the measured copy rate; one token of
// one sequence 3.2 us and of 64 sequences 3.0 us, a launch and its loads.  Into the
// INT8 cache 96 us and 4.5: a division an element and a reduction over a row's lanes.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "q8_quant.cuh"

namespace attn {
namespace {

constexpr int kBS = 16;        // tokens per cache block
constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens per CTA
constexpr int kSlot = 16;      // row elements per thread and step

struct Rows {  // a [B, H, T, D] view
  void* data;
  int64_t sb, sh, st;
  __device__ int64_t at(int b, int h, int t) const { return b * sb + h * sh + t * st; }
};

struct RopeParams {
  Rows in, out;       // queries (or rope_apply's tensor)
  Rows k, v;          // new keys and values, when there is a cache
  int B, T, D, n;     // n: rotated pairs per row
  int Hq, Hkv;        // Hkv = 0: no cache
  int tokens, heads;  // per CTA
  int slots;          // 16-element slots per row
  float sin_sign, magnitude;
  const int32_t* positions;
  int64_t pos_stride;
  const uint64_t* freqs;  // [n] turns per token, 64-bit fractions
  void* kc;
  void* vc;
  float* ks;  // INT8 cache: row scales
  float* vs;
  int64_t num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  int max_blocks;
  const int32_t* start_pos;
  uint32_t* status;
};

// cos and sin of position * f, f in 2^-64 turns
__device__ __forceinline__ float2 turn(int position, uint64_t f) {
  const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(position)) * f;
  const uint32_t quarter = static_cast<uint32_t>((frac + (uint64_t(1) << 61)) >> 62);  // nearest quarter turn
  const int64_t rest = static_cast<int64_t>(frac - (static_cast<uint64_t>(quarter) << 62));
  // rest in [-1/8, 1/8) turn; sincospif takes half turns
  const float x = static_cast<float>(static_cast<int32_t>(rest >> 32)) * 4.6566128730773926e-10f;  // 2^-31
  float s, c;
  sincospif(x, &s, &c);
  const bool odd = quarter & 1;
  const float cc = odd ? s : c, ss = odd ? c : s;
  // quarters 1, 2 turn the cosine's sign, quarters 2, 3 the sine's
  return make_float2(((quarter + 1) & 2) ? -cc : cc, (quarter & 2) ? -ss : ss);
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else
    return static_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
  if constexpr (BF16)
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
  else
    static_cast<float*>(p)[i] = x;
}

// 8 elements from 16-byte words
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4* w, float* x) {
  if constexpr (BF16) {
    x[0] = bf16lo_to_f32(w->x), x[1] = bf16hi_to_f32(w->x), x[2] = bf16lo_to_f32(w->y), x[3] = bf16hi_to_f32(w->y);
    x[4] = bf16lo_to_f32(w->z), x[5] = bf16hi_to_f32(w->z), x[6] = bf16lo_to_f32(w->w), x[7] = bf16hi_to_f32(w->w);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(w[i].x), x[4 * i + 1] = __uint_as_float(w[i].y);
      x[4 * i + 2] = __uint_as_float(w[i].z), x[4 * i + 3] = __uint_as_float(w[i].w);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* x) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Where the 16 elements of a slot sit in the row: elements 0..7 from e0, 8..15
// from e1.  Half layout: slots below n / 8 hold eight pairs (element e with
// element 8 + e); every other slot is 16 neighbouring dims.
struct SlotAt {
  int e0, e1;
  bool half_pairs;
};

template <bool INTER>
__device__ __forceinline__ SlotAt slot_at(int s, int n) {
  if (INTER) return {s * kSlot, s * kSlot + 8, false};
  if (s < n / 8) return {s * 8, n + s * 8, true};
  const int e = 2 * n + (s - n / 8) * kSlot;
  return {e, e + 8, false};
}

// Rotate a slot's 16 values; cs points at the token's (cos, sin) of pair 0.
template <bool INTER>
__device__ __forceinline__ void rotate16(float (&x)[16], const SlotAt& at, const float2* cs, int n) {
  if (INTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pair = at.e0 / 2 + j;
      if (pair < n) {
        const float2 t = cs[pair];
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * t.x - b * t.y;
        x[2 * j + 1] = a * t.y + b * t.x;
      }
    }
  } else if (at.half_pairs) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = cs[at.e0 + j];
      const float a = x[j], b = x[8 + j];
      x[j] = a * t.x - b * t.y;
      x[8 + j] = a * t.y + b * t.x;
    }
  }
}

// Q8: codes and row scale of a row whose S (4 or 8) slots sit in S neighbouring
// lanes, exactly as quantise_lane_q8 does from bf16 rows.
__device__ __forceinline__ void store_q8(float (&x)[16], int8_t* dst, float* scale_out, const SlotAt& at, int S,
                                         bool first) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const uint32_t w = pack_bf16x2(x[e], x[e + 1]);  // the values a bf16 cache would hold
    x[e] = bf16lo_to_f32(w), x[e + 1] = bf16hi_to_f32(w);
    a = fmaxf(a, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
  }
  const uint32_t row_lanes = ((1u << S) - 1u) << ((threadIdx.x & 31) / S * S);
  for (int o = S / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(row_lanes, a, o));
  const float scale = __fdiv_rn(a, 127.0f);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float c = scale > 0.f ? rintf(__fdiv_rn(x[4 * k + e], scale)) : 0.f;
      c = fminf(fmaxf(c, -127.f), 127.f);
      w[k] |= (static_cast<uint32_t>(static_cast<int32_t>(c)) & 0xffu) << (8 * e);
    }
  }
  if (dst == nullptr) return;  // this row is not cached (the lanes stay for the shuffle)
  *reinterpret_cast<uint2*>(dst + at.e0) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(dst + at.e1) = make_uint2(w[2], w[3]);
  if (first) *scale_out = scale;
}

// grid (token groups, head ranges).  VEC: 16-byte rows and whole slots; else
// element by element (odd strides, or a half layout whose n is no multiple
// of 8).  ONE (and VEC): a thread has one row, whose loads need not wait for the
// sines: 25 MB in 7.5 instead of 8.6 us; with more rows a thread the registers cost
// more than that saves (16 x 1024 tokens 73.4 instead of 67.6 us).  There bf16 rows
// take 32 registers, so that an SM holds 8 CTAs (65.8 us; with 34, 68.7).
template <bool BF16, bool INTER, bool VEC, bool Q8, bool ONE>
__global__ void __launch_bounds__(kThreads, BF16 && VEC && !ONE && !Q8 ? 8 : 4)
    rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs[];  // [tokens][n]
  __shared__ int64_t row_base[kMaxTokens];  // cache row of (token, KV head 0), -1: not cached
  wait_for_launch_ahead();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tokens), static_cast<int64_t>(p.B) * p.T - first));
  const int h0 = blockIdx.y * p.heads;
  const int nh = min(p.heads, p.Hq + 2 * p.Hkv - h0);

  const int S = p.slots;
  const int s = threadIdx.x % S;   // this thread's slot of every row it moves
  const int step = kThreads / S;   // rows per pass; an S that does not divide the CTA leaves threads over
  const SlotAt at = slot_at<INTER>(s, p.n);
  const bool spare = threadIdx.x >= step * S;  // never with Q8: S is 4 or 8 there
  const int rows_all = ntok * nh;
  int tok = 0, h = threadIdx.x / S;  // this thread's row; VEC: its 16 elements in w
  auto settle = [&] {
    while (h >= nh && tok < ntok) h -= nh, ++tok;
    return tok < ntok && !spare;
  };
  constexpr int EB = BF16 ? 2 : 4, kWords = EB;
  uint4 w[kWords] = {};
  auto fetch = [&] {
    const int64_t token = first + tok;
    const int b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
    const int head = h0 + h, kv = head - p.Hq;
    const Rows& src = kv < 0 ? p.in : (kv < p.Hkv ? p.k : p.v);
    const uint8_t* row = static_cast<const uint8_t*>(src.data) +
                         src.at(b, kv < 0 ? head : (kv < p.Hkv ? kv : kv - p.Hkv), t) * EB;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = *reinterpret_cast<const uint4*>(row + (i < kWords / 2 ? at.e0 : at.e1) * EB + i % (kWords / 2) * 16);
  };
  if constexpr (ONE) {  // it sets out before the sines
    if (settle()) fetch();
  }

  for (int i = threadIdx.x; i < ntok * p.n; i += kThreads) {
    const int64_t tok = first + i / p.n;
    float2 t = turn(p.positions[(tok / p.T) * p.pos_stride + tok % p.T], p.freqs[i % p.n]);
    cs[i] = make_float2(t.x * p.magnitude, t.y * p.magnitude * p.sin_sign);
  }
  if (p.Hkv > 0 && threadIdx.x < ntok) {
    const int64_t tok = first + threadIdx.x;
    const int b = static_cast<int>(tok / p.T), i = static_cast<int>(tok % p.T);
    const int start = p.start_pos[b];
    int64_t base = -1;
    if (start >= 0) {  // negative: an idle sequence
      if (static_cast<int64_t>(start) + p.T > static_cast<int64_t>(p.max_blocks) * kBS) {
        report(p.status, kStatusBounds);  // the whole sequence is skipped
      } else {
        const int slot = start + i;
        const int blk = p.bt[b * p.bt_stride + slot / kBS];
        if (blk < 0 || blk >= p.num_blocks)
          report(p.status, kStatusBounds);
        else
          base = static_cast<int64_t>(blk) * p.Hkv * kBS + slot % kBS;
      }
    }
    row_base[threadIdx.x] = base;
  }
  __syncthreads();

  for (int r = 0; r < rows_all; r += step, h += step) {  // the same trips for every thread: Q8 shuffles
    const bool there = settle();
    if constexpr (VEC) {
      if (!ONE && there) fetch();
    }
    if (!Q8 && !there) continue;
    const int tk = there ? tok : 0, head = h0 + (there ? h : 0);
    const int64_t token = first + tk;
    const int b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
    const Rows* src = &p.in;
    int hh = head;
    void* to = p.out.data;
    int64_t dst = 0;
    bool rot = true, write = there, cached = false;
    float* scale = nullptr;
    if (head >= p.Hq) {
      hh = head - p.Hq;
      const bool is_v = hh >= p.Hkv;
      if (is_v) hh -= p.Hkv;
      src = is_v ? &p.v : &p.k;
      rot = !is_v;
      cached = true;
      write = there && row_base[tk] >= 0;
      const int64_t row = row_base[tk] + static_cast<int64_t>(hh) * kBS;
      to = is_v ? p.vc : p.kc;
      dst = row * p.D;
      if constexpr (Q8) scale = (is_v ? p.vs : p.ks) + row;
    } else {
      dst = p.out.at(b, hh, t);
    }
    const void* from = src->data;
    const int64_t o = src->at(b, hh, t);
    const float2* tcs = cs + tk * p.n;
    if constexpr (VEC) {
      if (Q8 && cached) {
        // Not reached by every row of a warp at once: the S lanes of a row do
        // so together, and the shuffles below stay within them.
        float x[16];
        unpack8<BF16>(w, x);
        unpack8<BF16>(w + kWords / 2, x + 8);
        if (rot) rotate16<INTER>(x, at, tcs, p.n);
        store_q8(x, write ? static_cast<int8_t*>(to) + dst : nullptr, scale, at, S, s == 0);
      } else if (write) {
        const bool turned = rot && (INTER ? at.e0 < 2 * p.n : at.half_pairs);
        if (turned) {
          float x[16];
          unpack8<BF16>(w, x);
          unpack8<BF16>(w + kWords / 2, x + 8);
          rotate16<INTER>(x, at, tcs, p.n);
          store8<BF16>(to, dst + at.e0, x);
          store8<BF16>(to, dst + at.e1, x + 8);
        } else {  // values and dims past rotary_dim: a bit copy
          uint8_t* g = static_cast<uint8_t*>(to);
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            *reinterpret_cast<uint4*>(g + (dst + (i < kWords / 2 ? at.e0 : at.e1)) * EB + i % (kWords / 2) * 16) = w[i];
        }
      }
    } else if (write) {
      // slots of the half layout: ceil(n / 8) groups of eight pairs, then 16 dims
      // each; interleaved: 16 dims each
      const int pair_slots = INTER ? 0 : (p.n + 7) / 8;
      auto copy = [&](int e) {
        if constexpr (BF16)
          static_cast<uint16_t*>(to)[dst + e] = static_cast<const uint16_t*>(from)[o + e];
        else
          static_cast<uint32_t*>(to)[dst + e] = static_cast<const uint32_t*>(from)[o + e];
      };
      auto turn_pair = [&](int e, int f, int i) {
        const float a = load1<BF16>(from, o + e), c = load1<BF16>(from, o + f);
        store1<BF16>(to, dst + e, a * tcs[i].x - c * tcs[i].y);
        store1<BF16>(to, dst + f, a * tcs[i].y + c * tcs[i].x);
      };
      if (s < pair_slots) {
        for (int i = s * 8; i < min(p.n, s * 8 + 8); ++i) {
          if (rot)
            turn_pair(i, p.n + i, i);
          else
            copy(i), copy(p.n + i);
        }
      } else {
        const int e0 = INTER ? s * kSlot : 2 * p.n + (s - pair_slots) * kSlot;
        for (int e = e0; e < min(p.D, e0 + kSlot); e += 2) {
          if (INTER && rot && e < 2 * p.n)
            turn_pair(e, e + 1, e / 2);
          else
            for (int f = e; f < min(p.D, e + 2); ++f) copy(f);
        }
      }
    }
  }
}

bool rows_vec16(const View4& t) {
  const int eb = t.dtype == ATTN_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(t.data) % 16 != 0) return false;
  for (int i = 0; i < 3; ++i)
    if (t.shape[i] > 1 && (t.stride[i] * eb) % 16 != 0) return false;
  return true;
}

Rows rows(const View4& t) { return {t.data, t.stride[0], t.stride[1], t.stride[2]}; }

template <bool BF16, bool INTER, bool VEC, bool Q8, bool ONE>
cudaError_t launch(const RopeParams& p, dim3 grid, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.tokens) * p.n * sizeof(float2);
  return launch_early(rope_kernel<BF16, INTER, VEC, Q8, ONE>, grid, kThreads, smem, stream, p);
}

template <bool BF16, bool INTER, bool Q8>
cudaError_t pick(const RopeParams& p, bool vec, dim3 grid, cudaStream_t stream) {
  if (vec)
    return p.tokens * p.heads <= kThreads / p.slots ? launch<BF16, INTER, true, Q8, true>(p, grid, stream)
                                                    : launch<BF16, INTER, true, Q8, false>(p, grid, stream);
  if constexpr (Q8)
    return cudaErrorNotSupported;
  else
    return launch<BF16, INTER, false, false, false>(p, grid, stream);
}

}  // namespace

bool rope_rows_in_vectors(const RopeArgs& a) {
  const int64_t D = a.x.shape[3];
  bool vec = D % kSlot == 0 && (a.interleaved || (a.rotary_dim / 2) % 8 == 0) && rows_vec16(a.x) && rows_vec16(a.out);
  if (a.k_new.data != nullptr) vec = vec && rows_vec16(a.k_new) && rows_vec16(a.v_new);
  return vec;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const bool vec = rope_rows_in_vectors(a);
  RopeParams p = {};
  p.in = rows(a.x);
  p.out = rows(a.out);
  p.B = static_cast<int>(a.x.shape[0]);
  p.Hq = static_cast<int>(a.x.shape[1]);
  p.T = static_cast<int>(a.x.shape[2]);
  p.D = static_cast<int>(a.x.shape[3]);
  p.n = a.rotary_dim / 2;
  p.sin_sign = a.inverse ? -1.f : 1.f;
  p.magnitude = a.magnitude;
  p.positions = a.positions;
  p.pos_stride = a.pos_stride;
  p.freqs = a.freqs;
  const bool append = a.k_new.data != nullptr;
  if (append) {
    p.k = rows(a.k_new);
    p.v = rows(a.v_new);
    p.Hkv = a.cache.Hkv;
    p.kc = a.cache.k;
    p.vc = a.cache.v;
    p.ks = const_cast<float*>(a.cache.k_scale);
    p.vs = const_cast<float*>(a.cache.v_scale);
    p.num_blocks = a.cache.num_blocks;
    p.bt = a.block_table;
    p.bt_stride = a.bt_stride;
    p.max_blocks = a.max_blocks;
    p.start_pos = a.start_pos;
    p.status = a.status;
  }
  if (vec || a.interleaved)
    p.slots = (p.D + kSlot - 1) / kSlot;
  else
    p.slots = (p.n + 7) / 8 + (p.D - 2 * p.n + kSlot - 1) / kSlot;
  // Few tokens: one per CTA and the heads spread over CTAs, one row a thread
  // group, so that the call is one round trip to memory.  Many: kMaxTokens per
  // CTA with all their heads, so that a token's sines are computed once.
  const int64_t tokens = static_cast<int64_t>(p.B) * p.T;
  const int all_heads = p.Hq + 2 * p.Hkv;
  const int rows_per_pass = std::max(1, kThreads / p.slots);
  const int64_t ctas = 2 * static_cast<int64_t>(std::max(1, device_sm_count()));
  p.tokens = tokens >= ctas * kMaxTokens ? kMaxTokens : 1;
  p.heads = tokens >= ctas ? all_heads : std::min(all_heads, rows_per_pass);
  const int64_t gx = (tokens + p.tokens - 1) / p.tokens;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((all_heads + p.heads - 1) / p.heads));
  if (append && a.cache.k_scale != nullptr)
    return a.interleaved ? pick<true, true, true>(p, vec, grid, stream) : pick<true, false, true>(p, vec, grid, stream);
  if (a.x.dtype == ATTN_BF16)
    return a.interleaved ? pick<true, true, false>(p, vec, grid, stream)
                         : pick<true, false, false>(p, vec, grid, stream);
  return a.interleaved ? pick<false, true, false>(p, vec, grid, stream)
                       : pick<false, false, false>(p, vec, grid, stream);
}

}  // namespace attn
