// pa_fp8_append.cu -- pa_v2_qk_rope_append_fp8: per-head norm of q and k, rotation by
// position, and the append of k and v to pools of e4m3 codes with one power-of-two
// exponent for each page, KV head and side.
//
//   norm      x <- x * w / sqrt(mean(x^2) + eps)                (f32)
//   rotation  (x, y) <- (x cos a - y sin a, y cos a + x sin a),  a_j = pos * inv_freq[j]
//   exponent  need = least e in [-15, 7] with max |x| <= 448 2^e over the page's new tokens;
//             need where they begin the page, else max(old, need)
//   code      round(x 2^-e) to nearest even, once, from f32
//
// The new tokens of one page are a run of neighbours in the call, so one warp sees all of
// them for a head and side and decides the exponent alone: no atomics, no second
// launch, the same result in every call.  A run that skipped tokens split from an earlier one
// of its page is refused.  Where the exponent of a begun page grows, that
// warp also rescales the page's earlier codes.  A code is a 4-bit number times a power of
// two, so that step is exact except for codes that turn subnormal.
//
// HBM bound: q, k and v are read once and q_out and the codes written once.  Some CTAs walk
// q's tokens, a warp a token and all its heads with one computation of a lane's cosines
// and sines, the next rows on their way.  The others take stretches of tokens and handle
// the runs that begin in theirs, a warp a head of a side (a run's angles are computed once,
// by the CTA, while its K rows are on their way).  Rows are held as in pa_qk_rope.cu: 16
// bytes per lane in two pieces that hold both elements of each of the lane's pairs.  A run
// that fits a warp's registers as loaded (16 tokens of 128 elements) is read once and normed
// and rotated twice, for the maximum and for the codes; a longer one is read again, out of L2.
//
// 16384 tokens of 48 heads take 78 us of 54 (4.7 TB/s of 6.8): alone q takes 52 (5.2 TB/s)
// and the runs 45, which wait for their data, a run's steps one after the other (8 us a
// CTA, three CTAs an SM).  2048 tokens 19 us of 7, 1024 of as many requests 20 of 3.4: few rows for a run's steps
// to hide behind, or many runs one after the other.  Pages longer than a stretch leave CTAs without a run, and of 256 tokens
// (128 KB of angles) one CTA fits an SM instead of three: 16384 tokens 97, 134 and 199 us with pages of 64, 128 and
// 256, 2048 tokens 33, 35 and 29, 64 requests of one token 5.9, 5.9 and 6.5 (5.7 with pages of 16).  Kept in shared
// memory between maximum and codes K costs q more than it saves (93 us); held in registers it
// leaves two CTAs an SM (106); angles by every warp for itself spill (146); 64 registers for
// four CTAs spill (118).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.cuh"
#include "pa_mma.cuh"
#include "pa_rope.cuh"
#include "pa_tc05.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kApThreads = 256;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApMaxPage = 256;
constexpr int kApStretch = 16;  // tokens of a CTA's stretch, at most
constexpr int kApCtas = 3;      // per SM

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const int32_t* slots;
  const float* inv_freq;
  const void* q_weight;
  const void* k_weight;
  void* q_out;
  uint8_t* k_pool;
  uint8_t* v_pool;
  int8_t* k_exp;
  int8_t* v_exp;
  int32_t* status;
  int64_t num_rows;  // pool rows
  float eps;
  int32_t tokens, hq, hkv, rot, page_size;
  uint32_t ps_magic, ps_shift, half_magic, half_shift;
  int32_t stretch, kv_splits;           // tokens per KV CTA, and CTAs that share a stretch's heads
  int32_t q_from, q_ctas, q_warps, q_splits, q_share;  // warps with q rows, and warps that share a token's heads, so many each
};

__device__ __forceinline__ uint32_t codes_of(float a, float b) {  // a in the lower byte
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b), "f"(a));
  return y;
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// Two codes times f (a power of two, both halves), rounded to codes again.
__device__ __forceinline__ uint32_t rescaled(uint16_t x, __half2 f) {
  uint32_t h;
  uint16_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(x));
  const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&h), f);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(*reinterpret_cast<const uint32_t*>(&z)));
  return y;
}

// The least exponent whose largest code holds `top` (finite, not negative).
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);  // 448 = 1.75 2^8
  return min(max(e, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX);
}

// A lane's share of head rows of T.  PAIRED: its two pieces are partners (half split); else they are neighbours and
// pairs are neighbouring elements (interleaved).
template <typename T, int D, bool PAIRED>
struct Row {
  static constexpr int N = Vec<T>::N, P = N / 2;  // elements per lane; per piece, and pairs per lane
  static constexpr int kLanes = D / N;            // lanes per row (8, 16 or 32)
  static constexpr int kAtOnce = 32 / kLanes;     // rows a warp holds at once
  int e0, e1;      // the pieces' places in the row
  int pair0;       // the first pair of the lane
  bool rotated;
  __device__ __forceinline__ explicit Row(int rot) {
    const int lane = threadIdx.x & (kLanes - 1), half = rot / 2;
    rotated = lane * P < half;
    e0 = PAIRED && rotated ? lane * P : lane * N;
    e1 = PAIRED && rotated ? e0 + half : e0 + P;
    pair0 = lane * P;
  }
  __device__ __forceinline__ uint4 load(const T* row) const {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + e0)), b = __ldg(reinterpret_cast<const uint2*>(row + e1));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  // Norm with weights g, over the row's lanes, all of which call it.
  __device__ __forceinline__ static void norm(float (&x)[N], const float (&g)[N], float eps) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; i += 2) s2 = fma2(make_float2(x[i], x[i + 1]), make_float2(x[i], x[i + 1]), s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int s = kLanes / 2; s >= 1; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
    const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 y = mul2(mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv)), make_float2(g[i], g[i + 1]));
      x[i] = y.x;
      x[i + 1] = y.y;
    }
  }
  // cs: cosines, then sines `half` floats behind (elements that are not rotated are left out of it: 0 times an
  // infinity next to them is NaN)
  __device__ __forceinline__ void rotate(float (&x)[N], const float* cs, int half) const {
    if (!rotated) return;
    float2 co[P / 2], si[P / 2];  // half is a multiple of 8, and a lane's pairs of 4 or 2
    angles_at(cs, half, co, si);
    turn(x, co, si);
  }
  __device__ __forceinline__ void angles_at(const float* cs, int half, float2 (&co)[P / 2], float2 (&si)[P / 2]) const {
    if (P == 4) {
      const float4 c = *reinterpret_cast<const float4*>(cs + pair0), s = *reinterpret_cast<const float4*>(cs + half + pair0);
      co[0] = make_float2(c.x, c.y);
      si[0] = make_float2(s.x, s.y);
      co[P / 2 - 1] = make_float2(c.z, c.w);
      si[P / 2 - 1] = make_float2(s.z, s.w);
    } else {
      co[0] = *reinterpret_cast<const float2*>(cs + pair0);
      si[0] = *reinterpret_cast<const float2*>(cs + half + pair0);
    }
  }
  __device__ __forceinline__ static void turn(float (&x)[N], const float2 (&co)[P / 2], const float2 (&si)[P / 2]) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {  // two pairs: their first elements in u, their second ones in w
      const int a = PAIRED ? 2 * i : 4 * i, b = PAIRED ? a + P : a + 1, next = PAIRED ? 1 : 2;
      const float2 u = make_float2(x[a], x[a + next]), w = make_float2(x[b], x[b + next]);
      const float2 nu = fma2(make_float2(-w.x, -w.y), si[i], mul2(u, co[i]));
      const float2 nw = fma2(u, si[i], mul2(w, co[i]));
      x[a] = nu.x;
      x[a + next] = nu.y;
      x[b] = nw.x;
      x[b + next] = nw.y;
    }
  }
};

// The largest magnitude of a row's lane, infinities with it (NaN is left out); for V straight from the loaded bits.
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N], float top) {
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
  return top;
}
template <int N>
__device__ __forceinline__ float largest_finite(const float (&x)[N], float top) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (fabsf(x[i]) <= 3.402823466e38f) top = fmaxf(top, fabsf(x[i]));
  return top;
}

template <typename T, typename TQ, int D, bool PAIRED>
__global__ void __launch_bounds__(kApThreads, kApCtas) pa_v2_qk_rope_append_fp8_kernel(const AppendParams p) {
  using R = Row<T, D, PAIRED>;
  constexpr int N = R::N, P = R::P, kLanes = R::kLanes, kAtOnce = R::kAtOnce;
  constexpr int kHeld = 8;  // passes of a run that registers hold
  extern __shared__ __align__(16) float cs[];  // [tokens][2][rot / 2]: cosines, sines
  __shared__ uint64_t turns[D / 2];
  __shared__ int32_t slot_of[1 + kApStretch + kApMaxPage];  // from the token before the stretch on
  __shared__ int32_t pos_of[1 + kApStretch + kApMaxPage];

  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2, sub = lane / kLanes;
  const R row(p.rot);
  const bool is_q = (int)blockIdx.x >= p.q_from && (int)blockIdx.x < p.q_from + p.q_ctas;
  const int kv_block = (int)blockIdx.x - (p.q_from == 0 ? p.q_ctas : 0);
  const T* norm_weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
  float weight[N];
  if (norm_weight) Vec<T>::unpack(row.load(norm_weight), weight);

  if (is_q) {
    // ------------------------------------------------------------------ q: a warp walks tokens, all their heads with one
    // computation of a lane's cosines and sines, the next rows on their way
    const int first = ((int)blockIdx.x - p.q_from) * kApWarps + warp;
    constexpr int kBatch = 4;  // passes of rows under way per lane, and as many ahead
    const int h0 = first % p.q_splits * p.q_share, heads = min(p.q_share, p.hq - h0);
    const int batches = (heads + kBatch * kAtOnce - 1) / (kBatch * kAtOnce);
    uint64_t lane_turns[P];
#pragma unroll
    for (int i = 0; i < P; ++i) lane_turns[i] = row.rotated ? turn_of(p.inv_freq[row.pair0 + i]) : 0;
    int tok = first / p.q_splits;
    const int step = p.q_warps / p.q_splits;
    if (tok >= step) return;  // (a last warp of no whole group)
    auto fetch = [&](int t, int batch, uint4 (&raw)[kBatch]) {
      const T* q = static_cast<const T*>(p.q) + (int64_t)t * p.q_stride + (h0 + batch * kBatch * kAtOnce + sub) * D;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        raw[b] = make_uint4(0, 0, 0, 0);
        if (batch * kBatch * kAtOnce + b * kAtOnce + sub < heads) raw[b] = row.load(q + b * kAtOnce * D);
      }
    };
    uint4 raw[kBatch], ahead[kBatch];
    int32_t slot = -1, pos = 0;
    if (tok < p.tokens) {
      slot = __ldg(p.slots + tok);
      pos = __ldg(p.positions + tok);
      fetch(tok, 0, ahead);
    }
    while (tok < p.tokens) {
      float2 co[P / 2], si[P / 2];
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        const float2 a = rotation(pos, lane_turns[2 * i]), b = rotation(pos, lane_turns[2 * i + 1]);
        co[i] = make_float2(a.x, b.x);
        si[i] = make_float2(a.y, b.y);
      }
      const bool live = slot >= 0 && slot < p.num_rows;
      TQ* out = static_cast<TQ*>(p.q_out) + ((int64_t)tok * p.hq + h0 + sub) * D;
      const int next = tok + step;
      if (next < p.tokens) {
        slot = __ldg(p.slots + next);
        pos = __ldg(p.positions + next);
      }
      for (int batch = 0; batch < batches; ++batch) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) raw[b] = ahead[b];
        if (batch + 1 < batches) fetch(tok, batch + 1, ahead);
        else if (next < p.tokens) fetch(next, 0, ahead);
        // (a whole batch without a test between its passes: they run side by side)
        auto passes = [&](auto whole) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int h = (batch * kBatch + b) * kAtOnce;
          if (!decltype(whole)::value && h >= heads) break;
          float x[N];
          Vec<T>::unpack(raw[b], x);
          if (norm_weight) R::norm(x, weight, p.eps);
          if (row.rotated) R::turn(x, co, si);
          if (!live || (!decltype(whole)::value && h + sub >= heads)) continue;
          TQ* to = out + h * D;
          if (sizeof(TQ) != sizeof(T)) {  // f32 from 16 bits: a piece is 16 bytes
            *reinterpret_cast<float4*>(to + row.e0) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(to + row.e1) = make_float4(x[P], x[P + 1], x[N - 2], x[N - 1]);
          } else {
            const uint4 y = Vec<T>::pack(x);
            *reinterpret_cast<uint2*>(to + row.e0) = make_uint2(y.x, y.y);
            *reinterpret_cast<uint2*>(to + row.e1) = make_uint2(y.z, y.w);
          }
        }
        };
        if ((batch + 1) * kBatch * kAtOnce <= heads) passes(std::true_type());
        else passes(std::false_type());
      }
      tok = next;
    }
    return;
  }

  // -------------------------------------------------------------------- k and v: a warp takes a head of a side through the
  // runs that begin in the CTA's stretch of tokens
  const int task0 = kv_block % p.kv_splits * kApWarps, task = task0 + warp;
  const bool is_v = task >= p.hkv, has_k = task0 < p.hkv && half > 0;  // has_k: of the CTA, whose warps then share angles
  const int head = is_v ? task - p.hkv : task;
  const int w0 = kv_block / p.kv_splits * p.stretch, w1 = min(w0 + p.stretch, p.tokens);
  const int ahead = min(p.stretch + p.page_size, p.tokens - w0);
  for (int i = threadIdx.x; i < ahead + 1; i += kApThreads) {
    int32_t s = -1;
    if (w0 + i > 0) s = __ldg(p.slots + w0 - 1 + i);
    if (has_k && i > 0) pos_of[i] = __ldg(p.positions + w0 - 1 + i);
    if (s >= p.num_rows) {
      if (i > 0 && i <= w1 - w0 && task0 == 0) report(p.status, PA_DEVICE_BAD_SLOT);
      s = -1;
    }
    slot_of[i] = s;
  }
  if (has_k)
    for (int i = threadIdx.x; i < half; i += kApThreads) turns[i] = turn_of(p.inv_freq[i]);
  __syncthreads();
  const int64_t stride = is_v ? p.v_stride : p.k_stride, pitch = (int64_t)p.hkv * D;
  const T* in = static_cast<const T*>(is_v ? p.v : p.k) + head * D;
  uint8_t* pool = (is_v ? p.v_pool : p.k_pool) + head * D;
  int8_t* exps = (is_v ? p.v_exp : p.k_exp) + head;
  auto page_of = [&](int i) -> int32_t {  // of slot_of[i], -1 for none
    const int32_t s = slot_of[i];
    return s < 0 ? -1 : (int32_t)fast_div((uint32_t)s, p.ps_magic, p.ps_shift);
  };
  // (a lane a token of the stretch: kApStretch <= 32)
  const int32_t lane_page = lane < w1 - w0 ? page_of(lane + 1) : -1;
  uint32_t starts = __ballot_sync(0xffffffffu, lane_page >= 0 && page_of(lane) != lane_page);
  // Skipped tokens before a start, and before those a token of the same page: that one's run has decided the page, and
  // beside it this one would race for its exponent and codes.  It is refused.
  for (uint32_t gaps = starts & __ballot_sync(0xffffffffu, slot_of[lane & (kApStretch - 1)] < 0); gaps; gaps &= gaps - 1) {
    const int at = __ffs(gaps);
    int32_t last = -1;  // the page of the nearest token before that is not skipped
    for (int i = w0 + at - 3; i >= 0 && last < 0; i -= 32) {
      const int32_t s = i >= lane ? __ldg(p.slots + i - lane) : -1;
      const uint32_t live = __ballot_sync(0xffffffffu, s >= 0 && s < p.num_rows);
      if (live) last = (int32_t)fast_div((uint32_t)__shfl_sync(0xffffffffu, s, __ffs(live) - 1), p.ps_magic, p.ps_shift);
    }
    if (last != page_of(at)) continue;
    starts &= ~(1u << (at - 1));
    if (task0 == 0 && threadIdx.x == 0) report(p.status, PA_DEVICE_BAD_SLOT);
  }
  for (; starts; starts &= starts - 1) {
    const int at = __ffs(starts), t = w0 + at - 1;
    const int32_t page = page_of(at);
    // the run: how many tokens, and the least entry
    int len = 1, least = INT_MAX;
    for (int i = 0;; i += 32) {
      const bool in_run = i + lane < p.page_size && at + i + lane <= ahead && page_of(at + i + lane) == page;
      const uint32_t run = __ballot_sync(0xffffffffu, in_run);
      len = i + (run == 0xffffffffu ? 32 : __ffs(~run) - 1);
      if (i + lane < len) least = min(least, slot_of[at + i + lane] - page * p.page_size);
      if (run != 0xffffffffu) break;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    const bool busy = task < 2 * p.hkv;
    const T* src = in + (int64_t)t * stride;
    uint4 raw[kHeld];
    auto fetch = [&](int first) {  // rows first .. of the run
#pragma unroll
      for (int b = 0; b < kHeld; ++b)
        if (first + b * kAtOnce < len) raw[b] = row.load(src + min(first + b * kAtOnce + sub, len - 1) * stride);
    };
    if (busy) fetch(0);
    if (has_k) {
      __syncthreads();  // the run before is done with its angles
      for (int i = threadIdx.x; i < len * half; i += kApThreads) {
        const int tok = (int)fast_div((uint32_t)i, p.half_magic, p.half_shift), j = i - tok * half;
        const float2 r = rotation(pos_of[at + tok], turns[j]);
        cs[2 * half * tok + j] = r.x;
        cs[2 * half * tok + half + j] = r.y;
      }
      __syncthreads();
    }
    if (!busy) continue;
    int8_t* exp = exps + (int64_t)page * p.hkv;
    const int before = least > 0 ? min(max((int)*exp, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX) : 0;
    // Row b of those fetched, normed and rotated: computed twice, for the maximum and for the codes, where holding it
    // would take twice the registers (and leave two CTAs an SM instead of three).
    auto make = [&](int first, int b, float (&x)[N]) {
      Vec<T>::unpack(raw[b], x);
      if (!is_v) {
        if (norm_weight) R::norm(x, weight, p.eps);
        row.rotate(x, cs + 2 * half * min(first + b * kAtOnce + sub, len - 1), half);
      }
    };
    const bool again = len > kHeld * kAtOnce;
    float top = 0.f;
    for (int first = 0; first < len; first += kHeld * kAtOnce) {
      if (first > 0) fetch(first);
      auto passes = [&](auto whole) {
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          if (!decltype(whole)::value && first + b * kAtOnce >= len) break;
          float x[N];
          make(first, b, x);
          top = largest(x, top);
        }
      };
      if (first + kHeld * kAtOnce <= len) passes(std::true_type());
      else passes(std::false_type());
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const bool infinite = top > 3.402823466e38f;
    if (infinite) {  // infinities become NaN and do not count
      top = 0.f;
#pragma unroll 1
      for (int first = 0; first < len; first += kAtOnce) {
        raw[0] = row.load(src + min(first + sub, len - 1) * stride);
        float x[N];
        make(first, 0, x);
        top = largest_finite(x, top);
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    }
    int e = top > 0.f ? exponent_for(top) : PA_V2_FP8_EXP_MIN;
    if (least > 0) {
      e = max(e, before);
      if (e > before) {  // the page's earlier tokens
        const __half2 f = __float2half2_rn(power2(before - e));
        constexpr int kChunks = D / 16;
        for (int i = lane; i < least * kChunks; i += 32) {
          uint4* at16 = reinterpret_cast<uint4*>(pool + ((int64_t)page * p.page_size + i / kChunks) * pitch) + i % kChunks;
          uint4 u = *at16;
          uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = rescaled((uint16_t)w[j], f) | rescaled((uint16_t)(w[j] >> 16), f) << 16;
          *at16 = u;
        }
      }
    }
    if (lane == 0) *exp = (int8_t)e;
    const float down = power2(-e);
    for (int first = 0; first < len; first += kHeld * kAtOnce) {
      if (again || infinite) fetch(first);
      auto passes = [&](auto whole) {
#pragma unroll
      for (int b = 0; b < kHeld; ++b) {
        const int i = first + b * kAtOnce + sub;
        if (!decltype(whole)::value && i - sub >= len) break;
        float x[N];
        make(first, b, x);
        if (infinite) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (!(fabsf(x[j]) <= 3.402823466e38f)) x[j] = NAN;
        }
        uint32_t y[N / 4];
#pragma unroll
        for (int j = 0; j < N; j += 4) {
          const float2 z0 = mul2(make_float2(x[j], x[j + 1]), make_float2(down, down));
          const float2 z1 = mul2(make_float2(x[j + 2], x[j + 3]), make_float2(down, down));
          y[j / 4] = codes_of(z0.x, z0.y) | codes_of(z1.x, z1.y) << 16;
        }
        if (!decltype(whole)::value && i >= len) continue;
        uint8_t* to = pool + (int64_t)slot_of[at + i] * pitch;
        if (N == 8) {
          *reinterpret_cast<uint32_t*>(to + row.e0) = y[0];
          *reinterpret_cast<uint32_t*>(to + row.e1) = y[N / 4 - 1];
        } else {  // f32: two elements per piece
          *reinterpret_cast<uint16_t*>(to + row.e0) = (uint16_t)y[0];
          *reinterpret_cast<uint16_t*>(to + row.e1) = (uint16_t)(y[0] >> 16);
        }
      }
      };
      if (first + kHeld * kAtOnce <= len) passes(std::true_type());
      else passes(std::false_type());
    }
  }
}

using AppendKernel = void (*)(const AppendParams);

template <typename T, typename TQ>
AppendKernel pick_append(int D, bool paired) {
  if (D == 64) return paired ? pa_v2_qk_rope_append_fp8_kernel<T, TQ, 64, true> : pa_v2_qk_rope_append_fp8_kernel<T, TQ, 64, false>;
  return paired ? pa_v2_qk_rope_append_fp8_kernel<T, TQ, 128, true> : pa_v2_qk_rope_append_fp8_kernel<T, TQ, 128, false>;
}

bool on16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_qk_rope_append_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                              const void* v, int64_t v_stride, int32_t dtype, int32_t num_tokens,
                                              int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                              const int32_t* positions, const int32_t* slots, const float* inv_freq,
                                              int32_t rot_dim, int32_t interleaved, const void* q_weight,
                                              const void* k_weight, float eps, void* q_out, int32_t q_dtype,
                                              void* k_pool, void* v_pool, int8_t* k_exp, int8_t* v_exp,
                                              int64_t num_pages, int32_t page_size, int32_t* status,
                                              void* cuda_stream) {
  using namespace pa;
  if (num_tokens < 0 || num_qo_heads < 1 || num_kv_heads < 1 || rot_dim < 0 || num_pages < 1 || page_size < 1 ||
      !std::isfinite(eps) || eps < 0.f)
    return PA_EINVAL;
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return PA_EUNSUPPORTED;
  if (q_dtype != dtype && q_dtype != PA_F32) return PA_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  if (rot_dim > head_dim || rot_dim % 16 != 0) return PA_EUNSUPPORTED;
  if (num_qo_heads > 16384 || num_kv_heads > 16384 || page_size > kApMaxPage) return PA_EUNSUPPORTED;
  if ((int64_t)num_tokens * num_kv_heads > INT32_MAX) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !positions || !slots || !q_out || !k_pool || !v_pool || !k_exp || !v_exp ||
      (rot_dim > 0 && !inv_freq))
    return PA_EINVAL;
  const int64_t esize = dtype == PA_F32 ? 4 : 2;
  const int64_t q_row = (int64_t)num_qo_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (q_stride * esize > INT32_MAX || k_stride * esize > INT32_MAX || v_stride * esize > INT32_MAX)
    return PA_EUNSUPPORTED;
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride * esize % 16 || k_stride * esize % 16 ||
      v_stride * esize % 16)
    return PA_EINVAL;
  for (const void* x : {q, k, v, q_weight, k_weight, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (!on16(x)) return PA_EINVAL;
  AppendParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.q_out = q_out;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.k_exp = k_exp;
  p.v_exp = v_exp;
  p.status = status;
  p.num_rows = num_pages * page_size;
  p.eps = eps;
  p.tokens = num_tokens;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.rot = rot_dim;
  p.page_size = page_size;
  const FastDiv fd = FastDiv::make((uint32_t)page_size);
  p.ps_magic = fd.magic;
  p.ps_shift = fd.shift;
  const FastDiv fr = FastDiv::make((uint32_t)(rot_dim > 0 ? rot_dim / 2 : 1));
  p.half_magic = fr.magic;
  p.half_shift = fr.shift;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  // Stretches of as many tokens as leave two CTAs an SM for them all, a stretch's heads shared out in eights: with shorter
  // ones a CTA's begin, a few loads one after the other, is most of its time (2048 tokens 19.1 us, with a third of the
  // tokens 20.4), with longer ones runs wait behind one another (1024 requests of one token 20.3 us, twice the tokens 36).
  // For q as many warps as are resident, or, while the tokens alone do not give them work, several to a token.
  const int per = num_tokens / (kApCtas * sms);
  p.kv_splits = (2 * num_kv_heads + kApWarps - 1) / kApWarps;
  p.stretch = (int)std::min<int64_t>(std::max<int64_t>((int64_t)num_tokens * p.kv_splits / (2 * sms), 1), kApStretch);
  const int stretches = (num_tokens + p.stretch - 1) / p.stretch;
  const int kv_ctas = stretches * p.kv_splits;
  // With many tokens q's CTAs come first and leave a third of each SM to the stretches', which wait for their data most of
  // the time, so that the two run side by side (16384 tokens 78 us; q last and on all of the SM 84); with few the
  // stretches, which take longest, come first (777 tokens 6.4 us, last 8.0).
  const bool q_first = per >= kApStretch;
  const int q_most = (q_first ? kApCtas - 1 : kApCtas) * sms;
  const int resident = q_most * kApWarps, share = 4;  // heads that are worth a warp
  p.q_splits = num_tokens < resident ? std::min(resident / num_tokens, (num_qo_heads + share - 1) / share) : 1;
  p.q_share = (num_qo_heads + p.q_splits - 1) / p.q_splits;
  p.q_splits = (num_qo_heads + p.q_share - 1) / p.q_share;
  p.q_ctas = (int)std::min<int64_t>(q_most, ((int64_t)num_tokens * p.q_splits + kApWarps - 1) / kApWarps);
  p.q_warps = p.q_ctas * kApWarps;
  p.q_from = q_first ? 0 : kv_ctas;
  const bool paired = !interleaved, q32 = q_dtype == PA_F32;
  const AppendKernel fn =
      dtype == PA_F32   ? pick_append<float, float>(head_dim, paired)
      : dtype == PA_F16 ? (q32 ? pick_append<__half, float>(head_dim, paired) : pick_append<__half, __half>(head_dim, paired))
                        : (q32 ? pick_append<__nv_bfloat16, float>(head_dim, paired)
                               : pick_append<__nv_bfloat16, __nv_bfloat16>(head_dim, paired));
  const size_t most = (size_t)kApMaxPage * 2 * (head_dim / 2) * sizeof(float);
  if (!prepare_kernel(reinterpret_cast<const void*>(fn), most)) return PA_ECUDA;
  const size_t smem = (size_t)page_size * rot_dim * sizeof(float);
  const cudaError_t rc = launch_dependent(fn, dim3((unsigned)(kv_ctas + p.q_ctas)), dim3(kApThreads), smem,
                                          static_cast<cudaStream_t>(cuda_stream), p);
  if (rc != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
