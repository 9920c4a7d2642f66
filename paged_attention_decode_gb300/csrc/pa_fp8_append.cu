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
// launch, the same result in every call.  Where the exponent of a begun page grows, that
// warp also rescales the page's earlier codes.  A code is a 4-bit number times a power of
// two, so that step is exact except for codes that turn subnormal.
//
// HBM bound: q, k and v are read once and q_out and the codes written once.  The first CTAs
// take stretches of tokens and handle the runs that begin in theirs (a run's cosines
// and sines are computed once, for all heads); the others take q's rows.  Rows are held
// as in pa_qk_rope.cu: 16 bytes per lane in two pieces that hold both elements of each
// of the lane's pairs.  A run that fits a warp's registers (kHeld passes) is read once;
// a longer one is read again, out of L2, after its maximum is known.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.cuh"
#include "pa_mma.cuh"
#include "pa_rope.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kApThreads = 256;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApMaxPage = 256;
constexpr int kApStretch = 16;  // tokens of a CTA's stretch, at most
constexpr int kApQTile = 8;     // tokens of a q CTA, at most

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
  uint32_t ps_magic, ps_shift;
  int32_t stretch, kv_ctas, kv_splits;  // tokens per KV CTA, CTAs with runs, and CTAs that share a stretch's heads
  int32_t q_tile;
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
  // Norm (w non-null: weights as loaded) over the row's lanes, all of which call it.
  __device__ __forceinline__ static void norm(float (&x)[N], const uint4& w, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int s = kLanes / 2; s >= 1; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
    const float inv = rsqrtf(ss * (1.0f / D) + eps);
    float g[N];
    Vec<T>::unpack(w, g);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * inv * g[i];
  }
  // cs: cosines, then sines `half` floats behind (elements that are not rotated are left out of it: 0 times an
  // infinity next to them is NaN)
  __device__ __forceinline__ void rotate(float (&x)[N], const float* cs, int half) const {
    if (!rotated) return;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int a = PAIRED ? i : 2 * i, b = PAIRED ? i + P : 2 * i + 1;
      const float c = cs[pair0 + i], s = cs[half + pair0 + i];
      const float u = x[a], w = x[b];
      x[a] = fmaf(-w, s, u * c);
      x[b] = fmaf(u, s, w * c);
    }
  }
};

template <typename T, typename TQ, int D, bool PAIRED>
__global__ void __launch_bounds__(kApThreads, 2) pa_v2_qk_rope_append_fp8_kernel(const AppendParams p) {
  using R = Row<T, D, PAIRED>;
  constexpr int N = R::N, P = R::P, kLanes = R::kLanes, kAtOnce = R::kAtOnce;
  constexpr int kHeld = 64 / N;  // passes of a run that registers hold
  extern __shared__ float cs[];  // [tokens][2][rot / 2]: cosines, sines
  __shared__ uint64_t turns[D / 2];
  __shared__ int32_t slot_of[1 + kApStretch + kApMaxPage];  // from the token before the stretch on

  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2, sub = lane / kLanes;
  const R row(p.rot);
  for (int i = threadIdx.x; i < half; i += kApThreads) turns[i] = turn_of(p.inv_freq[i]);
  // cosines and sines of tokens [t0, t0 + n)
  auto angles = [&](int t0, int n) {
    for (int i = threadIdx.x; i < n * half; i += kApThreads) {
      const int tok = i / half, j = i - tok * half;
      const float2 r = rotation(p.positions[t0 + tok], turns[j]);
      cs[2 * half * tok + j] = r.x;
      cs[2 * half * tok + half + j] = r.y;
    }
  };

  if ((int)blockIdx.x >= p.kv_ctas) {
    // ------------------------------------------------------------------ q
    const int t0 = ((int)blockIdx.x - p.kv_ctas) * p.q_tile, n = min(p.q_tile, p.tokens - t0);
    const T* w = static_cast<const T*>(p.q_weight);
    const uint4 weight = w ? row.load(w) : make_uint4(0, 0, 0, 0);
    __syncthreads();
    angles(t0, n);
    __syncthreads();
    const int rows = n * p.hq;
    constexpr int kBatch = 4;  // rows under way per lane
    for (int base = warp * kAtOnce; base < rows; base += kBatch * kApWarps * kAtOnce) {
      uint4 raw[kBatch];
      int32_t tok[kBatch], head[kBatch];
      bool live[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = min(base + b * kApWarps * kAtOnce + sub, rows - 1);
        tok[b] = i / p.hq;
        head[b] = i - tok[b] * p.hq;
        const int32_t slot = __ldg(p.slots + t0 + tok[b]);
        live[b] = base + b * kApWarps * kAtOnce + sub < rows && slot >= 0 && slot < p.num_rows;
        raw[b] = row.load(static_cast<const T*>(p.q) + (int64_t)(t0 + tok[b]) * p.q_stride + head[b] * D);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float x[N];
        Vec<T>::unpack(raw[b], x);
        if (w) R::norm(x, weight, p.eps);
        row.rotate(x, cs + 2 * half * tok[b], half);
        if (!live[b]) continue;
        TQ* to = static_cast<TQ*>(p.q_out) + ((int64_t)(t0 + tok[b]) * p.hq + head[b]) * D;
        if (sizeof(TQ) != sizeof(T)) {  // f32 from 16 bits: a piece is 16 bytes
          *reinterpret_cast<float4*>(to + row.e0) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(to + row.e1) = make_float4(x[P], x[P + 1], x[N - 2], x[N - 1]);
        } else {
          const uint4 y = Vec<T>::pack(x);
          *reinterpret_cast<uint2*>(to + row.e0) = make_uint2(y.x, y.y);
          *reinterpret_cast<uint2*>(to + row.e1) = make_uint2(y.z, y.w);
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------------- k and v
  const int part = (int)blockIdx.x % p.kv_splits;
  const int w0 = (int)blockIdx.x / p.kv_splits * p.stretch, w1 = min(w0 + p.stretch, p.tokens);
  const int ahead = min(p.stretch + p.page_size, p.tokens - w0);
  for (int i = threadIdx.x; i < ahead + 1; i += kApThreads) {
    int32_t s = -1;
    if (w0 + i > 0) s = __ldg(p.slots + w0 - 1 + i);
    if (s >= p.num_rows) {
      if (i > 0 && i <= w1 - w0 && part == 0) report(p.status, PA_DEVICE_BAD_SLOT);
      s = -1;
    }
    slot_of[i] = s;
  }
  const T* kw = static_cast<const T*>(p.k_weight);
  const uint4 weight = kw ? row.load(kw) : make_uint4(0, 0, 0, 0);
  __syncthreads();
  auto page_of = [&](int i) -> int32_t {  // of slot_of[i], -1 for none
    const int32_t s = slot_of[i];
    return s < 0 ? -1 : (int32_t)fast_div((uint32_t)s, p.ps_magic, p.ps_shift);
  };
  for (int t = w0; t < w1; ++t) {
    const int at = t - w0 + 1;
    const int32_t page = page_of(at);
    if (page < 0 || page_of(at - 1) == page) continue;
    // the run: how many tokens, and the least entry
    int len = 1;
    while (len < p.page_size && at + len <= ahead && page_of(at + len) == page) ++len;
    int least = INT_MAX;
    for (int i = lane; i < len; i += 32) least = min(least, slot_of[at + i] - page * p.page_size);
    least = __reduce_min_sync(0xffffffffu, least);
    __syncthreads();  // the run before is done with its angles
    angles(t, len);
    __syncthreads();
    for (int task = part * kApWarps + warp; task < 2 * p.hkv; task += p.kv_splits * kApWarps) {
      const bool is_v = task >= p.hkv;
      const int head = is_v ? task - p.hkv : task;
      const T* src = static_cast<const T*>(is_v ? p.v : p.k) + (int64_t)t * (is_v ? p.v_stride : p.k_stride) + head * D;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      int8_t* exps = (is_v ? p.v_exp : p.k_exp) + (int64_t)page * p.hkv + head;
      uint8_t* pool = (is_v ? p.v_pool : p.k_pool) + head * D;
      const int64_t pitch = (int64_t)p.hkv * D;
      const int old = least > 0 ? min(max((int)*exps, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX) : 0;
      float x[kHeld][N];
      auto fetch = [&](int first) {  // tokens first .. of the run, normed and rotated
        uint4 raw[kHeld];
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          raw[b] = make_uint4(0, 0, 0, 0);
          if (first + b * kAtOnce < len) raw[b] = row.load(src + (int64_t)min(first + b * kAtOnce + sub, len - 1) * stride);
        }
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          if (first + b * kAtOnce >= len) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[b][i] = 0.f;
            continue;
          }
          Vec<T>::unpack(raw[b], x[b]);
          if (!is_v) {
            if (kw) R::norm(x[b], weight, p.eps);
            row.rotate(x[b], cs + 2 * half * min(first + b * kAtOnce + sub, len - 1), half);
          }
        }
      };
      float top = 0.f;
      for (int first = 0; first < len; first += kHeld * kAtOnce) {
        fetch(first);
#pragma unroll
        for (int b = 0; b < kHeld; ++b)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float a = fabsf(x[b][i]);
            if (a <= 3.402823466e38f) top = fmaxf(top, a);
          }
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      int e = top > 0.f ? exponent_for(top) : PA_V2_FP8_EXP_MIN;
      if (least > 0) {
        e = max(e, old);
        if (e > old) {  // the page's earlier tokens
          const __half2 f = __float2half2_rn(power2(old - e));
          constexpr int kChunks = D / 16;
          for (int i = lane; i < least * kChunks; i += 32) {
            uint4* at16 = reinterpret_cast<uint4*>(pool + ((int64_t)page * p.page_size + i / kChunks) * pitch) + i % kChunks;
            uint4 u = *at16;
            uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = rescaled((uint16_t)w[k], f) | rescaled((uint16_t)(w[k] >> 16), f) << 16;
            *at16 = u;
          }
        }
      }
      if (lane == 0) *exps = (int8_t)e;
      const float down = power2(-e);
      for (int first = 0; first < len; first += kHeld * kAtOnce) {
        if (len > kHeld * kAtOnce) fetch(first);
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
          const int i = first + b * kAtOnce + sub;
          if (i >= len) continue;
          uint8_t* to = pool + (int64_t)slot_of[at + i] * pitch;
          uint32_t y[N / 4];
#pragma unroll
          for (int k = 0; k < N; k += 4) {
            float z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = fabsf(x[b][k + j]) <= 3.402823466e38f ? x[b][k + j] * down : NAN;
            y[k / 4] = codes_of(z[0], z[1]) | codes_of(z[2], z[3]) << 16;
          }
          if (N == 8) {
            *reinterpret_cast<uint32_t*>(to + row.e0) = y[0];
            *reinterpret_cast<uint32_t*>(to + row.e1) = y[N / 4 - 1];
          } else {  // f32: two elements per piece
            *reinterpret_cast<uint16_t*>(to + row.e0) = (uint16_t)y[0];
            *reinterpret_cast<uint16_t*>(to + row.e1) = (uint16_t)(y[0] >> 16);
          }
        }
      }
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  // Stretches and q tiles: short enough that the CTAs fill the GPU, and, while the stretches alone do not, the heads of
  // one are shared out.
  const int per = num_tokens / (2 * sms);
  p.stretch = per < 1 ? 1 : per < kApStretch ? per : kApStretch;
  p.q_tile = per < 1 ? 1 : per < kApQTile ? per : kApQTile;
  const int stretches = (num_tokens + p.stretch - 1) / p.stretch;
  p.kv_splits = stretches < sms ? (2 * num_kv_heads + kApWarps - 1) / kApWarps : 1;
  if ((int64_t)stretches * p.kv_splits > INT32_MAX / 2) p.kv_splits = 1;
  p.kv_ctas = stretches * p.kv_splits;
  const int q_ctas = (num_tokens + p.q_tile - 1) / p.q_tile;
  const bool paired = !interleaved, q32 = q_dtype == PA_F32;
  const AppendKernel fn =
      dtype == PA_F32   ? pick_append<float, float>(head_dim, paired)
      : dtype == PA_F16 ? (q32 ? pick_append<__half, float>(head_dim, paired) : pick_append<__half, __half>(head_dim, paired))
                        : (q32 ? pick_append<__nv_bfloat16, float>(head_dim, paired)
                               : pick_append<__nv_bfloat16, __nv_bfloat16>(head_dim, paired));
  const size_t most = (size_t)kApMaxPage * 2 * (head_dim / 2) * sizeof(float);
  if (!prepare_kernel(reinterpret_cast<const void*>(fn), most)) return PA_ECUDA;
  const size_t smem = (size_t)(page_size > kApQTile ? page_size : kApQTile) * rot_dim * sizeof(float);
  const cudaError_t rc = launch_dependent(fn, dim3((unsigned)(p.kv_ctas + q_ctas)), dim3(kApThreads), smem,
                                          static_cast<cudaStream_t>(cuda_stream), p);
  if (rc != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
