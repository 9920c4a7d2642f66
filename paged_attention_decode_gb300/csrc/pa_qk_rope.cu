// pa_qk_rope.cu -- pa_v2_qk_rope_append: per-head norm of q and k, rotation by
// position, and the append of k and v to the paged pools, in one pass.
//
//   norm      x <- x * w / sqrt(mean(x^2) + eps)                (f32)
//   rotation  (x, y) <- (x cos a - y sin a, y cos a + x sin a),  a_j = pos * inv_freq[j]
//
// The angle is reduced in 64 bits before the sine is taken: pos * inv_freq in
// turns, minus its nearest integer, leaves a fraction of a turn that f32 holds
// to 2^-25, so a position of a million costs no accuracy (in f32 the product
// alone would be off by 0.06 radians there).
//
// One CTA per token.  A head's row is read as 16-byte pieces, one per lane, so
// a row takes head_dim / (16 / esize) lanes and the CTA's lanes hold several
// heads at once; a lane keeps the same place in the row for every head, so its
// cosines and sines are read once from shared memory, where the token's angles
// were computed once for all heads.  Half-split pairs sit (rot_dim / 2)
// elements apart, a whole number of lanes (rot_dim is a multiple of 16), and
// meet through one shuffle per element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kQkThreads = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

struct QkParams {
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
  void* k_pool;
  void* v_pool;
  int32_t* status;
  int64_t num_rows;  // pool rows
  float eps;
  int32_t hq, hkv, rot, interleaved;
};

// 16 bytes of T as floats, and back.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  __device__ __forceinline__ static uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Vec<__half> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Cosine and sine of pos * inv_freq radians.
__device__ __forceinline__ float2 rotation(int32_t pos, float inv_freq) {
  double turns = (double)pos * ((double)inv_freq * kInvTwoPi);
  turns -= rint(turns);
  float s, c;
  sincospif(2.0f * (float)turns, &s, &c);
  return make_float2(c, s);
}

template <typename T, typename TQ, int D>
__global__ void __launch_bounds__(kQkThreads) pa_v2_qk_rope_append_kernel(const QkParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int kLanes = D / N;                    // lanes per head row (8, 16 or 32)
  constexpr int kRows = kQkThreads / kLanes;       // head rows in flight per CTA
  __shared__ float2 cs[D / 2];

  pdl_launch_dependents();
  pdl_wait_prerequisites();

  const int t = blockIdx.x;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.num_rows) {  // padding, or a slot outside the pools
    if (slot >= p.num_rows && threadIdx.x == 0) report(p.status, PA_DEVICE_BAD_SLOT);
    return;
  }
  const int half = p.rot / 2;
  if ((int)threadIdx.x < half) cs[threadIdx.x] = rotation(p.positions[t], p.inv_freq[threadIdx.x]);
  __syncthreads();

  const int lane = threadIdx.x & (kLanes - 1);     // place in the row
  const int e0 = lane * N;
  const bool rotated = e0 < p.rot;                 // rot is a multiple of 2 N or of N: never inside a lane's piece
  const int hl = half / N;                         // lanes between the halves of a pair
  float2 r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r[i] = make_float2(1.f, 0.f);
    if (rotated) r[i] = p.interleaved ? cs[(e0 + i) >> 1] : cs[(e0 + i) < half ? e0 + i : e0 + i - half];
  }
  const bool upper = !p.interleaved && e0 >= half;

  const int heads = p.hq + 2 * p.hkv;
  for (int h0 = 0; h0 < heads; h0 += kRows) {
    const int h = h0 + (int)threadIdx.x / kLanes;
    const bool live = h < heads;
    const int kind = h < p.hq ? 0 : h < p.hq + p.hkv ? 1 : 2;  // q, k, v
    const int hh = kind == 0 ? h : kind == 1 ? h - p.hq : h - p.hq - p.hkv;
    const T* src = kind == 0   ? static_cast<const T*>(p.q) + t * p.q_stride
                   : kind == 1 ? static_cast<const T*>(p.k) + t * p.k_stride
                               : static_cast<const T*>(p.v) + t * p.v_stride;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(src + (int64_t)hh * D + e0);
    float x[N];
    Vec<T>::unpack(raw, x);
    // norm: every lane of the warp takes part in the shuffles, whatever its head's kind
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int w = kLanes / 2; w >= 1; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
    const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
    if (live && weight) {
      const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
      float g[N];
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(weight + e0), g);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = x[i] * inv * g[i];
    }
    if (p.rot > 0) {
      float y[N];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = x[i ^ 1];
      } else {
        const int warp_lane = threadIdx.x & 31;
        const int from = rotated ? (upper ? warp_lane - hl : warp_lane + hl) : warp_lane;
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
      }
      if (kind < 2 && rotated) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          // first of a pair: x cos - y sin; second: x cos + y sin (y its partner)
          const bool second = p.interleaved ? (i & 1) : upper;
          x[i] = fmaf(second ? y[i] : -y[i], r[i].y, x[i] * r[i].x);
        }
      }
    }
    if (!live) continue;
    if (kind == 0) {
      TQ* dst = static_cast<TQ*>(p.q_out) + ((int64_t)t * p.hq + hh) * D + e0;
#pragma unroll
      for (int j = 0; j < N / Vec<TQ>::N; ++j) {
        float z[Vec<TQ>::N];
#pragma unroll
        for (int i = 0; i < Vec<TQ>::N; ++i) z[i] = x[j * Vec<TQ>::N + i];
        reinterpret_cast<uint4*>(dst)[j] = Vec<TQ>::pack(z);
      }
    } else {
      T* pool = static_cast<T*>(kind == 1 ? p.k_pool : p.v_pool);
      *reinterpret_cast<uint4*>(pool + (slot * p.hkv + hh) * D + e0) = kind == 1 ? Vec<T>::pack(x) : raw;
    }
  }
}

using QkKernel = void (*)(const QkParams);

template <typename T>
QkKernel pick(int D, bool q32) {
  if (D == 64) return q32 ? pa_v2_qk_rope_append_kernel<T, float, 64> : pa_v2_qk_rope_append_kernel<T, T, 64>;
  return q32 ? pa_v2_qk_rope_append_kernel<T, float, 128> : pa_v2_qk_rope_append_kernel<T, T, 128>;
}

bool aligned(const void* x, int64_t a) { return reinterpret_cast<uintptr_t>(x) % a == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_qk_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                          const void* v, int64_t v_stride, int32_t dtype, int32_t num_tokens,
                                          int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                          const int32_t* positions, const int32_t* slots, const float* inv_freq,
                                          int32_t rot_dim, int32_t interleaved, const void* q_weight,
                                          const void* k_weight, float eps, void* q_out, int32_t q_dtype,
                                          void* k_pool, void* v_pool, int64_t num_pages, int32_t page_size,
                                          int32_t* status, void* cuda_stream) {
  if (num_tokens < 0 || num_qo_heads < 1 || num_kv_heads < 1 || rot_dim < 0 || num_pages < 1 || page_size < 1 ||
      !std::isfinite(eps) || eps < 0.f)
    return PA_EINVAL;
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return PA_EUNSUPPORTED;
  if (q_dtype != dtype && q_dtype != PA_F32) return PA_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  if (rot_dim > head_dim || rot_dim % 16 != 0) return PA_EUNSUPPORTED;
  if (num_qo_heads > 65536 || num_kv_heads > 65536) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !positions || !slots || !q_out || !k_pool || !v_pool || (rot_dim > 0 && !inv_freq))
    return PA_EINVAL;
  const int64_t esize = dtype == PA_F32 ? 4 : 2;
  const int64_t q_row = (int64_t)num_qo_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride * esize % 16 || k_stride * esize % 16 ||
      v_stride * esize % 16)
    return PA_EINVAL;
  for (const void* x : {q, k, v, q_weight, k_weight, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (!pa::aligned(x, 16)) return PA_EINVAL;
  pa::QkParams p;
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
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.status = status;
  p.num_rows = num_pages * page_size;
  p.eps = eps;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.rot = rot_dim;
  p.interleaved = interleaved ? 1 : 0;
  const bool q32 = q_dtype == PA_F32;
  const pa::QkKernel fn = dtype == PA_F32   ? pa::pick<float>(head_dim, true)
                          : dtype == PA_F16 ? pa::pick<__half>(head_dim, q32)
                                            : pa::pick<__nv_bfloat16>(head_dim, q32);
  const cudaError_t rc = pa::launch_dependent(fn, dim3(num_tokens), dim3(pa::kQkThreads), 0,
                                              static_cast<cudaStream_t>(cuda_stream), p);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
