// pa_tree.cu -- pa_v2_tree_attention: attention of several query tokens per
// request (a tree or a chain of new tokens) over the paged cache.
//
// Query token i of request r sees the L - n earlier visible tokens and the new
// tokens its mask row (or the chain rule j <= i) allows:
//   s = scale * q . k,  out = sum 2^(s' - m) v / sum 2^(s' - m),  s' = s * log2(e),
// one pass with a running maximum m and sum, all in f32.
//
// One warp per (token, query head): a lane holds head_dim / 32 elements of q
// and of the accumulator, a key's score is one shuffle reduction.
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

struct TreeParams {
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* indices;
  const int32_t* indptr;
  const int32_t* last_page_len;
  const int32_t* first_page_offset;
  const int32_t* qo_indptr;
  const int32_t* tree_mask;
  void* out;
  float* lse_out;
  int32_t* status;
  int64_t num_pages, num_indices;
  int32_t batch, num_tokens, mask_words, page_size, hq, hkv, group;
  float scale_log2;
};

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, __half* y) { *y = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(128) pa_v2_tree_attention_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);  // token * hq + head
  const int t = (int)(row / p.hq), h = (int)(row % p.hq);
  if (t >= p.num_tokens) return;
  // the token's request
  int r = -1, t0 = 0, n = 0;
  for (int i = 0; i < p.batch; ++i) {
    const int a = p.qo_indptr[i], b = p.qo_indptr[i + 1];
    if (a < 0 || b < a || b > p.num_tokens) {
      if (lane == 0) report(p.status, PA_DEVICE_BAD_INDPTR);
      continue;
    }
    if (t >= a && t < b) {
      r = i;
      t0 = a;
      n = b - a;
      break;
    }
  }
  if (r < 0) return;
  const int64_t base = p.indptr[r];
  const int64_t pages = (int64_t)p.indptr[r + 1] - base;
  const int lpl = p.last_page_len[r], fpo = p.first_page_offset[r];
  int64_t seen = 0;
  bool bad = base < 0 || pages < 0 || base + pages > p.num_indices;
  if (bad) {
    if (lane == 0) report(p.status, PA_DEVICE_BAD_SLOT);
  } else {
    if (pages > 0) {
      seen = (pages - 1) * p.page_size + lpl - fpo;
      bad = lpl < 1 || lpl > p.page_size || fpo < 0 || fpo >= p.page_size || seen < 1;
    }
    if (bad || n > seen || (p.tree_mask && n > 32 * p.mask_words)) {
      bad = true;
      if (lane == 0) report(p.status, PA_DEVICE_BAD_TREE);
    }
  }
  const int kvh = h / p.group;
  const T* q = static_cast<const T*>(p.q) + row * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f32(q[e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t i = 0; !bad && i < seen; ++i) {
    const int64_t j = i - (seen - n);  // new-token index when >= 0
    if (j >= 0) {
      const bool sees = p.tree_mask ? (p.tree_mask[(int64_t)t * p.mask_words + (j >> 5)] >> (j & 31)) & 1 : j <= t - t0;
      if (!sees) continue;
    }
    const int32_t page = p.indices[base + (fpo + i) / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) report(p.status, PA_DEVICE_BAD_PAGE);
      continue;
    }
    const int64_t at = (((int64_t)page * p.page_size + (fpo + i) % p.page_size) * p.hkv + kvh) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], to_f32(static_cast<const T*>(p.k_pool)[at + e]), s);
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float c = fast_exp2(m - mu), pr = fast_exp2(s - mu);
    l = l * c + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + pr * to_f32(static_cast<const T*>(p.v_pool)[at + e]);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + row * D + lane * E;
  const bool empty = l == 0.f;  // nothing visible (a NaN sum stays NaN)
#pragma unroll
  for (int e = 0; e < E; ++e) from_f32(empty ? 0.f : acc[e] / l, out + e);
  if (lane == 0) p.lse_out[row] = empty ? -INFINITY : m + fast_log2(l);
}

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_tree_attention_workspace(int32_t device, int32_t num_tokens, int32_t batch,
                                                    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                                    int64_t* bytes) {
  if (!bytes || device < 0 || num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads)
    return PA_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  *bytes = 32;
  return PA_OK;
}

extern "C" pa_status pa_v2_tree_attention(const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype,
                                          int64_t num_pages, int32_t page_size, int32_t num_qo_heads,
                                          int32_t num_kv_heads, int32_t head_dim, const int32_t* indices,
                                          int64_t num_indices, const int32_t* indptr, const int32_t* last_page_len,
                                          const int32_t* first_page_offset, int32_t batch, const int32_t* qo_indptr,
                                          int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
                                          float sm_scale, void* out, float* lse2_out, void* workspace,
                                          int64_t workspace_bytes, int32_t* status, void* cuda_stream) {
  if (num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads || page_size < 1 || num_pages < 1 || num_indices < 0 || mask_words < 0 ||
      (tree_mask && mask_words < 1) || !std::isfinite(sm_scale))
    return PA_EINVAL;
  if (kv_dtype != PA_F16 && kv_dtype != PA_BF16) return PA_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  if (page_size > 256 || (page_size > 16 && page_size % 16 != 0)) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (tree_mask && mask_words > PA_V2_MAX_MASK_WORDS) return PA_EUNSUPPORTED;
  if (num_tokens == 0 || batch == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !indptr || !last_page_len || !first_page_offset || !qo_indptr || !out ||
      !lse2_out || !workspace || (num_indices > 0 && !indices))
    return PA_EINVAL;
  for (const void* x : {q, k_pool, v_pool, static_cast<const void*>(out), static_cast<const void*>(workspace)})
    if (!pa::aligned16(x)) return PA_EINVAL;
  int dev = 0;
  int64_t need = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
  const pa_status ws = pa_v2_tree_attention_workspace(dev, num_tokens, batch, num_qo_heads, num_kv_heads, head_dim,
                                                      &need);
  if (ws != PA_OK) return ws;
  if (workspace_bytes < need) return PA_ECAPACITY;
  pa::TreeParams p;
  p.q = q;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.indices = indices;
  p.indptr = indptr;
  p.last_page_len = last_page_len;
  p.first_page_offset = first_page_offset;
  p.qo_indptr = qo_indptr;
  p.tree_mask = tree_mask;
  p.out = out;
  p.lse_out = lse2_out;
  p.status = status;
  p.num_pages = num_pages;
  p.num_indices = num_indices;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.mask_words = mask_words;
  p.page_size = page_size;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.group = num_qo_heads / num_kv_heads;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  const int64_t rows = (int64_t)num_tokens * num_qo_heads;
  if ((rows + 3) / 4 > INT32_MAX) return PA_EUNSUPPORTED;
  void (*fn)(const pa::TreeParams) =
      kv_dtype == PA_F16
          ? (head_dim == 64 ? pa::pa_v2_tree_attention_kernel<__half, 64> : pa::pa_v2_tree_attention_kernel<__half, 128>)
          : (head_dim == 64 ? pa::pa_v2_tree_attention_kernel<__nv_bfloat16, 64>
                            : pa::pa_v2_tree_attention_kernel<__nv_bfloat16, 128>);
  const cudaError_t rc = pa::launch_dependent(fn, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0,
                                              static_cast<cudaStream_t>(cuda_stream), p);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
