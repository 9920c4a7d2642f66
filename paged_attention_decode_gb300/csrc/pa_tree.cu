// pa_tree.cu -- pa_v2_tree_attention, its _sliding and _sinks forms and its
// workspace: argument checks and launches of the kernels in pa_tree_body.cuh (those
// without a window are compiled here).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa_launch.h"
#include "pa_pool_map.h"
#include "pa_tree_body.cuh"

namespace pa {
namespace {

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

using MergeKernel = void (*)(const TreeParams);

int64_t slots_bytes(int32_t ctas, int32_t head_dim) {
  return (int64_t)ctas * kTrSlots * (int64_t)sizeof(float) *
         (head_dim == 64 ? TreeCfg<64>::kSlotFloats : TreeCfg<128>::kSlotFloats);
}

// CTAs of the attention kernel: one per SM.
pa_status tree_ctas(int32_t device, int32_t* ctas) {
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  *ctas = sms;
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_tree_attention_workspace(int32_t device, int32_t num_tokens, int32_t batch,
                                                    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                                    int64_t* bytes) {
  if (!bytes || device < 0 || num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads)
    return PA_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  int32_t ctas = 0;
  const pa_status rc = pa::tree_ctas(device, &ctas);
  if (rc != PA_OK) return rc;
  *bytes = pa::slots_bytes(ctas, head_dim) + ctas * (int64_t)sizeof(pa::TreeFold);
  return PA_OK;
}

namespace pa {

pa_status tree_attention(const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype, int64_t num_pages,
                         int32_t page_size, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                         const int32_t* indices, int64_t num_indices, const int32_t* indptr,
                         const int32_t* last_page_len, const int32_t* first_page_offset, int32_t batch,
                         const int32_t* qo_indptr, int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
                         const int32_t* positions, int32_t window, int32_t sinks, float sm_scale, void* out,
                         float* lse2_out, void* workspace, int64_t workspace_bytes, int32_t* status,
                         void* cuda_stream) {
  if (num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads || page_size < 1 || num_pages < 1 || num_indices < 0 || mask_words < 0 ||
      (tree_mask && mask_words < 1) || !std::isfinite(sm_scale))
    return PA_EINVAL;
  if (kv_dtype != PA_F16 && kv_dtype != PA_BF16) return PA_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  if (page_size > 256 || (page_size > 16 && page_size % 16 != 0)) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (tree_mask && mask_words > PA_V2_MAX_MASK_WORDS) return PA_EUNSUPPORTED;
  const float scale_log2 = std::fabs(sm_scale) * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return PA_EUNSUPPORTED;  // times a score of 0 it would be NaN
  if ((int64_t)num_tokens * (num_qo_heads / num_kv_heads) > INT32_MAX - 2 * kTrBlock) return PA_EUNSUPPORTED;
  if (num_tokens == 0 || batch == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !indptr || !last_page_len || !first_page_offset || !qo_indptr || !out ||
      !lse2_out || !workspace || (num_indices > 0 && !indices) || (window > 0 && !positions))
    return PA_EINVAL;
  for (const void* x : {q, k_pool, v_pool, static_cast<const void*>(out), static_cast<const void*>(workspace)})
    if (!aligned16(x)) return PA_EINVAL;
  int dev = 0;
  int64_t need = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
  const pa_status ws = pa_v2_tree_attention_workspace(dev, num_tokens, batch, num_qo_heads, num_kv_heads, head_dim,
                                                      &need);
  if (ws != PA_OK) return ws;
  if (workspace_bytes < need) return PA_ECAPACITY;
  alignas(64) CUtensorMap tm_k, tm_v;
  std::memset(&tm_k, 0, sizeof(tm_k));
  std::memset(&tm_v, 0, sizeof(tm_v));
  const bool tma = tc_uses_tma(page_size);
  int box_rows = 8;  // rows of a TMA box: the largest power of two that divides a page, up to a whole tile
  while (box_rows < kTrTile && page_size % (2 * box_rows) == 0) box_rows *= 2;
  if (tma) {
    if (!make_pool_map(&tm_k, k_pool, kv_dtype, num_pages * page_size, num_kv_heads, head_dim, 64, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_pool_map(&tm_v, v_pool, kv_dtype, num_pages * page_size, num_kv_heads, head_dim, 64, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B))
      return PA_ECUDA;
  }
  TreeParams p;
  std::memset(&p, 0, sizeof(p));
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
  p.slots = static_cast<float*>(workspace);
  p.status = status;
  p.num_pages = num_pages;
  p.num_indices = num_indices;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.positions = positions;
  p.window = window;
  p.sinks = sinks;
  p.sink_tiles = (int32_t)(((int64_t)sinks + kTrTile - 1) / kTrTile);
  p.mask_words = mask_words;
  p.page_size = page_size;
  p.box_rows = box_rows;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.group = num_qo_heads / num_kv_heads;
  const pa_status sm = tree_ctas(dev, &p.ctas);
  if (sm != PA_OK) return sm;
  p.folds = reinterpret_cast<TreeFold*>(static_cast<char*>(workspace) + slots_bytes(p.ctas, head_dim));
  const FastDiv fd = FastDiv::make((uint32_t)page_size), fg = FastDiv::make((uint32_t)p.group);
  p.ps_magic = fd.magic;
  p.ps_shift = fd.shift;
  p.g_magic = fg.magic;
  p.g_shift = fg.shift;
  // the work's units at most, for tables that list every page and token once: every block of the batch against every
  // key tile.  The blocks' starting costs are at most 6 / batch times that, and a broken table can claim all of it
  // again for each of 32 requests: (32 + 6) * 2^25 still fits 31 bits.
  const double units = ((double)num_indices * page_size / kTrTile + 2.0 * batch) *
                       ((double)num_tokens * p.group / kTrBlock + batch) * num_kv_heads;
  p.small = batch <= 32 && units < (double)(1 << 25);
  const bool flat = sm_scale == 0.f;  // every score is zero, behind a mask's -inf too, where 0 times it is NaN
  p.scale_log2 = flat ? 1.f : scale_log2;
  p.q_xor = sm_scale < 0.f ? 0x80008000u : 0u;
  p.q_and = flat ? 0u : 0xffffffffu;
  const bool f16 = kv_dtype == PA_F16;
  const int smem = head_dim == 64 ? TreeCfg<64>::kSmemAlloc : TreeCfg<128>::kSmemAlloc;
  const int win = sinks > 0 ? kSinks : window > 0 ? kWindow : kNoWindow;
  const TreeKernel fn = win == kSinks    ? tree_kernel_sinks(f16, head_dim, tma)
                        : win == kWindow ? tree_kernel_window(f16, head_dim, tma)
                                         : pick_tree<kNoWindow>(f16, head_dim, tma);
  if (!prepare_kernel(reinterpret_cast<const void*>(fn), smem)) return PA_ECUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  // Not a programmatic dependent: its CTAs want an SM each, and taking the SMs as the kernel before it frees them puts
  // the blocks that share keys far apart (16 ragged requests behind the q/k preparation: a step of 128 us, 150 with
  // the early launch).
  fn<<<dim3(p.ctas), dim3(kTrThreads), smem, stream>>>(p, tm_k, tm_v);
  if (cudaGetLastError() != cudaSuccess) return PA_ECUDA;
  const MergeKernel merge =
      f16 ? (head_dim == 64 ? pa_v2_tree_merge_kernel<__half, 64> : pa_v2_tree_merge_kernel<__half, 128>)
          : (head_dim == 64 ? pa_v2_tree_merge_kernel<__nv_bfloat16, 64>
                            : pa_v2_tree_merge_kernel<__nv_bfloat16, 128>);
  if (p.ctas > 1) {
    const cudaError_t rc = launch_dependent(merge, dim3(p.ctas, 4), dim3(kMergeThreads), 0, stream, p);
    if (rc != cudaSuccess) {
      cudaGetLastError();
      return PA_ECUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // namespace pa

extern "C" pa_status pa_v2_tree_attention(const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype,
                                          int64_t num_pages, int32_t page_size, int32_t num_qo_heads,
                                          int32_t num_kv_heads, int32_t head_dim, const int32_t* indices,
                                          int64_t num_indices, const int32_t* indptr, const int32_t* last_page_len,
                                          const int32_t* first_page_offset, int32_t batch, const int32_t* qo_indptr,
                                          int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
                                          float sm_scale, void* out, float* lse2_out, void* workspace,
                                          int64_t workspace_bytes, int32_t* status, void* cuda_stream) {
  return pa::tree_attention(q, k_pool, v_pool, kv_dtype, num_pages, page_size, num_qo_heads, num_kv_heads, head_dim,
                            indices, num_indices, indptr, last_page_len, first_page_offset, batch, qo_indptr,
                            num_tokens, tree_mask, mask_words, nullptr, 0, 0, sm_scale, out, lse2_out, workspace,
                            workspace_bytes, status, cuda_stream);
}

extern "C" pa_status pa_v2_tree_attention_sliding(
    const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype, int64_t num_pages, int32_t page_size,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, const int32_t* indices, int64_t num_indices,
    const int32_t* indptr, const int32_t* last_page_len, const int32_t* first_page_offset, int32_t batch,
    const int32_t* qo_indptr, int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
    const int32_t* positions, int32_t window, float sm_scale, void* out, float* lse2_out, void* workspace,
    int64_t workspace_bytes, int32_t* status, void* cuda_stream) {
  if (window < 1) return PA_EINVAL;
  return pa::tree_attention(q, k_pool, v_pool, kv_dtype, num_pages, page_size, num_qo_heads, num_kv_heads, head_dim,
                            indices, num_indices, indptr, last_page_len, first_page_offset, batch, qo_indptr,
                            num_tokens, tree_mask, mask_words, positions, window, 0, sm_scale, out, lse2_out,
                            workspace, workspace_bytes, status, cuda_stream);
}

extern "C" pa_status pa_v2_tree_attention_sinks(
    const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype, int64_t num_pages, int32_t page_size,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, const int32_t* indices, int64_t num_indices,
    const int32_t* indptr, const int32_t* last_page_len, const int32_t* first_page_offset, int32_t batch,
    const int32_t* qo_indptr, int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
    const int32_t* positions, int32_t window, int32_t sinks, float sm_scale, void* out, float* lse2_out,
    void* workspace, int64_t workspace_bytes, int32_t* status, void* cuda_stream) {
  if (window < 1 || sinks < 1) return PA_EINVAL;
  return pa::tree_attention(q, k_pool, v_pool, kv_dtype, num_pages, page_size, num_qo_heads, num_kv_heads, head_dim,
                            indices, num_indices, indptr, last_page_len, first_page_offset, batch, qo_indptr,
                            num_tokens, tree_mask, mask_words, positions, window, sinks, sm_scale, out, lse2_out,
                            workspace, workspace_bytes, status, cuda_stream);
}
