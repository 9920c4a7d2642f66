// pa_tables.cu -- pa_v2_build_tables: the page table, slot map, positions and
// tree masks of one step, built on the device from the requests' lengths.
//
// With c cached and n new tokens, s = page_size, t = c + n (per request):
//   pages taken    ceil(t/s) - ceil(c/s), handed out from the free list in request order;
//   window         the last w = min(t, max(window, n)) tokens, from token t - w on; a sliding window of W: what
//                  the first new token sees, from token max(0, c + 1 - W) on (c - W without a new token);
//   page list      entries (that token)/s .. ceil(t/s)-1 of the request's block-table row;
//   token i        row page((c+i)/s) * s + (c+i) % s, position c + depth(i).
//
// Three prefix sums over the requests (pages listed, pages taken, new tokens)
// tie the requests together.  Every CTA computes them for itself in shared
// memory (12 bytes per request) and then fills its share of the outputs, so
// one launch does the whole step and no CTA waits for another: a page taken in
// this step is recomputed from its place in the free list wherever it is
// needed, instead of being read back from the block table that another CTA is
// writing.  Bound by latency (cold code, the lengths' load, the scan's barriers,
// the page ids' load, the walk up a tree) up to a few MB of page ids.  Replayed from
// a graph: 32 trees of 64 tokens, 9.4 us; 512 decode requests of 4K to 128K tokens
// (9 MB read and written, 1.4 us at the HBM rate), 10.0 us.  64-bit divisions by the
// page size, 64-bit sums and one-entry-per-thread copies of the page lists took 15
// and 19 us; every division is now a 32-bit product, the sums saturate instead, and
// a warp copies runs of 256 entries with all its loads in flight.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabRun = 256;  // page-list entries a warp copies at a time

struct TableParams {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  const int32_t* parents;
  int32_t* block_table;
  int32_t* indptr;
  int32_t* indices;
  int32_t* last_page_len;
  int32_t* first_page_offset;
  int32_t* qo_indptr;
  int32_t* slots;
  int32_t* positions;
  int32_t* tree_mask;
  int32_t* pages_needed;
  int32_t* status;
  int32_t batch, width, num_free, page_size, window, mask_words;
  int32_t reach;  // sliding window: what a token sees of its line of ancestors, itself included; else 0
  int32_t index_cap, token_cap;
  uint32_t ps_magic, ps_shift;
};

// One request's share of the step.
struct ReqGeom {
  int32_t cached;   // c
  int32_t tokens;   // n
  int32_t have;     // block-table entries filled before the step
  int32_t need;     // entries after it
  int32_t first;    // first entry of the visible window
  int32_t fpo, lpl;
  bool bad;         // lengths out of range: no pages, no slots
};

__device__ __forceinline__ int32_t pages_of(const TableParams& p, int32_t rows) {  // ceil(rows / page_size)
  return rows > 0 ? (int32_t)fast_div((uint32_t)(rows - 1), p.ps_magic, p.ps_shift) + 1 : 0;
}

__device__ __forceinline__ ReqGeom request_geom(const TableParams& p, int r) {
  ReqGeom g;
  const int32_t c = p.cached[r], n = p.fresh[r];
  g.cached = max(c, 0);
  g.tokens = max(n, 0);
  g.have = g.need = g.first = g.fpo = g.lpl = 0;
  g.bad = c < 0 || n < 0 || (int64_t)c + n > INT32_MAX;
  if (!g.bad) {
    const int32_t t = c + n;
    const int32_t need = pages_of(p, t);
    g.bad = need > p.width;
    if (!g.bad && t > 0) {
      const int32_t span = max(p.window, n);  // new tokens are always among the visible ones
      int32_t start = p.window > 0 && t > span ? t - span : 0;
      if (p.reach > 0) start = max(c + (n > 0 ? 1 : 0) - p.reach, 0);
      g.have = pages_of(p, c);
      g.need = need;
      g.first = (int32_t)fast_div((uint32_t)start, p.ps_magic, p.ps_shift);
      g.fpo = start - g.first * p.page_size;
      g.lpl = t - (need - 1) * p.page_size;
    }
  }
  return g;
}

// Sums that stop at the largest value: a batch may claim more tokens than fit.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? 0xffffffffu : s;
}

// Last r in [0, n) with a[r] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int last_le(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;  // a[lo] <= x, a[hi] > x (or hi == n)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Physical page of entry `col` of request r's block-table row after the step.
__device__ __forceinline__ int32_t page_at(const TableParams& p, const int32_t* taken, const ReqGeom& g, int r,
                                           int32_t col) {
  if (p.free_pages && col >= g.have) {
    const int64_t at = (int64_t)taken[r] + (col - g.have);
    return at < p.num_free ? p.free_pages[at] : -1;
  }
  return p.block_table[(int64_t)r * p.width + col];
}

__global__ void __launch_bounds__(kTabThreads) pa_v2_build_tables_kernel(const TableParams p) {
  extern __shared__ int32_t sm[];
  const int B = p.batch;
  int32_t* ip = sm;               // [B + 1] page-list prefix
  int32_t* taken = ip + B + 1;    // [B + 1] taken-page prefix
  int32_t* qo = taken + B + 1;    // [B + 1] token prefix, clamped to the capacity
  __shared__ uint32_t warp_sum[3][kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_launch_dependents();
  pdl_wait_prerequisites();

  // ---- the three prefix sums: each thread a run of consecutive requests
  const int per = (B + kTabThreads - 1) / kTabThreads;
  const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
  // (page counts fit: batch * width does)
  uint32_t sum[3] = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    const ReqGeom g = request_geom(p, r);
    if (g.bad && blockIdx.x == 0) report(p.status, PA_DEVICE_BAD_LENGTH);
    const int32_t pages = g.need - g.first, take = p.free_pages ? g.need - g.have : 0;
    ip[r] = pages;
    taken[r] = take;
    qo[r] = g.tokens;
    sum[0] += pages;
    sum[1] += take;
    sum[2] = add_sat(sum[2], g.tokens);
  }
  uint32_t before[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t v = __shfl_up_sync(0xffffffffu, sum[k], 1);
    if (lane == 0) v = 0;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, w);
      if (lane >= w) v = add_sat(v, u);
    }
    before[k] = v;
    if (lane == 31) warp_sum[k][warp] = add_sat(v, sum[k]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t earlier = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w)
      if (w < warp) earlier = add_sat(earlier, warp_sum[k][w]);
    before[k] = add_sat(earlier, before[k]);
  }
  const uint32_t cap = (uint32_t)p.token_cap;
  for (int r = r0; r < r1; ++r) {
    const int32_t pages = ip[r], take = taken[r], n = qo[r];
    ip[r] = (int32_t)before[0];
    taken[r] = (int32_t)before[1];
    qo[r] = (int32_t)min(before[2], cap);
    before[0] += pages;
    before[1] += take;
    before[2] = add_sat(before[2], n);
  }
  if (tid == kTabThreads - 1) {  // the last thread's runs end at B
    ip[B] = (int32_t)before[0];
    taken[B] = (int32_t)before[1];
    qo[B] = (int32_t)min(before[2], cap);
    if (blockIdx.x == 0) {
      if (before[2] > cap || before[0] > (uint32_t)p.index_cap) report(p.status, PA_DEVICE_BAD_LENGTH);
      if (p.free_pages && before[1] > (uint32_t)p.num_free) report(p.status, PA_DEVICE_NO_PAGES);
      *p.pages_needed = (int32_t)before[1];
    }
  }
  __syncthreads();

  const int64_t gthreads = (int64_t)gridDim.x * kTabThreads;
  const int64_t gtid = (int64_t)blockIdx.x * kTabThreads + tid;

  // ---- per request
  for (int64_t r = gtid; r <= B; r += gthreads) {
    p.indptr[r] = ip[r];
    p.qo_indptr[r] = qo[r];
    if (r < B) {
      const ReqGeom g = request_geom(p, (int)r);
      p.last_page_len[r] = g.lpl;
      p.first_page_offset[r] = g.fpo;
    }
  }

  // ---- pages taken from the free list, into the block table
  for (int64_t e = gtid; e < taken[B]; e += gthreads) {
    const int r = last_le(taken, B, (int32_t)e);
    const ReqGeom g = request_geom(p, r);
    const int32_t col = g.have + (int32_t)e - taken[r];
    p.block_table[(int64_t)r * p.width + col] = e < p.num_free ? p.free_pages[e] : -1;
  }

  // ---- page lists: a warp copies runs of kTabRun entries
  const int32_t n_idx = min(ip[B], p.index_cap);
  const int64_t gwarps = (int64_t)gridDim.x * (kTabThreads / 32);
  for (int64_t run = (int64_t)blockIdx.x * (kTabThreads / 32) + warp; run * kTabRun < n_idx; run += gwarps) {
    const int32_t i0 = (int32_t)(run * kTabRun);
    const int32_t end = (int32_t)min((run + 1) * (int64_t)kTabRun, (int64_t)n_idx);
    int r = last_le(ip, B, i0);
    ReqGeom g = request_geom(p, r);
    int32_t col = g.first + i0 - ip[r];
    if (end - i0 == kTabRun && end <= ip[r + 1] && (!p.free_pages || col + kTabRun <= g.have)) {
      // one request's old pages: a plain copy, all loads in flight at once
      const int32_t* src = p.block_table + (int64_t)r * p.width + col + lane;
      int32_t x[kTabRun / 32];
#pragma unroll
      for (int k = 0; k < kTabRun / 32; ++k) x[k] = src[32 * k];
#pragma unroll
      for (int k = 0; k < kTabRun / 32; ++k) p.indices[i0 + lane + 32 * k] = x[k];
      continue;
    }
    int32_t r_end = ip[r + 1];
    for (int32_t i = i0 + lane; i < end; i += 32) {
      if (i >= r_end) {
        r = last_le(ip, B, i);
        r_end = ip[r + 1];
        g = request_geom(p, r);
      }
      p.indices[i] = page_at(p, taken, g, r, g.first + i - ip[r]);
    }
  }

  // ---- tokens
  for (int64_t t = gtid; t < p.token_cap; t += gthreads) {
    if (t >= qo[B]) {
      p.slots[t] = -1;
      p.positions[t] = 0;
      continue;
    }
    const int r = last_le(qo, B, (int32_t)t);
    const ReqGeom g = request_geom(p, r);
    const int32_t base = qo[r];
    const int32_t i = (int32_t)t - base;
    int64_t slot = -1;
    if (!g.bad) {
      const int32_t at = g.cached + i;
      const int32_t entry = (int32_t)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
      const int32_t page = page_at(p, taken, g, r, entry);
      slot = (int64_t)page * p.page_size + (at - entry * p.page_size);
      if (page < 0 || slot > INT32_MAX) {
        slot = -1;
        report(p.status, page == -1 && p.free_pages ? PA_DEVICE_NO_PAGES : PA_DEVICE_BAD_PAGE);
      }
    }
    p.slots[t] = (int32_t)slot;
    // ancestors, from the token up: indices fall on the way, so the mask's words come out last to first
    int32_t depth = 0, word = p.mask_words;
    uint32_t bits = 0;
    const int32_t reach = p.reach > 0 ? p.reach : INT32_MAX;
    int32_t* row = p.tree_mask ? p.tree_mask + t * p.mask_words : nullptr;
    bool bad_tree = row && i >= 32 * p.mask_words;
    if (p.parents || row) {
      int32_t j = i;
      while (true) {
        const int32_t w = j >> 5;
        if (row && w < p.mask_words && depth < reach) {
          while (word > w) {
            if (word < p.mask_words) row[word] = (int32_t)bits;
            bits = 0;
            --word;
          }
          bits |= 1u << (j & 31);
        }
        int32_t up = j - 1;
        if (p.parents) {
          up = p.parents[base + j];
          if (up < -1 || up >= j) {
            bad_tree = true;
            up = -1;
          }
        }
        if (up < 0) break;
        ++depth;
        j = up;
      }
      while (row && word > 0) {
        if (word < p.mask_words) row[word] = (int32_t)bits;
        bits = 0;
        --word;
      }
      if (row) row[0] = (int32_t)bits;
    } else {
      depth = i;
    }
    if (bad_tree) report(p.status, PA_DEVICE_BAD_TREE);
    p.positions[t] = g.bad ? 0 : g.cached + depth;
  }
}

pa_status build_tables(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch, int32_t* block_table,
                       int32_t table_width, const int32_t* free_pages, int32_t num_free, const int32_t* parents,
                       int32_t page_size, int32_t window, int32_t reach, int32_t* indptr, int32_t* indices,
                       int64_t index_capacity, int32_t* last_page_len, int32_t* first_page_offset,
                       int32_t* qo_indptr, int32_t* slots, int32_t* positions, int64_t token_capacity,
                       int32_t* tree_mask, int32_t mask_words, int32_t* pages_needed, int32_t* status,
                       void* cuda_stream) {
  if (batch < 0 || table_width < 0 || num_free < 0 || page_size < 1 || window < 0 || index_capacity < 0 ||
      token_capacity < 0 || mask_words < 0 || !indptr || !qo_indptr || !pages_needed)
    return PA_EINVAL;
  if (batch > 0 && (!cached_lens || !new_lens || !last_page_len || !first_page_offset)) return PA_EINVAL;
  if ((batch > 0 && table_width > 0 && !block_table) || (index_capacity > 0 && !indices)) return PA_EINVAL;
  if (token_capacity > 0 && (!slots || !positions)) return PA_EINVAL;
  if (tree_mask && mask_words < 1) return PA_EINVAL;
  if (batch > PA_V2_MAX_TABLE_BATCH || (int64_t)batch * table_width > INT32_MAX || index_capacity > INT32_MAX ||
      token_capacity > INT32_MAX || token_capacity * mask_words > INT32_MAX)
    return PA_EUNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ECUDA;
  TableParams p;
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.free_pages = free_pages;
  p.parents = parents;
  p.block_table = block_table;
  p.indptr = indptr;
  p.indices = indices;
  p.last_page_len = last_page_len;
  p.first_page_offset = first_page_offset;
  p.qo_indptr = qo_indptr;
  p.slots = slots;
  p.positions = positions;
  p.tree_mask = tree_mask;
  p.pages_needed = pages_needed;
  p.status = status;
  p.batch = batch;
  p.width = table_width;
  p.num_free = num_free;
  p.page_size = page_size;
  p.window = window;
  p.reach = reach;
  p.mask_words = mask_words;
  p.index_cap = (int32_t)index_capacity;
  p.token_cap = (int32_t)token_capacity;
  const FastDiv fd = FastDiv::make((uint32_t)page_size);
  p.ps_magic = fd.magic;
  p.ps_shift = fd.shift;
  const size_t smem = 3 * ((size_t)batch + 1) * sizeof(int32_t);
  constexpr size_t kMaxSmem = 3 * (PA_V2_MAX_TABLE_BATCH + 1) * sizeof(int32_t);
  if (!prepare_kernel(reinterpret_cast<const void*>(pa_v2_build_tables_kernel), kMaxSmem)) return PA_ECUDA;
  const int64_t work = index_capacity / 8 > token_capacity ? index_capacity / 8 : token_capacity;
  const int64_t want = (work + kTabThreads - 1) / kTabThreads;
  const int blocks = (int)(want < 1 ? 1 : want < sms ? want : sms);
  const cudaError_t rc = launch_dependent(pa_v2_build_tables_kernel, dim3(blocks), dim3(kTabThreads), smem,
                                          static_cast<cudaStream_t>(cuda_stream), p);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_build_tables(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch,
                                        int32_t* block_table, int32_t table_width, const int32_t* free_pages,
                                        int32_t num_free, const int32_t* parents, int32_t page_size, int32_t window,
                                        int32_t* indptr, int32_t* indices, int64_t index_capacity,
                                        int32_t* last_page_len, int32_t* first_page_offset, int32_t* qo_indptr,
                                        int32_t* slots, int32_t* positions, int64_t token_capacity,
                                        int32_t* tree_mask, int32_t mask_words, int32_t* pages_needed,
                                        int32_t* status, void* cuda_stream) {
  return pa::build_tables(cached_lens, new_lens, batch, block_table, table_width, free_pages, num_free, parents,
                          page_size, window, 0, indptr, indices, index_capacity, last_page_len, first_page_offset,
                          qo_indptr, slots, positions, token_capacity, tree_mask, mask_words, pages_needed, status,
                          cuda_stream);
}

extern "C" pa_status pa_v2_build_tables_sliding(
    const int32_t* cached_lens, const int32_t* new_lens, int32_t batch, int32_t* block_table, int32_t table_width,
    const int32_t* free_pages, int32_t num_free, const int32_t* parents, int32_t page_size, int32_t window,
    int32_t* indptr, int32_t* indices, int64_t index_capacity, int32_t* last_page_len, int32_t* first_page_offset,
    int32_t* qo_indptr, int32_t* slots, int32_t* positions, int64_t token_capacity, int32_t* tree_mask,
    int32_t mask_words, int32_t* pages_needed, int32_t* status, void* cuda_stream) {
  if (window < 1) return PA_EINVAL;
  return pa::build_tables(cached_lens, new_lens, batch, block_table, table_width, free_pages, num_free, parents,
                          page_size, 0, window, indptr, indices, index_capacity, last_page_len, first_page_offset,
                          qo_indptr, slots, positions, token_capacity, tree_mask, mask_words, pages_needed, status,
                          cuda_stream);
}
