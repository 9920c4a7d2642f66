// pa_tree.cu -- pa_v2_tree_attention: attention of several query tokens per
// request (a tree or a chain of new tokens) over the paged cache, on the
// fifth-generation tensor cores.
//
// Query token i of request r sees the L - n earlier visible tokens and the new
// tokens its mask row (or the chain rule j <= i) allows:
//   s = scale log2(e) q . k,  out = sum 2^(s - m) v / sum 2^(s - m),
// one pass over the keys with a running maximum m and sum in f32.  Under a sliding window
// of W a token at depth d below its request's first one sees of the earlier tokens the
// last W - 1 - d: the request's keys begin where its first token's window does, and up to
// where its last token's can begin each row has an edge of its own.
//
// Work.  The query rows of a KV head are its n * G (token, head) pairs; a block
// of up to 256 of them meets the request's keys in tiles of 128 pool rows (page
// order, so a tile is whole pages or whole slices of one).  One block against
// one tile is a unit, and every CTA (one per SM) gets the same number of them,
// `run`, whatever the lengths: no host plan, no wave tail.  A block's keys are
// cut into chunks of `run` tiles, one CTA each; what is left of the blocks (all
// of a short request) is strung together and dealt out in equal stretches to
// the other CTAs.  So the blocks of one request meet the same keys at the same
// time, out of L2, and a block costs one partial result more than it must.  A
// block that one CTA meets alone is written as the result; parts go to the
// workspace, and pa_v2_tree_merge_kernel folds them.
//
// A CTA holds a 256-row block as two M=128 tiles, A and B.  With 128 rows or
// fewer, A and B are the same rows against alternate key tiles (two streams,
// joined at the end), so that one stream's softmax always overlaps the other's
// products.  Roles (384 threads):
//  - warps 0-3 and 4-7: softmax of stream A and of B, one row per thread (S read
//    from tensor memory, P written back over it in the pool's 16-bit type, O
//    rescaled in place only when a row's maximum grows by more than kLazy);
//  - warp 8: one thread issues S = Q K^T (both operands in shared memory) and
//    O += P V (P in tensor memory);
//  - warps 9 and 10: load K and V tiles through a ring of shared-memory stages,
//    TMA boxes of 64 elements x the largest power of two of rows that divides a
//    page (K by warp 9, V by warp 10: issuing the 16 boxes of a tile of 16-row
//    pages takes a thread about 1000 cycles), or cp.async by both for page sizes
//    whose pages do not start on 8-row boundaries; both walk the CTA's share of
//    the work, and warp 9 hands its pieces to the other roles;
//  - warp 11: makes V tiles that hold rows outside the visible range, or rows that
//    not every new token sees, safe: 0 * NaN is NaN, so what a mask or a window hides
//    must not be left in V.  Outside rows become zeros; non-finite elements of the
//    others become zeros and are added back, in the epilogue, to the rows that do see
//    them.
//
// What bounds it.  A tile of two streams of 128 rows is 2500 cycles of products
// (S and PV, D = 128, at the cuBLAS burst rate) and, from HBM, 2900 cycles of K
// and V when nothing else reads them; it takes 3100-3250: a row's softmax (1550:
// reading S, the maximum, 128 exponentials, packing, writing P) and the PV and S
// products that need it and that it needs (1250) follow one another within a
// stream, and the other stream fills most of the gap.  Around the tiles stand 6 to
// 8 us of start (cold code, barriers, tensor memory, the cut, the page list, Q
// and the first K tile) and, after a cut block, 2-4 us of epilogue, 1.4 us between
// the kernels and 3-6 us of merge.  16 bits, 32 query heads on 8 KV heads, D = 128,
// replayed from a graph: 64 tokens over 32K 46.6 us (20 us of HBM reads), 4 x 256
// tokens over 32K 400 us (1.37 PFLOP/s of 1.92 measured with cuBLAS) at 2070 MHz
// and 440 where the power cap holds the clock at 1800, 16 ragged requests 100 us
// (4.4 TB/s), 32 chains of 5 tokens with a 4096-token window 73 us (5.2 TB/s), 8
// tokens over 1K 15.2 us (nearly all start and merge).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pa_internal.cuh"
#include "pa_mma.cuh"
#include "pa_pool_map.h"
#include "pa_tc05.cuh"

namespace pa {
namespace {

constexpr int kTrThreads = 384;
constexpr int kTrTile = 128;      // query rows of a tensor-core tile, and keys of a key tile
constexpr int kTrBlock = 256;     // query rows of a block
constexpr int kTrSlots = 2;       // partial results per CTA (see rest_slot)
// What starting on a left-over costs, in key tiles, for blocks of one and of two tiles of query rows: the result of the
// piece before written, Q fetched, the first tile's softmax and the edges of the request (5 to 7 us, about 1.5 us a
// tile), and, with two, keys that no CTA beside reads at the time.  Sweeps over 4 x 256 tokens and 64 tokens over 32K,
// 16 ragged requests and 32 windowed chains: 2 / 2 gives 493, 44.8, 136 and 92 us, 6 / 6 gives 436, 44.6, 105 and 80,
// 4 / 12 gives 400, 46.9, 99 and 72.5, 4 / 24 gives 415, 46.9, 104 and 72.6.  (D = 128; short contexts were not swept.)
constexpr int kTrCost1 = 4, kTrCost2 = 12;
constexpr int kTrMmaWarp = 8, kTrLoadWarp = 9, kTrFixWarp = 11;
constexpr int kTrLoadThreads = 64;  // loader threads without TMA
constexpr int kTrRing = 2;        // pieces handed out ahead
constexpr int kTrLag = 3;         // without TMA: loads in flight behind the newest (below kStages - 1)
constexpr int kMergeThreads = 256;

// Tensor-memory columns: S of both streams (P over its first 64), then O of both.
constexpr uint32_t kTrTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int w) { return 128u * w; }
__device__ __forceinline__ uint32_t col_o(int w) { return 256u + 128u * w; }

template <int D>
struct TreeCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTrTile * D * 2;
  // D = 128: all the shared memory that the Q tiles leave; D = 64: room for two more is left
  static constexpr int kStages = D == 128 ? 5 : 9;
  static constexpr int kOffKv = 2 * kTileBytes;     // Q tiles first
  static constexpr int kOffMisc = kOffKv + kStages * kTileBytes;
  static constexpr int kMisc = D == 128 ? 2048 : 4096;  // barriers, pieces, small exchanges
  static constexpr int kSmem = kOffMisc + kMisc;
  static constexpr int kSmemAlloc = kSmem + 1024;   // room to align the base
  static constexpr int64_t kSlotFloats = (int64_t)kTrBlock * (D + 1);
};

// P is rounded to 16 bits relative to 2^kShift at the row's offset, and the offset follows the running maximum
// with a lag of up to kLazy (log2 units).  bf16 has f32's range and takes a wide lag.  f16 holds nothing below
// 2^-24: the shift keeps weights down to 2^-35 of the largest (a long context can hold thousands of those), and
// 2^(kShift + kLazy) stays below its largest value.  One 16-bit term: a second one for what the rounding drops would
// be a second product of P and V, half as much tensor work again; the outputs' relative error is 1.1 to 1.4 times
// that of f32 weights (bf16 0.0023 against 0.0017, f16 0.00024 to 0.00028 against 0.00021).
template <typename T> struct PRange;
template <> struct PRange<__half> { static constexpr float kShift = 11.f, kLazy = 4.f; };
template <> struct PRange<__nv_bfloat16> { static constexpr float kShift = 0.f, kLazy = 8.f; };

struct TreeFold;

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
  const int32_t* positions;
  void* out;
  float* lse_out;
  float* slots;    // partial results: kTrSlots * ctas
  TreeFold* folds;  // what each CTA of the merge kernel has to do
  int32_t* status;
  int64_t num_pages, num_indices;
  int32_t batch, num_tokens, mask_words, page_size, box_rows, hq, hkv, group, ctas;
  uint32_t ps_magic, ps_shift, g_magic, g_shift;
  float scale_log2;   // |sm_scale| * log2(e), or 1 for a zero scale
  uint32_t q_xor;     // sign flip of both halves of a q word for a negative scale
  uint32_t q_and;     // 0 for a zero scale
  int32_t window;     // sliding window, 0 for none
  int32_t small;      // the batch's requests fit a warp's lanes and all units 32 bits
};

// The sliding window, in kernels that know one: the others are compiled without it (its rows' edges cost 8 tokens over
// 1K 0.8 us of 15.2, and 4 x 256 tokens over 32K 1 %).
template <bool SLIDING>
__device__ __forceinline__ int32_t window_of(const TreeParams& p) {
  return SLIDING ? p.window : 0;
}

// One request's share of the work.
struct TreeReq {
  int32_t slot_base;
  int32_t t0, n;       // its query tokens
  int32_t lo, hi, ds;  // pool rows in page order: visible [lo, hi), new tokens [ds, hi)
  int32_t blocks;      // blocks of query rows per KV head
  int32_t tile0;       // first key tile
  int32_t common;      // key tiles every block meets
  int32_t units;       // per KV head: blocks * common, and what chains add per block (a block stops at its last token)
  int32_t cost;        // of starting on a left-over of one of its blocks
  int32_t kind;        // 0 (no query), kReqEmpty (nothing visible or a bad table: zeros and -inf), kReqEven, kReqChain
};
constexpr int kReqEmpty = 1, kReqEven = 2, kReqChain = 3;

// Key tiles of block b behind the common ones.
__device__ __forceinline__ int32_t tail_of(const TreeReq& g, int group, int b) {
  if (g.kind != kReqChain) return 0;
  const int32_t tok = (int32_t)min((int64_t)g.n, ((int64_t)kTrBlock * (b + 1) + group - 1) / group);
  return (g.ds + tok + kTrTile - 1) / kTrTile - g.tile0 - g.common;
}

template <bool SLIDING>
__device__ __forceinline__ TreeReq tree_req(const TreeParams& p, int r, bool tell) {
  TreeReq g = {};
  const int32_t window = window_of<SLIDING>(p);
  const int32_t a = p.qo_indptr[r], b = p.qo_indptr[r + 1];
  const int32_t s0 = p.indptr[r], s1 = p.indptr[r + 1];
  const int32_t lpl = p.last_page_len[r], fpo = p.first_page_offset[r];
  if (a < 0 || b < a || b > p.num_tokens) {
    if (tell) report(p.status, PA_DEVICE_BAD_INDPTR);
    return g;
  }
  if (a == b) return g;
  g.slot_base = s0;
  g.t0 = a;
  g.n = b - a;
  g.blocks = (g.n * p.group + kTrBlock - 1) / kTrBlock;  // num_tokens * group fits (checked by the host)
  g.cost = g.n * p.group > kTrTile ? kTrCost2 : kTrCost1;
  g.kind = kReqEmpty;
  g.common = 1;  // one unit for an empty block
  g.units = g.blocks;
  const int64_t pages = (int64_t)s1 - s0;
  if (s0 < 0 || pages < 0 || s1 > p.num_indices || pages * p.page_size > INT32_MAX - 2 * kTrTile) {
    if (tell) report(p.status, PA_DEVICE_BAD_SLOT);
    return g;
  }
  const int32_t hi = pages > 0 ? ((int32_t)pages - 1) * p.page_size + lpl : 0;
  // a sliding window: the first row its first token sees
  const int32_t lo = window > 0 ? max(fpo, hi - g.n - window + 1) : fpo;
  const int32_t tile0 = lo / kTrTile;
  const int32_t all = (hi + kTrTile - 1) / kTrTile - tile0;
  if (pages == 0 || lpl < 1 || lpl > p.page_size || fpo < 0 || fpo >= p.page_size || hi - fpo < g.n ||
      (p.tree_mask && g.n > 32 * p.mask_words) || (int64_t)g.blocks * (all + kTrCost2) > INT32_MAX ||
      (window > 0 && hi - fpo - g.n < min(p.positions[a], window - 1))) {
    if (tell) report(p.status, PA_DEVICE_BAD_TREE);
    return g;
  }
  g.lo = lo;
  g.hi = hi;
  g.ds = hi - g.n;
  g.tile0 = tile0;
  g.kind = kReqEven;
  g.common = all;
  g.units = g.blocks * all;
  if (!p.tree_mask && g.blocks > 1) {
    g.kind = kReqChain;
    g.common = g.ds / kTrTile - tile0;
    g.units = g.blocks * g.common;
    for (int i = 0; i < g.blocks; ++i) g.units += tail_of(g, p.group, i);
  }
  return g;
}

// Key tiles that block b meets.
__device__ __forceinline__ int32_t tiles_of(const TreeReq& g, int group, int b) {
  return g.common + tail_of(g, group, b);
}

// A block's left-over tiles, weighed with the cost of starting on them.
__device__ __forceinline__ int32_t rest_weight(const TreeReq& g, int32_t tiles, int32_t run) {
  const int32_t rest = tiles % run;
  return rest ? rest + g.cost : 0;
}

// Chunks of `run` tiles and left-over weight per KV head.
struct HeadCut {
  int32_t chunks, weight;
};
__device__ __forceinline__ HeadCut head_cut(const TreeReq& g, int group, int32_t run) {
  HeadCut h = {g.blocks * (g.common / run), g.blocks * rest_weight(g, g.common, run)};
  if (g.kind == kReqChain) {
    h.chunks = h.weight = 0;
    for (int b = 0; b < g.blocks; ++b) {
      const int32_t t = tiles_of(g, group, b);
      h.chunks += t / run;
      h.weight += rest_weight(g, t, run);
    }
  }
  return h;
}

// a / b for 0 <= a, 0 < b; in 32 bits where a allows.
__device__ __forceinline__ int64_t div_units(int64_t a, int32_t b) {
  return (a >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The cut of the whole batch, and the place of one chunk or left-over position in it.  CTAs [0, chunks) take a
// chunk each, the others a stretch of `stretch` left-over weight.  run counts the start of every block in, so
// chunks * run + weight <= ctas * run, and as there is a block, chunks < ctas.
struct TreeCut {
  int64_t weight;         // all left-over weight
  int64_t off;            // the position inside request r: of chunks, or of left-over weight
  int64_t r_weight;       // left-over weight of the requests before r
  int32_t run, chunks, stretch;
  int32_t r, r_chunks;    // r: batch when the position is past the end; chunks of the requests before it
};

// The run length for `tiles` units and the cost of starting on every block's left-over.
__device__ __forceinline__ int32_t run_of(int64_t tiles, int64_t cost, int32_t ctas) {
  return (int32_t)min(max(div_units(tiles + cost + ctas - 1, ctas), (int64_t)1), (int64_t)INT32_MAX);
}
// The stretch length.
__device__ __forceinline__ void set_stretch(TreeCut* t, int32_t ctas) {
  t->stretch = t->chunks < ctas ? (int32_t)div_units(t->weight + (ctas - t->chunks) - 1, ctas - t->chunks) : 0;
}

__device__ __forceinline__ int64_t scan_add(int64_t v, int lane) {
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, w);
    if (lane >= w) v += u;
  }
  return v;
}

// The cut for a small batch, by one warp: lane r holds request r in `mine`.  c < chunks: chunk c; else left-over
// position (c - chunks) * stretch.
__device__ __forceinline__ TreeCut cut_warp(const TreeParams& p, int c, const TreeReq& mine, int lane) {
  int32_t tiles = (mine.units + mine.blocks * mine.cost) * p.hkv;  // and the cost of starting on every left-over
#pragma unroll 1
  for (int w = p.batch > 1 ? 16 : 0; w >= 1; w >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, w);
  }
  TreeCut t;
  t.run = (int32_t)max((uint32_t)(tiles + p.ctas - 1) / (uint32_t)p.ctas, 1u);
  t.run = __shfl_sync(0xffffffffu, t.run, 0);
  const HeadCut h = head_cut(mine, p.group, t.run);
  const int32_t chunks = h.chunks * p.hkv, weight = h.weight * p.hkv;
  int32_t chunks_to = chunks, weight_to = weight;
#pragma unroll 1
  for (int w = p.batch > 1 ? 1 : 32; w < 32; w <<= 1) {
    const int32_t a = __shfl_up_sync(0xffffffffu, chunks_to, w), b = __shfl_up_sync(0xffffffffu, weight_to, w);
    if (lane >= w) {
      chunks_to += a;
      weight_to += b;
    }
  }
  const int last = p.batch - 1;
  t.chunks = __shfl_sync(0xffffffffu, chunks_to, last);
  const int32_t all = __shfl_sync(0xffffffffu, weight_to, last);
  t.weight = all;
  t.stretch = (int32_t)((uint32_t)(all + (p.ctas - t.chunks) - 1) / (uint32_t)(p.ctas - t.chunks));
  const bool chunk = c < t.chunks;
  const int32_t at = chunk ? c : (c - t.chunks) * t.stretch;
  const uint32_t after = __ballot_sync(0xffffffffu, lane <= last && at < (chunk ? chunks_to : weight_to));
  t.r = after ? __ffs(after) - 1 : p.batch;
  const int src = after ? t.r : 0;
  t.r_chunks = __shfl_sync(0xffffffffu, chunks_to - chunks, src);
  t.r_weight = __shfl_sync(0xffffffffu, weight_to - weight, src);
  t.off = at - (chunk ? t.r_chunks : (int32_t)t.r_weight);
  return t;
}

// Exclusive prefix of v over the block's threads; *total receives the sum.  Two barriers.
template <int THREADS>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* warp_sum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t upto = scan_add(v, lane);
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t before = upto - v, sum = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    sum += warp_sum[w];
  }
  __syncthreads();
  *total = sum;
  return before;
}

// The same for any batch, by every thread of the block (each a run of consecutive requests).
template <int THREADS, bool SLIDING>
__device__ __forceinline__ void cut_block(const TreeParams& p, int c, bool tell, TreeCut* out,
                                          int64_t* warp_sum) {
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int r0 = (int)min((int64_t)threadIdx.x * per, (int64_t)p.batch), r1 = min(r0 + per, p.batch);
  int64_t tiles = 0, cost = 0;
  for (int r = r0; r < r1; ++r) {
    const TreeReq g = tree_req<SLIDING>(p, r, tell);
    tiles += (int64_t)g.units * p.hkv;
    cost += (int64_t)g.blocks * g.cost * p.hkv;
  }
  int64_t all_tiles, all_cost, all_chunks, all_weight;
  block_prefix<THREADS>(tiles, warp_sum, &all_tiles);
  block_prefix<THREADS>(cost, warp_sum, &all_cost);
  TreeCut t;
  t.run = run_of(all_tiles, all_cost, p.ctas);
  int64_t chunks = 0, weight = 0;
  for (int r = r0; r < r1; ++r) {
    const HeadCut h = head_cut(tree_req<SLIDING>(p, r, false), p.group, t.run);
    chunks += (int64_t)h.chunks * p.hkv;
    weight += (int64_t)h.weight * p.hkv;
  }
  int64_t chunks_at = block_prefix<THREADS>(chunks, warp_sum, &all_chunks);
  int64_t weight_at = block_prefix<THREADS>(weight, warp_sum, &all_weight);
  t.chunks = (int32_t)all_chunks;
  t.weight = all_weight;
  set_stretch(&t, p.ctas);
  const bool chunk = c < t.chunks;
  const int64_t at = chunk ? c : (int64_t)(c - t.chunks) * t.stretch;
  const int64_t begin = chunk ? chunks_at : weight_at;
  const int64_t mine = chunk ? chunks : weight;
  t.r = p.batch;
  t.off = t.r_weight = t.r_chunks = 0;
  if (at >= begin && at < begin + mine) {
    for (t.r = r0; t.r < r1; ++t.r) {
      const HeadCut h = head_cut(tree_req<SLIDING>(p, t.r, false), p.group, t.run);
      const int64_t u = (int64_t)(chunk ? h.chunks : h.weight) * p.hkv;
      t.off = at - (chunk ? chunks_at : weight_at);
      if (t.off < u) break;
      chunks_at += (int64_t)h.chunks * p.hkv;
      weight_at += (int64_t)h.weight * p.hkv;
    }
    t.r_chunks = (int32_t)chunks_at;
    t.r_weight = weight_at;
    *out = t;
  } else if (threadIdx.x == 0 && at >= (chunk ? all_chunks : all_weight)) {
    *out = t;
  }
  __syncthreads();
}

// Block, and what is before it in its KV head, of chunk or left-over position x of the head.
struct BlockAt {
  int32_t b, tiles, x;     // the block, its key tiles, the position inside it
  int32_t chunks, weight;  // of the head's blocks before it
};
__device__ __forceinline__ BlockAt block_at(const TreeReq& g, int group, int32_t run, int32_t x, bool chunk) {
  BlockAt k = {0, g.common, x, 0, 0};
  if (g.kind != kReqChain) {
    const int32_t chunks = g.common / run, weight = rest_weight(g, g.common, run);
    const int32_t each = chunk ? chunks : weight;
    k.b = x / each;
    k.x = x - k.b * each;
    k.chunks = k.b * chunks;
    k.weight = k.b * weight;
    return k;
  }
  for (;; ++k.b) {
    k.tiles = tiles_of(g, group, k.b);
    const int32_t chunks = k.tiles / run, weight = rest_weight(g, k.tiles, run);
    const int32_t each = chunk ? chunks : weight;
    if (k.x < each || k.b + 1 >= g.blocks) return k;
    k.x -= each;
    k.chunks += chunks;
    k.weight += weight;
  }
}

// Slot of a partial result.  A chunk's is its CTA's first, and so is that of a left-over piece that its CTA's
// stretch cuts off (only the stretch's last piece can be, and such a CTA has no chunk).  The piece that ends a
// block goes to a second slot: of the CTA of the block's first chunk, or, when it has none, of its own CTA (then
// it opens the stretch: the block was cut at the end of the stretch before).
__device__ __forceinline__ int rest_slot(bool ends, int32_t chunks, int first_chunk, int cta, int ctas) {
  return !ends ? cta : ctas + (chunks > 0 ? first_chunk : cta);
}

__device__ __forceinline__ TreeReq shfl_req(const TreeReq& g, int r) {
  TreeReq o;
  const int32_t* src = reinterpret_cast<const int32_t*>(&g);
  int32_t* dst = reinterpret_cast<int32_t*>(&o);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(TreeReq) / 4); ++i) dst[i] = __shfl_sync(0xffffffffu, src[i], r);
  return o;
}

// A block to fold, and one CTA's share of it, as the attention kernel leaves it for the merge kernel.  The parts lie,
// in the order of the keys, in slots first_chunk .. first_chunk + chunks - 1 and, for the left-over weight (which
// begins `lead` into the stretch of CTA cta0), in those of rest_slot.
struct alignas(16) TreeFold {
  int32_t shares;  // 0: nothing to fold here
  int32_t share;
  int32_t t0, row0, rows, kvh;
  int32_t first_chunk, chunks;
  int32_t weight, lead, cta0, stretch, cost;
};

// A run of key tiles of one block, as the loader hands it to the other roles.
struct TreePiece {
  int32_t kind;            // 0: no more, 1: key tiles, 2: nothing visible
  int32_t tile, tiles;     // key tiles [tile, tile + tiles)
  int32_t lo, hi, ds;
  int32_t all;             // rows [all, ds) are seen by every new token
  int32_t t0;
  int32_t slot_base;       // the request's first page-table slot
  int32_t row0, rows;      // query rows [row0, row0 + rows) of the request
  int32_t kvh, slot;       // slot < 0: the whole block, written as the result
  int32_t tainted;         // set by the fix warp: it took non-finite values out of V
};

constexpr int kPieceEnd = 0, kPieceTiles = 1, kPieceEmpty = 2;

__device__ __forceinline__ bool needs_fix(const TreePiece& d, int tile) {
  return tile * kTrTile < d.all || (tile + 1) * kTrTile > d.ds;
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Bits [a, b) of a word, a and b clamped to [0, 32].
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b >= 32 ? 0xffffffffu : ((1u << b) - 1u)) & ~((1u << a) - 1u);
}

// The first row that a query token sees: token `token` of the batch, new token i of a request whose visible rows
// begin at lo and whose new tokens begin at ds.  A sliding window of W ends W - 1 - depth rows before ds, the depth (at
// most i) being how far the token's position lies behind the request's first new token's.
template <bool SLIDING>
__device__ __forceinline__ int first_seen(const TreeParams& p, int lo, int ds, int token, int i) {
  if (!SLIDING) return lo;
  const int depth = p.tree_mask ? min(max(__ldg(p.positions + token) - __ldg(p.positions + token - i), 0), i) : i;
  return max(lo, ds + (depth + 1 - p.window));
}

// Which of the keys base .. base+31 (page order) it sees, from row `low` on, its request's visible rows ending at hi.
// (Of the new tokens a tree's mask holds the window's cut itself.)
template <bool SLIDING>
__device__ __forceinline__ uint32_t visible_bits(const TreeParams& p, int low, int ds, int hi, int token, int i,
                                                 int base) {
  uint32_t bits = bit_range(low - base, ds - base);
  if (base + 32 > ds && base < hi) {
    if (p.tree_mask) {
      const int32_t* row = p.tree_mask + (int64_t)token * p.mask_words;
      const int at = base - ds;  // new-token index of bit 0
      const int w = at >> 5, sh = at & 31;
      const uint32_t x0 = w >= 0 && w < p.mask_words ? (uint32_t)__ldg(row + w) : 0u;
      const uint32_t x1 = w + 1 >= 0 && w + 1 < p.mask_words ? (uint32_t)__ldg(row + w + 1) : 0u;
      bits |= __funnelshift_r(x0, x1, sh) & bit_range(ds - base, hi - base);
    } else {
      bits |= bit_range((SLIDING ? max(ds, low) : ds) - base, min(ds + i + 1, hi) - base);
    }
  }
  return bits;
}

// A shared-memory matrix descriptor (smem_desc) as two words: the upper one is the same for every operand here
// (stride 1024 bytes between 8-row groups, version 1, 128-byte swizzle), so only the lower one, address and
// leading offset in 16-byte units, is computed per product, in 32 bits.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }

// D[128 x N] (+)= A[128 x 16] B[16 x N]; A in shared memory, or in tensor memory.
__device__ __forceinline__ void umma_lo(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

// Instruction descriptor of kind::f16: f32 accumulate, A and B of format fmt (0 f16, 1 bf16), A K-major, B
// K-major or MN-major, M x N.
__host__ __device__ constexpr uint32_t tree_idesc(uint32_t fmt, int n, bool b_mn) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTrTile >> 4) << 24);
}

__device__ __forceinline__ uint32_t sat_mask(uint32_t w, uint32_t exp2x) {  // 0xffff per non-finite half
  return __vcmpeq2(w & exp2x, exp2x);
}
template <typename T> struct ExpBits;
template <> struct ExpBits<__half> { static constexpr uint32_t k = 0x7c007c00u; };
template <> struct ExpBits<__nv_bfloat16> { static constexpr uint32_t k = 0x7f807f80u; };

__device__ __forceinline__ float half_of(const __half* x) { return __half2float(*x); }
__device__ __forceinline__ float half_of(const __nv_bfloat16* x) { return __bfloat162float(*x); }

// No key was visible to the row (a NaN sum stays NaN).
__device__ __forceinline__ bool nothing_seen(float l) { return l == 0.f; }

// The non-finite values that the fix warp took out of V (of rows that not every new token sees), back into the O of
// the rows that see them (a converged warp: called under a condition that is the same for all its lanes; query token
// tok of the piece's request on this thread's lane).  Where two streams were joined, y is stream B's O of this row
// (D / 4 quads, kTrTile apart), and O becomes o s0 + y s1 first: an infinity added before would meet s0 = 0 in a row
// whose keys are all stream B's, and 0 times it is NaN.
template <typename T, int D, bool SLIDING>
__device__ __noinline__ void put_back(const TreeParams& p, const TreePiece& d, int tok, uint32_t t_o, const float4* y,
                                      float s0, float s1) {
  // of the rows that not every token sees, [lo, all) and [ds, hi)
  const int k0 = max(d.tile * kTrTile, d.lo), k1 = min((d.tile + d.tiles) * kTrTile, d.hi);
  const int low = first_seen<SLIDING>(p, d.lo, d.ds, d.t0 + tok, tok);
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    __syncwarp();
    tmem_ld32(t_o + 32 * c, o);
    if (y) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = y[(8 * c + i) * kTrTile];
        o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * s0 + b.x * s1);
        o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * s0 + b.y * s1);
        o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * s0 + b.z * s1);
        o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * s0 + b.w * s1);
      }
    }
    for (int k = k0; k < k1; ++k) {
      if (k >= d.all && k < d.ds) k = d.ds;
      if (k >= k1) break;
      if (!(visible_bits<SLIDING>(p, low, d.ds, d.hi, d.t0 + tok, tok, k) & 1u)) continue;
      const int sl = (int)fast_div((uint32_t)k, p.ps_magic, p.ps_shift);
      const int32_t page = __ldg(p.indices + d.slot_base + sl);
      if (page < 0 || page >= p.num_pages) continue;
      const T* src = static_cast<const T*>(p.v_pool) +
                     (((int64_t)page * p.page_size + (k - sl * p.page_size)) * p.hkv + d.kvh) * D + 32 * c;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = half_of(src + i);
        if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
      }
    }
    __syncwarp();
    tmem_st32(t_o + 32 * c, o);
  }
}

template <typename T, int D, bool TMA, bool SLIDING>
__global__ void __launch_bounds__(kTrThreads, 1)
    pa_v2_tree_attention_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tm_k,
                                const __grid_constant__ CUtensorMap tm_v) {
  using C = TreeCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffMisc);
  uint64_t* b_full = bars;
  uint64_t* b_empty = b_full + C::kStages;
  uint64_t* b_s = b_empty + C::kStages;   // 2: S of a stream is complete
  uint64_t* b_p = b_s + 2;                // 4: a half of a stream's P is written (one arrival per warp)
  uint64_t* b_o = b_p + 4;                // the piece's products are complete
  uint64_t* b_q = b_o + 1;                // the piece's Q is in shared memory
  uint64_t* b_fix = b_q + 1;              // kStages: the V tile in a stage was made safe
  uint64_t* b_x = b_fix + C::kStages;     // stream B's state is in shared memory
  uint64_t* b_xd = b_x + 1;               // ... and has been read
  uint64_t* b_pf = b_xd + 1;              // kTrRing: a piece is handed out
  uint64_t* b_pe = b_pf + kTrRing;        // kTrRing: every role is done with it
  uint64_t* b_drain = b_pe + kTrRing;
  TreePiece* ring = reinterpret_cast<TreePiece*>(b_drain + 1);
  TreeCut* start = reinterpret_cast<TreeCut*>(ring + kTrRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + 1);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
  float* xstate = reinterpret_cast<float*>(tmem_slot + 2);  // [2][128]: stream B's maxima and sums
  int64_t* warp_sum = reinterpret_cast<int64_t*>(xstate);   // before the first piece
  int32_t(*rows_of)[kTrTile / 2] = reinterpret_cast<int32_t(*)[kTrTile / 2]>(xstate + 2 * kTrTile);  // the loaders'
  static_assert((3 * C::kStages + 11 + 2 * kTrRing) * 8 + kTrRing * sizeof(TreePiece) + sizeof(TreeCut) +
                        8 + 2 * kTrTile * 4 + kTrTile * 4 <=
                    C::kMisc,
                "the area behind the stages");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_addr(smem);

  pdl_launch_dependents();
  if (TMA && threadIdx.x == kTrLoadWarp * 32) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b_full[i], TMA ? 1 : kTrLoadThreads);
      mbar_init(&b_empty[i], 2);  // the MMAs that read the stage, and the fix warp
      mbar_init(&b_fix[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&b_s[w], 1);
      mbar_init(&b_p[2 * w], 4);
      mbar_init(&b_p[2 * w + 1], 4);
    }
    mbar_init(b_o, 1);
    mbar_init(b_q, 8);
    mbar_init(b_x, 4);
    mbar_init(b_xd, 4);
    for (int i = 0; i < kTrRing; ++i) {
      mbar_init(&b_pf[i], 1);
      mbar_init(&b_pe[i], 10);  // 8 softmax warps, the MMA warp, the fix warp
    }
    mbar_init(b_drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == kTrMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(kTrTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the loader warp finds the CTA's place alone when a request fits a lane, else all threads do
  const bool small = p.small != 0;
  if (!small) cut_block<kTrThreads, SLIDING>(p, blockIdx.x, blockIdx.x == 0, start, warp_sum);

  // Registers follow the roles: 208 for the softmax threads, which hold a row of scores, 88 for the others
  // (256 * 208 + 128 * 88 = 384 * 168).  Each warpgroup sets its own count on its own path.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ----------------------------------------------------------------- softmax
    const int w = warp >> 2;                 // stream
    const int row = (warp & 3) * 32 + lane;  // tile row = tensor-memory lane
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + col_s(w), t_o = t_lane + col_o(w);
    constexpr float kShift = PRange<T>::kShift, kLazy = PRange<T>::kLazy;
    const float scale = p.scale_log2;
    uint32_t par_s = 0, par_o = 0, par_x = 0, par_xd = 0;
    bool alive = true, pending_x = false;
    for (int pc = 0; alive; ++pc) {
      const int at = pc % kTrRing;
      if (!wait_phase(&b_pf[at], (uint32_t)((pc / kTrRing) & 1), abort_flag, p.status)) break;
      // read again from shared memory where it is needed: kept in registers across the tiles it would be spilled
      const volatile TreePiece& d = ring[at];
      const int kind = d.kind, rows = d.rows;
      if (kind == kPieceEnd) break;
      const bool dual = rows > kTrTile;
      const int rr = (dual ? w * kTrTile : 0) + row;         // row of the block
      const bool busy = (rr & ~31) < rows;                   // a row of this warp is of the block
      const int tok = (int)fast_div((uint32_t)(d.row0 + min(rr, rows - 1)), p.g_magic, p.g_shift);
      float m = -INFINITY, l = 0.f;
      if (kind == kPieceTiles) {
        // ---- Q, swizzled like the key tiles; rows past the block repeat its last one (their results go nowhere)
        if (pending_x) {  // the exchanged state of the piece before shares the Q tiles' memory
          if (!wait_phase(b_xd, par_xd, abort_flag, p.status)) break;
          par_xd ^= 1;
          pending_x = false;
        }
        {
          // a row's 16-byte pieces on neighbouring lanes; a warp fills its own 32 rows of its stream's tile, or,
          // when both streams read tile A, 16 of them
          constexpr int kChunks = D / 8, kPass = 32 / kChunks;
          unsigned char* dst = smem + (dual ? w : 0) * C::kTileBytes;
          const int c = lane % kChunks;
          const int first = dual ? (warp & 3) * 32 : warp * 16, count = dual ? 32 : 16;
          const int row0 = d.row0, t0 = d.t0, kvh = d.kvh;
          constexpr int kBatch = 32 / kPass;  // all loads before the first store
          uint4 x[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i * kPass >= count) break;
            const int br = min((dual ? w * kTrTile : 0) + first + i * kPass + lane / kChunks, rows - 1);
            const int tk = (int)fast_div((uint32_t)(row0 + br), p.g_magic, p.g_shift);
            const int64_t qr = (int64_t)(t0 + tk) * p.hq + (int64_t)kvh * p.group + (row0 + br - tk * p.group);
            x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + qr * D) + c);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i * kPass >= count) break;
            const int tr = first + i * kPass + lane / kChunks;
            x[i].x = (x[i].x ^ p.q_xor) & p.q_and;
            x[i].y = (x[i].y ^ p.q_xor) & p.q_and;
            x[i].z = (x[i].z ^ p.q_xor) & p.q_and;
            x[i].w = (x[i].w ^ p.q_xor) & p.q_and;
            *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTrTile * 128) + sw128(tr, c & 7)) = x[i];
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_q);
        }
        // ---- key tiles
        const int tiles = d.tiles, tile0 = d.tile, clear0 = d.all, clear1 = d.ds;  // no mask inside [clear0, clear1)
        const int low = first_seen<SLIDING>(p, d.lo, clear1, d.t0 + tok, tok);
        for (int j = dual ? 0 : w; j < tiles; j += dual ? 1 : 2) {
          if (!wait_phase(&b_s[w], par_s, abort_flag, p.status)) {
            alive = false;
            break;
          }
          par_s ^= 1;
          tc_fence_after();
          if (busy) {
            const int c0 = (tile0 + j) * kTrTile;
            const bool edge = c0 < clear0 || c0 + kTrTile > clear1;
            uint32_t x[2][64];  // the row's scores
            __syncwarp();
            tmem_ld64(t_s, x[0]);
            tmem_ld64(t_s + 64, x[1]);
            tmem_wait64(x[0]);
            tmem_wait64(x[1]);
            if (edge) {
              const int hi = d.hi, t0 = d.t0;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t vis = visible_bits<SLIDING>(p, low, clear1, hi, t0 + tok, tok, c0 + 32 * c);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  x[c >> 1][(c & 1) * 32 + i] = (vis >> i) & 1u ? x[c >> 1][(c & 1) * 32 + i] : 0xff800000u;
              }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mx[k] = max3(mx[k], __uint_as_float(x[0][i + k]), __uint_as_float(x[1][i + k]));
            }
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
            const bool need = mt > m + kLazy;  // m = -inf at first: any finite maximum
            const float a = need ? (m == -INFINITY ? 0.f : fast_exp2(m - mt)) : 1.f;
            if (need) m = mt;
            l *= a;
            const bool first = j == (dual ? 0 : w);
            if (!first && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(t_o + 32 * c, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                tmem_st32(t_o + 32 * c, o);
              }
            }
            const float mu = (m == -INFINITY ? 0.f : m) - kShift;
            const float2 scale2 = make_float2(scale, scale), off2 = make_float2(-mu, -mu);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 64; i += 2) {
                float2 y = fma2(make_float2(__uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1])), scale2, off2);
                y.x = fast_exp2(y.x);
                y.y = fast_exp2(y.y);
                sum[i >> 1 & 1] = add2(sum[i >> 1 & 1], y);
                pk[i / 2] = TC<T>::pack(y.x, y.y);
              }
              __syncwarp();
              tmem_st32(t_s + 32 * h, pk);
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&b_p[2 * w + h]);
            }
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&b_p[2 * w]);
              mbar_arrive(&b_p[2 * w + 1]);
            }
          }
        }
        if (!alive) break;
        if (!wait_phase(b_o, par_o, abort_flag, p.status)) break;
        par_o ^= 1;
        tc_fence_after();
      }

      // ---- the piece's result
      const bool joined = kind == kPieceTiles && !dual && d.tiles > 1;  // two streams to join
      float4* xo = reinterpret_cast<float4*>(smem);                       // [D / 4][128], over the Q tiles
      if (joined && w == 1) {
        if (busy) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(t_o + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              xo[(8 * c + i) * kTrTile + row] =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                              __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
          xstate[row] = m;
          xstate[kTrTile + row] = l;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_x);
      }
      pending_x = pending_x || joined;
      if (joined && w == 0) {
        if (!wait_phase(b_x, par_x, abort_flag, p.status)) break;
        par_x ^= 1;
      }
      if (busy && (dual || w == 0)) {
        float s0 = 1.f, s1 = 0.f;
        if (joined) {
          const float m1 = xstate[row], l1 = xstate[kTrTile + row];
          const float M = fmaxf(m, m1);
          s0 = m == -INFINITY ? 0.f : fast_exp2(m - M);
          s1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - M);
          l = l * s0 + l1 * s1;
          m = M;
        }
        const bool nothing = nothing_seen(l);
        const float inv = nothing ? 0.f : fast_rcp(l);
        const float lse = nothing ? -INFINITY : m - kShift + fast_log2(l);
        // (the whole warp or none of it: tensor memory is read and written by converged warps only, and rows that see
        // nothing in this piece stand beside rows that do)
        const bool mended = kind == kPieceTiles && d.tainted != 0;
        if (mended) put_back<T, D, SLIDING>(p, ring[at], tok, t_o, joined ? xo + row : nullptr, s0, s1);
        const bool valid = rr < rows, whole = d.slot < 0;
        const int qrow = d.row0 + min(rr, rows - 1);  // row of the request
        const int64_t orow = (int64_t)(d.t0 + tok) * p.hq + (int64_t)d.kvh * p.group + (qrow - tok * p.group);
        T* out = static_cast<T*>(p.out) + orow * D;
        float* slot = p.slots + (int64_t)max(d.slot, 0) * C::kSlotFloats;
        float4* part = reinterpret_cast<float4*>(slot) + (rr >> 7) * (D / 4 * kTrTile) + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (kind == kPieceTiles) {
            __syncwarp();
            tmem_ld32(t_o + 32 * c, o);
          }
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = nothing ? 0.f : __uint_as_float(o[i]);
          if (joined && !mended && !nothing) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 y = xo[(8 * c + i) * kTrTile + row];
              v[4 * i] = v[4 * i] * s0 + y.x * s1;
              v[4 * i + 1] = v[4 * i + 1] * s0 + y.y * s1;
              v[4 * i + 2] = v[4 * i + 2] * s0 + y.z * s1;
              v[4 * i + 3] = v[4 * i + 3] * s0 + y.w * s1;
            }
          }
          if (valid && whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) =
                  make_uint4(TC<T>::pack(v[8 * i] * inv, v[8 * i + 1] * inv),
                             TC<T>::pack(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                             TC<T>::pack(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                             TC<T>::pack(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[(8 * c + i) * kTrTile] = make_float4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv,
                                                        v[4 * i + 3] * inv);
          }
        }
        if (valid) {
          if (whole)
            p.lse_out[orow] = lse;
          else
            slot[(int64_t)kTrBlock * D + rr] = lse;
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (joined && w == 0) mbar_arrive(b_xd);
        mbar_arrive(&b_pe[at]);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kTrLoadWarp || warp == kTrLoadWarp + 1) {
      // ------------------------------------------------------------------ loader
      const bool leader = warp == kTrLoadWarp;
      TreeReq mine = {};
      TreeCut cut;
      if (small) {
        if (lane < p.batch) mine = tree_req<SLIDING>(p, lane, leader && blockIdx.x == 0);
        cut = cut_warp(p, blockIdx.x, mine, lane);
      } else {
        cut = *start;
      }
      const int32_t run = cut.run;
      int stage = 0, pieces = 0, ops = 0;
      int published = 0;  // without TMA: the operations whose copies the other roles may use
      bool alive = true;
      const int u = (warp - kTrLoadWarp) * 32 + lane;
      TreeReq g = {};
      const int box_rows = p.box_rows;
      // keys that several blocks read stay in L2 as other data does, the others leave it first
      const uint64_t first = policy_evict_first(), normal = policy_evict_normal();

      auto publish = [&](int upto) {  // without TMA: the copies of the operations before `upto` have landed
        fence_proxy_async_smem();
        for (; published < upto; ++published) mbar_arrive(&b_full[published % C::kStages]);
      };
      // K (or V) rows [128 tile, 128 tile + 128) of the request's pages into the next stage
      auto load = [&](int tile, int kvh, bool is_v) {
        if (TMA && is_v == leader) {  // the other warp's
          ++ops;
          stage = stage + 1 == C::kStages ? 0 : stage + 1;
          return;
        }
        if (!wait_phase(&b_empty[stage], ((ops / C::kStages) & 1) ^ 1, abort_flag, p.status)) {
          alive = false;
          return;
        }
        const uint64_t policy = g.blocks > 1 ? normal : first;
        const uint32_t dst = sbase + C::kOffKv + stage * C::kTileBytes;
        const int row0 = tile * kTrTile;
        const int rows = min(kTrTile, g.hi - row0);
        if (TMA) {
          // lane i resolves box i; one thread issues them all (copies whose operands differ from lane to lane are
          // issued one lane at a time anyway, at several times the cost)
          const int boxes = (rows + box_rows - 1) / box_rows;
          int32_t mine_row = 0;
          if (lane < boxes) {
            const int at = row0 + lane * box_rows;
            const int slot = (int)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
            const int32_t page = __ldg(p.indices + g.slot_base + slot);
            if (page >= 0 && page < p.num_pages && (!SLIDING || at + box_rows > g.lo)) {
              mine_row = page * p.page_size + (at - slot * p.page_size);
            } else {
              // past the pool: the box is zero-filled (as are boxes before a sliding window, whose pages may be gone)
              mine_row = (int32_t)(p.num_pages * p.page_size);
              if (!is_v && (!SLIDING || at + box_rows > g.lo)) report(p.status, PA_DEVICE_BAD_PAGE);
            }
          }
          volatile int32_t* box_row = rows_of[u >> 5];
          if (lane < 16) box_row[lane] = mine_row;
          __syncwarp();
          if (elect_one()) {
            mbar_arrive_expect_tx(&b_full[stage], (uint32_t)(boxes * box_rows * D * 2));
            unsigned char* to = smem + C::kOffKv + stage * C::kTileBytes;
#pragma unroll 2
            for (int i = 0; i < boxes; ++i, to += box_rows * 128) {
              const int32_t row = box_row[i];
#pragma unroll
              for (int half = 0; half < C::kHalves; ++half)
                tma_load_3d(to + half * (kTrTile * 128), is_v ? &tm_v : &tm_k, &b_full[stage], half * 64, kvh, row,
                            policy);
            }
          }
          __syncwarp();
        } else {
          // a warp gathers half of the rows: first each lane resolves two, then all copy them, 16 bytes per lane
          constexpr int kChunks = D / 8, kPass = 32 / kChunks;  // pieces of a row; rows per pass
          volatile int32_t* row_of = rows_of[u >> 5];
          const int half0 = (u >> 5) * (kTrTile / 2);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = row0 + half0 + 32 * i + lane;
            int32_t from = -1;
            if (at >= g.lo && at < g.hi) {
              const int slot = (int)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
              const int32_t page = __ldg(p.indices + g.slot_base + slot);
              if (page >= 0 && page < p.num_pages)
                from = page * p.page_size + (at - slot * p.page_size);
              else if (!is_v)
                report(p.status, PA_DEVICE_BAD_PAGE);
            }
            row_of[32 * i + lane] = from;
          }
          __syncwarp();
          const int ch = lane % kChunks, sub = lane / kChunks;
          const T* pool = static_cast<const T*>(is_v ? p.v_pool : p.k_pool) + (int64_t)kvh * D + ch * 8;
          const uint32_t row_bytes = (uint32_t)p.hkv * D * sizeof(T);
          const uint32_t to0 = dst + (uint32_t)(ch >> 3) * (kTrTile * 128) + half0 * 128;
#pragma unroll 8
          for (int i = 0; i < kTrTile / 2; i += kPass) {
            const int32_t from = row_of[i + sub];
            const uint32_t to = to0 + sw128(i + sub, ch & 7);
            if (from >= 0)
              cp_async_16(to, reinterpret_cast<const char*>(pool) + (uint64_t)(uint32_t)from * row_bytes, policy);
            else
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0u) : "memory");
          }
          cp_async_commit();
          cp_async_wait<kTrLag>();
          publish(ops + 1 - kTrLag);
        }
        ++ops;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
      };
      auto hand_out = [&](const TreePiece& d) {
        const int at = pieces % kTrRing;
        // (a second loader warp does not wait here: pieces without key tiles could pass it by)
        if (leader && !wait_phase(&b_pe[at], ((pieces / kTrRing) & 1) ^ 1, abort_flag, p.status)) {
          alive = false;
          return;
        }
        if (leader && lane == 0) {
          ring[at] = d;
          mbar_arrive(&b_pf[at]);
        }
        __syncwarp();
        ++pieces;
      };

      // key tiles [t0, t0 + tiles) of block b
      auto piece = [&](int kvh, int b, int32_t t0, int32_t tiles, int slot) {
        TreePiece d;
        d.kind = g.kind == kReqEmpty ? kPieceEmpty : kPieceTiles;
        d.tile = g.tile0 + t0;
        d.tiles = tiles;
        d.lo = g.lo;
        d.hi = g.hi;
        d.ds = g.ds;
        d.all = SLIDING ? max(g.lo, min(g.ds, g.hi - p.window)) : g.lo;
        d.t0 = g.t0;
        d.slot_base = g.slot_base;
        d.row0 = b * kTrBlock;
        d.rows = min(kTrBlock, g.n * p.group - d.row0);
        d.kvh = kvh;
        d.slot = slot;
        d.tainted = 0;
        hand_out(d);
        if (!alive || d.kind == kPieceEmpty) return;
        const int ahead = d.rows > kTrTile ? 1 : 2;  // key tiles S runs ahead of O (as the MMA warp takes them)
        for (int j = 0; j < tiles + ahead && alive; ++j) {
          if (j >= ahead) load(d.tile + j - ahead, kvh, true);
          if (j < tiles && alive) load(d.tile + j, kvh, false);
        }
        if (!TMA && alive) {  // before the ring of pieces is waited for
          cp_async_wait<0>();
          publish(ops);
        }
      };

      // what the merge kernel's CTA of this number does: blocks with chunks are shared out over the CTAs of their
      // chunks, blocks without over the CTAs whose stretches cut them.  `at`: where the block's left-over weight
      // begins; share < 0: counted from the stretch ends behind the block's first tile.
      const bool writes = leader && lane == 0;
      if (writes) p.folds[blockIdx.x].shares = 0;
      auto fold = [&](int kvh, int b, int first_chunk, int32_t chunks, int share, int64_t at, int32_t weight) {
        TreeFold f;
        f.stretch = cut.stretch;
        f.cost = g.cost;
        f.t0 = g.t0;
        f.kvh = kvh;
        f.row0 = b * kTrBlock;
        f.rows = min(kTrBlock, g.n * p.group - f.row0);
        f.first_chunk = first_chunk;
        f.chunks = chunks;
        f.weight = weight;
        f.cta0 = f.lead = 0;
        if (weight > 0) {
          const int64_t i = div_units(at, cut.stretch);
          f.cta0 = cut.chunks + (int)i;
          f.lead = (int32_t)(at - i * cut.stretch);
        }
        f.shares = chunks;
        f.share = share;
        if (share < 0) {
          const int idle = (f.lead + g.cost) / cut.stretch;  // stretch ends at or before the first tile
          f.share = (int)blockIdx.x - f.cta0 - idle;
          f.shares = (f.lead + weight - 1) / cut.stretch - idle;
        }
        if (writes) p.folds[blockIdx.x] = f;
      };

      int r = cut.r;
      if (r < p.batch && (int)blockIdx.x < cut.chunks) {
        g = small ? shfl_req(mine, r) : tree_req<SLIDING>(p, r, false);
        const HeadCut h = head_cut(g, p.group, run);
        const int kvh = (int)div_units(cut.off, h.chunks);
        const BlockAt k = block_at(g, p.group, run, (int32_t)(cut.off - (int64_t)kvh * h.chunks), true);
        piece(kvh, k.b, k.x * run, run, k.tiles == run ? -1 : (int)blockIdx.x);
        if (k.tiles != run && g.kind != kReqEmpty)
          fold(kvh, k.b, (int)blockIdx.x - k.x, k.tiles / run, k.x,
               cut.r_weight + (int64_t)kvh * h.weight + k.weight, rest_weight(g, k.tiles, run));
      } else {
        int64_t off = cut.off, r_weight = cut.r_weight;
        int32_t left = (int32_t)min((int64_t)cut.stretch,
                                    cut.weight - (int64_t)((int)blockIdx.x - cut.chunks) * cut.stretch);
        int chunks_before = cut.r_chunks;
        for (; r < p.batch && left > 0 && alive; ++r, off = 0) {
          g = small ? shfl_req(mine, r) : tree_req<SLIDING>(p, r, false);
          const HeadCut h = head_cut(g, p.group, run);
          int kvh = h.weight > 0 ? (int)div_units(off, h.weight) : p.hkv;
          int32_t in_head = (int32_t)(off - (int64_t)kvh * h.weight);
          for (; kvh < p.hkv && left > 0 && alive; ++kvh, in_head = 0) {
            BlockAt k = block_at(g, p.group, run, in_head, false);
            while (left > 0 && alive) {
              const int32_t chunks = k.tiles / run;
              const int32_t weight = rest_weight(g, k.tiles, run);
              const int32_t take = min(weight - k.x, left);
              const int32_t t0 = max(k.x - g.cost, 0), t1 = max(k.x + take - g.cost, 0);
              const bool ends = k.x + take == weight;
              if (t1 > t0)
                piece(kvh, k.b, chunks * run + t0, t1 - t0,
                      ends && t0 == 0 && chunks == 0
                          ? -1
                          : rest_slot(ends, chunks, chunks_before + kvh * h.chunks + k.chunks, blockIdx.x, p.ctas));
              left -= take;
              // the stretch ends inside the block, behind its first tile
              if (!ends && chunks == 0 && t1 > 0 && g.kind != kReqEmpty)
                fold(kvh, k.b, 0, 0, -1, r_weight + (int64_t)kvh * h.weight + k.weight, weight);
              if (k.b + 1 >= g.blocks) break;
              k.chunks += chunks;
              k.weight += weight;
              ++k.b;
              k.tiles = tiles_of(g, p.group, k.b);
              k.x = 0;
            }
          }
          chunks_before += p.hkv * h.chunks;
          r_weight += (int64_t)p.hkv * h.weight;
        }
      }
      if (alive) {
        TreePiece d = {};
        d.kind = kPieceEnd;
        hand_out(d);
      }
      if (TMA) {  // no copy of this CTA is left in flight, whatever ended the loop
        for (int i = max(ops - C::kStages, 0); i < ops; ++i)
          mbar_wait_bounded(&b_full[i % C::kStages], (uint32_t)((i / C::kStages) & 1), kWaitLimitCycles);
      } else {
        cp_async_wait<0>();
      }
    } else if (warp == kTrMmaWarp) {
      // --------------------------------------------------------------------- MMA
      constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t id_s = tree_idesc(fmt, kTrTile, false);
      constexpr uint32_t id_o = tree_idesc(fmt, D, true);
      if (elect_one()) {
        int op = 0;
        uint32_t par_p[2] = {0, 0}, par_q = 0, par_fix = 0;  // par_fix: a bit per stage
        bool alive = true, issued = false;
        auto take = [&]() -> int {  // the next loaded stage
          const int st = op % C::kStages;
          if (!wait_one(&b_full[st], (uint32_t)((op / C::kStages) & 1), abort_flag, p.status)) alive = false;
          ++op;
          return st;
        };
        auto scores = [&](int w, int qt, int st) {
          const uint32_t qa = desc_lo(sbase + qt * C::kTileBytes, 16);
          const uint32_t ka = desc_lo(sbase + C::kOffKv + st * C::kTileBytes, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = ((kk >> 2) * (kTrTile * 128) + (kk & 3) * 32) >> 4;
            umma_lo(tmem + col_s(w), qa + at, ka + at, id_s, kk != 0);
          }
          umma_commit(&b_s[w]);
          issued = true;
        };
        auto values = [&](int w, int st, bool acc) {
          const uint32_t va = desc_lo(sbase + C::kOffKv + st * C::kTileBytes, kTrTile * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the first half of the keys while the softmax still works on the second
            if (!wait_one(&b_p[2 * w + h], par_p[w], abort_flag, p.status)) {
              alive = false;
              return;
            }
            tc_fence_after();
#pragma unroll
            for (int kt = 4 * h; kt < 4 * h + 4; ++kt)
              umma_ts(tmem + col_o(w), tmem + col_s(w) + 8 * kt, va + kt * (2048 >> 4), id_o, acc || kt != 0);
          }
          par_p[w] ^= 1;
        };
        auto release = [&](int st) { umma_commit(&b_empty[st]); };
        for (int pc = 0; alive; ++pc) {
          const int at = pc % kTrRing;
          if (!wait_one(&b_pf[at], (uint32_t)((pc / kTrRing) & 1), abort_flag, p.status)) break;
          const TreePiece d = ring[at];
          if (d.kind == kPieceEnd) break;
          if (d.kind == kPieceTiles) {
            const bool dual = d.rows > kTrTile;
            // Q is written, and both streams are done with the piece before
            if (!wait_one(b_q, par_q, abort_flag, p.status)) break;
            par_q ^= 1;
            tc_fence_after();
            auto wait_fix = [&](int tile, int st) {
              if (!needs_fix(d, tile)) return;
              if (!wait_one(&b_fix[st], par_fix >> st & 1u, abort_flag, p.status)) alive = false;
              par_fix ^= 1u << st;
            };
            if (dual) {
              // the next tile is waited for while the products before it still run
              int k = take();
              if (!alive) break;
              scores(0, 0, k);
              scores(1, 1, k);
              release(k);
              int v = take();
              for (int j = 0; j < d.tiles && alive; ++j) {
                const bool more = j + 1 < d.tiles;
                wait_fix(d.tile + j, v);
                if (alive) values(0, v, j > 0);
                if (alive && more) k = take();
                if (!alive) break;
                if (more) scores(0, 0, k);
                values(1, v, j > 0);
                if (!alive) break;
                release(v);
                if (more) {
                  v = take();
                  if (!alive) break;
                  scores(1, 1, k);
                  release(k);
                }
              }
            } else {
              for (int w = 0; w < min(2, d.tiles) && alive; ++w) {
                const int k = take();
                if (!alive) break;
                scores(w, 0, k);
                release(k);
              }
              for (int j = 0; j < d.tiles && alive; ++j) {
                const int v = take();
                if (alive) wait_fix(d.tile + j, v);
                if (alive) values(j & 1, v, j > 1);
                if (!alive) break;
                release(v);
                if (j + 2 < d.tiles) {
                  const int k = take();
                  if (!alive) break;
                  scores(j & 1, 0, k);
                  release(k);
                }
              }
            }
            if (!alive) break;
            umma_commit(b_o);
          }
          mbar_arrive(&b_pe[at]);
        }
        // every MMA of this CTA has completed before tensor memory is released
        if (issued) {
          umma_commit(b_drain);
          if (!mbar_wait_bounded(b_drain, 0, kWaitLimitCycles)) report(p.status, PA_DEVICE_WAIT_TIMEOUT);
        }
      }
      __syncwarp();
    } else if (warp == kTrFixWarp) {
      // --------------------------------------------------------- V tiles made safe
      int op = 0;
      bool alive = true;
      for (int pc = 0; alive; ++pc) {
        const int at = pc % kTrRing;
        if (!wait_phase(&b_pf[at], (uint32_t)((pc / kTrRing) & 1), abort_flag, p.status)) break;
        const TreePiece d = ring[at];
        if (d.kind == kPieceEnd) break;
        if (d.kind == kPieceTiles) {
          // every stage is waited for and released, K tiles too: a wait names a phase by its parity, which only
          // tells phases apart that are at most one apart
          auto stage_of = [&](bool last) -> int {
            const int st = op % C::kStages;
            if (!wait_phase(&b_full[st], (uint32_t)((op / C::kStages) & 1), abort_flag, p.status)) alive = false;
            ++op;
            if (last && alive && lane == 0) mbar_arrive(&b_empty[st]);
            return st;
          };
          const int ahead = d.rows > kTrTile ? 1 : 2;
          for (int j = 0; j < min(ahead, d.tiles) && alive; ++j) stage_of(true);
          for (int j = 0; j < d.tiles && alive; ++j) {
            const bool fix = needs_fix(d, d.tile + j);
            const int st = stage_of(!fix);
            if (!alive) break;
            const int c0 = (d.tile + j) * kTrTile;
            if (!fix) {
              if (j + ahead < d.tiles) stage_of(true);
              continue;
            }
            constexpr int kChunks = D / 8;
            const uint32_t base = sbase + C::kOffKv + st * C::kTileBytes;
            const int ch = lane % kChunks;
            const uint32_t col = base + (uint32_t)(ch >> 3) * (kTrTile * 128);
            constexpr int kPass = 32 / kChunks;  // rows per pass
            const int sub = lane / kChunks;
            auto zero_rows = [&](int r0, int r1) {
#pragma unroll 8
              for (int row = r0 + sub; row < r1; row += kPass)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(col + sw128(row, ch & 7)), "r"(0u)
                             : "memory");
            };
            uint32_t any = 0;
            auto check_rows = [&](int r0, int r1) {  // four passes' loads at once
              constexpr uint32_t e = ExpBits<T>::k;
              for (int base_row = r0; base_row < r1; base_row += 4 * kPass) {
                uint32_t x[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int row = min(base_row + k * kPass + sub, r1 - 1);
                  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(x[k][0]), "=r"(x[k][1]), "=r"(x[k][2]), "=r"(x[k][3])
                               : "r"(col + sw128(row, ch & 7))
                               : "memory");
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t n[4], bad = 0;
#pragma unroll
                  for (int i = 0; i < 4; ++i) bad |= n[i] = sat_mask(x[k][i], e);
                  if (bad) {
                    any = 1;
                    const int row = min(base_row + k * kPass + sub, r1 - 1);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(col + sw128(row, ch & 7)),
                                 "r"(x[k][0] & ~n[0]), "r"(x[k][1] & ~n[1]), "r"(x[k][2] & ~n[2]), "r"(x[k][3] & ~n[3])
                                 : "memory");
                  }
                }
              }
            };
            // rows of the tile: outside, earlier tokens that only some see, that all see (left alone), new tokens,
            // outside
            const int in0 = min(max(d.lo - c0, 0), kTrTile), in1 = min(max(d.hi - c0, in0), kTrTile);
            zero_rows(0, in0);
            if (SLIDING) check_rows(in0, min(max(d.all - c0, in0), kTrTile));
            check_rows(min(max(d.ds - c0, in0), in1), in1);
            zero_rows(in1, kTrTile);
            if (__any_sync(0xffffffffu, any != 0) && lane == 0)
              *reinterpret_cast<volatile int32_t*>(&ring[at].tainted) = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&b_fix[st]);
              mbar_arrive(&b_empty[st]);
            }
            __syncwarp();
            if (j + ahead < d.tiles) stage_of(true);
          }
        }
        if (!alive) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_pe[at]);
      }
    }
  }

  // ---- release tensor memory once every role is done with it
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == kTrMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTrTmemCols) : "memory");
  }
}

// Folds the partial results of blocks that were cut: weights 2^(lse_i - max) of the normalized parts, in the
// order of the keys.  CTA c does what CTA c of the attention kernel wrote down for it; a warp takes 32 rows x 8
// columns, one row per lane (the parts are stored column by column, so a warp's loads are contiguous), eight
// parts in flight.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) pa_v2_tree_merge_kernel(const TreeParams p) {
  using C = TreeCfg<D>;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const TreeFold f = p.folds[blockIdx.x];
  if (f.shares == 0) return;
  const int jobs = (f.rows + 31) / 32 * (D / 8);
  const int workers = f.shares * (int)gridDim.y * (kMergeThreads / 32);
  const int me = (f.share * (int)gridDim.y + (int)blockIdx.y) * (kMergeThreads / 32) + (int)(threadIdx.x >> 5);
  for (int job = me; job < jobs; job += workers) {
    const int rg = job / (D / 8), oct = job % (D / 8);
    const int in_block = rg * 32 + lane;
    const int row = f.row0 + in_block;
    const bool valid = in_block < f.rows;
    int i = 0;          // chunks taken
    int32_t at = 0;     // left-over weight taken
    int cta = f.cta0;
    auto next = [&]() -> int {  // slot of the next part in the order of the keys, or -1
      if (i < f.chunks) return f.first_chunk + i++;
      while (at < f.weight) {
        const int32_t end = min((cta - f.cta0 + 1) * f.stretch - f.lead, f.weight);
        const bool some = end > max(at, f.cost);
        const int slot = rest_slot(end == f.weight, f.chunks, f.first_chunk, cta, p.ctas);
        at = end;
        ++cta;
        if (some) return slot;
      }
      return -1;
    };
    bool more = true;
    float M = -INFINITY, L = 0.f;
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    while (more) {
      constexpr int kBatch = 8;
      float lse[kBatch];
      float4 x[kBatch][2];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int slot = next();
        more = slot >= 0;
        lse[q] = -INFINITY;
        x[q][0] = x[q][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= 0 && valid) {
          const float* base = p.slots + (int64_t)slot * C::kSlotFloats;
          lse[q] = __ldcg(base + (int64_t)kTrBlock * D + in_block);
          const float4* v =
              reinterpret_cast<const float4*>(base) + (in_block >> 7) * (D / 4 * kTrTile) + (in_block & 127);
          x[q][0] = __ldcg(v + (2 * oct) * kTrTile);
          x[q][1] = __ldcg(v + (2 * oct + 1) * kTrTile);
        }
      }
      float mb = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) mb = fmaxf(mb, lse[i]);
      const float mu = mb == -INFINITY ? 0.f : mb;
      const float sc = M == -INFINITY ? 0.f : fast_exp2(M - mu);
      L *= sc;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        acc[k].x *= sc;
        acc[k].y *= sc;
        acc[k].z *= sc;
        acc[k].w *= sc;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (lse[i] == -INFINITY) continue;
        const float wgt = fast_exp2(lse[i] - mu);
        L += wgt;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          acc[k].x = fmaf(wgt, x[i][k].x, acc[k].x);
          acc[k].y = fmaf(wgt, x[i][k].y, acc[k].y);
          acc[k].z = fmaf(wgt, x[i][k].z, acc[k].z);
          acc[k].w = fmaf(wgt, x[i][k].w, acc[k].w);
        }
      }
      M = mb;
    }
    if (!valid) continue;
    const int tok = (int)fast_div((uint32_t)row, p.g_magic, p.g_shift);
    const int64_t orow = (int64_t)(f.t0 + tok) * p.hq + (int64_t)f.kvh * p.group + (row - tok * p.group);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + orow * D + 8 * oct) =
        make_uint4(TC<T>::pack(acc[0].x * inv, acc[0].y * inv), TC<T>::pack(acc[0].z * inv, acc[0].w * inv),
                   TC<T>::pack(acc[1].x * inv, acc[1].y * inv), TC<T>::pack(acc[1].z * inv, acc[1].w * inv));
    if (oct == 0) p.lse_out[orow] = L == 0.f ? -INFINITY : M + fast_log2(L);
  }
}

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

using TreeKernel = void (*)(const TreeParams, const CUtensorMap, const CUtensorMap);
using MergeKernel = void (*)(const TreeParams);

template <typename T, int D, bool TMA>
TreeKernel pick_window(bool sliding) {
  return sliding ? pa_v2_tree_attention_kernel<T, D, TMA, true> : pa_v2_tree_attention_kernel<T, D, TMA, false>;
}
template <typename T>
TreeKernel pick_tree(int D, bool tma, bool sliding) {
  if (D == 64) return tma ? pick_window<T, 64, true>(sliding) : pick_window<T, 64, false>(sliding);
  return tma ? pick_window<T, 128, true>(sliding) : pick_window<T, 128, false>(sliding);
}

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
namespace {

// window 0: none, and positions are not read.
pa_status tree_attention(const void* q, const void* k_pool, const void* v_pool, int32_t kv_dtype, int64_t num_pages,
                         int32_t page_size, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                         const int32_t* indices, int64_t num_indices, const int32_t* indptr,
                         const int32_t* last_page_len, const int32_t* first_page_offset, int32_t batch,
                         const int32_t* qo_indptr, int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
                         const int32_t* positions, int32_t window, float sm_scale, void* out, float* lse2_out,
                         void* workspace, int64_t workspace_bytes, int32_t* status, void* cuda_stream) {
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
  const TreeKernel fn = f16 ? pick_tree<__half>(head_dim, tma, window > 0)
                            : pick_tree<__nv_bfloat16>(head_dim, tma, window > 0);
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

}  // namespace
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
                            num_tokens, tree_mask, mask_words, nullptr, 0, sm_scale, out, lse2_out, workspace,
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
                            num_tokens, tree_mask, mask_words, positions, window, sm_scale, out, lse2_out, workspace,
                            workspace_bytes, status, cuda_stream);
}
