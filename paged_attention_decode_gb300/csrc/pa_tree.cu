// pa_tree.cu -- pa_v2_tree_attention: attention of several query tokens per
// request (a tree or a chain of new tokens) over the paged cache, on the
// fifth-generation tensor cores.
//
// Query token i of request r sees the L - n earlier visible tokens and the new
// tokens its mask row (or the chain rule j <= i) allows:
//   s = scale log2(e) q . k,  out = sum 2^(s - m) v / sum 2^(s - m),
// one pass over the keys with a running maximum m and sum in f32.
//
// Work.  The query rows of a KV head are its n * G (token, head) pairs; a block
// of up to 256 of them meets the request's keys in tiles of 128 pool rows (page
// order, so a tile is whole pages or whole slices of one).  One block against
// one tile is a unit; the units of all (request, KV head, block) in order are
// cut into equal runs, one per CTA and one CTA per SM, whatever the lengths: no
// host plan, no wave tail.  A CTA's run meets several blocks or a part of one;
// a block whole inside a run is written as the result, parts go to the
// workspace and pa_v2_tree_merge_kernel folds them.  When a request has several
// blocks, its keys are cut into segments of about one run and the order is
// segment by segment, so the CTAs at work on one segment's blocks read the same
// keys at about the same time (out of L2).
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
//  - warp 9 (and 10): loads K and V tiles through a ring of shared-memory
//    stages, TMA boxes of up to 16 rows x 64 elements per page, or cp.async for
//    page sizes whose pages do not start on 8-row boundaries; it also walks the
//    CTA's run and hands the pieces to the other roles;
//  - warp 11: makes V tiles that hold rows outside the visible range or new
//    tokens safe: 0 * NaN is NaN, so what a mask hides must not be left in V.
//    Outside rows become zeros; non-finite elements of new tokens become zeros
//    and are added back, in the epilogue, to the rows that do see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pa_internal.cuh"
#include "pa_mma.cuh"
#include "pa_tc05.cuh"

namespace pa {
namespace {

constexpr int kTrThreads = 384;
constexpr int kTrTile = 128;      // query rows of a tensor-core tile, and keys of a key tile
constexpr int kTrBlock = 256;     // query rows of a block
constexpr int kTrSlots = 3;       // partial results a CTA can leave (see piece_slot)
constexpr int kTrMmaWarp = 8, kTrLoadWarp = 9, kTrFixWarp = 11;
constexpr int kTrLoadThreads = 64;  // loader threads without TMA
constexpr int kTrRing = 2;        // pieces handed out ahead
constexpr int kMergeThreads = 256;

// Tensor-memory columns: S of both streams (P over its first 64), then O of both.
constexpr uint32_t kTrTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int w) { return 128u * w; }
__device__ __forceinline__ uint32_t col_o(int w) { return 256u + 128u * w; }

template <int D>
struct TreeCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTrTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 9;  // all the shared memory that the Q tiles leave
  static constexpr int kOffKv = 2 * kTileBytes;     // Q tiles first
  static constexpr int kOffMisc = kOffKv + kStages * kTileBytes;
  static constexpr int kSmem = kOffMisc + 2048;
  static constexpr int kSmemAlloc = kSmem + 1024;   // room to align the base
  static constexpr int64_t kSlotFloats = (int64_t)kTrBlock * (D + 1);
};

// P is rounded to 16 bits relative to 2^kShift at the row's offset, and the offset follows the running maximum
// with a lag of up to kLazy (log2 units).  bf16 has f32's range and takes a wide lag.  f16 holds nothing below
// 2^-24: the shift keeps weights down to 2^-35 of the largest (a long context can hold thousands of those), and
// 2^(kShift + kLazy) stays below its largest value.
template <typename T> struct PRange;
template <> struct PRange<__half> { static constexpr float kShift = 11.f, kLazy = 4.f; };
template <> struct PRange<__nv_bfloat16> { static constexpr float kShift = 0.f, kLazy = 8.f; };

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
  float* slots;    // partial results: kTrSlots per CTA
  int32_t* status;
  int64_t num_pages, num_indices;
  int32_t batch, num_tokens, mask_words, page_size, hq, hkv, group, ctas;
  uint32_t ps_magic, ps_shift, g_magic, g_shift;
  float scale_log2;   // |sm_scale| * log2(e), or 1 for a zero scale
  uint32_t q_xor;     // sign flip of both halves of a q word for a negative scale
  uint32_t q_and;     // 0 for a zero scale
};

// One request's share of the work.
struct TreeReq {
  int32_t slot_base, pages;
  int32_t t0, n;       // its query tokens
  int32_t lo, hi, ds;  // pool rows in page order: visible [lo, hi), new tokens [ds, hi)
  int32_t blocks;      // blocks of query rows per KV head
  int32_t tile0;       // first key tile
  int32_t common;      // key tiles every block meets
  int32_t sum_tail;    // further key tiles, over all blocks (chains: a block stops at its last token)
  bool chain, empty;   // empty: nothing visible or a bad table: zeros and -inf

  __device__ __forceinline__ int64_t units() const { return (int64_t)blocks * common + sum_tail; }  // per KV head
};

__device__ __forceinline__ int32_t tail_of(const TreeReq& g, int group, int b) {
  if (!g.chain || g.empty) return 0;
  const int64_t tok = min((int64_t)g.n, ((int64_t)kTrBlock * (b + 1) + group - 1) / group);
  return (int32_t)((g.ds + tok + kTrTile - 1) / kTrTile) - g.tile0 - g.common;
}

__device__ __forceinline__ TreeReq tree_req(const TreeParams& p, int r, bool tell) {
  TreeReq g;
  const int32_t a = p.qo_indptr[r], b = p.qo_indptr[r + 1];
  const int32_t s0 = p.indptr[r], s1 = p.indptr[r + 1];
  const int32_t lpl = p.last_page_len[r], fpo = p.first_page_offset[r];
  g.t0 = a;
  g.n = b - a;
  g.lo = g.hi = g.ds = g.tile0 = g.sum_tail = 0;
  g.slot_base = s0;
  g.pages = 0;
  g.blocks = g.common = 0;
  g.chain = p.tree_mask == nullptr;
  g.empty = true;
  if (a < 0 || b < a || b > p.num_tokens) {
    if (tell) report(p.status, PA_DEVICE_BAD_INDPTR);
    g.n = 0;
  }
  if (g.n == 0) return g;
  g.blocks = (int32_t)(((int64_t)g.n * p.group + kTrBlock - 1) / kTrBlock);
  g.common = 1;  // one unit for an empty block
  const int64_t pages = (int64_t)s1 - s0;
  if (s0 < 0 || pages < 0 || s1 > p.num_indices || pages * p.page_size > INT32_MAX - 2 * kTrTile) {
    if (tell) report(p.status, PA_DEVICE_BAD_SLOT);
    return g;
  }
  const int64_t hi = pages > 0 ? (pages - 1) * p.page_size + lpl : 0;
  if (pages == 0 || lpl < 1 || lpl > p.page_size || fpo < 0 || fpo >= p.page_size || hi - fpo < g.n ||
      (p.tree_mask && g.n > 32 * p.mask_words)) {
    if (tell) report(p.status, PA_DEVICE_BAD_TREE);
    return g;
  }
  g.empty = false;
  g.pages = (int32_t)pages;
  g.lo = fpo;
  g.hi = (int32_t)hi;
  g.ds = g.hi - g.n;
  g.tile0 = g.lo / kTrTile;
  const int32_t all = (g.hi + kTrTile - 1) / kTrTile - g.tile0;
  if (g.blocks == 1 || !g.chain) {
    g.common = all;
    g.chain = g.chain && g.blocks > 1;
  } else {
    g.common = max(g.ds / kTrTile - g.tile0, 0);
    for (int b2 = 0; b2 < g.blocks; ++b2) g.sum_tail += tail_of(g, p.group, b2);
  }
  return g;
}

// Segments of a request's common key tiles: one when it has one block, else about one CTA's run each.
__device__ __forceinline__ int32_t segments(const TreeReq& g, int64_t run) {
  if (g.blocks <= 1 || g.common == 0) return 1;
  return (int32_t)((g.common + run - 1) / run);
}
__device__ __forceinline__ int32_t seg_begin(const TreeReq& g, int32_t S, int32_t s) {
  return (int32_t)((int64_t)s * g.common / S);
}

// Place of a partial result that starts `pos` units into its CTA's run of `run` units.  A run meets at most one
// piece at its start (pos 0) and pieces of at least ceil(run / 2) units, or the run's last one, after it: a block
// in one segment is cut only by the ends of a run, and a request is cut into several segments only when its
// common tiles exceed a run, which makes each at least ceil(run / 2) long.
__device__ __forceinline__ int piece_slot(int64_t pos, int64_t run) {
  return pos == 0 ? 0 : 1 + (int)((pos - 1) / ((run + 1) / 2));
}

// Where the block-wide scan below found a unit.
struct TreeStart {
  int64_t total, run;  // all units; units per CTA
  int64_t off;         // the unit's offset inside request r
  int32_t r;           // batch when the unit is past the end
};

// Every thread of the block: units of all requests, the run length, and the request of unit `cta * run`.
template <int THREADS>
__device__ __forceinline__ void tree_schedule(const TreeParams& p, int64_t cta, bool tell, TreeStart* out,
                                              int64_t* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int r0 = min((int64_t)tid * per, (int64_t)p.batch), r1 = min(r0 + per, p.batch);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += tree_req(p, r, tell).units() * p.hkv;
  int64_t v = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, w);
    if (lane >= w) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  int64_t before = v - mine, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t run = (total + p.ctas - 1) / p.ctas;
  const int64_t unit = cta * run;
  if (tid == 0) {
    out->total = total;
    out->run = run;
    if (unit >= total) {
      out->r = p.batch;
      out->off = 0;
    }
  }
  if (unit < total && unit >= before && unit < before + mine) {
    int64_t off = unit - before;
    int r = r0;
    for (; r < r1; ++r) {
      const int64_t u = tree_req(p, r, false).units() * p.hkv;
      if (off < u) break;
      off -= u;
    }
    out->r = r;
    out->off = off;
  }
  __syncthreads();
}

// A run of key tiles of one block, as the loader hands it to the other roles.
struct TreePiece {
  int32_t kind;            // 0: no more, 1: key tiles, 2: nothing visible
  int32_t tile, tiles;     // key tiles [tile, tile + tiles)
  int32_t lo, hi, ds;
  int32_t t0, n;
  int32_t slot_base;       // the request's first page-table slot
  int32_t row0, rows;      // query rows [row0, row0 + rows) of the request
  int32_t kvh, slot;       // slot < 0: the whole block, written as the result
  int32_t tainted;         // set by the fix warp: a visible new token has a non-finite value
};

constexpr int kPieceEnd = 0, kPieceTiles = 1, kPieceEmpty = 2;

__device__ __forceinline__ bool needs_fix(const TreePiece& d, int tile) {
  return tile * kTrTile < d.lo || (tile + 1) * kTrTile > d.ds;
}

// Bits [a, b) of a word, a and b clamped to [0, 32].
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b >= 32 ? 0xffffffffu : ((1u << b) - 1u)) & ~((1u << a) - 1u);
}

// Which of the keys base .. base+31 (page order) query token i of the piece sees.
__device__ __forceinline__ uint32_t visible_bits(const TreeParams& p, const TreePiece& d, int i, int base) {
  uint32_t bits = bit_range(d.lo - base, d.ds - base);
  if (base + 32 > d.ds && base < d.hi) {
    if (p.tree_mask) {
      const int32_t* row = p.tree_mask + (int64_t)(d.t0 + i) * p.mask_words;
      const int at = base - d.ds;  // new-token index of bit 0
      const int w = at >> 5, sh = at & 31;
      const uint32_t x0 = w >= 0 && w < p.mask_words ? (uint32_t)__ldg(row + w) : 0u;
      const uint32_t x1 = w + 1 >= 0 && w + 1 < p.mask_words ? (uint32_t)__ldg(row + w + 1) : 0u;
      bits |= __funnelshift_r(x0, x1, sh) & bit_range(d.ds - base, d.hi - base);
    } else {
      bits |= bit_range(d.ds - base, min(d.ds + i + 1, d.hi) - base);
    }
  }
  return bits;
}

// D[128 x N] (+)= A[128 x 16] B[16 x N], A in tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
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

template <typename T, int D, bool TMA>
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
  uint64_t* b_p = b_s + 2;                // 2: P of a stream is written (one arrival per warp)
  uint64_t* b_o = b_p + 2;                // the piece's products are complete
  uint64_t* b_q = b_o + 1;                // the piece's Q is in shared memory
  uint64_t* b_fix = b_q + 1;              // kStages: the V tile in a stage was made safe
  uint64_t* b_x = b_fix + C::kStages;     // stream B's state is in shared memory
  uint64_t* b_xd = b_x + 1;               // ... and has been read
  uint64_t* b_pf = b_xd + 1;              // kTrRing: a piece is handed out
  uint64_t* b_pe = b_pf + kTrRing;        // kTrRing: every role is done with it
  uint64_t* b_drain = b_pe + kTrRing;
  TreePiece* ring = reinterpret_cast<TreePiece*>(b_drain + 1);
  TreeStart* start = reinterpret_cast<TreeStart*>(ring + kTrRing);
  int64_t* warp_sum = reinterpret_cast<int64_t*>(start + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(warp_sum + kTrThreads / 32);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
  float* xstate = reinterpret_cast<float*>(tmem_slot + 2);  // [2][128]: stream B's maxima and sums
  static_assert((3 * C::kStages + 9 + 2 * kTrRing) * 8 + kTrRing * sizeof(TreePiece) + sizeof(TreeStart) +
                        kTrThreads / 32 * 8 + 8 + 2 * kTrTile * 4 <=
                    2048,
                "the area behind the stages");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_addr(smem);

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b_full[i], TMA ? 1 : kTrLoadThreads);
      mbar_init(&b_empty[i], 2);  // the MMAs that read the stage, and the fix warp
      mbar_init(&b_fix[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&b_s[w], 1);
      mbar_init(&b_p[w], 4);
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
  pdl_wait_prerequisites();
  tree_schedule<kTrThreads>(p, blockIdx.x, blockIdx.x == 0, start, warp_sum);

  if (warp == kTrLoadWarp || (!TMA && warp == kTrLoadWarp + 1)) {
    // ------------------------------------------------------------------ loader
    const bool leader = warp == kTrLoadWarp;
    const int64_t run = start->run;
    int64_t left = min(run, start->total - (int64_t)blockIdx.x * run);  // units to go (<= 0: none)
    int r = start->r;
    int64_t off = start->off;
    int stage = 0, pieces = 0, ops = 0;
    int pend = -1;  // without TMA: the stage whose copies are not published yet
    bool alive = true;
    const int u = (warp - kTrLoadWarp) * 32 + lane;
    TreeReq g = {};
    const int box_rows = p.page_size < 16 ? p.page_size : 16;
    const uint64_t policy = policy_evict_first();

    auto publish = [&]() {  // without TMA: the pending stage's copies have landed
      fence_proxy_async_smem();
      mbar_arrive(&b_full[pend]);
      pend = -1;
    };
    // K (or V) rows [128 tile, 128 tile + 128) of the request's pages into the next stage
    auto load = [&](int tile, int kvh, bool is_v) {
      if (!wait_phase(&b_empty[stage], ((ops / C::kStages) & 1) ^ 1, abort_flag, p.status)) {
        alive = false;
        return;
      }
      const uint32_t dst = sbase + C::kOffKv + stage * C::kTileBytes;
      const int row0 = tile * kTrTile;
      const int rows = min(kTrTile, g.hi - row0);
      if (TMA) {
        const int boxes = (rows + box_rows - 1) / box_rows;
        if (lane == 0) mbar_arrive_expect_tx(&b_full[stage], (uint32_t)(boxes * box_rows * D * 2));
        __syncwarp();
        for (int i = lane; i < boxes * C::kHalves; i += 32) {
          const int box = i / C::kHalves, half = i % C::kHalves;
          const int at = row0 + box * box_rows;
          const int slot = (int)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
          const int32_t page = __ldg(p.indices + g.slot_base + slot);
          int32_t row;
          if (page >= 0 && page < p.num_pages) {
            row = page * p.page_size + (at - slot * p.page_size);
          } else {
            row = (int32_t)(p.num_pages * p.page_size);  // past the pool: the box is zero-filled
            if (!is_v && half == 0) report(p.status, PA_DEVICE_BAD_PAGE);
          }
          tma_load_3d(smem + C::kOffKv + stage * C::kTileBytes + half * (kTrTile * 128) + box * box_rows * 128,
                      is_v ? &tm_v : &tm_k, &b_full[stage], half * 64, kvh, row, policy);
        }
        __syncwarp();
      } else {
        constexpr int kChunks = D / 8;                       // 16-byte pieces of a row
        constexpr int kPass = kTrLoadThreads / kChunks;      // rows per pass
        const int ch = u % kChunks;
        const uint32_t col = (uint32_t)(ch >> 3) * (kTrTile * 128);
        const T* pool = static_cast<const T*>(is_v ? p.v_pool : p.k_pool) + (int64_t)kvh * D + ch * 8;
#pragma unroll 8
        for (int i = 0; i < kTrTile / kPass; ++i) {
          const int row = i * kPass + u / kChunks;
          const int at = row0 + row;
          const uint32_t to = dst + col + sw128(row, ch & 7);
          bool have = at >= g.lo && at < g.hi;
          if (have) {
            const int slot = (int)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
            const int32_t page = __ldg(p.indices + g.slot_base + slot);
            have = page >= 0 && page < p.num_pages;
            if (have)
              cp_async_16(to, pool + ((int64_t)page * p.page_size + (at - slot * p.page_size)) * p.hkv * D, policy);
            else if (ch == 0 && !is_v)
              report(p.status, PA_DEVICE_BAD_PAGE);
          }
          if (!have) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0u) : "memory");
        }
        cp_async_commit();
        if (pend >= 0) {
          cp_async_wait<1>();
          publish();
        }
        pend = stage;
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

    int64_t pos = 0;  // units done
    while (left > 0 && alive && r < p.batch) {
      g = tree_req(p, r, false);
      const int64_t per_head = g.units();
      const int32_t S = segments(g, run);
      int kvh = per_head > 0 ? (int)(off / per_head) : p.hkv;
      int64_t x = per_head > 0 ? off % per_head : 0;
      for (; kvh < p.hkv && left > 0 && alive; ++kvh, x = 0) {
        for (int s = 0; s < S && left > 0 && alive; ++s) {
          const int32_t t_begin = seg_begin(g, S, s);
          const int32_t len_s = seg_begin(g, S, s + 1) - t_begin;
          const int64_t seg_units = (int64_t)g.blocks * len_s + (s == S - 1 ? g.sum_tail : 0);
          if (x >= seg_units) {
            x -= seg_units;
            continue;
          }
          int b = 0;
          if (len_s > 0 && (s < S - 1 || g.sum_tail == 0)) {
            b = (int)(x / len_s);
            x -= (int64_t)b * len_s;
          }
          for (; b < g.blocks && left > 0 && alive; ++b) {
            const int32_t len = len_s + (s == S - 1 ? tail_of(g, p.group, b) : 0);
            if (x >= len) {
              x -= len;
              continue;
            }
            TreePiece d;
            d.kind = g.empty ? kPieceEmpty : kPieceTiles;
            d.tile = g.tile0 + t_begin + (int32_t)x;
            d.tiles = (int32_t)min((int64_t)len - x, left);
            d.lo = g.lo;
            d.hi = g.hi;
            d.ds = g.ds;
            d.t0 = g.t0;
            d.n = g.n;
            d.slot_base = g.slot_base;
            d.row0 = b * kTrBlock;
            d.rows = min(kTrBlock, g.n * p.group - d.row0);
            d.kvh = kvh;
            d.slot = S == 1 && x == 0 && d.tiles == len ? -1 : (int)blockIdx.x * kTrSlots + piece_slot(pos, run);
            d.tainted = 0;
            hand_out(d);
            if (!alive) break;
            if (d.kind == kPieceTiles) {
              const int ahead = d.rows > kTrTile ? 1 : 2;  // key tiles S runs ahead of O (as the MMA warp takes them)
              for (int j = 0; j < min(ahead, d.tiles) && alive; ++j) load(d.tile + j, kvh, false);
              for (int j = 0; j < d.tiles && alive; ++j) {
                load(d.tile + j, kvh, true);
                if (j + ahead < d.tiles && alive) load(d.tile + j + ahead, kvh, false);
              }
              if (!TMA && pend >= 0) {
                cp_async_wait<0>();
                publish();
              }
            }
            left -= d.tiles;
            pos += d.tiles;
            x = 0;
          }
          x = 0;
        }
      }
      ++r;
      off = 0;
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
    int op = 0;
    uint32_t par_p[2] = {0, 0}, par_q = 0, par_fix = 0;  // par_fix: a bit per stage
    bool alive = true, issued = false;
    auto take = [&]() -> int {  // the next loaded stage
      const int st = op % C::kStages;
      if (!wait_phase(&b_full[st], (uint32_t)((op / C::kStages) & 1), abort_flag, p.status)) alive = false;
      ++op;
      return st;
    };
    auto scores = [&](int w, int qt, int st) {
      if (lane == 0) {
        const uint32_t qa = sbase + qt * C::kTileBytes, ka = sbase + C::kOffKv + st * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk >> 2) * (kTrTile * 128) + (kk & 3) * 32;
          umma(tmem + col_s(w), smem_desc(qa + at, 16, 1024), smem_desc(ka + at, 16, 1024), id_s, kk != 0);
        }
        umma_commit(&b_s[w]);
        issued = true;
      }
      __syncwarp();
    };
    auto values = [&](int w, int st, bool acc) {
      if (!wait_phase(&b_p[w], par_p[w], abort_flag, p.status)) {
        alive = false;
        return;
      }
      par_p[w] ^= 1;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t va = sbase + C::kOffKv + st * C::kTileBytes;
#pragma unroll
        for (int kt = 0; kt < kTrTile / 16; ++kt)
          umma_ts(tmem + col_o(w), tmem + col_s(w) + 8 * kt, smem_desc(va + kt * 2048, kTrTile * 128, 1024), id_o,
                  acc || kt != 0);
      }
      __syncwarp();
    };
    auto release = [&](int st) {
      if (lane == 0) umma_commit(&b_empty[st]);
      __syncwarp();
    };
    for (int pc = 0; alive; ++pc) {
      const int at = pc % kTrRing;
      if (!wait_phase(&b_pf[at], (uint32_t)((pc / kTrRing) & 1), abort_flag, p.status)) break;
      const TreePiece d = ring[at];
      if (d.kind == kPieceEnd) break;
      if (d.kind == kPieceTiles) {
        const bool dual = d.rows > kTrTile;
        // Q is written, and both streams are done with the piece before
        if (!wait_phase(b_q, par_q, abort_flag, p.status)) break;
        par_q ^= 1;
        tc_fence_after();
        auto wait_fix = [&](int tile, int st) {
          if (!needs_fix(d, tile)) return;
          if (!wait_phase(&b_fix[st], par_fix >> st & 1u, abort_flag, p.status)) alive = false;
          par_fix ^= 1u << st;
        };
        if (dual) {
          int k = take();
          if (!alive) break;
          scores(0, 0, k);
          scores(1, 1, k);
          release(k);
          for (int j = 0; j < d.tiles && alive; ++j) {
            const int v = take();
            if (alive) wait_fix(d.tile + j, v);
            if (alive) values(0, v, j > 0);
            if (alive && j + 1 < d.tiles) {
              k = take();
              if (alive) scores(0, 0, k);
            }
            if (alive) values(1, v, j > 0);
            if (!alive) break;
            release(v);
            if (j + 1 < d.tiles) {
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
        if (lane == 0) umma_commit(b_o);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&b_pe[at]);
      __syncwarp();
    }
    // every MMA of this CTA has completed before tensor memory is released
    if (lane == 0 && issued) umma_commit(b_drain);
    __syncwarp();
    if (__shfl_sync(0xffffffffu, issued ? 1 : 0, 0)) {
      if (!mbar_wait_bounded(b_drain, 0, kWaitLimitCycles) && lane == 0) report(p.status, PA_DEVICE_WAIT_TIMEOUT);
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
          uint32_t any = 0;
          auto fix_rows = [&](int r0, int r1) {
#pragma unroll 4
            for (int row = r0 + lane / kChunks; row < r1; row += 32 / kChunks) {
              const uint32_t a = col + sw128(row, ch & 7);
              uint32_t x0, x1, x2, x3;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                           : "r"(a)
                           : "memory");
              const int pr = c0 + row;
              const bool inside = pr >= d.lo && pr < d.hi;
              constexpr uint32_t e = ExpBits<T>::k;
              const uint32_t n0 = sat_mask(x0, e), n1 = sat_mask(x1, e), n2 = sat_mask(x2, e), n3 = sat_mask(x3, e);
              const uint32_t bad = n0 | n1 | n2 | n3;
              if (inside) any |= bad;
              if (!inside || bad) {
                const uint32_t keep = inside ? 0xffffffffu : 0u;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x0 & ~n0 & keep),
                             "r"(x1 & ~n1 & keep), "r"(x2 & ~n2 & keep), "r"(x3 & ~n3 & keep)
                             : "memory");
              }
            }
          };
          const int head = min(max(d.lo - c0, 0), kTrTile), tail = min(max(d.ds - c0, head), kTrTile);
          fix_rows(0, head);
          fix_rows(tail, kTrTile);
          if (__any_sync(0xffffffffu, any != 0) && lane == 0) *reinterpret_cast<volatile int32_t*>(&ring[at].tainted) = 1;
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
  } else if (warp < 8) {
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
      const TreePiece d = ring[at];
      if (d.kind == kPieceEnd) break;
      const bool dual = d.rows > kTrTile;
      const int rr = (dual ? w * kTrTile : 0) + row;         // row of the block
      const bool valid = rr < d.rows;
      const bool busy = (rr & ~31) < d.rows;                 // a row of this warp is
      const int qrow = d.row0 + min(rr, d.rows - 1);         // row of the request
      const int tok = (int)fast_div((uint32_t)qrow, p.g_magic, p.g_shift);
      const int64_t orow = (int64_t)(d.t0 + tok) * p.hq + (int64_t)d.kvh * p.group + (qrow - tok * p.group);
      float m = -INFINITY, l = 0.f;
      if (d.kind == kPieceTiles) {
        // ---- Q, swizzled like the key tiles; rows past the block are zeros
        if (pending_x) {  // the exchanged state of the piece before shares the Q tiles' memory
          if (!wait_phase(b_xd, par_xd, abort_flag, p.status)) break;
          par_xd ^= 1;
          pending_x = false;
        }
        {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + orow * D);
          unsigned char* dst = smem + (dual ? w : 0) * C::kTileBytes;
          constexpr int kChunks = D / 8;
          const int c_begin = dual ? 0 : w * (kChunks / 2), c_end = dual ? kChunks : c_begin + kChunks / 2;
#pragma unroll 8
          for (int c = c_begin; c < c_end; ++c) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (valid) {
              x = __ldg(src + c);
              x.x = (x.x ^ p.q_xor) & p.q_and;
              x.y = (x.y ^ p.q_xor) & p.q_and;
              x.z = (x.z ^ p.q_xor) & p.q_and;
              x.w = (x.w ^ p.q_xor) & p.q_and;
            }
            *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTrTile * 128) + sw128(row, c & 7)) = x;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_q);
        }
        // ---- key tiles
        for (int j = dual ? 0 : w; j < d.tiles; j += dual ? 1 : 2) {
          if (!wait_phase(&b_s[w], par_s, abort_flag, p.status)) {
            alive = false;
            break;
          }
          par_s ^= 1;
          tc_fence_after();
          if (busy) {
            const int c0 = (d.tile + j) * kTrTile;
            const bool edge = needs_fix(d, d.tile + j);
            uint32_t vis[4];
            if (edge) {
#pragma unroll
              for (int c = 0; c < 4; ++c) vis[c] = visible_bits(p, d, tok, c0 + 32 * c);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x[32];
              __syncwarp();
              tmem_ld32(t_s + 32 * c, x);
              if (edge) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  mx = fmaxf(mx, (vis[c] >> i) & 1u ? __uint_as_float(x[i]) : -INFINITY);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(x[i]));
              }
            }
            const float mt = mx * scale;
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
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[32];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t x[32];
                __syncwarp();
                tmem_ld32(t_s + 64 * h + 32 * c, x);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float y0 = fast_exp2(fmaf(__uint_as_float(x[i]), scale, -mu));
                  float y1 = fast_exp2(fmaf(__uint_as_float(x[i + 1]), scale, -mu));
                  if (edge) {
                    y0 = (vis[2 * h + c] >> i) & 1u ? y0 : 0.f;
                    y1 = (vis[2 * h + c] >> (i + 1)) & 1u ? y1 : 0.f;
                  }
                  sum[i & 2] += y0;
                  sum[(i & 2) + 1] += y1;
                  pk[16 * c + i / 2] = TC<T>::pack(y0, y1);
                }
              }
              __syncwarp();
              tmem_st32(t_s + 32 * h, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_p[w]);
        }
        if (!alive) break;
        if (!wait_phase(b_o, par_o, abort_flag, p.status)) break;
        par_o ^= 1;
        tc_fence_after();
      }

      // ---- the piece's result
      const bool joined = d.kind == kPieceTiles && !dual && d.tiles > 1;  // two streams to join
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
        const bool nothing = l == 0.f;  // no visible key (a NaN sum stays NaN)
        const float inv = nothing ? 0.f : 1.f / l;
        const float lse = nothing ? -INFINITY : m - kShift + fast_log2(l);
        const bool tainted = d.kind == kPieceTiles && *reinterpret_cast<volatile int32_t*>(&ring[at].tainted) != 0;
        T* out = static_cast<T*>(p.out) + orow * D;
        float* slot = p.slots + (int64_t)max(d.slot, 0) * C::kSlotFloats;
        float4* part = reinterpret_cast<float4*>(slot) + (rr >> 7) * (D / 4 * kTrTile) + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (d.kind == kPieceTiles) {
            __syncwarp();
            tmem_ld32(t_o + 32 * c, o);
          }
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = nothing ? 0.f : __uint_as_float(o[i]);
          if (joined && !nothing) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 y = xo[(8 * c + i) * kTrTile + row];
              v[4 * i] = v[4 * i] * s0 + y.x * s1;
              v[4 * i + 1] = v[4 * i + 1] * s0 + y.y * s1;
              v[4 * i + 2] = v[4 * i + 2] * s0 + y.z * s1;
              v[4 * i + 3] = v[4 * i + 3] * s0 + y.w * s1;
            }
          }
          if (tainted && !nothing) {
            // the non-finite values the fix warp took out, back to the rows that see them
            const int k0 = max(d.tile * kTrTile, d.ds), k1 = min((d.tile + d.tiles) * kTrTile, d.hi);
            for (int k = k0; k < k1; ++k) {
              if (!(visible_bits(p, d, tok, k) & 1u)) continue;
              const int sl = (int)fast_div((uint32_t)k, p.ps_magic, p.ps_shift);
              const int32_t page = __ldg(p.indices + d.slot_base + sl);
              if (page < 0 || page >= p.num_pages) continue;
              const T* src = static_cast<const T*>(p.v_pool) +
                             (((int64_t)page * p.page_size + (k - sl * p.page_size)) * p.hkv + d.kvh) * D + 32 * c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = half_of(src + i);
                if (!isfinite(y)) v[i] += y;
              }
            }
          }
          if (valid && d.slot < 0) {
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
          if (d.slot < 0)
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
// order of the keys.  A KV head of a request with cuts is shared out over the CTAs of the cuts inside it (cut c
// is unit c * run); a warp takes 32 rows x 8 columns, one row per lane (the parts are stored column by column, so
// a warp's loads are contiguous), eight parts in flight.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) pa_v2_tree_merge_kernel(const TreeParams p) {
  __shared__ TreeStart start;
  __shared__ int64_t warp_sum[kMergeThreads / 32];
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int64_t cut = (int64_t)blockIdx.x + 1;
  tree_schedule<kMergeThreads>(p, cut, false, &start, warp_sum);
  if (start.r >= p.batch) return;
  const int64_t run = start.run, unit = cut * run;
  const TreeReq g = tree_req(p, start.r, false);
  if (g.empty) return;
  const int64_t per_head = g.units();
  const int kvh = (int)(start.off / per_head);
  const int64_t first = unit - start.off % per_head;  // first unit of this KV head
  if (first == unit) return;                          // the cut falls between two heads
  const int64_t c_first = first / run + 1, c_last = (first + per_head - 1) / run;
  const int32_t S = segments(g, run);
  const int rows = g.n * p.group;
  const int64_t jobs = (int64_t)((rows + 31) / 32) * (D / 8);
  const int64_t workers = (c_last - c_first + 1) * gridDim.y * (kMergeThreads / 32);
  const int64_t me = ((cut - c_first) * gridDim.y + blockIdx.y) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  using C = TreeCfg<D>;
  for (int64_t job = me; job < jobs; job += workers) {
    const int rg = (int)(job / (D / 8)), oct = (int)(job % (D / 8));
    const int row = rg * 32 + lane;
    const int b = rg * 32 / kTrBlock;
    const int in_block = row - b * kTrBlock;
    const bool valid = row < rows;
    // the block's parts: for each segment, the runs its units fall into
    int s = 0;
    int64_t at = 0, end = 0;  // units of the current segment still to visit
    int64_t seg_first = 0;
    bool more = true, whole = false;
    auto enter = [&]() {  // unit range of block b in segment s
      const int32_t t0 = seg_begin(g, S, s), len_s = seg_begin(g, S, s + 1) - t0;
      int64_t lead = (int64_t)b * len_s;
      int32_t len = len_s;
      if (s == S - 1) {
        for (int i = 0; g.sum_tail && i < b; ++i) lead += tail_of(g, p.group, i);
        len += tail_of(g, p.group, b);
      }
      seg_first = at = first + (int64_t)g.blocks * t0 + lead;
      end = at + len;
    };
    enter();
    whole = S == 1 && at / run == (end - 1) / run;  // one piece: already written as the result
    if (whole) continue;
    auto next = [&]() -> int64_t {  // slot of the next part, or -1
      while (more && at >= end) {
        if (++s >= S) {
          more = false;
          break;
        }
        enter();
      }
      if (!more) return -1;
      const int64_t cta = at / run;
      const int64_t slot = cta * kTrSlots + piece_slot(at - cta * run, run);
      at = min((cta + 1) * run, end);
      return slot;
    };
    float M = -INFINITY, L = 0.f;
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    while (more) {
      constexpr int kBatch = 8;
      float lse[kBatch];
      float4 x[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t slot = next();
        lse[i] = -INFINITY;
        x[i][0] = x[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= 0 && valid) {
          const float* base = p.slots + slot * C::kSlotFloats;
          lse[i] = __ldcg(base + (int64_t)kTrBlock * D + in_block);
          const float4* v = reinterpret_cast<const float4*>(base) + (in_block >> 7) * (D / 4 * kTrTile) + (in_block & 127);
          x[i][0] = __ldcg(v + (2 * oct) * kTrTile);
          x[i][1] = __ldcg(v + (2 * oct + 1) * kTrTile);
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
    const int64_t orow = (int64_t)(g.t0 + tok) * p.hq + (int64_t)kvh * p.group + (row - tok * p.group);
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

template <typename T>
TreeKernel pick_tree(int D, bool tma) {
  if (D == 64) return tma ? pa_v2_tree_attention_kernel<T, 64, true> : pa_v2_tree_attention_kernel<T, 64, false>;
  return tma ? pa_v2_tree_attention_kernel<T, 128, true> : pa_v2_tree_attention_kernel<T, 128, false>;
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
  *bytes = (int64_t)ctas * pa::kTrSlots * (int64_t)sizeof(float) *
           (head_dim == 64 ? pa::TreeCfg<64>::kSlotFloats : pa::TreeCfg<128>::kSlotFloats);
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
  if ((int64_t)num_tokens * (num_qo_heads / num_kv_heads) > INT32_MAX - 2 * pa::kTrBlock) return PA_EUNSUPPORTED;
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
  alignas(64) CUtensorMap tm_k, tm_v;
  std::memset(&tm_k, 0, sizeof(tm_k));
  std::memset(&tm_v, 0, sizeof(tm_v));
  const bool tma = pa::tc_uses_tma(page_size);
  if (tma) {
    const int box_rows = page_size < 16 ? page_size : 16;
    if (!pa::make_pool_map(&tm_k, k_pool, kv_dtype, num_pages * page_size, num_kv_heads, head_dim, 64, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pa::make_pool_map(&tm_v, v_pool, kv_dtype, num_pages * page_size, num_kv_heads, head_dim, 64, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B))
      return PA_ECUDA;
  }
  pa::TreeParams p;
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
  p.mask_words = mask_words;
  p.page_size = page_size;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.group = num_qo_heads / num_kv_heads;
  const pa_status sm = pa::tree_ctas(dev, &p.ctas);
  if (sm != PA_OK) return sm;
  const pa::FastDiv fd = pa::FastDiv::make((uint32_t)page_size), fg = pa::FastDiv::make((uint32_t)p.group);
  p.ps_magic = fd.magic;
  p.ps_shift = fd.shift;
  p.g_magic = fg.magic;
  p.g_shift = fg.shift;
  const bool flat = std::fabs(sm_scale) < 1e-30f;  // every score is zero
  p.scale_log2 = flat ? 1.f : std::fabs(sm_scale) * 1.4426950408889634f;
  p.q_xor = sm_scale < 0.f ? 0x80008000u : 0u;
  p.q_and = flat ? 0u : 0xffffffffu;
  const bool f16 = kv_dtype == PA_F16;
  const int smem = head_dim == 64 ? pa::TreeCfg<64>::kSmemAlloc : pa::TreeCfg<128>::kSmemAlloc;
  const pa::TreeKernel fn = f16 ? pa::pick_tree<__half>(head_dim, tma) : pa::pick_tree<__nv_bfloat16>(head_dim, tma);
  if (!pa::prepare_kernel(reinterpret_cast<const void*>(fn), smem)) return PA_ECUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (pa::launch_dependent(fn, dim3(p.ctas), dim3(pa::kTrThreads), smem, stream, p, tm_k, tm_v) != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  const pa::MergeKernel merge =
      f16 ? (head_dim == 64 ? pa::pa_v2_tree_merge_kernel<__half, 64> : pa::pa_v2_tree_merge_kernel<__half, 128>)
          : (head_dim == 64 ? pa::pa_v2_tree_merge_kernel<__nv_bfloat16, 64>
                            : pa::pa_v2_tree_merge_kernel<__nv_bfloat16, 128>);
  if (p.ctas > 1) {
    const cudaError_t rc = pa::launch_dependent(merge, dim3(p.ctas - 1, 2), dim3(pa::kMergeThreads), 0, stream, p);
    if (rc != cudaSuccess) {
      cudaGetLastError();
      return PA_ECUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
