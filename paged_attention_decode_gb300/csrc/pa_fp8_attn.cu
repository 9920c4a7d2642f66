// pa_fp8_attn.cu -- pa_v2_attention_fp8: attention of each request's new tokens (one,
// a chain or a tree of them) over a paged cache of e4m3 codes with a power-of-two
// exponent for each page and KV head.
//
//   k_j = 2^ek(page of j) kc_j,   v_j likewise,
//   s_ij = scale log2(e) 2^ek(j) q_i . kc_j,  out_i = sum 2^(s_ij - m_i) v_j / sum 2^(s_ij - m_i),
// one pass over the keys with a running maximum m and sum in f32.  The codes become f16
// in registers (exactly), q is f16 times a power of two of its row (exact but for
// elements 2^-24 of the row's largest and below), and the exponents, -15 .. 7, keep every
// 2^ev vc a binary16 number: both products of m16n8k16 have exact operands but for P,
// which is rounded to f16 once, 2^kF8Shift at the row's offset: by 2^-11 of a weight down to
// 2^-25 of the offset's, where f16 is normal (the f16 or bf16 output rounds by 2^-11 or 2^-8
// anyhow), and by 2^-36 of the offset's below, 2^20 keys of it together 2^-16 of the largest
// value; scores, statistics and sums, of weights before that rounding, are f32.
//
// Work.  The query rows of a KV head (n * G pairs of new token and head) are taken in
// blocks of 8 NT; one block against one tile of 32 pool rows (page order) is a unit.  The
// units of the batch in order (request, KV head, block, tile) are cut into equal runs over
// the warps of one CTA per SM: no host plan, no wave tail, whatever the lengths.  A warp
// that meets a block's tiles alone writes its result; the others leave partial results,
// which pa_v2_fp8_merge_kernel folds.  Where runs are long, a run belongs to a team of
// warps, one for each KV head: a page's rows of all heads lie side by side, and asked for
// at the same time HBM serves them at 6.2 TB/s, one head after the other at 5.2.  Where
// runs are short, partial results cost more than that gains: there neighbouring runs of a
// head go to the warps of a CTA, which joins their parts in shared memory first.
//
// A warp owns a ring of stages (a stage: 32 K rows and 32 V rows of D bytes) and walks
// its units without a block barrier: TMA boxes, 128- or 64-byte swizzled, or 16-byte
// cp.async copies for page sizes that do not start on 8-row boundaries.  S^T = K Q^T takes
// the K rows as the A operand: a lane's fragment is the 16 dims of one LDS.128 per four
// k-steps, since the order of the dims is free as long as q's is the same.  O^T += V^T P^T
// takes V through ldmatrix.trans of byte pairs: a register holds two tokens x two dims,
// one byte permutation apart from the two A registers it becomes.  P^T goes from the
// accumulator's layout to the B operand's by movmatrix.
//
// What bounds it (GB300, 32 query heads on 8 KV heads, D = 128, page size 16, replayed over
// three sets of inputs in turn): 64 ragged requests of 1K-32K, one token each, 214-229 us,
// 5.9-6.2 TB/s of 6.8 measured: HBM; 52 % of the issue slots.  32 chains of 5 tokens in a
// window of 4096 with 4 sinks 78 us of 29: 20 of 24 columns of products, two warps a scheduler
// that wait for one another's shuffles and conversions, 35 % of the issue slots.  One token over
// 32K 25 us (10 of HBM), over 1K 13 us: starts (8 us: cold code, tables, pages, tiles, one after the other),
// joining 2-3, the merge kernel 4.  More warps help while registers allow them (12 at 168
// for one block of 8 rows: 26 -> 23 us over 32K; the wider blocks need 255); q in registers
// up to 16 rows, in shared memory for 24.  Measured and not kept: blocks of 32 rows (spills); the
// same code for a request's geometry called, not inlined (+2 us everywhere); lanes as parts in
// the joining (equal).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pa_internal.cuh"
#include "pa_launch.h"
#include "pa_mma.cuh"
#include "pa_pool_map.h"
#include "pa_tc05.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kF8MaxWarps = 12;
constexpr int kF8Tile = 32;       // keys of a unit
constexpr int kF8Infos = 8;       // requests a warp's ring can have under way, a power of two
constexpr float kF8Shift = 11.f;  // P is rounded relative to 2^kF8Shift at the row's offset,
constexpr float kF8Lazy = 4.f;    // which follows the running maximum with a lag of up to kF8Lazy (log2 units)
constexpr int kF8MaxRows = 24;    // query rows of a block, at most
constexpr int kMergeWarps = 8;
constexpr int kMergeFew = 16;     // parts that one warp folds alone
constexpr int kMergeCtas = 2;     // per SM
constexpr int kF8PartRows = 192;  // rows of a CTA's runs, at most: 12 warps of 8, 8 of 24
constexpr int64_t kF8Spread = 16;  // units of a run from which on heads are taken side by side
constexpr int64_t kF8MaxUnits = 1ll << 40;  // units of one request, at most

template <int D, int NT>
struct F8Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kSide = kF8Tile * D;    // bytes of a stage's K, or V
  static constexpr bool kQSmem = NT > 2;       // q's fragments live in shared memory: 16 NT registers are too many
  // 64 K registers: 168 a thread for 12 warps, 255 for 8
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kStages = (D == 128 ? 1 : 2) * (kQSmem || kWarps == 12 ? 2 : 3);
  static constexpr int kRing = kStages * 2 * kSide;
  static constexpr int kQ = kQSmem ? kRows * D * 2 : 0;
  // floats of a row of a partial result in the ring: shifted by 4 banks a row where there is room
  static constexpr int kPartRow = kRows * (D + 4) * 4 <= kRing ? D + 4 : D;
  static constexpr int kOffQ = kWarps * kRing;
  static constexpr int kOffMeta = kOffQ + kWarps * kQ;
};

// A block that several runs (or CTAs) met, for the merge kernel: `parts` partial results, the first in place `first` of
// F8Params::parts, the others in next, next + step, ...
struct alignas(16) F8Header {
  int32_t t0, row0, kvh, rows;
  int32_t parts, first, next, step;
};

struct F8Params {
  const void* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int8_t* k_exp;
  const int8_t* v_exp;
  const int32_t* indices;
  const int32_t* indptr;
  const int32_t* last_page_len;
  const int32_t* first_page_offset;
  const int32_t* qo_indptr;
  const int32_t* tree_mask;
  const int32_t* positions;
  void* out;
  float* lse_out;
  float* parts;        // [workers * 2][part_rows * (head_dim + 1)]: values, then lse (log2)
  int32_t* counts;     // [workers]: what the merge kernel has to do for the header, in CTA's turns; [workers]: 1 where
                       // only every CTA's first warp has one
  F8Header* headers;   // [workers]
  int32_t* status;
  int64_t num_pages, num_indices;
  int32_t part_rows;  // rows of a part
  int32_t batch, num_tokens, mask_words, page_size, box_rows, hq, hkv, group, workers, q_bf16;
  int32_t team, teams, groups;  // heads side by side, the teams of so many warps, and teams that share a request's heads
  uint32_t ps_magic, ps_shift, g_magic, g_shift, team_magic, team_shift;
  float scale_log2;
  int32_t window, sinks;  // 0: no window
};

// One request: rows are pool rows in page order, counted from its first listed page.
struct F8Req {
  int32_t kind;        // 0: no new token, 1: nothing visible or a bad table (zeros and -inf), 2: keys
  int32_t slot_base, t0, n;
  int32_t lo, hi, ds;  // listed rows [lo, hi), new tokens [ds, hi)
  int32_t sink_end;    // rows [lo, sink_end) are seen by all, as far as they come before a token (sink_end <= hi)
  int32_t win0;        // the first row that the window of the first new token shows
  int32_t ns, gap;     // the first ns tiles hold sinks, the others lie `gap` further on
  int32_t tiles, blocks;
  __device__ __forceinline__ int32_t tile(int32_t v) const { return v < ns ? v : v + gap; }
  // some new token sees row x
  __device__ __forceinline__ bool seen(int32_t x) const { return x < hi && (x >= win0 || (x >= lo && x < sink_end)); }
};
constexpr int kF8Empty = 1, kF8Keys = 2;

template <int ROWS>
__device__ __forceinline__ F8Req f8_req(const F8Params& p, int r, bool tell) {
  F8Req g = {};
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
  g.blocks = (int32_t)(((int64_t)g.n * p.group + ROWS - 1) / ROWS);  // num_tokens * group fits 31 bits (checked by the host)
  g.kind = kF8Empty;
  g.tiles = 1;
  const int64_t pages = (int64_t)s1 - s0;
  if (s0 < 0 || pages < 0 || s1 > p.num_indices || pages * p.page_size > INT32_MAX - 2 * kF8Tile) {
    if (tell) report(p.status, PA_DEVICE_BAD_SLOT);
    return g;
  }
  const int32_t hi = pages > 0 ? ((int32_t)pages - 1) * p.page_size + lpl : 0;
  const int32_t ds = hi - g.n;
  bool bad = pages == 0 || lpl < 1 || lpl > p.page_size || fpo < 0 || fpo >= p.page_size || ds < fpo ||
             (p.tree_mask && g.n > 32 * p.mask_words);
  if (!bad && p.window > 0) {
    // sinks are the request's first tokens, so all of it is listed; else what the first new token's window shows
    if (p.sinks > 0) bad = fpo != 0 || (p.positions && p.positions[a] != ds);
    else bad = p.positions && ds - fpo < min(p.positions[a], p.window - 1);
  }
  const int32_t win0 = p.window > 0 ? (int32_t)max((int64_t)fpo, (int64_t)ds + 1 - p.window) : fpo;
  const int32_t sink_end = p.window > 0 && p.sinks > 0 ? min(p.sinks, hi) : fpo;
  const int32_t last = (hi + kF8Tile - 1) / kF8Tile, near = win0 / kF8Tile;
  const int32_t ns = sink_end > fpo ? min((sink_end + kF8Tile - 1) / kF8Tile, near) : 0;
  const int32_t first = ns > 0 ? 0 : near;  // sinks mean fpo = 0
  const int32_t tiles = ns + last - max(ns, near);
  if (!bad && (int64_t)g.blocks * tiles > kF8MaxUnits / p.hkv) bad = true;
  if (bad) {
    if (tell) report(p.status, PA_DEVICE_BAD_TREE);
    return g;
  }
  g.kind = kF8Keys;
  g.lo = fpo;
  g.hi = hi;
  g.ds = ds;
  g.sink_end = sink_end;
  g.win0 = win0;
  g.ns = ns > 0 ? ns : 0;
  g.gap = ns > 0 ? max(ns, near) - ns : first;
  g.tiles = tiles;
  return g;
}

// a / b for 0 <= a, 0 < b; in 32 bits where they allow.
__device__ __forceinline__ int64_t div_units(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Units of a KV head.
__device__ __forceinline__ int64_t units_of(const F8Req& g) { return g.kind == 0 ? 0 : (int64_t)g.blocks * g.tiles; }

// What the loading side of a warp tells the computing side of a stage.
struct F8Unit {
  int32_t base;   // its first row
  int32_t flags;  // kUnit* and, above them, its request's place in the warp's infos
  int32_t kvh, blk;
};
constexpr int kUnitBegins = 1, kUnitEnds = 2, kUnitShift = 2;  // the first, the last unit of its block
struct alignas(16) F8Meta {
  float k_scale[kF8Tile];
  __half v_scale[kF8Tile];
  F8Unit unit;
};

// A block's keys that a warp met only part of, where a CTA joins its warps' parts.
struct F8Part {
  int32_t valid, from_prev, to_next;
  int32_t t0, row0, rows, kvh;
  int64_t end;  // the unit behind the block's last
};

// Turns of a merge CTA for a block: one per row, or, with few parts, one per kMergeWarps rows.
__device__ __forceinline__ int32_t merge_turns(int32_t rows, int32_t parts) {
  return parts > kMergeFew ? rows : (rows + kMergeWarps - 1) / kMergeWarps;
}

// Bits [a, b) of a word, a and b clamped to [0, 32].
__device__ __forceinline__ uint32_t bits_between(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b >= 32 ? 0xffffffffu : ((1u << b) - 1u)) & ~((1u << a) - 1u);
}

// The first row that new token i of the request sees through its window: at depth d behind the request's first new
// token (a chain: d = i) rows up to ds + d - window are hidden.
__device__ __forceinline__ int32_t window_from(const F8Params& p, const F8Req& g, int32_t i) {
  if (p.window == 0) return g.lo;
  const int32_t depth =
      p.tree_mask ? min(max(__ldg(p.positions + g.t0 + i) - __ldg(p.positions + g.t0), 0), i) : i;
  return (int32_t)max((int64_t)g.lo, (int64_t)g.ds + depth + 1 - p.window);
}

// Which of the rows base .. base + 31 new token i sees, its window beginning at `low`.
__device__ __forceinline__ uint32_t seen_bits(const F8Params& p, const F8Req& g, int32_t i, int32_t low, int32_t base) {
  uint32_t bits = bits_between(low - base, g.ds - base) | bits_between(g.lo - base, min(g.sink_end, g.ds) - base);
  if (base + kF8Tile > g.ds && base < g.hi) {
    if (p.tree_mask) {  // the mask holds the window's cut of the new tokens itself
      const int32_t* row = p.tree_mask + (int64_t)(g.t0 + i) * p.mask_words;
      const int at = base - g.ds;  // new-token number of bit 0
      const int w = at >> 5, sh = at & 31;
      const uint32_t x0 = w >= 0 && w < p.mask_words ? (uint32_t)__ldg(row + w) : 0u;
      const uint32_t x1 = w + 1 >= 0 && w + 1 < p.mask_words ? (uint32_t)__ldg(row + w + 1) : 0u;
      bits |= __funnelshift_r(x0, x1, sh) & bits_between(g.ds - base, g.hi - base);
    } else {
      const int32_t end = min(g.ds + i + 1, g.hi);
      bits |= bits_between(max(g.ds, low) - base, end - base) | bits_between(g.ds - base, min(g.sink_end, end) - base);
    }
  }
  return bits;
}

// Two e4m3 codes as f16, exactly.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {  // once this thread's cp.async copies so far have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Byte offset of 16-byte chunk `ch` of row `row` of a side.
template <int D>
__device__ __forceinline__ uint32_t side_at(int row, int ch) {
  return D == 128 ? (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t pack16(const F8Params& p, float a, float b) {
  return p.q_bf16 ? TC<__nv_bfloat16>::pack(a, b) : TC<__half>::pack(a, b);
}

// Row `row` of a request's rows of KV head kvh, as a row of q and out.
__device__ __forceinline__ int64_t out_row_of(const F8Params& p, int32_t t0, int32_t kvh, int32_t row) {
  const int32_t tok = (int32_t)fast_div((uint32_t)row, p.g_magic, p.g_shift);
  return (int64_t)(t0 + tok) * p.hq + (int64_t)kvh * p.group + (row - tok * p.group);
}

template <int D, int NT, bool TMA>
__global__ void __launch_bounds__(32 * F8Cfg<D, NT>::kWarps, 1)
    pa_v2_attention_fp8_kernel(const F8Params p, const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v) {
  using C = F8Cfg<D, NT>;
  constexpr int S = C::kStages, R = C::kRows, KS = D / 16, W = C::kWarps;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[W][S];
  __shared__ F8Req infos[W][kF8Infos];
  __shared__ F8Part parts[W][2];
  __shared__ float stats[W][2][2][R];  // [part][maxima, sums]
  __shared__ int64_t warp_sum[W];
  __shared__ int64_t ends[32 * W];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * C::kRing;
  F8Meta* meta = reinterpret_cast<F8Meta*>(smem + C::kOffMeta) + warp * S;
  uint64_t* full = bars[warp];

  pdl_launch_dependents();
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&full[i], TMA ? 1 : 32);
    fence_barrier_init();
    parts[warp][0].valid = parts[warp][1].valid = 0;
  }
  pdl_wait_prerequisites();

  // ---- the cut: every warp's first unit.  A warp finds it alone where a lane holds a request, else all threads do
  // (their barriers and second look at the request cost one token over 1K 0.6 us).
  const bool alone = p.batch <= 32;
  int64_t units = 0, upto;
  F8Req own = {};
  const int per_thread = (p.batch + (32 * W) - 1) / (32 * W);
  if (alone) {
    if (lane < p.batch) own = f8_req<R>(p, lane, blockIdx.x == 0 && warp == 0);
    upto = units_of(own);
  } else {
    const int r0 = (int)min((int64_t)threadIdx.x * per_thread, (int64_t)p.batch), r1 = min(r0 + per_thread, p.batch);
    upto = 0;
    for (int r = r0; r < r1; ++r) upto += units_of(f8_req<R>(p, r, blockIdx.x == 0));
  }
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, w);
    if (lane >= w) upto += x;
  }
  if (alone) {
    units = __shfl_sync(0xffffffffu, upto, 31);
  } else {
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    for (int w = 0; w < W; ++w) {
      if (w < warp) upto += warp_sum[w];
      units += warp_sum[w];
    }
    ends[threadIdx.x] = upto;  // units of a KV head up to this thread's last request
    __syncthreads();
  }
  // Warps of a team take the same run of units of neighbouring heads, side by side: their rows lie side by side too, and
  // HBM serves them so (64 ragged requests of 8 KV heads 255 -> 214 us, 5.2 -> 6.2 TB/s).  Then every warp leaves its own
  // partial results.  Where runs are short those cost more than that gains (a request of 32K tokens: 205 parts a head, 30
  // against 22 us): there each team is one warp, the warps of a CTA take neighbouring runs and join their parts.  (Runs
  // of 16 and more units side by side against joined: 4 x 32K tokens 55 and 65 us, 64 x 1-4K 63 and 74, a request of
  // 128K 58 and 65; of 9, a request of 64K, 45 and 37.)
  const int32_t worker0 = (int)blockIdx.x * W, worker = worker0 + warp;
  const bool join = units * p.groups < (int64_t)kF8Spread * p.teams;
  const int32_t size = join ? 1 : p.team, teams = join ? p.workers : p.teams, groups = join ? p.hkv : p.groups;
  const int32_t team = join ? worker : (int32_t)fast_div((uint32_t)worker, p.team_magic, p.team_shift);
  const int32_t in_team = worker - team * size;
  units *= groups;
  const int64_t run = max(div_units(units + teams - 1, teams), (int64_t)1);
  const int64_t u0 = team * run;
  const int64_t count = max(min(run, units - u0), (int64_t)0);
  if (lane == 0) p.counts[worker] = 0;
  if (worker0 == 0 && threadIdx.x == 0) p.counts[p.workers] = join;

  // ---- the loading side: units are taken (their pages asked for) and then loaded
  // (requests are read from shared memory where they are needed: in registers, twice, they crowd out the accumulators)
  int32_t l_r = 0, l_kvh = 0, l_blk = 0, l_v = 0, l_info = 0;  // the unit taken last
  int32_t l_tiles = 0, l_base = 0, l_sinks = 0, l_win = 0, l_hi = 0;  // of its block: units left behind it, its first
                                                                      // row, tiles of sinks left, rows [l_win, l_hi)
  int32_t pend_k = 0, pend_v = 0, pend_stage = -1;
  const uint64_t policy = policy_evict_first(), keep = policy_evict_normal();
  struct Taken {
    int32_t page, entry;  // of this lane's row; page -2: nobody sees it
    uint32_t vis;         // rows that somebody sees, whole boxes
    F8Unit unit;
  };
  auto enter_block = [&](int v) {
    const F8Req& q = infos[warp][l_info];
    l_tiles = q.tiles - 1 - v;
    l_base = q.tile(v) * kF8Tile;
    l_sinks = q.ns - v;
    l_win = q.kind == kF8Keys ? q.win0 : INT_MAX;
    l_hi = q.hi;
  };
  auto take = [&](Taken& n, bool first) {  // the unit behind the one taken last (first: that one)
    int flags = 0;
    if (!first) {
      if (l_tiles > 0) {
        --l_tiles;
        l_base += kF8Tile;
        if (--l_sinks == 0) l_base += infos[warp][l_info].gap * kF8Tile;
      } else {
        if (++l_blk == infos[warp][l_info].blocks) {
          l_blk = 0;
          if ((l_kvh += size) >= p.hkv) {
            l_kvh = in_team;
            F8Req q;
            do q = f8_req<R>(p, ++l_r, false);  // (there is one with units: this one is in it)
            while (q.kind == 0);
            l_info = (l_info + 1) & (kF8Infos - 1);
            __syncwarp();
            if (lane == 0) infos[warp][l_info] = q;
            __syncwarp();
          }
        }
        enter_block(0);
        flags = kUnitBegins;
      }
    } else if (l_v == 0) {
      flags = kUnitBegins;
    }
    if (l_tiles == 0) flags |= kUnitEnds;
    n.unit = F8Unit{l_base, flags | l_info << kUnitShift, l_kvh, l_blk};
    const int32_t at = l_base + lane;
    n.page = -2;
    n.entry = 0;
    n.vis = 0xffffffffu;
    if (l_base < l_win || l_base + kF8Tile > l_hi) {  // some rows nobody sees
      const F8Req& q = infos[warp][l_info];
      n.vis = __ballot_sync(0xffffffffu, q.kind == kF8Keys && q.seen(at));
      if (TMA) {  // whole boxes
        const int b = lane & -p.box_rows;
        n.vis = __ballot_sync(0xffffffffu, (n.vis & bits_between(b, b + p.box_rows)) != 0);
      }
    }
    if (n.vis >> lane & 1u) {
      const int32_t slot = (int32_t)fast_div((uint32_t)at, p.ps_magic, p.ps_shift);
      n.entry = at - slot * p.page_size;
      n.page = __ldg(p.indices + infos[warp][l_info].slot_base + slot);
    }
  };
  auto load = [&](const Taken& n, int stage, int32_t& ek, int32_t& ev) {  // and ask for its rows' exponents
    unsigned char* kd = ring + stage * 2 * C::kSide;
    // a bad page: past the pool, where a box is zero-filled
    int32_t row = TMA ? (int32_t)(p.num_pages * p.page_size) : -1;
    ek = ev = 0;
    if (n.page >= 0 && n.page < p.num_pages) {
      row = n.page * p.page_size + n.entry;
      const int64_t e = (int64_t)n.page * p.hkv + n.unit.kvh;
      ek = __ldg(p.k_exp + e);
      ev = __ldg(p.v_exp + e);
    } else if (n.page != -2) {
      report(p.status, PA_DEVICE_BAD_PAGE);
    }
    if (lane == 0) meta[stage].unit = n.unit;
    // rows that several blocks read stay in L2 as other data does, the others leave it first
    const uint64_t pol = infos[warp][n.unit.flags >> kUnitShift].blocks > 1 ? keep : policy;
    if (TMA) {
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)__popc(n.vis) * D * 2;
        if (bytes) mbar_arrive_expect_tx(&full[stage], bytes);
        else arrive(&full[stage]);
      }
      for (int b = 0; b < kF8Tile; b += p.box_rows) {
        const int32_t y = __shfl_sync(0xffffffffu, row, b);
        if (lane == 0 && (n.vis >> b & 1u)) {
          tma_load_3d(kd + b * D, &tm_k, &full[stage], 0, n.unit.kvh, y, pol);
          tma_load_3d(kd + C::kSide + b * D, &tm_v, &full[stage], 0, n.unit.kvh, y, pol);
        }
      }
    } else {
      constexpr int kChunks = D / 16, kPass = 32 / kChunks;
      const int ch = lane % kChunks, sub = lane / kChunks;
      const int64_t pitch = (int64_t)p.hkv * D;
      const uint32_t to = smem_addr(kd);
#pragma unroll
      for (int i = 0; i < kF8Tile; i += kPass) {
        const int32_t y = __shfl_sync(0xffffffffu, row, i + sub);
        const uint32_t d = to + side_at<D>(i + sub, ch);
        if (y >= 0) {
          const int64_t from = y * pitch + (int64_t)n.unit.kvh * D + ch * 16;
          cp_async_16(d, p.k_pool + from, pol);
          cp_async_16(d + C::kSide, p.v_pool + from, pol);
        } else {
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(d), "r"(0u) : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(d + C::kSide), "r"(0u) : "memory");
        }
      }
      copies_arrive(&full[stage]);
    }
  };
  auto store_exponents = [&](int stage, int32_t ek, int32_t ev) {
    meta[stage].k_scale[lane] = power_of_two(min(max(ek, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX));
    meta[stage].v_scale[lane] = __float2half_rn(power_of_two(min(max(ev, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX)));
  };

  // ---- the computing side's view of its block, and Q
  uint32_t qb[C::kQSmem ? 1 : KS][C::kQSmem ? 1 : NT][2];
  float qf[NT][2];              // scale of the columns' scores
  uint2* qs = reinterpret_cast<uint2*>(smem + C::kOffQ + warp * C::kQ);  // [KS][NT][32], with kQSmem
  int32_t low = 0, tok = -1, clear0 = 0;  // of the row on this lane; rows [clear0, ds) are seen by all of the block's
  int32_t c_info = 0, c_ds = 0, c_sinks = 0, rows = 0, row0 = 0, kvh = 0, v_first = 0;
  bool c_keys = false;
  int64_t block_end = 0;        // the unit behind the block's last
  auto begin = [&](const F8Unit& unit, int64_t j) {  // a block, at the warp's unit j
    c_info = unit.flags >> kUnitShift;
    const F8Req& q = infos[warp][c_info];
    kvh = unit.kvh;
    block_end = u0 + j + q.tiles - v_first;
    c_keys = q.kind == kF8Keys;
    c_ds = q.ds;
    c_sinks = min(q.sink_end, c_ds);
    row0 = unit.blk * R;
    rows = (int32_t)min((int64_t)R, (int64_t)q.n * p.group - row0);
    const int32_t last_tok = (int32_t)fast_div((uint32_t)(row0 + rows - 1), p.g_magic, p.g_shift);
    tok = lane < rows ? (int32_t)fast_div((uint32_t)(row0 + lane), p.g_magic, p.g_shift) : -1;
    low = c_keys && tok >= 0 ? window_from(p, q, tok) : 0;
    clear0 = p.window > 0 ? (int32_t)max((int64_t)q.lo, (int64_t)q.ds + last_tok + 1 - p.window) : q.lo;
  };
  constexpr int kMine = D / 4;  // dims of a lane: t D / 4 ..
  auto fetch_q = [&](uint4 (&raw)[NT][D / 32]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int32_t c = nt * 8 + g;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) + out_row_of(p, infos[warp][c_info].t0, kvh, row0 + c) * D + t * kMine);
#pragma unroll
      for (int i = 0; i < kMine / 8; ++i) raw[nt][i] = c_keys && c < rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    }
  };
  auto take_q = [&](const uint4 (&raw)[NT][D / 32]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[kMine];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kMine / 8; ++i) {
        const uint32_t w[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 f;
          if (p.q_bf16) f = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
          else f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          x[8 * i + 2 * k] = f.x;
          x[8 * i + 2 * k + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row's largest element to [2^13, 2^14); rows that f16 holds as they are are not made smaller, and what is
      // given back to the scores stays finite, so that one of zero stays zero at every scale
      int e = 13;
      if (top > 0.f && top <= 3.4028234e38f) e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
      if (e <= 15) e = min(e, 13);
      const float up = power_of_two(13 - e);
      const float down = fminf(fmaxf(power_of_two(e - 13) * p.scale_log2, -3.4028234e38f), 3.4028234e38f);
      qf[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      qf[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t b0 = TC<__half>::pack(x[4 * k] * up, x[4 * k + 1] * up);
        const uint32_t b1 = TC<__half>::pack(x[4 * k + 2] * up, x[4 * k + 3] * up);
        if (C::kQSmem) {
          qs[(k * NT + nt) * 32 + lane] = make_uint2(b0, b1);
        } else {
          qb[k][nt][0] = b0;
          qb[k][nt][1] = b1;
        }
      }
    }
  };

  int64_t issued = min(count, (int64_t)S);
  Taken next;
  if (count > 0) {
    // the request that holds unit u0, searched by the warp's lanes: its lane, or its thread and, where a thread has
    // several, it
    int64_t off;
    if (alone) {
      l_r = __ffs(__ballot_sync(0xffffffffu, upto * groups > u0)) - 1;
      const int64_t before = __shfl_sync(0xffffffffu, upto, max(l_r - 1, 0));
      off = u0 - (l_r > 0 ? before * groups : 0);
      if (lane == l_r) infos[warp][0] = own;
    } else {
      int first = 0;
      while (!__any_sync(0xffffffffu, ends[first + lane] * groups > u0)) first += 32;
      first += __ffs(__ballot_sync(0xffffffffu, ends[first + lane] * groups > u0)) - 1;
      l_r = min(first * per_thread, p.batch - 1);
      off = u0 - (first > 0 ? ends[first - 1] * groups : 0);
      F8Req q = f8_req<R>(p, l_r, false);
      while (off >= units_of(q) * groups) {
        off -= units_of(q) * groups;
        q = f8_req<R>(p, ++l_r, false);
      }
      if (lane == 0) infos[warp][0] = q;
    }
    __syncwarp();
    const F8Req& q = infos[warp][0];
    const int32_t tiles = q.tiles;
    const int64_t head = (int64_t)q.blocks * tiles;
    const int32_t heads = (int32_t)div_units(off, head);  // groups of heads before
    const int64_t in_head = off - heads * head;
    l_kvh = heads * size + in_team;
    l_blk = (int32_t)div_units(in_head, tiles);
    l_v = (int32_t)(in_head - (int64_t)l_blk * tiles);
    enter_block(l_v);
    // each step for all stages before the next: their loads' latencies pass together
    Taken n[S];
    int32_t ek[S], ev[S];
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < issued) take(n[i], i == 0);
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < issued) load(n[i], i, ek[i], ev[i]);
    v_first = l_v;
    begin(n[0].unit, 0);
    uint4 raw[NT][D / 32];
    fetch_q(raw);
    if (issued < count) take(next, false);
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < issued) store_exponents(i, ek[i], ev[i]);
    take_q(raw);
    __syncwarp();
  }

  // ---- the computing side
  float o[KS][NT][4];           // O^T: dims 16 c + 2 g, + 1 (elements 0, 2 and 1, 3's rows), columns 2 t, 2 t + 1
  float m[NT][2], l[NT][2];     // of columns 2 t and 2 t + 1; sums over this lane's keys
  auto reset = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[c][nt][i] = 0.f;
    }
  };
  reset();
  bool alive = true;
  int stage = 0;
  uint32_t parity = 0;
  for (int64_t j = 0; j < count; ++j) {
    const F8Unit unit = meta[stage].unit;
    if (j > 0 && (unit.flags & kUnitBegins)) {
      v_first = 0;
      begin(unit, j);
      uint4 raw[NT][D / 32];
      fetch_q(raw);
      take_q(raw);
      reset();
    }

    // every row of the block sees every row of the tile: behind the last one's window's begin, or among the sinks (which
    // begin at row 0; without them sink_end is the first listed row, in the first tile)
    const int32_t base = unit.base;
    const bool clear = base + kF8Tile <= c_ds && (base >= clear0 || base + kF8Tile <= c_sinks);
    uint32_t mine_bits = 0, some = 0xffffffffu;
    bool skip = !c_keys;
    if (!clear && !skip) {
      if (tok >= 0) mine_bits = seen_bits(p, infos[warp][c_info], tok, low, base);
      some = __reduce_or_sync(0xffffffffu, mine_bits);
      skip = some == 0;
    }
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], parity, kWaitLimitCycles))) {
      report(p.status, PA_DEVICE_WAIT_TIMEOUT);
      alive = false;
      break;
    }
    if (!skip) {
      const uint32_t kb = smem_addr(ring + stage * 2 * C::kSide), vb = kb + C::kSide;
      // ---- S^T
      float s[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[i][h][0]), "=r"(x[i][h][1]), "=r"(x[i][h][2]), "=r"(x[i][h][3])
                         : "r"(kb + side_at<D>(16 * i + 8 * h + g, t * (D / 64) + c))
                         : "memory");
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int k = 4 * c + w;
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (C::kQSmem) {
              const uint2 u = qs[(k * NT + nt) * 32 + lane];
              b[nt][0] = u.x;
              b[nt][1] = u.y;
            } else {
              b[nt][0] = qb[k][nt][0];
              b[nt][1] = qb[k][nt][1];
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {codes_lo(x[i][0][w]), codes_lo(x[i][1][w]), codes_hi(x[i][0][w]),
                                   codes_hi(x[i][1][w])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) TC<__half>::mma(s[i][nt], a, b[nt][0], b[nt][1]);
          }
        }
      }
      // ---- scores in log2 units, softmax
      float ks[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = meta[stage].k_scale[8 * i + g];
      // (each step for all columns before the next: 2 warps a scheduler do not hide one column's chain of shuffles)
      float mt[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t see[2] = {0xffffffffu, 0xffffffffu};
        if (!clear) {
          see[0] = __shfl_sync(0xffffffffu, mine_bits, 8 * nt + 2 * t);
          see[1] = __shfl_sync(0xffffffffu, mine_bits, 8 * nt + 2 * t + 1);
        }
        mt[nt][0] = mt[nt][1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // token 16 i + 8 (k >> 1) + g, column 2 t + (k & 1)
            const int q4 = 2 * i + (k >> 1);
            float y = s[i][nt][k] * ks[q4] * qf[nt][k & 1];  // (2^ek first: both factors together could overflow)
            if (!clear) y = see[k & 1] >> (8 * q4 + g) & 1u ? y : -INFINITY;
            s[i][nt][k] = y;
            mt[nt][k & 1] = fmaxf(mt[nt][k & 1], y);
          }
      }
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mt[nt][0] = fmaxf(mt[nt][0], __shfl_xor_sync(0xffffffffu, mt[nt][0], x));
          mt[nt][1] = fmaxf(mt[nt][1], __shfl_xor_sync(0xffffffffu, mt[nt][1], x));
        }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        grow |= mt[nt][0] > m[nt][0] + kF8Lazy || mt[nt][1] > m[nt][1] + kF8Lazy;
      if (__any_sync(0xffffffffu, grow)) {  // m = -inf at first: any finite maximum
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float scale[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool need = mt[nt][k] > m[nt][k] + kF8Lazy;
            scale[k] = !need ? 1.f : m[nt][k] == -INFINITY ? 0.f : fast_exp2(m[nt][k] - mt[nt][k]);
            if (need) m[nt][k] = mt[nt][k];
            l[nt][k] *= scale[k];
          }
#pragma unroll
          for (int c = 0; c < KS; ++c) {
            o[c][nt][0] *= scale[0];
            o[c][nt][1] *= scale[1];
            o[c][nt][2] *= scale[0];
            o[c][nt][3] *= scale[1];
          }
        }
      }
      uint32_t pb[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float off[2] = {(m[nt][0] == -INFINITY ? 0.f : m[nt][0]) - kF8Shift,
                              (m[nt][1] == -INFINITY ? 0.f : m[nt][1]) - kF8Shift};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = fast_exp2(s[i][nt][2 * h] - off[0]), e1 = fast_exp2(s[i][nt][2 * h + 1] - off[1]);
            l[nt][0] += e0;
            l[nt][1] += e1;
            pb[nt][2 * i + h] = TC<__half>::pack(e0, e1);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) pb[nt][i] = transposed(pb[nt][i]);
      // ---- O^T += V^T P^T, 16 dims at a time
      uint32_t vs[4];  // tokens 8 i + 2 t, + 1
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vs[i] = *reinterpret_cast<const uint32_t*>(&meta[stage].v_scale[8 * i + 2 * t]);
      // what a row does not see must not meet its zero weight as a NaN: rows that nobody sees become zeros, and NaN
      // codes of the others zeros that are put back below for the rows that see them
      uint32_t vm[4] = {}, taint = 0;
      if (!clear) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = some >> (8 * i + 2 * t);
          vm[i] = (u & 1u ? 0x00ff00ffu : 0u) | (u & 2u ? 0xff00ff00u : 0u);
        }
      }
      auto values = [&](bool safe) {
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          uint32_t x[4];
          ldsm_x4_trans(x, vb + side_at<D>(lane, c));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = __byte_perm(x[i], 0, 0x3120);
            if (safe) {
              x[i] &= vm[i];
              const uint32_t nan = __vcmpeq4(x[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              taint |= nan;
              x[i] &= ~nan;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = 2 * h;
            const uint32_t a[4] = {mul_f16(codes_lo(x[2 * h]), vs[k]), mul_f16(codes_hi(x[2 * h]), vs[k]),
                                   mul_f16(codes_lo(x[2 * h + 1]), vs[k + 1]),
                                   mul_f16(codes_hi(x[2 * h + 1]), vs[k + 1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) TC<__half>::mma(o[c][nt], a, pb[nt][k], pb[nt][k + 1]);
          }
        }
      };
      if (clear) {
        values(false);
      } else {
        values(true);
        if (__any_sync(0xffffffffu, taint != 0)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t see0 = __shfl_sync(0xffffffffu, mine_bits, 8 * nt + 2 * t);
            const uint32_t see1 = __shfl_sync(0xffffffffu, mine_bits, 8 * nt + 2 * t + 1);
#pragma unroll
            for (int c = 0; c < KS; ++c) {
#pragma unroll 1
              for (int k = 0; k < kF8Tile; ++k) {
                uint16_t pair;  // dims 16 c + 2 g, + 1 of token k
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(pair) : "r"(vb + side_at<D>(k, c) + 2 * g) : "memory");
                const bool n0 = (pair & 0x7f) == 0x7f, n1 = (pair >> 8 & 0x7f) == 0x7f;
                if (see0 >> k & 1u) {
                  if (n0) o[c][nt][0] = NAN;
                  if (n1) o[c][nt][2] = NAN;
                }
                if (see1 >> k & 1u) {
                  if (n0) o[c][nt][1] = NAN;
                  if (n1) o[c][nt][3] = NAN;
                }
              }
            }
          }
        }
      }
    }
    __syncwarp();

    // ---- the block's last unit, or this warp's
    const bool ends = (unit.flags & kUnitEnds) != 0;
    const bool last = j + 1 == count;
    if (ends || last) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 4);
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 8);
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 16);
        }
      if (ends && v_first == 0) {  // all of it was met here
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int32_t c = 8 * nt + 2 * t + k;
            if (c >= rows) continue;
            const int64_t row = out_row_of(p, infos[warp][c_info].t0, kvh, row0 + c);
            const float sum = l[nt][k], inv = sum == 0.f ? 0.f : 1.f / sum;
            uint32_t* to = static_cast<uint32_t*>(p.out) + row * (D / 2) + g;
#pragma unroll
            for (int i = 0; i < KS; ++i) to[8 * i] = pack16(p, o[i][nt][k] * inv, o[i][nt][2 + k] * inv);
            if (g == 0) p.lse_out[row] = sum == 0.f ? -INFINITY : m[nt][k] - kF8Shift + fast_log2(sum);
          }
      } else {
        // a part: of a block that began in the run before, or of one that goes on in the next
        const int part = last ? 1 : 0;  // to be joined: the warp's last in its ring, which nothing loads into any more
        float* to = join && last ? reinterpret_cast<float*>(ring)
                                 : p.parts + ((int64_t)worker * 2 + (join || v_first == 0 ? 1 : 0)) * (p.part_rows * (D + 1));
        const int pitch = join && last ? C::kPartRow : D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int32_t c = 8 * nt + 2 * t + k;
            if (c >= rows) continue;
            const float sum = l[nt][k], by = join ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int i = 0; i < KS; ++i)
              *reinterpret_cast<float2*>(to + c * pitch + 16 * i + 2 * g) = make_float2(o[i][nt][k] * by, o[i][nt][2 + k] * by);
            if (g == 0 && join) {
              stats[warp][part][0][c] = m[nt][k];
              stats[warp][part][1][c] = sum;
            } else if (g == 0) {
              to[p.part_rows * D + c] = sum == 0.f ? -INFINITY : m[nt][k] - kF8Shift + fast_log2(sum);
            }
          }
        if (lane == 0 && join) {
          parts[warp][part] = F8Part{1, v_first != 0, !ends, infos[warp][c_info].t0, row0, rows, kvh, block_end};
        } else if (lane == 0 && v_first == 0) {
          const int32_t n = (int32_t)(div_units(block_end - 1, run) - team) + 1;
          p.counts[worker] = merge_turns(rows, n);
          p.headers[worker] = F8Header{infos[warp][c_info].t0, row0, kvh, rows, n, worker * 2 + 1, (worker + size) * 2, size * 2};
        }
      }
    }
    if (pend_stage >= 0) store_exponents(pend_stage, pend_k, pend_v);  // of the unit loaded last
    pend_stage = -1;
    if (issued < count) {
      load(next, stage, pend_k, pend_v);
      pend_stage = stage;
      if (++issued < count) take(next, false);
    }
    __syncwarp();
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
  }
  if (!alive) {  // no copy of this warp is left in flight
    for (int i = 0; i < S; ++i) {
      mbar_wait_bounded(&full[stage], parity, kWaitLimitCycles);
      if (++stage == S) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (!TMA) cp_async_wait<0>();
    if (lane == 0) {
      p.counts[worker] = 0;
      parts[warp][0].valid = parts[warp][1].valid = 0;
    }
  }
  if (!join) return;
  __syncthreads();
  // ---- parts of the same block are joined: with those of other CTAs still to come, or as the result.  Part 2 w + k is
  // warp w's; parts whose block goes on in the next one form a chain.
  const F8Part& mine_part = parts[min(lane >> 1, W - 1)][lane & 1];
  const uint32_t valid = __ballot_sync(0xffffffffu, lane < 2 * W && mine_part.valid);
  const uint32_t goes_on = __ballot_sync(0xffffffffu, lane < 2 * W && mine_part.valid && mine_part.to_next);
  auto next_chain = [&](uint32_t& left) {
    uint32_t chain = left & -left;
    left &= left - 1;
    while (left && (goes_on & (1u << (31 - __clz(chain))))) {
      chain |= left & -left;
      left &= left - 1;
    }
    return chain;
  };
  auto slot_of = [&](const F8Part& a) {
    return p.parts + (int64_t)(worker0 + (a.from_prev ? 0 : 1)) * 2 * (p.part_rows * (D + 1));
  };
  // the parts' weights, normalized: a warp a chain, a lane a row
  int number = 0;
  for (uint32_t left = valid; left; ++number) {
    const uint32_t chain = next_chain(left);
    if (number % W != warp) continue;
    const F8Part& a = parts[(__ffs(chain) - 1) >> 1][(__ffs(chain) - 1) & 1];
    const bool cut = a.from_prev || (goes_on >> (31 - __clz(chain)) & 1u);
    if (lane < a.rows) {
      float M = -INFINITY, sum = 0.f;
      for (uint32_t b = chain; b;) {  // four parts' loads at once
        float mk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mk[i] = -INFINITY;
          if (b) {
            const int k = __ffs(b) - 1;
            b &= b - 1;
            mk[i] = stats[k >> 1][k & 1][0][lane];
          }
        }
        M = fmaxf(M, fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])));
      }
      for (uint32_t b = chain; b;) {
        float mk[4], lk[4];
        float* at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mk[i] = -INFINITY;
          lk[i] = 0.f;
          at[i] = nullptr;
          if (b) {
            const int k = __ffs(b) - 1;
            b &= b - 1;
            at[i] = &stats[k >> 1][k & 1][0][lane];
            mk[i] = *at[i];
            lk[i] = stats[k >> 1][k & 1][1][lane];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = mk[i] == -INFINITY ? 0.f : fast_exp2(mk[i] - M);
          if (at[i]) *at[i] = w;
          sum += w * lk[i];
        }
      }
      stats[(__ffs(chain) - 1) >> 1][(__ffs(chain) - 1) & 1][1][lane] = sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : M - kF8Shift + fast_log2(sum);
      if (cut) slot_of(a)[p.part_rows * D + lane] = lse;
      else p.lse_out[out_row_of(p, a.t0, a.kvh, a.row0 + lane)] = lse;
    }
    if (lane == 0 && !a.from_prev && cut) {
      const int32_t n = (int32_t)div_units(a.end - 1, run * W) - (int)blockIdx.x + 1;
      p.counts[worker0] = merge_turns(a.rows, n);
      p.headers[worker0] = F8Header{a.t0, a.row0, a.kvh, a.rows, n, (worker0 + 1) * 2, (worker0 + W) * 2, W * 2};
    }
  }
  __syncthreads();
  // the values: 32 / (D / 4) rows a warp
  constexpr int kQuads = D / 4;
  const int d = lane % kQuads * 4;
  for (uint32_t left = valid; left;) {
    const uint32_t chain = next_chain(left);
    const F8Part& a = parts[(__ffs(chain) - 1) >> 1][(__ffs(chain) - 1) & 1];
    const bool cut = a.from_prev || (goes_on >> (31 - __clz(chain)) & 1u);
    for (int c = warp * (32 / kQuads) + lane / kQuads; c < a.rows; c += W * (32 / kQuads)) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t b = chain; b;) {  // four parts' loads at once
        float w[4];
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = 0.f;
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (b) {
            const int k = __ffs(b) - 1;
            b &= b - 1;
            w[i] = stats[k >> 1][k & 1][0][c];
            x[i] = k & 1 ? *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + (k >> 1) * C::kRing) +
                                                            c * C::kPartRow + d)
                         : __ldcg(reinterpret_cast<const float4*>(
                               p.parts + ((int64_t)(worker0 + (k >> 1)) * 2 + 1) * (p.part_rows * (D + 1)) + c * D + d));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc.x += w[i] * x[i].x;
          acc.y += w[i] * x[i].y;
          acc.z += w[i] * x[i].z;
          acc.w += w[i] * x[i].w;
        }
      }
      const float inv = stats[(__ffs(chain) - 1) >> 1][(__ffs(chain) - 1) & 1][1][c];
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (cut) {
        *reinterpret_cast<float4*>(slot_of(a) + c * D + d) = acc;
      } else {
        const int64_t row = out_row_of(p, a.t0, a.kvh, a.row0 + c);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + d) =
            make_uint2(pack16(p, acc.x, acc.y), pack16(p, acc.z, acc.w));
      }
    }
  }
}

// Folds the parts of the blocks that several runs met: weights 2^(lse_i - max) of the normalized parts.  A turn of a CTA
// is a row whose parts its warps share, joined in a fixed order, or, where the parts are few, a row for each warp.
// Where CTAs have joined their warps' parts, kMergeCtas CTAs share each one's header; else every CTA adds up all turns
// and takes every gridDim.x-th (4 us that the first case does not need).
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, kMergeCtas) pa_v2_fp8_merge_kernel(const F8Params p) {
  constexpr int V = D / 32;  // dims of a lane
  constexpr int kThreads = 32 * kMergeWarps;
  extern __shared__ uint8_t counts[];  // [workers]: at most kF8MaxRows each
  __shared__ int32_t turns_to[kThreads], warp_turns[kMergeWarps];
  __shared__ float sm[kMergeWarps], sl[kMergeWarps], so[kMergeWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_prerequisites();

  auto fold = [&](const F8Header& h, int turn) {
    const bool few = h.parts <= kMergeFew;
    const int c = few ? turn * kMergeWarps + warp : turn;
    float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    constexpr int kBatch = 8;
    const int stride = few ? 1 : kMergeWarps;
    for (int k0 = few ? 0 : warp; k0 < h.parts && c < h.rows; k0 += kBatch * stride) {
      float lse[kBatch], x[kBatch][V];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = k0 + b * stride;
        lse[b] = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) x[b][i] = 0.f;
        if (k < h.parts) {
          const float* part = p.parts + (int64_t)(k == 0 ? h.first : h.next + (k - 1) * h.step) * (p.part_rows * (D + 1));
          lse[b] = __ldcg(part + p.part_rows * D + c);
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(part + c * D + V * lane + i));
            x[b][i] = y.x;
            x[b][i + 1] = y.y;
          }
        }
      }
      float mb = M;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) mb = fmaxf(mb, lse[b]);
      const float mu = mb == -INFINITY ? 0.f : mb;
      const float sc = M == -INFINITY ? 0.f : fast_exp2(M - mu);
      L *= sc;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] *= sc;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (lse[b] == -INFINITY) continue;
        const float w = fast_exp2(lse[b] - mu);
        L += w;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(w, x[b][i], acc[i]);
      }
      M = mb;
    }
    if (few) {
      if (c >= h.rows) return;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int64_t row = out_row_of(p, h.t0, h.kvh, h.row0 + c);
#pragma unroll
      for (int i = 0; i < V; i += 2)
        static_cast<uint32_t*>(p.out)[row * (D / 2) + (V * lane + i) / 2] = pack16(p, acc[i] * inv, acc[i + 1] * inv);
      if (lane == 0) p.lse_out[row] = L == 0.f ? -INFINITY : M + fast_log2(L);
      return;
    }
    if (lane == 0) {
      sm[warp] = M;
      sl[warp] = L;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) so[warp][V * lane + i] = acc[i];
    __syncthreads();
    if (threadIdx.x < D / 2) {
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, sm[w]);
      float sum = 0.f;
      float2 out = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = sm[w] == -INFINITY ? 0.f : fast_exp2(sm[w] - mx);
        sum += f * sl[w];
        out.x += f * so[w][2 * threadIdx.x];
        out.y += f * so[w][2 * threadIdx.x + 1];
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int64_t row = out_row_of(p, h.t0, h.kvh, h.row0 + c);
      static_cast<uint32_t*>(p.out)[row * (D / 2) + threadIdx.x] = pack16(p, out.x * inv, out.y * inv);
      if (threadIdx.x == 0) p.lse_out[row] = sum == 0.f ? -INFINITY : mx + fast_log2(sum);
    }
    __syncthreads();
  };

  const int ctas = gridDim.x / kMergeCtas, mine = (int)blockIdx.x % ctas * (p.workers / ctas);
  const int joined = __ldcg(p.counts + p.workers), turns = __ldcg(p.counts + mine);
  const F8Header h = p.headers[mine];  // (asked for with the counts: whether it holds anything they tell)
  if (joined) {
    for (int turn = (int)blockIdx.x / ctas; turn < turns; turn += kMergeCtas) fold(h, turn);
    return;
  }
  for (int i = threadIdx.x; i < p.workers; i += kThreads) counts[i] = (uint8_t)__ldcg(p.counts + i);
  __syncthreads();
  // turns up to each thread's stretch of workers
  const int per = (p.workers + kThreads - 1) / kThreads;
  int32_t upto = 0;
  for (int i = threadIdx.x * per; i < min((int)(threadIdx.x + 1) * per, p.workers); ++i) upto += counts[i];
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, upto, w);
    if (lane >= w) upto += x;
  }
  if (lane == 31) warp_turns[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += warp_turns[w];
  turns_to[threadIdx.x] = upto;
  __syncthreads();
  const int total = turns_to[kThreads - 1];
  for (int turn = blockIdx.x; turn < total; turn += gridDim.x) {
    int lo = 0;  // the first stretch that ends behind the turn
    for (int step = kThreads / 2; step >= 1; step >>= 1)
      if (turns_to[lo + step - 1] <= turn) lo += step;
    int worker = lo * per, c = turn - (lo ? turns_to[lo - 1] : 0);
    while (c >= counts[worker]) c -= counts[worker++];
    fold(p.headers[worker], c);
  }
}

// ---- many query rows per request
//
// A prompt's chunk meets each key with hundreds of query rows, in blocks of kRows: the tensor cores bound it, and the warp's
// ones at that.  So the pages that some token sees are written out once in q's 16-bit type (exactly: an element is a
// binary16 number of 4 significant bits, and a bfloat16 one) and the tree attention runs over them, tcgen05 products and
// all: 4 x 256 tokens over 8K take 197 us (expansion 36, attention 153) where blocks of few rows took 815.  The rule counts
// rows, averaged over the requests, and not keys, so that it loses on one side of the border and gains on the other: 100 rows
// of one request over 1K, 8K and 32K tokens 25, 44 and 87 us (96 rows, in blocks: 19, 38 and 95), 100 rows of each of 32
// requests over 1K 106 (in blocks 132); 68 rows this way 24, 39 and 83 (in blocks 19, 33 and 79), of 32 requests 101 (90).
//
// The tree attention rounds P to the pages' type, which is q's: with bf16 by 2^-8 of each weight, where the blocks of few
// rows round it by 2^-11.  Against 64 bits the outputs' relative error is then 0.0021 where their own rounding alone gives
// 0.0017.  Pages in f16 for a bf16 q would keep the 2^-11, but q's rows would each need a power of two that the tree
// attention's scores do not have.
struct F8Wide {
  int32_t* qo_wide;     // qo_indptr for the tree attention, all zero when the pages do not fit
  int32_t* qo_narrow;   // and for the blocks of few rows, all zero when they do
  int32_t* indptr;      // the page tables of the requests one behind the other, a refused one's empty
  int32_t* table;       // pages of k and v
  void* k;
  void* v;
  int64_t max_slots, max_pages;
  bool last;            // no blocks of few rows follow: the listed pages are fewer, so only lists that overlap pass them
  uint32_t hkv_magic, hkv_shift;
};
constexpr int kWideThreads = 256;
constexpr int kWideCtas = 6;                  // per SM
constexpr int kWideChunks = 512;              // 8-byte pieces of a side that a warp takes at once
constexpr int64_t kWideElements = 1ll << 28;  // of k, and of v: 262144 tokens of 8 heads of 128
constexpr int64_t kWideSlots = 1ll << 20;
constexpr int64_t kWideRows = 96;             // query rows of a KV head: more of them take this way

// Pages [0, a) and [b, pages) of the request are seen by some token.
struct F8Pages {
  int32_t pages, a, b;
  __device__ __forceinline__ int32_t seen() const { return a + pages - max(a, b); }
};
__device__ __forceinline__ F8Pages f8_pages(const F8Params& p, const F8Req& g, int r) {
  if (g.kind != kF8Keys) return {0, 0, 0};
  return {p.indptr[r + 1] - p.indptr[r], g.sink_end > g.lo ? (g.sink_end + p.page_size - 1) / p.page_size : 0,
          g.win0 / p.page_size};
}

// 8 codes times 2^e as T: a lane's 16 bytes, so that a warp writes whole lines (16 codes a lane, 32 bytes in two stores,
// 209 us for 4 x 256 tokens over 8K and 287 for 25 over 128K, so 197 and 237).
template <typename T>
__device__ __forceinline__ uint4 widen(const uint2& c, int e) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t y[4];
  const float f = power_of_two(min(max(e, PA_V2_FP8_EXP_MIN), PA_V2_FP8_EXP_MAX));
  const __half2 h = __float2half2_rn(f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y[2 * i] = mul_f16(codes_lo(w[i]), *reinterpret_cast<const uint32_t*>(&h));
    y[2 * i + 1] = mul_f16(codes_hi(w[i]), *reinterpret_cast<const uint32_t*>(&h));
  }
  if (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
      y[i] = TC<__nv_bfloat16>::pack(x.x, x.y);
    }
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads) pa_v2_fp8_expand_kernel(const F8Params p, const F8Wide w) {
  constexpr int W = kWideThreads / 32;
  __shared__ int64_t warp_sum[2][W], ends[2][kWideThreads];  // slots, seen pages
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int per_thread = (p.batch + kWideThreads - 1) / kWideThreads;
  const int r0 = (int)min((int64_t)threadIdx.x * per_thread, (int64_t)p.batch), r1 = min(r0 + per_thread, p.batch);
  int64_t mine[2] = {0, 0}, total[2] = {0, 0}, upto[2];
  for (int r = r0; r < r1; ++r) {
    const F8Pages n = f8_pages(p, f8_req<kF8MaxRows>(p, r, blockIdx.x == 0), r);
    mine[0] += n.pages;
    mine[1] += n.seen();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    upto[k] = mine[k];
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto[k], i);
      if (lane >= i) upto[k] += x;
    }
    if (lane == 31) warp_sum[k][warp] = upto[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    for (int i = 0; i < W; ++i) {
      if (i < warp) upto[k] += warp_sum[k][i];
      total[k] += warp_sum[k][i];
    }
    ends[k][threadIdx.x] = upto[k];
  }
  __syncthreads();
  const bool fits = total[0] <= w.max_slots && total[1] <= w.max_pages;
  if (blockIdx.x == 0) {
    int64_t at = upto[0] - mine[0];
    for (int r = r0; r < r1; ++r) {
      const int32_t qo = p.qo_indptr[r];
      w.qo_wide[r] = fits || w.last ? qo : 0;  // (not fitting, with empty tables, which are refused)
      w.qo_narrow[r] = fits ? 0 : qo;
      w.indptr[r] = fits ? (int32_t)at : 0;
      at += f8_pages(p, f8_req<kF8MaxRows>(p, r, false), r).pages;
    }
    if (threadIdx.x == 0) {
      const int32_t qo = p.qo_indptr[p.batch];
      w.qo_wide[p.batch] = fits || w.last ? qo : 0;
      w.qo_narrow[p.batch] = fits ? 0 : qo;
      w.indptr[p.batch] = fits ? (int32_t)total[0] : 0;
    }
  }
  if (!fits) return;
  // a run of slots' parts of 4096 elements for every warp (whole slots left most warps of 2K slots without one: 85 us)
  const int64_t page_elements = (int64_t)p.page_size * p.hkv * D;
  const int chunks = (int)(page_elements / 8), parts = (chunks + kWideChunks - 1) / kWideChunks;
  const int64_t workers = (int64_t)gridDim.x * W, run = div_units(total[0] * parts + workers - 1, workers);
  const int64_t begin = ((int64_t)blockIdx.x * W + warp) * run, behind = min(begin + run, total[0] * parts);
  if (begin >= behind) return;
  int64_t u = div_units(begin, parts);
  int part = (int)(begin - u * parts);
  int first = 0;  // the thread of the request that holds slot u
  while (!__any_sync(0xffffffffu, ends[0][first + lane] > u)) first += 32;
  first += __ffs(__ballot_sync(0xffffffffu, ends[0][first + lane] > u)) - 1;
  int r = first * per_thread;
  int64_t slot0 = first > 0 ? ends[0][first - 1] : 0, page0 = first > 0 ? ends[1][first - 1] : 0;
  F8Pages n = f8_pages(p, f8_req<kF8MaxRows>(p, r, false), r);
  for (int64_t i = begin; i < behind; ++i) {
    while (u - slot0 >= n.pages) {
      slot0 += n.pages;
      page0 += n.seen();
      ++r;
      n = f8_pages(p, f8_req<kF8MaxRows>(p, r, false), r);
    }
    const int32_t s = (int32_t)(u - slot0);
    const int64_t slot = u;
    const int c0 = part * kWideChunks, c1 = min(c0 + kWideChunks, chunks);
    if (++part == parts) {
      part = 0;
      ++u;
    }
    const int32_t page = __ldg(p.indices + p.indptr[r] + s);
    const bool copied = (s < n.a || s >= n.b) && page >= 0 && page < p.num_pages;  // (the attention reports bad pages)
    const int64_t id = page0 + (s < n.a ? s : s - max(n.a, n.b) + n.a);
    if (lane == 0 && c0 == 0) w.table[slot] = copied ? (int32_t)id : -1;
    if (!copied) continue;
    const uint2* k = reinterpret_cast<const uint2*>(p.k_pool + page * page_elements);
    const uint2* v = reinterpret_cast<const uint2*>(p.v_pool + page * page_elements);
    uint4* ko = reinterpret_cast<uint4*>(static_cast<T*>(w.k) + id * page_elements);
    uint4* vo = reinterpret_cast<uint4*>(static_cast<T*>(w.v) + id * page_elements);
    const int8_t* ke = p.k_exp + (int64_t)page * p.hkv;
    const int8_t* ve = p.v_exp + (int64_t)page * p.hkv;
#pragma unroll 4
    for (int c = c0 + lane; c < c1; c += 32) {
      const uint32_t row = (uint32_t)c / (D / 8);  // of the page's rows and heads
      const uint32_t head = row - fast_div(row, w.hkv_magic, w.hkv_shift) * p.hkv;
      ko[c] = widen<T>(__ldg(k + c), __ldg(ke + head));
      vo[c] = widen<T>(__ldg(v + c), __ldg(ve + head));
    }
  }
}

using F8Kernel = void (*)(const F8Params, const CUtensorMap, const CUtensorMap);

struct F8Pick {
  F8Kernel fn;
  int rows, smem, threads;
};
template <int D, int NT>
F8Pick pick_f8(bool tma) {
  using C = F8Cfg<D, NT>;
  return {tma ? pa_v2_attention_fp8_kernel<D, NT, true> : pa_v2_attention_fp8_kernel<D, NT, false>, C::kRows,
          C::kOffMeta + (int)(C::kWarps * C::kStages * sizeof(F8Meta)) + 1024, 32 * C::kWarps};
}
// Rows of a block.  One of 24 rows takes 1.2 times one of 16 where a warp meets many (32 requests over 8K: 20 rows 160
// us, as two blocks 247; 64 rows 440 and 474; but 32 rows 300 and 250), and where it meets few, the units one after the
// other are what a call takes, and narrow blocks make more and shorter ones (20 rows over 1K 17.7 us and 14.2, 64 rows of 8
// requests over 1K 35 and 31; 32 requests over 512, just below the limit, 20 rows 34 and 36, 64 rows 64 and 57).
// Blocks of 32 rows spill (32 rows over 8K 254 us, 64 rows 479).
template <int D>
F8Pick pick_f8(int64_t rows, bool few, bool tma) {
  if (rows <= 8) return pick_f8<D, 1>(tma);
  return rows <= 16 || few || 5 * ((rows + 15) / 16) <= 6 * ((rows + 23) / 24) ? pick_f8<D, 2>(tma) : pick_f8<D, 3>(tma);
}
constexpr int64_t kF8Few = 4;  // tiles of keys per warp, up to which few

bool f8_aligned(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// The workspace: partial results, headers and counts.
int64_t parts_bytes(int32_t ctas, int32_t head_dim) {
  return (int64_t)ctas * kF8PartRows * 2 * (head_dim + 1) * (int64_t)sizeof(float);
}
int64_t all_bytes(int32_t ctas, int32_t head_dim) {
  return parts_bytes(ctas, head_dim) + (int64_t)ctas * kF8MaxWarps * (sizeof(F8Header) + sizeof(int32_t)) + 16;
}

// For many query rows per request: the tables, and k and v.
struct WideLayout {
  int64_t qo_wide, qo_narrow, indptr, table, k, v, tree, bytes;  // byte offsets behind the workspace of few rows
};
WideLayout wide_layout(int32_t batch, int64_t tree_bytes) {
  WideLayout l;
  int64_t at = 0;
  auto part = [&](int64_t bytes) {
    const int64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  const int64_t ints = ((int64_t)batch + 1) * 4;
  l.qo_wide = part(ints);
  l.qo_narrow = part(ints);
  l.indptr = part(ints);
  l.table = part(kWideSlots * 4);
  l.k = part(kWideElements * 2);
  l.v = part(kWideElements * 2);
  l.tree = part(tree_bytes);
  l.bytes = at;
  return l;
}
int64_t few_rows_bytes(int32_t ctas, int32_t head_dim) { return (all_bytes(ctas, head_dim) + 255) / 256 * 256; }
// Query rows of a KV head and request, were the tokens spread evenly (the lengths are on the device).
int64_t rows_of(int32_t num_tokens, int32_t batch, int32_t group) {
  return batch > 0 ? ((int64_t)num_tokens + batch - 1) / batch * group : 0;
}

// Heads that a team of warps takes side by side: the largest divisor of the KV heads up to 64.
int32_t team_of(int32_t hkv, int32_t workers) {
  int32_t n = hkv < 64 ? hkv : 64;
  if (n > workers) n = workers;
  while (hkv % n) --n;
  return n;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_v2_attention_fp8_workspace(int32_t device, int32_t num_tokens, int32_t batch,
                                                   int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                                   int64_t* bytes) {
  if (!bytes || device < 0 || num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads)
    return PA_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  *bytes = pa::few_rows_bytes(sms, head_dim);
  if (pa::rows_of(num_tokens, batch, num_qo_heads / num_kv_heads) > pa::kWideRows) {
    int64_t tree = 0;
    const pa_status rc =
        pa_v2_tree_attention_workspace(device, num_tokens, batch, num_qo_heads, num_kv_heads, head_dim, &tree);
    if (rc != PA_OK) return rc;
    *bytes += pa::wide_layout(batch, tree).bytes;
  }
  return PA_OK;
}

extern "C" pa_status pa_v2_attention_fp8(const void* q, int32_t q_dtype, const void* k_pool, const void* v_pool,
                                         const int8_t* k_exp, const int8_t* v_exp, int64_t num_pages,
                                         int32_t page_size, int32_t num_qo_heads, int32_t num_kv_heads,
                                         int32_t head_dim, const int32_t* indices, int64_t num_indices,
                                         const int32_t* indptr, const int32_t* last_page_len,
                                         const int32_t* first_page_offset, int32_t batch, const int32_t* qo_indptr,
                                         int32_t num_tokens, const int32_t* tree_mask, int32_t mask_words,
                                         const int32_t* positions, int32_t window, int32_t sinks, float sm_scale,
                                         void* out, float* lse2_out, void* workspace, int64_t workspace_bytes,
                                         int32_t* status, void* cuda_stream) {
  using namespace pa;
  if (num_tokens < 0 || batch < 0 || num_kv_heads < 1 || num_qo_heads < num_kv_heads ||
      num_qo_heads % num_kv_heads || page_size < 1 || num_pages < 1 || num_indices < 0 || mask_words < 0 ||
      (tree_mask && mask_words < 1) || window < 0 || sinks < 0 || (sinks > 0 && window == 0) || !std::isfinite(sm_scale))
    return PA_EINVAL;
  if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_EUNSUPPORTED;
  if (page_size > 256 || (page_size > 16 && page_size % 16 != 0)) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (tree_mask && mask_words > PA_V2_MAX_MASK_WORDS) return PA_EUNSUPPORTED;
  if (batch > (1 << 20)) return PA_EUNSUPPORTED;
  const float scale_log2 = sm_scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return PA_EUNSUPPORTED;
  const int32_t group = num_qo_heads / num_kv_heads;
  if ((int64_t)num_tokens * group > INT32_MAX - 2 * kF8MaxRows) return PA_EUNSUPPORTED;
  if (num_tokens == 0 || batch == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !k_exp || !v_exp || !indptr || !last_page_len || !first_page_offset || !qo_indptr ||
      !out || !lse2_out || !workspace || (num_indices > 0 && !indices) || (window > 0 && tree_mask && !positions))
    return PA_EINVAL;
  for (const void* x : {q, k_pool, v_pool, static_cast<const void*>(out), static_cast<const void*>(workspace)})
    if (!f8_aligned(x)) return PA_EINVAL;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  const int64_t rows = rows_of(num_tokens, batch, group);
  if (workspace_bytes < few_rows_bytes(sms, head_dim)) return PA_ECAPACITY;
  alignas(64) CUtensorMap tm_k, tm_v;
  std::memset(&tm_k, 0, sizeof(tm_k));
  std::memset(&tm_v, 0, sizeof(tm_v));
  const bool tma = tc_uses_tma(page_size);
  int box_rows = 8;  // rows of a TMA box: the largest power of two that divides a page, up to a whole tile
  while (box_rows < kF8Tile && page_size % (2 * box_rows) == 0) box_rows *= 2;
  if (tma) {
    const CUtensorMapSwizzle sw = head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_pool_map(&tm_k, k_pool, PA_E4M3, num_pages * page_size, num_kv_heads, head_dim, head_dim, box_rows, sw) ||
        !make_pool_map(&tm_v, v_pool, PA_E4M3, num_pages * page_size, num_kv_heads, head_dim, head_dim, box_rows, sw))
      return PA_ECUDA;
  }
  F8Params p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_exp = k_exp;
  p.v_exp = v_exp;
  p.indices = indices;
  p.indptr = indptr;
  p.last_page_len = last_page_len;
  p.first_page_offset = first_page_offset;
  p.qo_indptr = qo_indptr;
  p.tree_mask = tree_mask;
  p.positions = positions;
  p.out = out;
  p.lse_out = lse2_out;
  p.parts = static_cast<float*>(workspace);
  p.headers = reinterpret_cast<F8Header*>(static_cast<char*>(workspace) + parts_bytes(sms, head_dim));
  p.counts = reinterpret_cast<int32_t*>(p.headers + sms * kF8MaxWarps);
  p.status = status;
  p.num_pages = num_pages;
  p.num_indices = num_indices;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.mask_words = mask_words;
  p.page_size = page_size;
  p.box_rows = box_rows;
  p.hq = num_qo_heads;
  p.hkv = num_kv_heads;
  p.group = group;
  p.q_bf16 = q_dtype == PA_BF16;
  const FastDiv fd = FastDiv::make((uint32_t)page_size), fg = FastDiv::make((uint32_t)group);
  p.ps_magic = fd.magic;
  p.ps_shift = fd.shift;
  p.g_magic = fg.magic;
  p.g_shift = fg.shift;
  p.scale_log2 = scale_log2;
  p.window = window;
  p.sinks = sinks;
  // the keys that are listed, or that windows show, at most
  int64_t keys = std::min(num_indices, (int64_t)1 << 40) * page_size;
  if (window > 0) keys = std::min(keys, ((int64_t)window + sinks) * batch + num_tokens);
  const bool few = keys <= kF8Few * kF8Tile * 8 * sms / num_kv_heads;
  const F8Pick pick = head_dim == 64 ? pick_f8<64>(rows, few, tma) : pick_f8<128>(rows, few, tma);
  if (!prepare_kernel(reinterpret_cast<const void*>(pick.fn), pick.smem)) return PA_ECUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t rc = cudaSuccess;
  const int64_t page_elements = (int64_t)page_size * num_kv_heads * head_dim;
  // many rows, where the workspace has room for their pages (it may be one for other sizes); a window's depths come from
  // the positions there, for chains too
  int64_t tree_bytes = 0;
  pa_status ws = PA_OK;
  if (rows > kWideRows && (window == 0 || positions) && page_elements <= kWideElements) {
    ws = pa_v2_tree_attention_workspace(dev, num_tokens, batch, num_qo_heads, num_kv_heads, head_dim, &tree_bytes);
    if (ws != PA_OK) return ws;
  }
  const WideLayout l = wide_layout(batch, tree_bytes);
  if (tree_bytes > 0 && workspace_bytes - few_rows_bytes(sms, head_dim) >= l.bytes) {
    char* base = static_cast<char*>(workspace) + few_rows_bytes(sms, head_dim);
    F8Wide w;
    w.qo_wide = reinterpret_cast<int32_t*>(base + l.qo_wide);
    w.qo_narrow = reinterpret_cast<int32_t*>(base + l.qo_narrow);
    w.indptr = reinterpret_cast<int32_t*>(base + l.indptr);
    w.table = reinterpret_cast<int32_t*>(base + l.table);
    w.k = base + l.k;
    w.v = base + l.v;
    w.max_slots = kWideSlots;
    w.max_pages = kWideElements / page_elements;
    w.last = num_indices <= w.max_slots && num_indices <= w.max_pages;
    const FastDiv fk = FastDiv::make((uint32_t)num_kv_heads);
    w.hkv_magic = fk.magic;
    w.hkv_shift = fk.shift;
    auto expand = p.q_bf16 ? (head_dim == 64 ? pa_v2_fp8_expand_kernel<__nv_bfloat16, 64> : pa_v2_fp8_expand_kernel<__nv_bfloat16, 128>)
                           : (head_dim == 64 ? pa_v2_fp8_expand_kernel<__half, 64> : pa_v2_fp8_expand_kernel<__half, 128>);
    rc = launch_dependent(expand, dim3(sms * kWideCtas), dim3(kWideThreads), 0, stream, p, w);
    if (rc != cudaSuccess) {
      cudaGetLastError();
      return PA_ECUDA;
    }
    ws = tree_attention(q, w.k, w.v, q_dtype, w.max_pages, page_size, num_qo_heads, num_kv_heads, head_dim, w.table,
                        kWideSlots, w.indptr, last_page_len, first_page_offset, batch, w.qo_wide, num_tokens, tree_mask,
                        mask_words, positions, window, sinks, sm_scale, out, lse2_out, base + l.tree, tree_bytes, status,
                        cuda_stream);
    if (ws != PA_OK || w.last) return ws;
    p.qo_indptr = w.qo_narrow;
  }
  p.workers = sms * (pick.threads / 32);
  p.team = team_of(num_kv_heads, p.workers);
  p.teams = p.workers / p.team;
  p.groups = num_kv_heads / p.team;
  const FastDiv ft = FastDiv::make((uint32_t)p.team);
  p.team_magic = ft.magic;
  p.team_shift = ft.shift;
  p.part_rows = pick.rows;
  rc = launch_dependent(pick.fn, dim3(sms), dim3(pick.threads), pick.smem, stream, p, tm_k, tm_v);
  if (rc == cudaSuccess)
    rc = launch_dependent(head_dim == 64 ? pa_v2_fp8_merge_kernel<64> : pa_v2_fp8_merge_kernel<128>,
                          dim3(sms * kMergeCtas), dim3(32 * kMergeWarps), p.workers, stream, p);
  if (rc != cudaSuccess) {
    cudaGetLastError();
    return PA_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
