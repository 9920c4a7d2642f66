// pa_qk_rope.cu -- pa_v2_qk_rope_append: per-head norm of q and k, rotation by
// position, and the append of k and v to the paged pools, in one pass.
//
//   norm      x <- x * w / sqrt(mean(x^2) + eps)                (f32)
//   rotation  (x, y) <- (x cos a - y sin a, y cos a + x sin a),  a_j = pos * inv_freq[j]
//
// The angle is reduced in 64 bits before the sine is taken: a frequency is kept as
// the fraction of a turn that one position adds, times 2^64, so an integer product
// with the position wraps around whole turns by itself and leaves a fraction of a
// turn that f32 holds to 2^-26; a position of a million costs no accuracy (in f32
// the product alone would be off by 0.06 radians there).
//
// HBM bound: every row is read and written once.  A lane holds 16 bytes of a head's
// row as two 8-byte pieces, so a row takes head_dim / (16 / esize) lanes and a CTA's
// lanes hold several heads at once.  The two pieces are chosen so that a lane has
// both elements of each of its pairs: half-split pairs sit rot_dim / 2 elements
// apart, so its second piece is the first one's partner (with one 16-byte piece per
// lane every element had to be shuffled across lanes, and the kernel was bound by
// its instructions: 115 us for 16384 tokens of 48 heads).  A CTA walks
// tiles of up to four tokens, each lane keeping the same heads and the same places in
// the row: its pieces of the next two tokens are on their way into a ring in shared
// memory (its own places there: no barrier), and the next tile's cosines and sines are
// computed by all threads, one angle each, into the other half of a shared buffer (one
// barrier per tile; with one per token, behind the two warps that computed its angles,
// the kernel took 86 us).  A frequency is converted once per CTA.
//
// 16384 tokens of 48 heads take 73 us, 5.5 TB/s (81 % of the measured copy rate).  With
// one token ahead in registers 24 KB per SM were under way, too little for the memory's
// latency: 80 us, and 74.5 with the ring; norm and rotation two elements an instruction
// took the rest.  A ring of four tokens is equal, of six slower (78), three CTAs per SM
// with the registers that leaves slower too (90).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.cuh"
#include "pa_mma.cuh"
#include "pa_tc05.cuh"
#include "pa_v2.h"

namespace pa {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkPasses = 3;  // heads a lane holds at once, at most (four do not fit its registers)
constexpr int kQkTile = 4;    // tokens per tile, at most: one angle per thread
constexpr int kQkSlots = 3;   // tokens whose pieces a thread has room for in the ring
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
  int32_t tokens, hq, hkv, rot, tile;
};

// Two 8-byte pieces of T as floats, and back (one rounding).
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

// The part of a turn that one position adds, times 2^64.
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
  const double f = (double)inv_freq * kInvTwoPi;
  return __double2ull_rd((f - floor(f)) * 18446744073709551616.0);
}

// Cosine and sine after pos positions.
__device__ __forceinline__ float2 rotation(int32_t pos, uint64_t turn) {
  const int32_t part = (int32_t)(uint32_t)(((uint64_t)(int64_t)pos * turn) >> 32);  // [-1/2, 1/2) turns, times 2^32
  float s, c;
  sincospif((float)part * 4.656612873077393e-10f, &s, &c);  // 2^-31: sincospif takes half turns
  return make_float2(c, s);
}

__device__ __forceinline__ void copy_piece(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}

// NP: heads per lane (blockIdx.y takes the next NP * kRows heads).  PAIRED: the lane's pieces are partners (half
// split); else they are neighbours and pairs are neighbouring elements (interleaved).
template <typename T, typename TQ, int D, int NP, bool PAIRED>
__global__ void __launch_bounds__(kQkThreads, 2) pa_v2_qk_rope_append_kernel(const QkParams p) {
  constexpr int N = Vec<T>::N, P = N / 2;     // elements per lane; per piece, and pairs per lane
  constexpr int kLanes = D / N;               // lanes per head row (8, 16 or 32)
  constexpr int kRows = kQkThreads / kLanes;  // head rows in flight per CTA and pass
  __shared__ __align__(16) float cs[2][kQkTile][2][D / 2];  // cosines, sines
  extern __shared__ uint2 ring[];  // [kQkSlots][NP][2][kQkThreads]: each thread's own pieces

  pdl_launch_dependents();
  pdl_wait_prerequisites();

  const int half = p.rot / 2;
  const int lane = threadIdx.x & (kLanes - 1);
  const bool rotated = lane * P < half;
  // the places of the two pieces: partners while there are any, then neighbours
  const int e0 = PAIRED && rotated ? lane * P : lane * N, e1 = PAIRED && rotated ? e0 + half : e0 + P;
  const int heads = p.hq + 2 * p.hkv;

  // this lane's heads: where they are read and written (bytes; a row's place is base + index * step, both steps
  // below 2^31), and their norm weights
  const char* src[NP];
  char* dst[NP];
  uint32_t src_step[NP], dst_step[NP];
  uint4 weight[NP];
  int kind[NP];  // q, k, v or none
  bool normed[NP];
  const int gap = e1 - e0;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int h = ((int)blockIdx.y * NP + i) * kRows + (int)threadIdx.x / kLanes;
    kind[i] = h < p.hq ? 0 : h < p.hq + p.hkv ? 1 : h < heads ? 2 : 3;
    const int hh = kind[i] == 0 ? h : kind[i] == 1 ? h - p.hq : h - p.hq - p.hkv;
    const int at = hh * D + e0;
    const T* base = static_cast<const T*>(kind[i] == 0 ? p.q : kind[i] == 1 ? p.k : p.v) + at;
    src[i] = reinterpret_cast<const char*>(base);
    src_step[i] = (uint32_t)((kind[i] == 0 ? p.q_stride : kind[i] == 1 ? p.k_stride : p.v_stride) * sizeof(T));
    dst[i] = kind[i] == 0 ? reinterpret_cast<char*>(static_cast<TQ*>(p.q_out) + at)
                          : reinterpret_cast<char*>(static_cast<T*>(kind[i] == 1 ? p.k_pool : p.v_pool) + at);
    dst_step[i] = kind[i] == 0 ? (uint32_t)(p.hq * D * sizeof(TQ)) : (uint32_t)(p.hkv * D * sizeof(T));
    const T* w = static_cast<const T*>(kind[i] == 0 ? p.q_weight : kind[i] == 1 ? p.k_weight : nullptr);
    normed[i] = w != nullptr;
    weight[i] = make_uint4(0, 0, 0, 0);
    if (w) {
      const uint2 a = *reinterpret_cast<const uint2*>(w + e0), b = *reinterpret_cast<const uint2*>(w + e1);
      weight[i] = make_uint4(a.x, a.y, b.x, b.y);
    }
  }

  // this thread's angle: one frequency of one token of a tile
  const int angle = threadIdx.x % (D / 2), angle_tok = threadIdx.x / (D / 2);
  const bool has_angle = angle < half && angle_tok < p.tile;
  const uint64_t turn = has_angle ? turn_of(p.inv_freq[angle]) : 0;
  auto angles = [&](int first, int buf) {  // of the tile whose first token is `first`
    if (has_angle && first + angle_tok < p.tokens) {
      const float2 r = rotation(p.positions[first + angle_tok], turn);
      cs[buf][angle_tok][0][angle] = r.x;
      cs[buf][angle_tok][1][angle] = r.y;
    }
  };
  int t = blockIdx.x * p.tile, in_tile = 0;
  const int jump = ((int)gridDim.x - 1) * p.tile + 1;  // from a tile's last token to the next tile's first
  auto skip_of = [&](int place) { return place + 1 == p.tile ? jump : 1; };
  // the pieces of the next tokens are under way to the ring, kQkSlots - 1 tokens ahead
  const uint32_t mine = smem_addr(ring + threadIdx.x);
  constexpr uint32_t kPiece = kQkThreads * sizeof(uint2), kSlot = NP * 2 * kPiece;
  int ahead = t, ahead_place = 0;
  uint32_t fill = mine, drain = mine;
  auto next_slot_of = [&](uint32_t at) { return at + kSlot == mine + kQkSlots * kSlot ? mine : at + kSlot; };
  auto fetch = [&]() {  // one more token's pieces, if there is one
    if (ahead < p.tokens) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (kind[i] < 3) {
          const char* from = src[i] + (uint64_t)(uint32_t)ahead * src_step[i];
          copy_piece(fill + 2 * i * kPiece, from);
          copy_piece(fill + (2 * i + 1) * kPiece, from + gap * (int)sizeof(T));
        }
      }
      ahead += skip_of(ahead_place);
      ahead_place = ahead_place + 1 == p.tile ? 0 : ahead_place + 1;
    }
    cp_async_commit();
    fill = next_slot_of(fill);
  };
  int32_t next_slot = 0;
  if (t < p.tokens) {
#pragma unroll
    for (int i = 0; i < kQkSlots - 1; ++i) fetch();
    next_slot = p.slots[t];
    angles(t, 0);
  }
  __syncthreads();
  for (int buf = 0; t < p.tokens;) {
    cp_async_wait<kQkSlots - 2>();
    uint4 raw[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      uint2 a, b;
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a.x), "=r"(a.y) : "r"(drain + 2 * i * kPiece) : "memory");
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(b.x), "=r"(b.y)
                   : "r"(drain + (2 * i + 1) * kPiece)
                   : "memory");
      raw[i] = make_uint4(a.x, a.y, b.x, b.y);
    }
    drain = next_slot_of(drain);
    fetch();  // into the slot that was read a token ago
    const int64_t slot = next_slot;
    const int place = in_tile, after = t + skip_of(place);
    in_tile = place + 1 == p.tile ? 0 : place + 1;
    if (after < p.tokens) next_slot = p.slots[after];
    if (place == 0) angles(t + (int)gridDim.x * p.tile, buf ^ 1);
    if (slot >= 0 && slot < p.num_rows) {
      float2 co[P / 2], si[P / 2];  // the pairs' cosines and sines
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        co[i] = si[i] = make_float2(0.f, 0.f);
        if (rotated) {
          co[i] = *reinterpret_cast<const float2*>(&cs[buf][place][0][lane * P + 2 * i]);
          si[i] = *reinterpret_cast<const float2*>(&cs[buf][place][1][lane * P + 2 * i]);
        }
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        if (__any_sync(0xffffffffu, kind[k] < 2)) {  // a warp of v heads alone has nothing to compute
          float x[N];
          Vec<T>::unpack(raw[k], x);
          if (__any_sync(0xffffffffu, normed[k])) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N; i += 2) s2 = fma2(make_float2(x[i], x[i + 1]), make_float2(x[i], x[i + 1]), s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int w = kLanes / 2; w >= 1; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
            if (normed[k]) {
              const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
              float g[N];
              Vec<T>::unpack(weight[k], g);
#pragma unroll
              for (int i = 0; i < N; i += 2) {
                const float2 y = mul2(mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv)),
                                      make_float2(g[i], g[i + 1]));
                x[i] = y.x;
                x[i + 1] = y.y;
              }
            }
          }
          if (rotated) {  // the other elements are left out of it: 0 times an infinity next to them is NaN
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
          if (kind[k] == 0 && sizeof(TQ) != sizeof(T)) {  // f32 from 16 bits: a piece is 16 bytes
            char* to = dst[k] + (uint64_t)(uint32_t)t * dst_step[k];
            *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(to + gap * (int)sizeof(TQ)) = make_float4(x[P], x[P + 1], x[N - 2], x[N - 1]);
          } else if (kind[k] < 2) {
            raw[k] = Vec<T>::pack(x);
          }
        }
        if (kind[k] < 3 && !(kind[k] == 0 && sizeof(TQ) != sizeof(T))) {
          char* to = dst[k] + (uint64_t)(uint32_t)(kind[k] == 0 ? t : (int)slot) * dst_step[k];
          *reinterpret_cast<uint2*>(to) = make_uint2(raw[k].x, raw[k].y);
          *reinterpret_cast<uint2*>(to + gap * (int)sizeof(T)) = make_uint2(raw[k].z, raw[k].w);
        }
      }
    } else if (slot >= p.num_rows && threadIdx.x == 0) {
      report(p.status, PA_DEVICE_BAD_SLOT);
    }
    t = after;
    if (in_tile == 0) {
      __syncthreads();
      buf ^= 1;
    }
  }
}

using QkKernel = void (*)(const QkParams);

template <typename T, typename TQ, int D, bool PAIRED>
QkKernel pick_passes(int np) {
  return np == 1   ? pa_v2_qk_rope_append_kernel<T, TQ, D, 1, PAIRED>
         : np == 2 ? pa_v2_qk_rope_append_kernel<T, TQ, D, 2, PAIRED>
                   : pa_v2_qk_rope_append_kernel<T, TQ, D, 3, PAIRED>;
}
template <typename T, typename TQ>
QkKernel pick_layout(int D, bool paired, int np) {
  if (D == 64) return paired ? pick_passes<T, TQ, 64, true>(np) : pick_passes<T, TQ, 64, false>(np);
  return paired ? pick_passes<T, TQ, 128, true>(np) : pick_passes<T, TQ, 128, false>(np);
}
template <typename T>
QkKernel pick(int D, bool q32, bool paired, int np) {
  return q32 ? pick_layout<T, float>(D, paired, np) : pick_layout<T, T>(D, paired, np);
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
  if (num_qo_heads > 16384 || num_kv_heads > 16384) return PA_EUNSUPPORTED;
  if (num_pages >= (1ll << 31) || num_pages * page_size >= (1ll << 31)) return PA_EUNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !positions || !slots || !q_out || !k_pool || !v_pool || (rot_dim > 0 && !inv_freq))
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
  p.tokens = num_tokens;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ECUDA;
  // Head passes of a token: as few CTAs per token as hold them, or, while the tokens alone do not fill the GPU, a
  // CTA per pass (8 tokens of 48 heads: 24 CTAs instead of 8).
  const bool q32 = q_dtype == PA_F32;
  const int rows = (int)(pa::kQkThreads / (head_dim * esize / 16));
  const int passes = (num_qo_heads + 2 * num_kv_heads + rows - 1) / rows;
  int groups = (passes + pa::kQkPasses - 1) / pa::kQkPasses;
  if ((int64_t)num_tokens * groups < sms) groups = passes;
  const int np = (passes + groups - 1) / groups;
  const pa::QkKernel fn = dtype == PA_F32   ? pa::pick<float>(head_dim, true, !interleaved, np)
                          : dtype == PA_F16 ? pa::pick<__half>(head_dim, q32, !interleaved, np)
                                            : pa::pick<__nv_bfloat16>(head_dim, q32, !interleaved, np);
  const size_t smem = sizeof(uint2) * pa::kQkSlots * np * 2 * pa::kQkThreads;  // with the angles below 48 KB
  const int per_sm = np == 1 ? 3 : 2;  // CTAs that registers allow (about 70, 100 and 120 a thread); asking costs time in every call
  const int64_t wave = ((int64_t)sms * per_sm + groups - 1) / groups;  // CTAs along the tokens: one wave
  int tile = (int)(num_tokens / wave);  // whole tiles only where every CTA still gets some
  p.tile = tile < 1 ? 1 : tile < pa::kQkTile ? tile : pa::kQkTile;
  const int64_t tiles = ((int64_t)num_tokens + p.tile - 1) / p.tile;
  const cudaError_t rc = pa::launch_dependent(fn, dim3((unsigned)(tiles < wave ? tiles : wave), groups),
                                              dim3(pa::kQkThreads), smem, static_cast<cudaStream_t>(cuda_stream), p);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}
