// k_logprobs.cu -- log probabilities of given tokens, entropy and the k
// largest of logits rows, in one pass over the logits.
//
//   s = sum e^(x-m),  t = sum e^(x-m) (x-m) log2 e,  m a logit near the largest
//   log p_i = (x_i - m) - ln s,   H = ln 2 (log2 s - t / s)
//
// A row is cut into parts, one CTA each.  Every thread keeps a running
// (reference, s, t); a warp reads blocks of 2 KB and keeps the largest logit of
// each chunk of 512.  The CTA that finishes a row last
// (a counter per row) joins the parts' sums and finds the k largest logits.
// A bound that at least k chunks' maxima reach is reached by at least k logits,
// all of them in those chunks; halving finds one that few more than k chunks
// reach, without a sort.  These chunks are read again, 512 k of the row's logits,
// out of L2, and those of their logits that reach the bound are ranked by
// counting.  The streaming part so carries one warp-wide maximum per 512 logits
// and nothing else for the top k, whatever the values are.
//
// Pairs (value, id) are compared as one 64-bit key, the value's
// order-preserving bits above the complemented id: keys are distinct, and equal
// values rank by ascending id whatever the order in which they are met.
//
// Measured on a GB300 (us a call, device): 512 f32 rows of 151,936, k = 20, 54 (311
// MB, 5.8 TB/s, 85% of the measured copy), without a top k 47.5 (97%); as many bf16
// rows 36 and 28 (5.6 TB/s); 65 bf16 rows of 150,001, k = 8, 12.3; one f32 row, k =
// 5, 7.2, without a top k 4.3.  f32 streams are bound by HBM, 16-bit ones by 7
// instructions a logit next to it: two logits in a multiply-add, maxima and clamps
// of two 16-bit or three f32 values, and blocks of two 16-bit chunks, over which a
// step's 60 other instructions are spread (logit by logit and chunk by chunk the
// bf16 rows took 48 and 36).  A row's join adds 4 us of dependent steps, and for the
// 512 f32 rows 16 MB that have left L2; rows that end together hide nothing of it.
// With a ring of 8 KB a warp and three CTAs per SM the 512 f32 rows took 60 and 53.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;         // logits of a chunk, of which the maximum is kept
constexpr int kVecs = 4;            // 16-byte vectors of a lane in a block: one f32 chunk or two 16-bit ones
constexpr int kBlockBytes = kVecs * 512;
constexpr int kCtasPerSm = 4;       // resident
constexpr int kRing = 6144;         // bytes of a warp's ring: 4 CTAs of 8 warps have 192 KB in flight or at work
constexpr int kMostPicks = kLogprobsMaxTop + kWarps;  // chunks that are read again
constexpr int kHeld = 512;          // chunk maxima that a CTA, or a warp's registers, hold
constexpr int kWaves = 2;
constexpr int kWorth = 64;          // blocks of a part, at least, where the rows alone fill the GPU
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max and clamp that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two f32 values in one register pair: one instruction for two logits.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ void unpair(uint64_t x, float* a, float* b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
  return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}

// Order-preserving bits: a < b as floats <=> key(a) < key(b); +0 and -0 equal;
// NaN above everything.  0 is below every value's key: "nothing".
__device__ __forceinline__ uint32_t key32(float x) {
  if (x != x) return 0xFFFFFFFEu;  // (a NaN; all bits set is kept for "above every key")
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t id) {
  return ((uint64_t)key32(x) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t key_id(uint64_t k) { return ~(uint32_t)k; }

// (m, s, t) of a set of logits; m = -inf: empty or all masked.
struct Stat {
  float m, s, t;
};
// The joined sums of a warp's lanes, in every lane: all move to the largest
// reference first.
__device__ __forceinline__ Stat warp_join(Stat v) {
  const float m = key_value(__reduce_max_sync(0xffffffffu, key32(v.m)));
  // an empty side contributes nothing; its shift would be -inf
  const float d = v.m == -INFINITY ? 0.f : (v.m - m) * kLog2e, c = ex2(d);
  float s = v.s * c;
  // the terms' shift d moves t by d s; far below, c = 0 and d may overflow: no term
  float t = c == 0.f ? 0.f : c * fmaf(d, v.s, v.t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  return Stat{m, s, t};
}

// Two sets' sums in one (as warp_join, without the lanes).
__device__ __forceinline__ Stat join2(Stat a, Stat b) {
  const float m = max_nan(a.m, b.m);
  const float da = a.m == -INFINITY ? 0.f : (a.m - m) * kLog2e, ca = ex2(da);
  const float db = b.m == -INFINITY ? 0.f : (b.m - m) * kLog2e, cb = ex2(db);
  return Stat{m, a.s * ca + b.s * cb, (ca == 0.f ? 0.f : ca * fmaf(da, a.s, a.t)) + (cb == 0.f ? 0.f : cb * fmaf(db, b.s, b.t))};
}

// 16-byte vectors of T.  top: the largest value of a lane's vectors of a chunk; clamp: values
// raised to kLow, where infinities would make 0 * -inf of a term; pairs: two values
// each as f32.  kNear: up to this size of the reference, what kLow stands for is so
// far below it that its terms are 0.
template <typename T>
struct Loader;
template <>
struct Loader<float> {
  static constexpr int kVec = 4;
  static constexpr float kNear = 0x1p20f;
  __device__ static float top(const uint4* u) {
    float y = -INFINITY;
#pragma unroll
    for (int i = 0; i < kChunk / 32 / kVec; ++i)
      y = max_nan(max_nan(y, __uint_as_float(u[i].x), __uint_as_float(u[i].y)), __uint_as_float(u[i].z), __uint_as_float(u[i].w));
    return y;
  }
  __device__ static void pairs(const uint4& u, uint64_t* p) {  // raised to -2^100
    p[0] = pair(max_nan(__uint_as_float(u.x), -0x1p100f), max_nan(__uint_as_float(u.y), -0x1p100f));
    p[1] = pair(max_nan(__uint_as_float(u.z), -0x1p100f), max_nan(__uint_as_float(u.w), -0x1p100f));
  }
  __device__ static void get(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  __device__ static float one(const float* p) { return *p; }
  __device__ static float none() { return -INFINITY; }
};
template <>
struct Loader<__half> {
  static constexpr int kVec = 8;
  static constexpr float kNear = 0x1p15f;
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
  __device__ static float2 two(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  __device__ static float top(const uint4* u) {
    uint32_t y = max2(max2(u[0].x, u[0].y), max2(u[0].z, u[0].w));
#pragma unroll
    for (int i = 1; i < kChunk / 32 / kVec; ++i) y = max2(y, max2(max2(u[i].x, u[i].y), max2(u[i].z, u[i].w)));
    const float2 f = two(y);
    return max_nan(f.x, f.y);
  }
  __device__ static void pairs(const uint4& u, uint64_t* p) {  // raised to -65504
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(max2(w[i], 0xFBFFFBFFu));
      p[i] = pair(f.x, f.y);
    }
  }
  __device__ static void get(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static float one(const __half* p) { return __half2float(*p); }
  __device__ static __half none() { return __ushort_as_half(0xFC00); }
};
template <>
struct Loader<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr float kNear = 0x1p20f;
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
  __device__ static float2 two(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
  __device__ static float top(const uint4* u) {
    uint32_t y = max2(max2(u[0].x, u[0].y), max2(u[0].z, u[0].w));
#pragma unroll
    for (int i = 1; i < kChunk / 32 / kVec; ++i) y = max2(y, max2(max2(u[i].x, u[i].y), max2(u[i].z, u[i].w)));
    const float2 f = two(y);
    return max_nan(f.x, f.y);
  }
  __device__ static void pairs(const uint4& u, uint64_t* p) {  // raised to -2^100
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(max2(w[i], 0xF180F180u));
      p[i] = pair(f.x, f.y);
    }
  }
  __device__ static void get(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __nv_bfloat16 none() { return __ushort_as_bfloat16(0xFF80); }
};

// Keys held by a warp, `Regs` in every lane (0: none); each(f) calls f(number, key)
// for one key per lane, in the order of the numbers.  The search finds a bound that
// at least k of all `count` keys reach, but no more than `enough` if it can: halving
// between the least of the lanes' largest (32 keys reach it, or all) and the largest.
struct Bound {
  uint32_t floor, above;  // above: larger than every key
  int reach;              // keys that reach the floor
};
template <typename Each>
__device__ __forceinline__ int keys_reach(Each each, uint32_t bound) {
  int n = 0;
  each([&](int, uint32_t key) { n += key >= bound; });
  return (int)__reduce_add_sync(0xffffffffu, n);
}
template <typename Each>
__device__ __forceinline__ Bound find_bound(Each each, int count, int k, int enough) {
  uint32_t most = 0;
  each([&](int, uint32_t key) { most = max(most, key); });
  Bound b{1u, __reduce_max_sync(0xffffffffu, most) + 1, count};
  if (count < k) return b;
  b.floor = __reduce_min_sync(0xffffffffu, most ? most : 0xFFFFFFFFu);
  b.reach = keys_reach(each, b.floor);
  uint32_t hi = b.above;
  while (b.reach > enough && hi - b.floor > 1) {
    const uint32_t mid = b.floor + (hi - b.floor) / 2;
    const int n = keys_reach(each, mid);
    if (n >= k) {
      b.floor = mid;
      b.reach = n;
    } else {
      hi = mid;
    }
  }
  return b;
}

// How rows are cut, and where the workspace holds what: a counter per row (zero
// between calls; only rows of several parts have one, and there are fewer than
// num_sms * kCtasPerSm * kWaves of those, so their place is the same in every call), a
// Stat per part, the largest key32 of every chunk.
struct Plan {
  int chunks;  // of a row's blocks, at the worst alignment
  int parts;   // of a row
  int per;     // blocks of a part
  int64_t stats, keys, bytes;  // offsets and size
};

// One lane's N vectors of those from element e0 on, lane after lane; e0 plus the row's
// first address is a multiple of 16 bytes.  -inf outside of the row.
template <typename T, int N>
__device__ __forceinline__ void load_vectors(const T* x, int64_t vocab, int64_t e0, uint4* u) {
  using L = Loader<T>;
  constexpr int V = L::kVec;
  const int lane = threadIdx.x & 31;
  if (e0 >= 0 && e0 + N * 32 * V <= vocab) {
    const uint4* p = reinterpret_cast<const uint4*>(x + e0) + lane;
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = __ldcg(p + i * 32);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      alignas(16) T t[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int64_t e = e0 + (i * 32 + lane) * V + k;
        t[k] = e >= 0 && e < vocab ? x[e] : L::none();
      }
      u[i] = *reinterpret_cast<const uint4*>(t);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_kernel(const __grid_constant__ LogprobsArgs a, const Plan plan) {
  using L = Loader<T>;
  // values of a vector, logits of a block, its chunks, a lane's vectors of a chunk
  constexpr int V = L::kVec, kBlock = 32 * kVecs * V, S = kBlock / kChunk, U = kVecs / S;
  extern __shared__ __align__(128) unsigned char lp_smem[];
  __shared__ uint64_t s_list[kThreads];
  __shared__ uint32_t s_keys[kHeld];
  __shared__ int s_pick[kMostPicks];
  __shared__ Stat s_stat[kWarps];
  __shared__ int s_last, s_n, s_count, s_taken;
  __shared__ uint32_t s_floor, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / plan.parts;
  const int part = (int)(blockIdx.x - row * plan.parts);
  const int k = a.k;
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  float4* stats = reinterpret_cast<float4*>(ws + plan.stats) + row * plan.parts;
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + plan.keys) + row * plan.chunks;
  pdl_trigger();
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
  const int head = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int chunks = (int)((a.vocab + head + kChunk - 1) / kChunk);
  const int b1 = min((chunks + S - 1) / S, (part + 1) * plan.per);
  // the maxima of a row that this CTA has alone stay in shared memory, if they fit
  // (512 rows: 2 us less than with a store of 4 bytes per chunk)
  const bool alone = plan.parts == 1 && plan.chunks <= kHeld;

  // r: the reference, a logit near the largest so far (-inf: none yet).  Up to
  // |r| = kNear the terms are 2^(x L - z), one multiply-add each, with z = r L
  // rounded: z stands for itself and the sums are corrected by 2^(z - r L) at
  // the end.  Beyond, where that factor is no longer near 1, x - r comes first.
  float r = -INFINITY, z = 0.f;
  bool near = true;              // |r| <= kNear, or no reference yet
  uint64_t s2 = 0, t2 = 0;       // s and t, the logits of even and of odd places apart
  auto scale = [&](float d, float c) {  // from one reference to another that is d above: c = 2^d
    float s0, s1, t0, t1;
    unpair(s2, &s0, &s1);
    unpair(t2, &t0, &t1);
    t0 = c == 0.f ? 0.f : c * fmaf(d, s0, t0);
    t1 = c == 0.f ? 0.f : c * fmaf(d, s1, t1);
    s2 = pair(s0 * c, s1 * c);
    t2 = pair(t0, t1);
  };
  auto exact = [&] {  // from reference z to reference r
    const float d = -fmaf(r, kLog2e, -z);
    scale(d, ex2(d));
  };
  // Blocks that lie inside the row come through a ring in shared memory, kStages
  // - 1 of them on their way.  A lane copies the 16-byte vectors that it reads
  // itself, so a wait for its own copies is all the synchronization there is.
  constexpr int kStages = kRing / kBlockBytes;
  const uint32_t ring = smem_u32(lp_smem) + warp * kRing + lane * 16, ring_end = ring + kStages * kBlockBytes;
  const int in0 = head ? 1 : 0, in1 = min((int)((a.vocab + head) / kBlock), b1);
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  int b = part * plan.per + warp;
  // the block that is fetched next: its number, this lane's first vector, its place
  int fb = b;
  const unsigned char* from = reinterpret_cast<const unsigned char*>(x - head + (int64_t)b * kBlock) + lane * 16;
  uint32_t to = ring;
  auto fetch = [&] {
    if (fb >= in0 && fb < in1) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(to + i * 512), "l"(from + i * 512), "l"(policy)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fb += kWarps;
    from += kWarps * kBlockBytes;
    to += kBlockBytes;
    if (to == ring_end) to = ring;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();
  int id = -1;
  if (a.ids) {
    id = a.ids[row];
    if (id < 0 || id >= a.vocab) {  // padding, or refused
      if (id >= 0 && part == 0 && tid == 0) set_error(a.status, MINFER_ERR_TOKEN_OOB);
      asm volatile("cp.async.wait_all;" ::: "memory");
      return;
    }
  }
  float given = 0.f;  // the given token's logit, on its way until the end
  if (a.ids && tid == kThreads - 32) given = L::one(x + id);
  uint32_t at = ring;
#pragma unroll 1
  for (; b < b1; b += kWarps) {
    fetch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    uint4 u[kVecs];
    if (b >= in0 && b < in1) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w)
                     : "r"(at + i * 512)
                     : "memory");
    } else {
      load_vectors<T, kVecs>(x, a.vocab, (int64_t)b * kBlock - head, u);
    }
    at += kBlockBytes;
    if (at == ring_end) at = ring;
    float top = L::top(u), top1 = S > 1 ? L::top(u + kVecs - U) : top;
    if (k > 0) {
      uint32_t best = __reduce_max_sync(0xffffffffu, key32(top));
      if (S > 1) {
        const uint32_t best1 = __reduce_max_sync(0xffffffffu, key32(top1));
        if (lane == 1) best = best1;
      }
      const int c = b * S + lane;
      if (lane < S && c < chunks) *(alone ? s_keys + c : keys + c) = best;
    }
    if (S > 1) top = max_nan(top, top1);
    // a new reference only when the terms get large: 2^(4 L) at most
    if (!(top <= r + 4.f)) {
      if (r != -INFINITY) {
        if (near) exact();
        const float d = (r - top) * kLog2e;
        scale(d, ex2(d));
      }
      r = top;
      z = r * kLog2e;
      near = fabsf(r) <= L::kNear;
      if (near) {
        const float d = fmaf(r, kLog2e, -z);
        scale(d, ex2(d));
      }
    }
    auto add = [&](float d0, float d1) {
      const uint64_t e2 = pair(ex2(d0), ex2(d1));
      s2 = add2(s2, e2);
      t2 = fma2(e2, pair(d0, d1), t2);
    };
    if (near) {
      const uint64_t scale2 = pair(kLog2e, kLog2e), minus2 = pair(-z, -z);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        uint64_t f[V / 2];
        L::pairs(u[i], f);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float d0, d1;
          unpair(fma2(f[e], scale2, minus2), &d0, &d1);
          add(d0, d1);
        }
      }
    } else {
      // 2^-200 is 0 in f32: the clamp changes no sum and keeps 0 * -inf out of t
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        float f[V];
        L::get(u[i], f);
#pragma unroll
        for (int e = 0; e < V; e += 2) add(max_nan((f[e] - r) * kLog2e, -200.f), max_nan((f[e + 1] - r) * kLog2e, -200.f));
      }
    }
  }
  if (near && r != -INFINITY) exact();
  float s0, s1, t0, t1;
  unpair(s2, &s0, &s1);
  unpair(t2, &t0, &t1);
  Stat v = warp_join(Stat{r, s0 + s1, t0 + t1});
  if (lane == 0) s_stat[warp] = v;
  __syncthreads();
  // the last warp has the row's sums (alone: it writes what depends on them)
  constexpr int kSumWarp = kWarps - 1;
  if (warp == kSumWarp) v = warp_join(lane < kWarps ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f});
  if (plan.parts > 1) {
    if (tid == kSumWarp * 32) {
      stats[part] = make_float4(v.m, v.s, v.t, 0.f);
      __threadfence();  // also the other threads' keys: they came before the barrier
      unsigned* counter = reinterpret_cast<unsigned*>(ws) + row;
      s_last = atomicAdd(counter, 1u) == (unsigned)plan.parts - 1;
      if (s_last) *counter = 0;
      __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
  }

  if (warp == kSumWarp) {
    if (plan.parts > 1) {
      v = Stat{-INFINITY, 0.f, 0.f};
      for (int p = lane; p < plan.parts; p += 32) {
        const float4 q = __ldcg(stats + p);
        v = join2(v, Stat{q.x, q.y, q.z});
      }
      v = warp_join(v);
    }
    const float log2s = log2f(v.s);
    if (lane == 0) {
      s_stat[0] = Stat{v.m, log2s, 0.f};  // for every warp, behind the barriers below
      const bool none = v.m == -INFINITY;
      if (a.ids) a.logprob[row] = none ? -INFINITY : (given - v.m) - kLn2 * log2s;
      if (a.entropy) a.entropy[row] = none ? 0.f : kLn2 * (log2s - v.t / v.s);
    }
  }
  if (k == 0) return;

  // Meanwhile one warp finds a bound `floor` that at least k chunks' maxima reach, but
  // few more.  With fewer than k chunks all count.  (In every warp, which saves a
  // barrier, it cost 512 rows 3 us of issue slots.)
  if (warp == 0) {
    // the first maxima in registers, further ones (of vocabularies past 262,144)
    // are read again whenever they are counted
    uint32_t held[kHeld / 32];
    if (alone) {
#pragma unroll
      for (int i = 0; i < kHeld / 32; ++i) held[i] = i * 32 + lane < chunks ? s_keys[i * 32 + lane] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < kHeld / 32; ++i) held[i] = i * 32 + lane < chunks ? __ldcg(keys + i * 32 + lane) : 0u;
    }
    auto each = [&](auto f) {  // the chunks' maxima
#pragma unroll
      for (int i = 0; i < kHeld / 32; ++i)
        if (i * 32 < chunks) f(i * 32 + lane, held[i]);
      for (int c = kHeld; c < chunks; c += 32) f(c + lane, c + lane < chunks ? __ldcg(keys + c + lane) : 0u);
    };
    // (as many picks for every warp, kMostPicks for k = kLogprobsMaxTop)
    const Bound b = find_bound(each, chunks, k, (k + 3 + kWarps - 1) / kWarps * kWarps);
    // Those chunks, in the order of their ids.  If more than kMostPicks have
    // the same maximum, the first of them do: each holds one such logit, fewer than
    // k chunks have a larger maximum, and equal logits rank by their ids.
    int equals = b.reach > kMostPicks ? kMostPicks - keys_reach(each, b.floor + 1) : kMostPicks;
    int taken = 0;
    each([&](int c, uint32_t key) {
      const unsigned lower = (1u << lane) - 1, eq = __ballot_sync(0xffffffffu, key == b.floor);
      const bool take = key > b.floor || (key == b.floor && __popc(eq & lower) < equals);
      const unsigned all = __ballot_sync(0xffffffffu, take);
      if (take) s_pick[taken + __popc(all & lower)] = c;
      taken += __popc(all);
      equals -= min(__popc(eq), equals);
    });
    if (lane == 0) {
      s_taken = taken;
      s_floor = b.floor;
      s_above = b.above;
      s_n = s_count = 0;
    }
  }
  __syncthreads();
  const int taken = s_taken;

  // Those chunks come into the warps' rings, kPicks a warp together (all of them, but
  // of more than 24 f32 chunks).
  constexpr int kChunkBytes = kChunk * (int)sizeof(T);
  const int cin1 = (int)((a.vocab + head) / kChunk);
  auto inside = [&](int c) { return c >= in0 && c < cin1; };
  constexpr int kPicks = kRing / kChunkBytes * kWarps < kMostPicks ? kRing / kChunkBytes : kMostPicks / kWarps;
  bool resident = false;
  const unsigned char* const mine = lp_smem + warp * kRing + lane * 16;
  auto fetch_picks = [&](int p0) {
    if (resident) return;
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      if (p0 + j * kWarps >= taken) break;
      const int cp = s_pick[p0 + j * kWarps];
      if (inside(cp)) {
        const unsigned char* p = reinterpret_cast<const unsigned char*>(x + ((int64_t)cp * kChunk - head)) + lane * 16;
#pragma unroll
        for (int i = 0; i < U; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + j * kChunkBytes + i * 512), "l"(p + i * 512) : "memory");
      } else {
        uint4 edge[U];
        load_vectors<T, U>(x, a.vocab, (int64_t)cp * kChunk - head, edge);
#pragma unroll
        for (int i = 0; i < U; ++i) *reinterpret_cast<uint4*>(lp_smem + warp * kRing + j * kChunkBytes + i * 512 + lane * 16) = edge[i];
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    resident = taken <= kPicks * kWarps;
  };
  // The warp's logits that reach a bound: their number, and, with `list`, they
  // themselves at the end of s_list as long as there is room (in an order of
  // arrival: the ranks do not depend on it).
  auto sweep = [&](uint32_t bound, bool list) {
    int n = 0;
    for (int p0 = warp; p0 < taken; p0 += kPicks * kWarps) {
      fetch_picks(p0);
      unsigned large[kPicks];
      int own = 0;
      auto id_of = [&](int j, int i) {
        return (int64_t)s_pick[p0 + j * kWarps] * kChunk - head + ((i / V) * 32 + lane) * V + i % V;
      };
#pragma unroll
      for (int j = 0; j < kPicks; ++j) {
        large[j] = 0;
        if (p0 + j * kWarps >= taken) continue;
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float y[V];
          L::get(*reinterpret_cast<const uint4*>(mine + j * kChunkBytes + i * 512), y);
#pragma unroll
          for (int e = 0; e < V; ++e) m |= (unsigned)(key32(y[e]) >= bound) << (i * V + e);
        }
        if (!inside(s_pick[p0 + j * kWarps])) {
          for (unsigned all = m; all; all &= all - 1) {
            const int64_t id = id_of(j, __ffs(all) - 1);
            if (id < 0 || id >= a.vocab) m &= ~(all & -all);
          }
        }
        large[j] = m;
        own += __popc(m);
      }
      int at = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += y;
      }
      const int all = __shfl_sync(0xffffffffu, at, 31);
      n += all;
      if (!list) continue;
      int base = 0;
      if (lane == 0 && all) base = atomicAdd(&s_n, all);
      base = __shfl_sync(0xffffffffu, base, 0);
      at += base - own;
      if (base + all <= kThreads) {
#pragma unroll
        for (int j = 0; j < kPicks; ++j)
          for (unsigned m = large[j]; m; m &= m - 1, ++at) {
            const int i = __ffs(m) - 1;
            s_list[at] = make_key(L::one(reinterpret_cast<const T*>(mine + j * kChunkBytes + (i / V) * 512) + i % V), (uint32_t)id_of(j, i));
          }
      }
    }
    return n;
  };
  uint32_t floor = s_floor;
  const bool all_count = floor == 1 && a.vocab > kThreads;  // fewer than k chunks: no use in a list of everything
  if (!all_count) sweep(floor, true);
  __syncthreads();
  int n = all_count ? kThreads + 1 : s_n;
  const uint32_t above = s_above;
  if (n > kThreads && floor + 1 < above) {
    // A better floor from the largest logit of every thread's share of the chunks:
    // at least 32 threads have one.  (What is -inf behind a row's ends counts only
    // for a floor that every logit reaches.)
    uint32_t best = 0;
    for (int p0 = warp; p0 < taken; p0 += kPicks * kWarps) {
      fetch_picks(p0);
#pragma unroll 1
      for (int j = 0; j < kPicks && p0 + j * kWarps < taken; ++j)
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float y[V];
          L::get(*reinterpret_cast<const uint4*>(mine + j * kChunkBytes + i * 512), y);
#pragma unroll
          for (int e = 0; e < V; ++e) best = max(best, key32(y[e]));
        }
    }
    s_keys[tid] = best;
    __syncthreads();
    if (warp == 0) {
      uint32_t held[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) held[i] = s_keys[i * 32 + lane];
      auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) f(i * 32 + lane, held[i]);
      };
      const Bound b = find_bound(each, kThreads, k, k + 8);
      if (lane == 0) {
        s_floor = b.floor;
        s_n = 0;
      }
    }
    __syncthreads();
    floor = s_floor;
    sweep(floor, true);
    __syncthreads();
    n = s_n;
  }
  if (n > kThreads) {
    // Many logits reach the floor: equal ones (rows of which a mask leaves little),
    // or large ones side by side.  The least bound above it that no more than
    // kThreads reach; if fewer than k do, those equal to the bound below follow in
    // the order of their ids.
    auto total = [&](uint32_t bound) {
      const int own = sweep(bound, false);
      if (lane == 0 && own) atomicAdd(&s_count, own);
      __syncthreads();
      const int sum = s_count;
      __syncthreads();
      if (tid == 0) s_count = 0;
      __syncthreads();
      return sum;
    };
    uint32_t hi = floor + 1;
    n = hi == above ? 0 : total(hi);
    if (n > kThreads) {
      floor = hi;
      hi = above;
      n = 0;
      while (hi - floor > 1) {
        const uint32_t mid = floor + (hi - floor) / 2;
        const int at_mid = total(mid);
        if (at_mid > kThreads) {
          floor = mid;
        } else {
          hi = mid;
          n = at_mid;
          if (n >= k) break;
        }
      }
    }
    __syncthreads();  // s_n has been read
    if (tid == 0) s_n = 0;
    __syncthreads();
    if (n > 0) sweep(hi, true);
    if (n < k && warp == 0) {
      int at = n;
      for (int p = 0; p < taken && at < k; ++p) {
        uint4 u[U];
        load_vectors<T, U>(x, a.vocab, (int64_t)s_pick[p] * kChunk - head, u);
#pragma unroll
        for (int i = 0; i < U; ++i) {  // a vector of every lane: neighbouring logits
          const int64_t e0 = (int64_t)s_pick[p] * kChunk - head + (i * 32 + lane) * V;
          unsigned eq = 0;
          float f[V];
          L::get(u[i], f);
#pragma unroll
          for (int e = 0; e < V; ++e) eq |= (unsigned)(key32(f[e]) == floor && e0 + e >= 0 && e0 + e < a.vocab) << e;
          int to = __popc(eq);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, to, o);
            if (lane >= o) to += y;
          }
          const int all = __shfl_sync(0xffffffffu, to, 31);
          to += at - __popc(eq);
          for (; eq && to < k; eq &= eq - 1) s_list[to++] = (uint64_t)floor << 32 | (uint32_t)~(uint32_t)(e0 + __ffs(eq) - 1);
          at += all;
        }
      }
    }
    n = max(n, k);
    __syncthreads();
  }
  // a key's place is the number of keys above it
  if (tid < n) {
    const uint64_t own = s_list[tid];
    int at = 0;
    for (int i = 0; i < n; ++i) at += s_list[i] > own;
    if (at < k) {
      const float m = s_stat[0].m, log2s = s_stat[0].s;
      a.top_ids[row * k + at] = (int32_t)key_id(own);
      a.top_logprobs[row * k + at] = m == -INFINITY ? -INFINITY : (key_value((uint32_t)(own >> 32)) - m) - kLn2 * log2s;
    }
  }
}

// Parts of a row: with fewer rows than the GPU holds CTAs, as many as it holds (340
// rows: 42 us; one part more, so that a second round begins, 45; 65 rows 14.2
// against 16.3); with more, so many that it is filled kWaves times, for the last
// round's idle share (620 rows: once 60 us, twice 53) as long as a part is worth its
// join (1,000 bf16 rows of 18,000: 15 us whole, 20 in halves).  None has less than a
// block per warp.
Plan plan_of(int64_t rows, int64_t vocab, int vec, int k, int num_sms) {
  Plan p;
  const int block = 32 * kVecs * vec;  // logits
  const int blocks = (int)((vocab + vec - 1 + block - 1) / block);
  const int64_t resident = (int64_t)num_sms * kCtasPerSm;
  const int64_t want = rows <= resident ? resident / rows : (resident * kWaves + rows - 1) / rows;
  const int64_t most = rows <= resident ? (blocks + kWarps - 1) / kWarps : std::max(1, blocks / kWorth);
  const int64_t parts = std::min(want, most);
  p.per = (int)((blocks + parts - 1) / parts);
  p.parts = (blocks + p.per - 1) / p.per;
  p.chunks = blocks * (block / kChunk);
  p.stats = ((int64_t)num_sms * kCtasPerSm * kWaves * 4 + 15) / 16 * 16;
  p.keys = p.stats + rows * p.parts * 16;
  p.bytes = p.keys + (k > 0 ? rows * p.chunks * 4 : 0);
  return p;
}

template <typename T>
cudaError_t launch(const LogprobsArgs& a, int num_sms, cudaStream_t st) {
  const Plan plan = plan_of(a.rows, a.vocab, Loader<T>::kVec, a.k, num_sms);
  const cudaError_t e = allow_smem<logprobs_kernel<T>>(kWarps * kRing);
  if (e != cudaSuccess) return e;
  return launch_pdl(logprobs_kernel<T>, dim3((unsigned)(a.rows * plan.parts)), dim3(kThreads), kWarps * kRing, st, a, plan);
}

}  // namespace

int64_t logprobs_workspace(int64_t rows, int64_t vocab, int k, int num_sms) {
  // the size does not depend on the logits' type: enough for vectors of 4 and of 8 values
  return std::max(plan_of(rows, vocab, 4, k, num_sms).bytes, plan_of(rows, vocab, 8, k, num_sms).bytes);
}

cudaError_t logprobs_launch(const LogprobsArgs& a, int type, int num_sms, cudaStream_t stream) {
  if (type == MINFER_F32) return launch<float>(a, num_sms, stream);
  if (type == MINFER_F16) return launch<__half>(a, num_sms, stream);
  return launch<__nv_bfloat16>(a, num_sms, stream);
}

}  // namespace minfer
