// k_sample.cu -- the next token of logits rows: top-k, top-p and min-p, temperature,
// and the draw from a given random number.
//
//   order    tokens by descending logit, equal ones by ascending id
//   top-k    the first k
//   top-p    of those the shortest beginning whose weights exp((x - max) / t) reach top_p
//            of their sum
//   min-p    those with exp((x - max) / t) >= min_p            (t: 1, or the temperature)
//   draw     weights w = exp((x - max) / temperature) of what is left, in the order of
//            their ids: the first token whose inclusive sum of weights exceeds u times
//            the whole
//
// A token depends on sums over a whole row to a precision that f32 does not have: a
// border between two tokens of 150,000 lies within 1e-6 of any random number, so sums
// that are off by 1e-7 give another token in one row of ten.  Weights are therefore whole
// numbers: 2^t is put together from a table of 2^(j/256) and a quadratic (to 2^-31 of
// itself) and shifted to a fixed point that is the same for the whole row; their sums
// are exact in 64 bits and do not depend on who adds what first.
//
// A thread-block cluster does a row, and keeps it: a CTA copies its slice of the row
// into shared memory (cp.async, all of it on its way at once; a thread reads what it
// has copied itself), so further passes cost no memory traffic.  What lies behind the
// room in shared memory (vocabularies past 8 x 25,600 f32) is read again from L2.
//
// Most rows need two or three exchanges in the cluster: (1) the maximum, and a bound
// under which nothing can be among the first k: the k-th largest of the maxima of a
// CTA's threads; (2) with top-p and no top-k, the sum of all weights; (3) what lies
// above the bound goes to the first CTA, which sorts it (a few hundred tokens), cuts it
// by the three filters, sorts what is left by id and draws.  Rows for which that list
// overflows or does not reach (no filter, high temperatures, large k) go the wide way:
// the border of a filter is bracketed by passes over the row with three thresholds each
// until a list holds what lies between, and the draw goes segment by segment.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;      // tokens that the first CTA sorts
constexpr int kGuess = 128;      // of top-p alone: tokens that the first bound aims at
constexpr int kCopies = 8;       // of the table, against bank conflicts
constexpr int kSlots = 6;        // numbers of one exchange
constexpr int kRoom = 77824;     // bytes of a row's slice that a CTA keeps, at most
constexpr float kLowest = -3.402823466e38f;

typedef unsigned long long u64;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the address of p's counterpart in CTA r
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t r) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
  return a;
}
__device__ __forceinline__ void put(uint32_t a, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }
__device__ __forceinline__ int peer_add(uint32_t a, int v) {
  int before;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(before) : "r"(a), "r"(v) : "memory");
  return before;
}
__device__ __forceinline__ int peer_get(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// f32 as an unsigned number of the same order (-0 as 0; a NaN as max_nan gives it last)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// floor(n * f) for 0 <= f < 1, exactly; *rest: whether something was cut off
__device__ __forceinline__ u64 times(u64 n, float f, bool* rest) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  const u64 mant = (u64)(e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu);  // f = mant 2^(max(e, 1) - 150)
  const int down = 126 - (int)max(e, 1u);                                  // f = (mant << 40) 2^-64 2^-down, down >= 0
  const u64 hi = __umul64hi(n, mant << 40), lo = n * (mant << 40);
  if (down >= 64) {
    *rest = (hi | lo) != 0;
    return 0;
  }
  *rest = lo != 0 || (hi & ((1ull << down) - 1)) != 0;
  return hi >> down;
}

// ------------------------------------------------------------------ weights
// 2^(a/16) and 2^(b/256), times 2^63
__constant__ u64 c_coarse[16] = {0x8000000000000000ull, 0x85AAC367CC487B15ull, 0x8B95C1E3EA8BD6E7ull, 0x91C3D373AB11C336ull,
                                 0x9837F0518DB8A96Full, 0x9EF5326091A111AEull, 0xA5FED6A9B15138EAull, 0xAD583EEA42A14AC6ull,
                                 0xB504F333F9DE6484ull, 0xBD08A39F580C36BFull, 0xC5672A115506DADDull, 0xCE248C151F8480E4ull,
                                 0xD744FCCAD69D6AF4ull, 0xE0CCDEEC2A94E111ull, 0xEAC0C6E7DD24392Full, 0xF5257D152486CC2Cull};
__constant__ u64 c_fine[16] = {0x8000000000000000ull, 0x8058D7D2D5E5F6B1ull, 0x80B1ED4FD999AB6Cull, 0x810B40A1D81406D4ull,
                               0x8164D1F3BC030773ull, 0x81BEA1708DDE6056ull, 0x8218AF4373FC25ECull, 0x8272FB97B2A5894Cull,
                               0x82CD8698AC2BA1D7ull, 0x83285071E0FC4547ull, 0x8383594EEFB6EE37ull, 0x83DEA15B9541B132ull,
                               0x843A28C3ACDE4046ull, 0x8495EFB3303EFD30ull, 0x84F1F656379C1A29ull, 0x854E3CD8F9C8C95Dull};
constexpr float kStep = 0x1.8p15f;   // adding it rounds to 1/256
constexpr float kUnit = 0x1.8p-7f;   // adding it rounds to 2^-30

// The weights of a row under one temperature: exp((x - m) / T) as a whole number in
// units of 2^-point of a power of two near the maximum's.
struct Weigh {
  float c, c_low;  // log2(e) / T as a sum
  float m;
  float lim;       // what lies below weighs nothing: x below lim, or x - m
  int top;         // whole part of the maximum's exponent
  int down;        // 62 - point
  bool apart;      // |m| c is large: x - m is taken first

  // What does not depend on the maximum is set before.  An exponent below -62 (which a
  // sum of 2^31 weights does not notice) counts as -62: its weight is 0, and -inf and
  // huge differences stay out of the arithmetic.
  __device__ __forceinline__ void at(float max, float t) {
    m = max;
    apart = !(fabsf(max * c) <= 8192.f);
    lim = apart ? -43.f * t : max - 43.f * t;  // 62 ln 2 = 42.98
    top = 0;
    top = -shift(max);
  }
  // t = (x or x - m) log2(e) / T as th + tl
  __device__ __forceinline__ void exponent(float x, float* th, float* tl) const {
    if (!apart) {
      x = fmaxf(x, lim);
      *th = __fmul_rn(x, c);
      *tl = fmaf(x, c_low, fmaf(x, c, -*th));
    } else {
      float d = __fsub_rn(x, m);
      const float b = __fsub_rn(d, x);
      float low = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
      if (!(d > lim)) d = lim, low = 0.f;
      *th = __fmul_rn(d, c);
      *tl = fmaf(low, c, fmaf(d, c_low, fmaf(d, c, -*th)));
    }
  }
  // top less the whole part of t
  __device__ __forceinline__ int shift(float x) const {
    float th, tl;
    exponent(x, &th, &tl);
    return top - ((int)(__float_as_uint(th + kStep) - __float_as_uint(kStep)) >> 8);
  }
  // table: a lane's copy, entry j at j * kCopies
  __device__ __forceinline__ u64 operator()(float x, const uint2* table) const {
    float th, tl;
    exponent(x, &th, &tl);
    const float k = __fadd_rn(th, kStep);
    const uint32_t bits = __float_as_uint(k);
    // t = whole + j / 256 + r, |r| <= 2^-9 and what tl brings
    const float r = __fadd_rn(__fsub_rn(th, __fsub_rn(k, kStep)), tl);
    const int whole = (int)(bits - __float_as_uint(kStep)) >> 8;
    const uint2 e = table[(bits & 255u) * kCopies];
    const float p = r * fmaf(r, 0.24022651f, 0.69314718f);  // 2^r - 1
    const uint32_t mant = e.y + __float_as_uint(fmaf(__uint_as_float(e.x), p, kUnit));  // 2^30 2^(j/256 + r)
    u64 w;  // rounded: cut off, 150,000 small weights would lose 2^-28 of the largest
    asm("shr.b64 %0, %1, %2;" : "=l"(w) : "l"((u64)mant << 32), "r"(top - whole + down - 1));
    return (w + 1) >> 1;
  }
};

// ln of a weight's share of `whole`; c: log2(e) / T
__device__ float log_share(const Weigh& w, double c, float x, u64 one, u64 whole) {
  if (one >= whole) return 0.f;
  if (one >= whole - one) return (float)log1p(-(double)(whole - one) / (double)whole);  // (near 0, where ln loses digits)
  const double t = (w.apart ? (double)x - w.m : (double)x) * c;
  return (float)(0.6931471805599453 * (t - w.top + (62 - w.down)) - log((double)whole));
}

// ------------------------------------------------------------------ the kernel
struct SampleShared {
  uint2 table[256 * kCopies];
  u64 list[kList];
  u64 ex[2][kSlots][kMaxCluster];  // what the CTAs of the cluster tell, by turns
  u64 red[kWarps][kSlots];
  u64 found;                       // a token that one CTA told all: logit bits, id
  double log_min, flush, c[2];     // t ln min_p; -60 ln 2 times the temperature; log2(e) / T
  Weigh w[2];                      // filters, draw (without what depends on the maximum)
  float floor;                     // logits below are out
  int count;                       // entries of list
  uint32_t keys[2][kWarps];
};

// What a cluster works on.
template <typename T>
struct Row {
  static constexpr int E = 16 / (int)sizeof(T);
  const T* x;           // its first logit
  int64_t first;        // first vector of this CTA's slice begins at logit `first` (of the first CTA maybe below 0)
  int64_t vocab;
  int vectors, kept;    // of the slice; of them in shared memory
  int seg;              // vectors of a warp, a multiple of 32
  const uint4* slice;

  __device__ __forceinline__ uint4 edge(int v) const {  // a vector that may reach over the row's ends
    union {
      uint4 q;
      T e[E];
    } u;
    const int64_t i0 = first + (int64_t)v * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = i0 + e;
      if (i >= 0 && i < vocab) {
        u.e[e] = x[i];
      } else if constexpr (sizeof(T) == 4) {
        u.e[e] = -INFINITY;
      } else {
        reinterpret_cast<unsigned short*>(u.e)[e] = std::is_same<T, __half>::value ? 0xFC00 : 0xFF80;
      }
    }
    return u.q;
  }
  __device__ __forceinline__ bool inside(int v) const {
    const int64_t i0 = first + (int64_t)v * E;
    return i0 >= 0 && i0 + E <= vocab;
  }
  __device__ __forceinline__ void load(int v, float (&y)[E]) const {
    uint4 q;
    if (v < kept)
      q = slice[v];
    else if (inside(v))
      q = *reinterpret_cast<const uint4*>(x + first + (int64_t)v * E);
    else
      q = edge(v);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        y[j] = __uint_as_float(u[j]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        y[2 * j] = f.x, y[2 * j + 1] = f.y;
      } else {
        y[2 * j] = __uint_as_float(u[j] << 16), y[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    }
  }
  // this warp's vectors, 32 at a time: f(values, id of the first)
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int warp = threadIdx.x >> 5, end = min((warp + 1) * seg, vectors);
    for (int v = warp * seg + (threadIdx.x & 31); v < end; v += 32) {
      float y[E];
      load(v, y);
      f(y, (int)(first + (int64_t)v * E));
    }
  }
};

// Adds up (or, with kMax, takes the largest of) N numbers of every thread of the
// cluster; part: this CTA's and those of the CTAs before it.
template <int N, bool kMax = false>
__device__ __forceinline__ void exchange(SampleShared& s, u64 (&v)[N], uint32_t rank, int cluster, int& turn, u64* before = nullptr, u64* own = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (kMax)
      v[i] = __reduce_max_sync(0xffffffffu, (unsigned)v[i]);
    else
      v[i] = warp_sum(v[i]);
    if (lane == 0) s.red[warp][i] = v[i];
  }
  __syncthreads();
  if (tid < N * cluster) {
    const int i = tid % N;
    u64 t = 0;
    for (int w = 0; w < kWarps; ++w) t = kMax ? max(t, s.red[w][i]) : t + s.red[w][i];
    put(peer(&s.ex[turn][i][rank], tid / N), t);
  }
  cluster_sync();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0;
    if (i == 0 && before) *before = 0;
    for (int c = 0; c < cluster; ++c) {
      const u64 x = s.ex[turn][i][c];
      v[i] = kMax ? max(v[i], x) : v[i] + x;
      if (i == 0 && before && c < (int)rank) *before += x;
    }
    if (i == 0 && own) *own = s.ex[turn][0][rank];
  }
  turn ^= 1;
}

// Sorts list[0, n), n a power of two, ascending.  The pairs of a warp's threads lie in
// the same 64 entries while they are up to 32 apart.
__device__ void sort_list(u64* list, int n) {
  const int t = threadIdx.x;
  __syncthreads();
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int q = t; q < n / 2; q += kThreads) {
        const int i = 2 * q - (q & (j - 1));
        const u64 a = list[i], b = list[i + j];
        if ((a > b) == ((i & k) == 0)) list[i] = b, list[i + j] = a;
      }
      const int next = j > 1 ? j >> 1 : k;
      if (j > 32 || next > 32)
        __syncthreads();
      else
        __syncwarp();
    }
  }
  __syncthreads();
}
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// Inclusive sums over entries 2 tid and 2 tid + 1 of all threads; returns the whole.
__device__ __forceinline__ u64 scan_pairs(SampleShared& s, u64 (&w)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 both = w[0] + w[1];
  const u64 incl = warp_scan(both, lane);
  if (lane == 31) s.red[warp][0] = incl;
  __syncthreads();
  u64 before = 0, whole = 0;
  for (int i = 0; i < kWarps; ++i) {
    const u64 x = s.red[i][0];
    if (i < warp) before += x;
    whole += x;
  }
  __syncthreads();
  w[1] = before + incl;
  w[0] = w[1] - both + w[0];
  return whole;
}

__device__ __forceinline__ u64 by_logit(float x, int id) { return (u64)~key_of(x) << 32 | (uint32_t)id; }
__device__ __forceinline__ float logit_of(u64 e) { return of_key(~(uint32_t)(e >> 32)); }

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int cluster, int64_t slice_vectors, int room_vectors, int down) {
  constexpr int E = Row<T>::E;
  extern __shared__ __align__(16) unsigned char smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  uint4* slice = reinterpret_cast<uint4*>(smem + (sizeof(SampleShared) + 15) / 16 * 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const uint2* table = s.table + (lane & (kCopies - 1));

  pdl_trigger();
  cluster_arrive();  // waited for before a peer's memory is touched
  for (int i = tid; i < 256 * kCopies; i += kThreads) {
    const int j = i / kCopies;
    const uint32_t t = (uint32_t)((__umul64hi(c_coarse[j >> 4], c_fine[j & 15]) + 0x80000000ull) >> 32);  // 2^30 2^(j/256)
    s.table[i] = make_uint2(__float_as_uint((float)t * 0x1p-30f), t - __float_as_uint(kUnit));
  }
  pdl_wait();
  cluster_wait();

  int turn = 0;
  for (int64_t row = blockIdx.x / cluster; row < a.rows; row += gridDim.x / cluster) {
    // ---- settings
    const float u = a.u[row], temp = a.temperature ? a.temperature[row] : 1.f;
    const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
    const int want_k = a.top_k ? a.top_k[row] : 0;
    if (u < 0.f) continue;  // padding
    if (!(u < 1.f) || !(temp == 0.f || (temp >= 1e-6f && temp <= 1e6f)) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f)) {
      if (rank == 0 && tid == 0) set_error(a.status, MINFER_ERR_ARG);
      continue;
    }
    const bool greedy = temp == 0.f;
    const int k = want_k > 0 && want_k < a.vocab ? want_k : 0;
    const float sharp = a.temperature_first ? temp : 1.f;  // what the filters see

    // ---- the row
    Row<T> r;
    r.x = static_cast<const T*>(a.x) + row * a.row_stride;
    r.vocab = a.vocab;
    const int head = (int)((reinterpret_cast<uintptr_t>(r.x) & 15) / sizeof(T));  // logits before the first in its vector
    r.first = (int64_t)rank * slice_vectors * E - head;
    const int64_t all = (head + a.vocab + E - 1) / E;
    r.vectors = (int)max((int64_t)0, min(slice_vectors, all - (int64_t)rank * slice_vectors));
    r.kept = min(r.vectors, room_vectors);
    r.seg = ((r.vectors + kWarps - 1) / kWarps + 31) / 32 * 32;
    r.slice = slice;
    const int begin = warp * r.seg + lane, end = min((warp + 1) * r.seg, r.vectors);
    {
      // all copies at once, in four groups
      const int quarter = max(32, (r.seg / 4 + 31) / 32 * 32);
      int v = begin;
#pragma unroll
      for (int q = 1; q <= 4; ++q) {
        const int stop = q == 4 ? end : min(end, warp * r.seg + q * quarter);
        for (; v < stop; v += 32) {
          if (v >= r.kept) continue;
          if (r.inside(v))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slice + v)), "l"(r.x + r.first + (int64_t)v * E) : "memory");
          else
            slice[v] = r.edge(v);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (tid == 0) {
        s.count = 0;
        if (!greedy) {
          const double log2e = 1.4426950408889634, ln2 = 0.6931471805599453;
          for (int i = 0; i < 2; ++i) {
            const double c = log2e / (double)(i ? temp : sharp);
            s.c[i] = c;
            s.w[i].c = (float)c;
            s.w[i].c_low = (float)(c - (double)(float)c);
          }
          s.flush = -60 * ln2 * (double)temp;
          s.log_min = min_p > 0.f ? (double)sharp * log((double)min_p) : -1e300;
        }
      }
      float top = -INFINITY;
      v = begin;
#pragma unroll
      for (int q = 1; q <= 4; ++q) {
        if (q == 1) asm volatile("cp.async.wait_group 3;" ::: "memory");
        if (q == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
        if (q == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (q == 4) asm volatile("cp.async.wait_group 0;" ::: "memory");
        const int stop = q == 4 ? end : min(end, warp * r.seg + q * quarter);
        for (; v < stop; v += 32) {
          float y[E];
          r.load(v, y);
#pragma unroll
          for (int e = 0; e < E; ++e) top = max_nan(top, y[e]);
        }
      }
      // ---- the maximum, and the bound
      const uint32_t key = key_of(top);
      const int aim = greedy ? 0 : k > 0 ? (k <= kThreads ? k : 0) : top_p < 1.f ? kGuess : 0;
      uint32_t bound = 0;
      if (aim > 0) {
        const uint32_t hi_w = __reduce_max_sync(0xffffffffu, key), lo_w = __reduce_min_sync(0xffffffffu, key);
        if (lane == 0) s.keys[0][warp] = lo_w, s.keys[1][warp] = hi_w;
        __syncthreads();
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        for (int i = 0; i < kWarps; ++i) lo = min(lo, s.keys[0][i]), hi = max(hi, s.keys[1][i]);
        // at least `aim` threads have a maximum of lo or more, fewer one of `over` or more
        for (uint32_t over = hi == 0xFFFFFFFFu ? hi : hi + 1; over - lo > 1;) {
          const uint32_t mid = lo + (over - lo) / 2;
          const int n = __syncthreads_count(key >= mid);
          if (n >= aim) {
            lo = mid;
            if (n <= aim + aim / 4 + 2) break;
          } else {
            over = mid;
          }
        }
        bound = lo;
      }
      u64 v2[2] = {key, bound};
      exchange<2, true>(s, v2, rank, cluster, turn);
      const float m = of_key((uint32_t)v2[0]);
      const float b = v2[1] ? fmaxf(of_key((uint32_t)v2[1]), kLowest) : kLowest;  // -inf is no candidate

      auto write = [&](int token, float logprob) {
        a.token[row] = token;
        if (a.logprob) a.logprob[row] = logprob;
      };
      bool done = true;
      if (!(m < INFINITY)) {  // a NaN or +inf
        if (rank == 0 && tid == 0) set_error(a.status, MINFER_ERR_ARG);
      } else if (m == -INFINITY) {
        if (rank == 0 && tid == 0) write(-1, -INFINITY);
      } else if (greedy) {
        int id = 0x7FFFFFFF;
        r.each([&](const float (&y)[E], int i0) {
#pragma unroll
          for (int e = E - 1; e >= 0; --e)
            if (y[e] == m) id = min(id, i0 + e);
        });
        u64 v1[1] = {0x7FFFFFFFu - (unsigned)id};
        exchange<1, true>(s, v1, rank, cluster, turn);
        if (rank == 0 && tid == 0) write((int)(0x7FFFFFFFu - (unsigned)v1[0]), 0.f);
      } else {
        done = false;
      }
      if (done) {
        cluster_sync();
        continue;
      }

      // ---- the weights' scale; logits below `floor` are out for min-p or weigh nothing
      Weigh wf = s.w[0], wd = s.w[1];
      wf.down = wd.down = down;
      wf.at(m, sharp);
      wd.at(m, temp);
      if (tid == 0) s.floor = fmaxf(__double2float_ru((double)m + fmax(s.log_min, s.flush)), kLowest);

      u64 need = 0;  // of top-p: tokens are kept while the weights before them are less
      bool covered = true;
      auto set_need = [&](u64 total) {
        bool rest;
        need = times(total, top_p, &rest);
        need = max(need + rest, (u64)1);
      };
      if (k == 0 && top_p < 1.f) {
        u64 v3[2] = {0, 0};
        r.each([&](const float (&y)[E], int) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const u64 w = wf(y[e], table);
            v3[0] += w;
            v3[1] += y[e] >= b ? w : 0;
          }
        });
        exchange<2>(s, v3, rank, cluster, turn);
        set_need(v3[0]);
        covered = v3[1] >= need;
      } else {
        __syncthreads();  // s.floor
      }
      const float floor_x = s.floor;

      // logits in [from, below) that `kept` leaves, to the first CTA's list, in any order;
      // returns how many there are
      auto gather = [&](float from, float below, auto kept) {
        r.each([&](const float (&y)[E], int i0) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (y[e] >= from && y[e] < below && kept(y[e], i0 + e)) {
              const int at = peer_add(peer(&s.count, 0), 1);
              if (at < kList) put(peer(&s.list[at], 0), by_logit(y[e], i0 + e));
            }
        });
        cluster_sync();
        return peer_get(peer(&s.count, 0));
      };

      // ---- the short way
      bool wide = false;
      float from;
      if (a.vocab <= kList)
        from = kLowest;
      else if (k > 0) {
        wide = aim == 0;
        from = top_p < 1.f ? b : fmaxf(b, floor_x);
      } else if (top_p < 1.f) {
        wide = !covered && floor_x < b;
        from = fmaxf(b, floor_x);
      } else {
        wide = min_p == 0.f;
        from = floor_x;
      }
      if (!wide) {
        const int n = gather(from, INFINITY, [](float, int) { return true; });
        wide = n > kList;
        if (!wide && rank == 0) {
          const int size = power_of_two(n);
          for (int i = n + tid; i < size; i += kThreads) s.list[i] = ~0ull;
          sort_list(s.list, size);
          const int first_k = k > 0 ? min(k, n) : n;
          int left = first_k;
          if (top_p < 1.f) {
            u64 w[2], one[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) one[i] = w[i] = 2 * tid + i < first_k ? wf(logit_of(s.list[2 * tid + i]), table) : 0;
            const u64 whole = scan_pairs(s, w);
            if (k > 0 || a.vocab <= kList) set_need(whole);
            const int c0 = __syncthreads_count(2 * tid < first_k && w[0] - one[0] < need);
            const int c1 = __syncthreads_count(2 * tid + 1 < first_k && w[1] - one[1] < need);
            left = max(1, c0 + c1);
          }
          {
            const int c0 = __syncthreads_count(2 * tid < left && logit_of(s.list[min(2 * tid, kList - 1)]) >= floor_x);
            const int c1 = __syncthreads_count(2 * tid + 1 < left && logit_of(s.list[min(2 * tid + 1, kList - 1)]) >= floor_x);
            left = max(1, c0 + c1);
          }
          if (left == 1) {
            if (tid == 0) write((int)(uint32_t)s.list[0], 0.f);
          } else {
            // in the order of ids
            const int size2 = power_of_two(left);
            for (int i = tid; i < size2; i += kThreads) {
              const u64 e = s.list[i];
              s.list[i] = i < left ? e << 32 | e >> 32 : ~0ull;
            }
            sort_list(s.list, size2);
            u64 w[2], one[2];
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int at = 2 * tid + i;
              x[i] = at < left ? of_key(~(uint32_t)s.list[at]) : 0.f;
              one[i] = w[i] = at < left ? wd(x[i], table) : 0;
            }
            const u64 whole = scan_pairs(s, w);
            bool rest;
            const u64 target = times(whole, u, &rest);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (u > 0.f ? w[i] - one[i] <= target && target < w[i] : 2 * tid + i == 0)  // (u 0: the first, however little it weighs)
                write((int)(s.list[2 * tid + i] >> 32), log_share(wd, s.c[1], x[i], one[i], whole));
          }
        }
      }

      // ---- the wide way
      if (wide) {
        float xb = -INFINITY;  // kept: what is larger, and of its equals the ids up to idb
        int idb = 0x7FFFFFFF;
        auto kept = [&](float x, int id) { return x > xb || (x == xb && id <= idb && x > -INFINITY); };

        // The first token, in the order of ids, at which the sum of weigh(x, id) exceeds
        // target(whole): to all threads of the cluster, with the whole.
        auto locate = [&](auto weigh, auto target, u64* whole) {
          u64 mine = 0;
          r.each([&](const float (&y)[E], int i0) {
#pragma unroll
            for (int e = 0; e < E; ++e) mine += weigh(y[e], i0 + e);
          });
          const u64 seg_sum = warp_sum(mine);
          u64 v1[1] = {mine}, before, own;
          exchange<1>(s, v1, rank, cluster, turn, &before, &own);
          const u64 t = target(v1[0]);
          *whole = v1[0];
          (void)seg_sum;
          if (t >= before && t < before + own) {  // in this CTA (s.red holds its warps' sums)
            for (int i = 0; i < warp; ++i) before += s.red[i][0];
            if (t >= before && t < before + seg_sum) {
              const int end_w = min((warp + 1) * r.seg, r.vectors);
              for (int v0 = warp * r.seg; v0 < end_w; v0 += 32) {
                float y[E];
                u64 w[E], sum = 0;
                const bool there = v0 + lane < end_w;
                if (there) r.load(v0 + lane, y);
                const int i0 = (int)(r.first + (int64_t)(v0 + lane) * E);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  w[e] = there ? weigh(y[e], i0 + e) : 0;
                  sum += w[e];
                }
                const u64 incl = warp_scan(sum, lane) + before;
                if (incl - sum <= t && t < incl) {
                  u64 at = incl - sum;
                  bool hit = false;
#pragma unroll
                  for (int e = 0; e < E; ++e) {
                    at += w[e];
                    if (!hit && t < at) {
                      hit = true;
                      for (int c = 0; c < cluster; ++c) put(peer(&s.found, c), (u64)__float_as_uint(y[e]) << 32 | (uint32_t)(i0 + e));
                    }
                  }
                }
                before = __shfl_sync(0xffffffffu, incl, 31);
                if (t < before) break;
              }
            }
          }
          cluster_sync();
          return s.found;
        };

        // Moves the border (xb, idb) to the last token, in descending order, before
        // which less than `goal` is kept: tokens (kMass false) or weights.
        auto cut = [&](auto is_mass, u64 goal) {
          constexpr bool kMass = decltype(is_mass)::value;
          uint32_t lo = key_of(kLowest), hi = key_of(m) + 1;  // `goal` is reached at lo, not at hi
          u64 n_lo = ~0ull, n_hi = 0, f_hi = 0;  // tokens of that size or larger, and the measure
          for (int step = 0; step == 0 || (n_lo - n_hi > kList && hi - lo > 1); ++step) {
            uint32_t at[3];
            if (step == 0) {
              at[0] = lo, at[1] = max(lo, key_of(fmaxf(m - 16.f * sharp, kLowest))), at[2] = max(lo, key_of(fmaxf(m - 4.f * sharp, kLowest)));
            } else {
              // by value and by bits in turn: the first closes in fast, the second ends
              const float x0 = of_key(lo), x1 = of_key(hi);
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const uint32_t by_bits = lo + (uint32_t)(((u64)(hi - lo) * (j + 1)) >> 2);
                const float x = x0 * (0.75f - 0.25f * j) + x1 * (0.25f + 0.25f * j);
                at[j] = step & 1 ? key_of(x) : by_bits;
                at[j] = min(max(at[j], lo + 1), hi - 1);
              }
            }
            const float t0 = of_key(at[0]), t1 = of_key(at[1]), t2 = of_key(at[2]);
            u64 v6[6] = {0, 0, 0, 0, 0, 0};
            r.each([&](const float (&y)[E], int i0) {
#pragma unroll
              for (int e = 0; e < E; ++e)
                if (y[e] >= t0 && kept(y[e], i0 + e)) {
                  const u64 w = kMass ? wf(y[e], table) : 1;
                  v6[0] += 1, v6[3] += w;
                  if (y[e] >= t1) v6[1] += 1, v6[4] += w;
                  if (y[e] >= t2) v6[2] += 1, v6[5] += w;
                }
            });
            exchange<6>(s, v6, rank, cluster, turn);
            if (step == 0) {
              if (v6[3] < goal) return;  // all of it is kept
              n_lo = v6[0];
            }
#pragma unroll
            for (int j = 0; j < 3; ++j)
              if (v6[3 + j] >= goal) lo = at[j], n_lo = v6[j];
#pragma unroll
            for (int j = 2; j >= 0; --j)
              if (v6[3 + j] < goal) hi = at[j], n_hi = v6[j], f_hi = v6[3 + j];
          }
          if (n_lo - n_hi <= kList) {
            if (tid == 0) s.count = 0;
            cluster_sync();
            const int n = gather(of_key(lo), of_key(hi), kept);
            if (rank == 0) {
              const int size = power_of_two(n);
              for (int i = n + tid; i < size; i += kThreads) s.list[i] = ~0ull;
              sort_list(s.list, size);
              u64 w[2], one[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) one[i] = w[i] = 2 * tid + i < n ? (kMass ? wf(logit_of(s.list[2 * tid + i]), table) : 1) : 0;
              scan_pairs(s, w);
#pragma unroll
              for (int i = 0; i < 2; ++i)  // the one whose weight reaches the goal
                if (f_hi + w[i] - one[i] < goal && f_hi + w[i] >= goal && one[i] > 0)
                  for (int c = 0; c < cluster; ++c) put(peer(&s.found, c), (u64)__float_as_uint(logit_of(s.list[2 * tid + i])) << 32 | (uint32_t)s.list[2 * tid + i]);
            }
            cluster_sync();
            xb = __uint_as_float((uint32_t)(s.found >> 32));
            idb = (int)(uint32_t)s.found;
          } else {
            // one value, more often than the list is long
            const float x = of_key(lo);
            const u64 w = kMass ? wf(x, table) : 1, nth = (goal - f_hi + w - 1) / w;
            u64 whole;
            const u64 found = locate([&](float y, int id) { return (u64)(y == x && kept(y, id)); }, [&](u64) { return nth - 1; }, &whole);
            xb = x;
            idb = (int)(uint32_t)found;
          }
          __syncthreads();  // s.found has been read
        };
        if (k > 0) cut(std::false_type(), (u64)k);
        if (top_p < 1.f) {
          if (k > 0) {
            u64 v1[1] = {0};
            r.each([&](const float (&y)[E], int i0) {
#pragma unroll
              for (int e = 0; e < E; ++e) v1[0] += kept(y[e], i0 + e) ? wf(y[e], table) : 0;
            });
            exchange<1>(s, v1, rank, cluster, turn);
            set_need(v1[0]);
          }
          cut(std::true_type(), need);
        }
        u64 whole, count;
        u64 found = locate([&](float y, int id) { return y >= floor_x && kept(y, id) ? wd(y, table) : 0; },
                                 [&](u64 n) {
                                   bool rest;
                                   return times(n, u, &rest);
                                 },
                                 &whole);
        if (u == 0.f) found = locate([&](float y, int id) { return (u64)(y >= floor_x && kept(y, id)); }, [](u64) { return (u64)0; }, &count);
        if (rank == 0 && tid == 0) {
          const float x = __uint_as_float((uint32_t)(found >> 32));
          write((int)(uint32_t)found, log_share(wd, s.c[1], x, wd(x, table), whole));
        }
      }
      cluster_sync();  // the next row's first words
    }
  }
}

template <typename T>
cudaError_t sample_typed(const SampleArgs& a, int num_sms, cudaStream_t st) {
  constexpr int E = Row<T>::E;
  const int64_t all = (a.vocab + 2 * E - 2) / E;  // vectors of a row, wherever it begins
  // As many CTAs as keep the row; more while they leave SMs idle and have something to do.
  int cluster = 1;
  auto slice = [&] { return (all + cluster - 1) / cluster; };
  while (cluster < kMaxCluster && (slice() * 16 > kRoom || (a.rows * cluster * 2 <= num_sms && slice() * 16 > 8192))) cluster *= 2;
  const int room = (int)std::min<int64_t>(slice(), kRoom / 16);
  const int smem = (int)((sizeof(SampleShared) + 15) / 16 * 16) + room * 16;
  const cudaError_t e = allow_smem<sample_kernel<T>>((int)((sizeof(SampleShared) + 15) / 16 * 16) + kRoom);
  if (e != cudaSuccess) return e;
  int down = 1;  // weights of 2^(63 - down) at most: the sum of all fits 64 bits
  while ((1ll << down) < a.vocab) ++down;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.rows, 1 << 24) * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, cluster, slice(), room, down);
}

}  // namespace

cudaError_t sample_launch(const SampleArgs& a, int type, int num_sms, cudaStream_t st) {
  return type == MINFER_F32   ? sample_typed<float>(a, num_sms, st)
         : type == MINFER_F16 ? sample_typed<__half>(a, num_sms, st)
                              : sample_typed<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace minfer
