// sample.cuh -- what the sampling kernels share: a row's settings, weights as whole
// numbers, and the end of a row whose candidates are in a list.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

typedef unsigned long long u64;
constexpr float kLowest = -3.402823466e38f;

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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// floor(n * f) for 0 <= f < 1 (and not -0), exactly; *rest: whether something was cut off
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

// ------------------------------------------------------------------ settings
struct Settings {
  float u, temp, top_p, min_p;
  float sharp;  // the temperature that the filters see
  int k;        // 0: off
  bool skip, bad, greedy;

  // The temperature of the weights whose sum over the whole row is wanted; 0: of none.
  __device__ __forceinline__ float whole_row() const { return greedy || k > 0 ? 0.f : top_p < 1.f ? sharp : min_p > 0.f ? 0.f : temp; }
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
  Settings s;
  s.u = a.u[row] + 0.f;  // (-0 as 0: `times` reads the bits)
  s.temp = a.temperature ? a.temperature[row] : 1.f;
  s.top_p = a.top_p ? a.top_p[row] + 0.f : 1.f;
  s.min_p = a.min_p ? a.min_p[row] : 0.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  s.k = k > 0 && k < a.vocab ? k : 0;
  s.sharp = a.temperature_first ? s.temp : 1.f;
  s.greedy = s.temp == 0.f;
  s.skip = s.u < 0.f;  // padding
  s.bad = !(s.u < 1.f) || !(s.greedy || (s.temp >= 1e-6f && s.temp <= 1e6f)) || !(s.top_p >= 0.f) || !(s.min_p >= 0.f && s.min_p <= 1.f);
  return s;
}
// The logit below which min-p leaves nothing, or a token weighs too little to be drawn;
// m: the largest.  In 64 bits, rounded up, so that f32 logits compare as if exact.
__device__ __noinline__ float floor_at(float temp, float sharp, float min_p, float m) {
  const double ln2 = 0.6931471805599453;
  double at = -60 * ln2 * (double)temp;
  if (min_p > 0.f) at = fmax(at, (double)sharp * log((double)min_p));
  return fmaxf(__double2float_ru((double)m + at), kLowest);
}
// (a function that is called takes values: what it took by reference would live in memory)
__device__ __forceinline__ float floor_of(const Settings& s, float m) { return floor_at(s.temp, s.sharp, s.min_p, m); }

// 8 or 4 logits of a vector; a vector that may reach over the row's ends, -inf outside
template <typename T>
struct Logits {
  static constexpr int E = 16 / (int)sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4& q, float (&y)[E]) {
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
  static __device__ __forceinline__ bool inside(int64_t i0, int64_t vocab) { return i0 >= 0 && i0 + E <= vocab; }
  static __device__ __noinline__ uint4 edge(const T* x, int64_t i0, int64_t vocab) {
    union {
      uint4 q;
      uint32_t w[4];
      unsigned short h[8];
    } u;
    u.q = make_uint4(0, 0, 0, 0);
    for (int e = 0; e < E; ++e) {
      const bool in = i0 + e >= 0 && i0 + e < vocab;
      if constexpr (sizeof(T) == 4)
        u.w[e] = in ? reinterpret_cast<const uint32_t*>(x)[i0 + e] : 0xFF800000u;
      else
        u.h[e] = in ? reinterpret_cast<const unsigned short*>(x)[i0 + e] : (unsigned short)(std::is_same<T, __half>::value ? 0xFC00 : 0xFF80);
    }
    return u.q;
  }
};

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

// Copies of the table of 2^(j/256), entry j at j * copies: as an f32, and as a whole
// number of 2^-30 less the bits of kUnit.
__device__ __forceinline__ void fill_table(uint2* table, int copies, int tid, int threads) {
  for (int i = tid; i < 256 * copies; i += threads) {
    const int j = i / copies;
    const uint32_t t = (uint32_t)((__umul64hi(c_coarse[j >> 4], c_fine[j & 15]) + 0x80000000ull) >> 32);
    table[i] = make_uint2(__float_as_uint((float)t * 0x1p-30f), t - __float_as_uint(kUnit));
  }
}

// The weights under one temperature: exp((x - m) / T) as a whole number in units of
// 2^(down - 62) of a power of two near the maximum's.  Before it is cut to these units a
// weight is off by at most, as a share of itself: 2^-31 for the table's entry and 2^-31 for the
// sum, each rounded to 2^-30; 0.0555 |r|^3 for the cubic term, which is left out, and 0.694 |r|
// 2^-22 for the steps of the others, with |r| <= 2^-9 + |t| 2^-23; and 1.5e-14 |t| for t itself.
// That is less than 2^-29 up to |t| = 1,050 and than 2^-28 up to the 8,254 of a row that is not
// apart (measured: 2^-29.3 and 2^-29.0).
struct Weigh {
  float c, c_low;  // log2(e) / T as a sum
  float m;
  float lim;       // what lies below weighs nothing: x below lim, or x - m
  int top;         // whole part of the maximum's exponent
  int down;
  bool apart;      // |m| c is large: x - m is taken first

  // An exponent below -62 (which a sum of 2^31 weights does not notice) counts as -62:
  // its weight is 0, and -inf and huge differences stay out of the arithmetic.
  __device__ __forceinline__ void at(float t, float max, int down_, float far = 8192.f) {
    const float hi = 1.44269502162933349609375f, low = 1.92596299112661746886e-8f;  // log2(e)
    c = __fdiv_rn(hi, t);
    c_low = __fdiv_rn(fmaf(-c, t, hi) + low, t);
    m = max;
    down = down_;
    apart = !(fabsf(max * c) <= far);
    lim = apart ? -43.f * t : max - 43.f * t;  // 62 ln 2 = 42.98
    top = 0;
    top = whole_of(max);
  }
  // What exponents are taken from, x (or x - m) as a sum of two; kApart false: the caller
  // knows that the row is not apart.
  template <int N, bool kApart>
  __device__ __forceinline__ void bases(const float (&x)[N], float (&v)[N], float (&low)[N]) const {
    if (kApart && apart) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[e] = __fsub_rn(x[e], m);
        const float b = __fsub_rn(v[e], x[e]);
        low[e] = __fadd_rn(__fsub_rn(x[e], __fsub_rn(v[e], b)), __fsub_rn(-m, b));
        if (!(v[e] > lim)) v[e] = lim, low[e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = fmaxf(x[e], lim), low[e] = 0.f;
    }
  }
  // t = (v + low) log2(e) / T as th + tl
  template <bool kApart>
  __device__ __forceinline__ void exponent(float v, float low, float* th, float* tl) const {
    *th = __fmul_rn(v, c);
    *tl = fmaf(v, c_low, fmaf(v, c, -*th));
    if (kApart) *tl = fmaf(low, c, *tl);
  }
  __device__ __forceinline__ int whole_of(float x) const {
    float at[1] = {x}, v[1], low[1], th, tl;
    bases<1, true>(at, v, low);
    exponent<true>(v[0], low[0], &th, &tl);
    return (int)(__float_as_uint(th + kStep) - __float_as_uint(kStep)) >> 8;
  }
  // N weights side by side.  table: the caller's copy, entry j at j * kCopies.  (One piece of
  // code for rows that are apart and rows that are not, with a branch for all N: the kernels
  // wait for their instructions.)
  template <int kCopies, bool kApart = true, int N>
  __device__ __forceinline__ void all(const float (&x)[N], u64 (&w)[N], const uint2* table) const {
    float v[N], low[N];
    bases<N, kApart>(x, v, low);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float th, tl;
      exponent<kApart>(v[i], low[i], &th, &tl);
      const float k = __fadd_rn(th, kStep);
      const uint32_t bits = __float_as_uint(k);
      // t = whole + j / 256 + r, |r| <= 2^-9 and what tl brings
      const float r = __fadd_rn(__fsub_rn(th, __fsub_rn(k, kStep)), tl);
      const int whole = (int)(bits - __float_as_uint(kStep)) >> 8;
      const uint2 e = table[(bits & 255u) * kCopies];
      const float p = r * fmaf(r, 0.24022651f, 0.69314718f);  // 2^r - 1
      const uint32_t mant = e.y + __float_as_uint(fmaf(__uint_as_float(e.x), p, kUnit));  // 2^30 2^(j/256 + r)
      u64 y;  // rounded: cut off, 150,000 small weights would lose 2^-28 of the largest
      asm("shr.b64 %0, %1, %2;" : "=l"(y) : "l"((u64)mant << 32), "r"(top - whole + down - 1));
      w[i] = (y + 1) >> 1;
    }
  }
  template <int kCopies, bool kApart = true>
  __device__ __forceinline__ u64 one(float x, const uint2* table) const {
    const float at[1] = {x};
    u64 w[1];
    all<kCopies, kApart>(at, w, table);
    return w[0];
  }
};

// ln of a weight's share of `whole`; from, power: log_share's
__device__ __noinline__ float log_share_of(float temp, float x, float from, int power, u64 one, u64 whole) {
  if (one >= whole) return 0.f;
  if (one >= whole - one) return (float)log1p(-(double)(whole - one) / (double)whole);  // (near 0, where ln loses digits)
  return (float)(((double)x - from) / temp + 0.6931471805599453 * power - log((double)whole));
}
__device__ __forceinline__ float log_share(const Weigh& w, float temp, float x, u64 one, u64 whole) {
  return log_share_of(temp, x, w.apart ? w.m : 0.f, 62 - w.down - w.top, one, whole);
}

// ------------------------------------------------------------------ lists
// Entries: logit and id, ascending in the order of the filters.
__device__ __forceinline__ u64 by_logit(float x, int id) { return (u64)~key_of(x) << 32 | (uint32_t)id; }
__device__ __forceinline__ float logit_of(u64 e) { return of_key(~(uint32_t)(e >> 32)); }
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// Sorts list[0, n) ascending, kPer entries to a thread (thread t has t + r kThreads), in
// registers: partners meet in a thread, by shuffles, or through the list.
template <int kThreads, int kPer>
__device__ __noinline__ void sort_wide(u64* list, int n) {
  const int t = threadIdx.x;
  u64 v[kPer];
#pragma unroll
  for (int r = 0; r < kPer; ++r) v[r] = t + r * kThreads < n ? list[t + r * kThreads] : ~0ull;
  for (int k = 2; k <= kThreads * kPer; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      u64 other[kPer];
      if (j >= kThreads) {
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          other[r] = 0;
#pragma unroll
          for (int q = 0; q < kPer; ++q)
            if ((r ^ q) * kThreads == j) other[r] = v[q];
        }
      } else if (j >= 32) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kPer; ++r) list[t + r * kThreads] = v[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kPer; ++r) other[r] = list[(t ^ j) + r * kThreads];
      } else {
#pragma unroll
        for (int r = 0; r < kPer; ++r) other[r] = __shfl_xor_sync(0xffffffffu, v[r], j);
      }
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int e = t + r * kThreads;
        const bool small = ((e & k) == 0) == ((e & j) == 0);  // keeps the smaller one
        v[r] = (v[r] < other[r]) == small ? v[r] : other[r];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPer; ++r) list[t + r * kThreads] = v[r];
  __syncthreads();
}
// Sorts list[0, n), n <= kEntries, entries distinct; of what follows nothing is left.  Up
// to 256 entries find their places by counting the smaller ones, as many threads to an
// entry as there are (64 entries: 0.2 us against 3 by exchanges).
template <int kThreads, int kEntries>
__device__ __forceinline__ void sort_list(u64* list, int n) {
  if (n > 256 || n > kThreads) {
    if (kThreads >= 512 && n <= kThreads)
      sort_wide<kThreads, 1>(list, n);
    else if (kEntries >= 2 * kThreads && n <= 2 * kThreads)
      sort_wide<kThreads, 2>(list, n);
    else if (kEntries > 4 * kThreads && n <= 4 * kThreads)
      sort_wide<kThreads, 4>(list, n);
    else
      sort_wide<kThreads, kEntries / kThreads>(list, n);
    return;
  }
  const int per = min(32, kThreads / power_of_two(n)), i = threadIdx.x / per;
  const u64 mine = i < n ? list[i] : 0;
  int c = 0;
  for (int j = threadIdx.x & (per - 1); j < n; j += per) c += list[j] < mine;
  for (int o = per >> 1; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  __syncthreads();
  if (i < n && (threadIdx.x & (per - 1)) == 0) list[c] = mine;
  __syncthreads();
}

// Inclusive sums over the kPer neighbouring numbers of all threads; returns the whole.
template <int kThreads, int kPer>
__device__ __forceinline__ u64 scan_all(u64* red, u64 (&w)[kPer]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 1; i < kPer; ++i) w[i] += w[i - 1];
  const u64 incl = warp_scan(w[kPer - 1], lane);
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  u64 before = incl - w[kPer - 1], whole = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    const u64 x = red[i];
    if (i < warp) before += x;
    whole += x;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) w[i] += before;
  return whole;
}

// The tokens before which weights of less than this many are kept: at least one.
__device__ __forceinline__ u64 need_of(u64 total, float top_p) {
  bool rest;
  const u64 n = times(total, top_p, &rest);
  return max(n + rest, (u64)1);
}

// The end of a row whose candidates, n of them, are in `list` in any order: they are the
// first n of the row's order, or, where fewer than that, all that weigh something.
// whole: the sum of the filters' weights over the row, if top-p is to be taken from it
// (0: from the list's own).  False if top-p reaches past the list and `open` says that
// there is something there.  All threads; write(token, log probability) by one.
template <int kThreads, int kPer, int kEntries, int kCopies, typename F>
__device__ __forceinline__ bool finish_sorted(u64* list, u64* red, int n, const Settings& s, const Weigh& wf, const Weigh& wd, const uint2* table, float floor_x,
                                              u64 whole, bool open, F write) {
  const int i0 = threadIdx.x * kPer;
  int left = s.k > 0 ? min(s.k, n) : n;
  if (s.top_p < 1.f) {
    u64 w[kPer], one[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) one[i] = w[i] = i0 + i < left ? wf.one<kCopies>(logit_of(list[i0 + i]), table) : 0;
    const u64 sum = scan_all<kThreads, kPer>(red, w);
    const u64 need = need_of(whole ? whole : sum, s.top_p);
    if (open && sum < need) return false;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += __syncthreads_count(i0 + i < left && w[i] - one[i] < need);
    left = max(1, c);
  }
  {
    int c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += __syncthreads_count(i0 + i < left && logit_of(list[i0 + i]) >= floor_x);
    left = max(1, c);
  }
  if (left == 1) {
    if (threadIdx.x == 0) write((int)(uint32_t)list[0], 0.f);
    return true;
  }
  // in the order of ids
  for (int i = threadIdx.x; i < left; i += kThreads) list[i] = list[i] << 32 | list[i] >> 32;
  __syncthreads();
  sort_list<kThreads, kEntries>(list, left);
  u64 w[kPer], one[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) one[i] = w[i] = i0 + i < left ? wd.one<kCopies>(of_key(~(uint32_t)list[i0 + i]), table) : 0;
  const u64 sum = scan_all<kThreads, kPer>(red, w);
  bool rest;
  const u64 target = times(sum, s.u, &rest);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (s.u > 0.f ? w[i] - one[i] <= target && target < w[i] : i0 + i == 0)  // (u 0: the first, however little it weighs)
      write((int)(list[i0 + i] >> 32), log_share(wd, s.temp, of_key(~(uint32_t)list[i0 + i]), one[i], sum));
  return true;
}
template <int kThreads, int kEntries, int kCopies, typename F>
__device__ __forceinline__ bool finish_list(u64* list, u64* red, int n, const Settings& s, const Weigh& wf, const Weigh& wd, const uint2* table, float floor_x,
                                            u64 whole, bool open, F write) {
  sort_list<kThreads, kEntries>(list, n);
  if (n <= kThreads) return finish_sorted<kThreads, 1, kEntries, kCopies>(list, red, n, s, wf, wd, table, floor_x, whole, open, write);
  if (kEntries > 2 * kThreads && n <= 2 * kThreads)
    return finish_sorted<kThreads, 2, kEntries, kCopies>(list, red, n, s, wf, wd, table, floor_x, whole, open, write);
  return finish_sorted<kThreads, kEntries / kThreads, kEntries, kCopies>(list, red, n, s, wf, wd, table, floor_x, whole, open, write);
}

}  // namespace
}  // namespace minfer
