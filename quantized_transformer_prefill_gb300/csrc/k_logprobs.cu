// k_logprobs.cu -- log probabilities of given tokens, entropy and the k
// largest of logits rows, in one pass over the logits.
//
//   m = max x,  s = sum e^(x-m),  t = sum e^(x-m) (x-m) log2 e
//   log p_i = (x_i - m) - ln s,   H = ln 2 (log2 s - t / s)
//
// x - m is taken before the factor log2 e: one multiply-add with a rounded
// m log2 e would be off by 2^-24 |m|, which for logits of 1e30, or for rows
// masked with the type's lowest value, is any power of two.
//
// A row is cut into parts, one CTA each; a part keeps a running (m, s, t) per
// thread and the k largest (value, id) pairs.  The pairs are compared as one
// 64-bit key, the value's order-preserving bits above the complemented id, so
// keys are distinct and equal values rank by ascending id whatever the order
// in which threads meet them.  logprobs_join_kernel adds up a row's parts.
//
// The k largest of a part: the k-th largest of the 32 lane maxima of a warp is
// a lower bound of the part's k-th largest value, so after the first tile only
// values from the best such bound on are collected; later tiles add what
// exceeds the bound, and the collected pairs are cut back to k whenever they
// pass a limit, which raises the bound.  Almost every value fails one compare.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 4096;            // values of a tile, kThreads x 16
constexpr int kPer = kTile / kThreads;  // values of a thread
constexpr int kCut = 512;               // collected pairs that trigger a cut back to k
constexpr int kCap = kCut + kTile;
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
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = max_nan(a.m, b.m);
  // an empty side contributes nothing; its shift would be -inf
  const float da = a.m == -INFINITY ? 0.f : (a.m - r.m) * kLog2e, db = b.m == -INFINITY ? 0.f : (b.m - r.m) * kLog2e;
  const float ca = ex2(da), cb = ex2(db);
  r.s = a.s * ca + b.s * cb;
  // the terms' shift d moves t by d s; far below, c = 0 and d may overflow: no term
  r.t = (ca == 0.f ? 0.f : ca * (a.t + da * a.s)) + (cb == 0.f ? 0.f : cb * (b.t + db * b.s));
  return r;
}
__device__ __forceinline__ Stat warp_join(Stat v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.t = __shfl_xor_sync(0xffffffffu, v.t, o);
    // both lanes of a pair join in the same order: the sum does not depend on the lane
    v = (threadIdx.x & o) ? join(w, v) : join(v, w);
  }
  return v;
}

// The lane-th largest of the warp's 32 keys (bitonic sort, descending).
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t w = __shfl_xor_sync(0xffffffffu, v, j);
      const bool desc = (lane & k) == 0, low = (lane & j) == 0;
      v = (desc == low) ? max(v, w) : min(v, w);
    }
  return v;
}

// The largest key of the CTA; every thread gets it.  s: one slot per warp.
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) v = s[i] > v ? s[i] : v;
  return v;
}

// The min(k, n) largest of the n distinct keys buf[0..n) to the front, in
// descending order.  All threads; ends with a barrier.
__device__ void cut_to_k(uint64_t* buf, int n, int k, uint64_t* s_best, uint64_t* s_red) {
  const int tid = threadIdx.x;
  if (n <= kThreads) {
    // a key's place is the number of keys above it
    const uint64_t own = tid < n ? buf[tid] : 0;
    int place = 0;
    for (int i = 0; i < n; ++i) place += buf[i] > own;
    __syncthreads();
    if (tid < n && place < k) buf[place] = own;
  } else {
    uint64_t last = ~0ull;  // the key taken in the round before
    for (int j = 0; j < k; ++j) {
      uint64_t best = 0;
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t v = buf[i];
        best = (v < last && v > best) ? v : best;
      }
      last = block_max(best, s_red);
      if (tid == 0) s_best[j] = last;
    }
    __syncthreads();
    if (tid < k) buf[tid] = s_best[tid];
  }
  __syncthreads();
}

template <typename T>
struct Loader;  // 16-byte vectors of T as floats
template <>
struct Loader<float> {
  static constexpr int kVec = 4;
  __device__ static void get(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  __device__ static float one(const float* p) { return *p; }
};
template <>
struct Loader<__half> {
  static constexpr int kVec = 8;
  __device__ static void get(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static float one(const __half* p) { return __half2float(*p); }
};
template <>
struct Loader<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static void get(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

// A part's result in the workspace: Stat, then (k > 0) k keys, descending;
// padded so that the next one is 16-byte aligned again.
struct Plan {
  int parts;      // per row
  int64_t vecs;   // 16-byte vectors of a part
};
__host__ __device__ inline int64_t part_bytes(int k) { return 16 + 16 * (int64_t)((k + 1) / 2); }

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobsArgs a, Plan plan) {
  using L = Loader<T>;
  constexpr int V = L::kVec, U = kPer / V;  // vectors of a thread per tile
  __shared__ uint64_t s_buf[kCap];
  __shared__ uint64_t s_best[kLogprobsMaxTop], s_red[kThreads / 32];
  __shared__ uint32_t s_thr[kThreads / 32];
  __shared__ Stat s_stat[kThreads / 32];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / plan.parts;
  const int part = (int)(blockIdx.x - row * plan.parts);
  const int k = a.k;
  if (tid == 0) s_n = 0;
  pdl_trigger();
  pdl_wait();
  if (a.ids) {
    const int id = a.ids[row];
    if (id < 0 || id >= a.vocab) return;  // padding, or refused (the join reports it)
  }
  // Vector v of the row covers the values [v*V - head, (v+1)*V - head): the
  // row's first address rounded down to 16 bytes is vector 0.
  const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
  const int head = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int64_t nvec = (a.vocab + head + V - 1) / V;
  const int64_t v0 = part * plan.vecs, v1 = min(nvec, v0 + plan.vecs);
  const T* base = x - head;

  float m = -INFINITY, s = 0.f, t = 0.f;
  float thr = -INFINITY;                  // values up to thr cannot be among the k largest
  bool have = false;                      // thr is set
  for (int64_t w0 = v0; w0 < v1; w0 += kThreads * U) {
    float f[kPer];
    // values outside the row: -inf for the sums, and never collected
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = w0 + u * kThreads + tid;
      const int64_t e0 = v * V - head;
      if (v < v1 && e0 >= 0 && e0 + V <= a.vocab) {
        L::get(__ldcs(reinterpret_cast<const uint4*>(base + v * V)), f + u * V);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          f[u * V + j] = (v < v1 && e0 + j >= 0 && e0 + j < a.vocab) ? L::one(x + e0 + j) : -INFINITY;
      }
    }
    float top = f[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) top = max_nan(top, f[i]);

    // running sums; one rescale per tile.  With nothing but -inf so far any
    // reference does, all terms are 0.
    const float mn = max_nan(m, top), z = mn == -INFINITY ? 0.f : mn;
    if (mn != m) {
      const float shift = m == -INFINITY ? 0.f : (m - mn) * kLog2e, c = ex2(shift);
      t = c == 0.f ? 0.f : c * fmaf(shift, s, t);
      s *= c;
      m = mn;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // 2^-200 is 0 in f32: the clamp changes no sum and keeps 0 * -inf out of t
      const float d = max_nan((f[i] - z) * kLog2e, -200.f);
      const float e = ex2(d);
      s += e;
      t = fmaf(e, d, t);
    }

    if (k > 0) {
      bool over = false;  // more than kCut pairs lie in the buffer
      auto collect = [&](bool strict) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (strict ? !(f[i] <= thr) : !(f[i] < thr)) {
            const int64_t id = (w0 + (i / V) * kThreads + tid) * V - head + i % V;
            if (id >= 0 && id < a.vocab && w0 + (i / V) * kThreads + tid < v1) {
              const int at = atomicAdd(&s_n, 1);
              s_buf[at] = make_key(f[i], (uint32_t)id);
              over |= at >= kCut;
            }
          }
        }
      };
      if (!have) {
        // the best k-th lane maximum of a warp (NaN ranks highest)
        const uint32_t sorted = warp_sort_desc(key32(top));
        const uint32_t kth = __shfl_sync(0xffffffffu, sorted, k - 1);
        if (lane == 0) s_thr[warp] = kth;
        __syncthreads();
        uint32_t best = s_thr[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) best = max(best, s_thr[i]);
        thr = key_value(best);
        have = true;
        if (!(top < thr)) collect(false);
      } else if (!(top <= thr)) {
        collect(true);
      }
      if (__syncthreads_or(over)) {
        cut_to_k(s_buf, s_n, k, s_best, s_red);
        thr = key_value((uint32_t)(s_buf[k - 1] >> 32));
        if (tid == 0) s_n = k;
        __syncthreads();
      }
    }
  }

  unsigned char* out = static_cast<unsigned char*>(a.ws) + (row * plan.parts + part) * part_bytes(k);
  if (k > 0) {
    __syncthreads();
    const int n = s_n;
    cut_to_k(s_buf, n, k, s_best, s_red);
    if (tid < k) reinterpret_cast<uint64_t*>(out + 16)[tid] = tid < n ? s_buf[tid] : 0;
  }
  Stat v = warp_join(Stat{m, s, t});
  if (lane == 0) s_stat[warp] = v;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v = join(v, s_stat[i]);
    *reinterpret_cast<float4*>(out) = make_float4(v.m, v.s, v.t, 0.f);
  }
}

// One CTA per row: the parts' sums, the k largest of the parts' lists, and the
// given token's log probability.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_join_kernel(const __grid_constant__ LogprobsArgs a, Plan plan) {
  __shared__ uint64_t s_red[kThreads / 32];
  __shared__ Stat s_stat[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int k = a.k;
  pdl_trigger();
  pdl_wait();
  int id = -1;
  if (a.ids) {
    id = a.ids[row];
    if (id >= a.vocab) {
      if (tid == 0) set_error(a.status, MINFER_ERR_TOKEN_OOB);
      return;
    }
    if (id < 0) return;
  }
  const unsigned char* in = static_cast<const unsigned char*>(a.ws) + row * plan.parts * part_bytes(k);
  Stat v{-INFINITY, 0.f, 0.f};
  for (int p = tid; p < plan.parts; p += kThreads) {
    const float4 q = *reinterpret_cast<const float4*>(in + p * part_bytes(k));
    v = join(v, Stat{q.x, q.y, q.z});
  }
  v = warp_join(v);
  if (lane == 0) s_stat[warp] = v;
  __syncthreads();
  v = s_stat[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) v = join(v, s_stat[i]);
  const bool none = v.m == -INFINITY;
  const float log2s = log2f(v.s);
  auto logp = [&](float x) { return none ? -INFINITY : (x - v.m) - kLn2 * log2s; };
  if (tid == 0) {
    if (a.ids) a.logprob[row] = logp(Loader<T>::one(static_cast<const T*>(a.x) + row * a.row_stride + id));
    if (a.entropy) a.entropy[row] = none ? 0.f : kLn2 * (log2s - v.t / v.s);
  }
  uint64_t last = ~0ull;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
    for (int p = tid; p < plan.parts; p += kThreads) {
      // the part's list is descending: its first key below the last one taken
      const uint64_t* list = reinterpret_cast<const uint64_t*>(in + p * part_bytes(k) + 16);
      for (int i = 0; i < k; ++i) {
        const uint64_t q = list[i];
        if (q < last) {
          best = q > best ? q : best;
          break;
        }
      }
    }
    last = block_max(best, s_red);
    if (tid == 0) {
      a.top_ids[row * k + j] = (int32_t)key_id(last);
      a.top_logprobs[row * k + j] = logp(key_value((uint32_t)(last >> 32)));
    }
  }
}

// Parts of a row: enough CTAs to fill the GPU several times over (the last
// wave's idle share shrinks with their number), none below one vector per
// thread.  vecs is the same for every row; a row's vectors vary by one with
// its alignment.
Plan plan_of(int64_t rows, int64_t vocab, int64_t vec, int num_sms) {
  const int64_t nvec = (vocab + vec - 1) / vec + 1;
  const int64_t want = std::max<int64_t>(1, ((int64_t)num_sms * 32 + rows - 1) / rows);
  Plan p;
  int64_t parts = std::min<int64_t>(want, (nvec + kThreads - 1) / kThreads);
  p.vecs = (nvec + parts - 1) / parts;
  p.parts = (int)((nvec + p.vecs - 1) / p.vecs);
  return p;
}

template <typename T>
cudaError_t launch(const LogprobsArgs& a, int num_sms, cudaStream_t st) {
  const Plan plan = plan_of(a.rows, a.vocab, Loader<T>::kVec, num_sms);
  cudaError_t e = launch_pdl(logprobs_kernel<T>, dim3((unsigned)(a.rows * plan.parts)), dim3(kThreads), 0, st, a, plan);
  if (e != cudaSuccess) return e;
  return launch_pdl(logprobs_join_kernel<T>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, plan);
}

}  // namespace

int64_t logprobs_workspace(int64_t rows, int64_t vocab, int k, int num_sms) {
  // the size does not depend on the logits' type: enough for vectors of 4 and of 8 values
  return rows * std::max(plan_of(rows, vocab, 4, num_sms).parts, plan_of(rows, vocab, 8, num_sms).parts) * part_bytes(k);
}

cudaError_t logprobs_launch(const LogprobsArgs& a, int type, int num_sms, cudaStream_t stream) {
  if (type == MINFER_F32) return launch<float>(a, num_sms, stream);
  if (type == MINFER_F16) return launch<__half>(a, num_sms, stream);
  return launch<__nv_bfloat16>(a, num_sms, stream);
}

}  // namespace minfer
