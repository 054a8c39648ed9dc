// paged_attn.cuh -- what the kernels of attention over paged K/V caches share: the
// walk over a ragged batch in equal shares, the partials that shares leave in the
// workspace and how they are joined, and the warp-level instructions.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kGroup = 16;              // neighbouring shares whose partials are joined first
constexpr int kMaxJoin = 64;            // partials of one join: kDirect, kGroup, or the number of groups
// Partials that are joined in one step (20 of them: 8.3 us a call, in two steps
// 9.8; 32 of them: 10.2 either way).
constexpr int kDirect = 32;

// What the threads of a CTA share while they join partials.
template <int R>
struct JoinShared {
  float* part[kMaxJoin];  // the partials, in the order of their shares
  float w[kMaxJoin][R];   // their weights
  float2 out[R];          // the joined (max, sum)
};

// The workspace: counters (zero between calls; one per share for a piece that
// starts in it, one per group for a piece that started before it, one per share
// for the groups of a piece), then per share two partials, slot 1 for the piece
// that starts in the share and slot 0 for the one that started before it: R
// (max, sum) pairs and R x HD.
constexpr int kMaxShares = kGroup * (kMaxJoin - 1);
constexpr int64_t kPartOffset = ((2 * kMaxShares + kMaxShares / kGroup + 1) * 4 + 255) / 256 * 256;  // the same for every call
__host__ __device__ constexpr int64_t part_floats(int rows, int hd) { return (int64_t)rows * (hd + 2); }

// Units of a request; a length out of range counts as none.
template <int kUnit>
__device__ __forceinline__ int units_of(int len, int cap) {
  return (len < 0 || len > cap) ? 0 : (int)(((unsigned)len + kUnit - 1) / kUnit);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The same for data that is read once: first to leave L2, where the page tables,
// the partials and the code of the join stay.
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp16_stream(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// the 8 x 8 matrix of 16-bit values whose row lane / 4, columns 2 (lane % 4) and
// the next a register holds, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void store_as(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Walks the units of the batch: request r, head block v (KV head and group of
// R query heads), unit u of it.  The next request's length is read one
// request ahead.
struct Walk {
  int r, v, u, units, len, next_len;
};
__device__ __forceinline__ int len_at(const PagedAttnRows& a, int r) { return r < a.n_req ? a.len[r] : 0; }
template <int kUnit>
__device__ __forceinline__ void walk_next(Walk& w, const PagedAttnRows& a, int nv, int cap) {
  if (++w.u < w.units) return;
  w.u = 0;
  if (++w.v < nv) return;
  w.v = 0;
  do {
    ++w.r;
    w.len = w.next_len;
    w.next_len = len_at(a, w.r + 1);
    w.units = units_of<kUnit>(w.len, cap);
  } while (w.units == 0 && w.r < a.n_req);
}

// How the units are cut into shares: as many as there are CTAs, none of them
// empty; the first `more` of them hold one unit more than the others.  (At least
// two units a share made a single request of 64 rows slower, 6.3 us against 4.2,
// for its two KV heads then share a CTA.)
struct Shares {
  int64_t total, each;
  int n, more;
  __device__ __forceinline__ Shares(int64_t units, int n_ctas) {
    total = units;
    n = (int)max((int64_t)1, min(units, (int64_t)n_ctas));
    // (64-bit divisions are long; few batches need one)
    each = total >> 32 ? total / n : (int64_t)((uint32_t)total / (uint32_t)n);
    more = (int)(total - each * n);
  }
  __device__ __forceinline__ int64_t begin(int c) const { return each * c + min(c, more); }
  // the share that holds unit x
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t low = (each + 1) * more, y = x < low ? x : x - low, d = x < low ? each + 1 : each;
    return (x < low ? 0 : more) + (int)(y >> 32 ? y / d : (int64_t)((uint32_t)y / (uint32_t)d));
  }
};

// Joins `count` partials.  Their outputs are copied to shared memory (ring, all
// of them at once or as many as fit) while the weights are worked out, a warp
// per row and a lane per partial; then every thread adds up four dims of a row
// at a time.  final: the result, over `scale` (weight_scale), goes to o and lse, else it replaces the first
// partial.  A sum below 0 marks a piece that met a bad page; it spoils the
// whole.  All threads; s.part is written before a barrier of the caller's.
template <typename T, int HD, int R, int kWarps>
__device__ void join_parts(JoinShared<R>& s, unsigned char* ring, int ring_bytes, int count, int rows, bool final, float scale, T* o, float* lse) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kItems = (R * HD / 4 + kWarps * 32 - 1) / (kWarps * 32);  // of a thread
  const int items = rows * HD / 4, fit = min(count, ring_bytes / (items * 16));
  auto copy = [&](int p0) {
    const int n = min(fit, count - p0);
    uint32_t dst = smem_u32(ring) + tid * 16;
#pragma unroll 4
    for (int p = 0; p < n; ++p, dst += items * 16) {
      const float4* src = reinterpret_cast<const float4*>(s.part[p0 + p] + 2 * R) + tid;
#pragma unroll
      for (int k = 0; k < kItems; ++k)
        if (tid + k * kWarps * 32 < items) cp16(dst + k * kWarps * 512, src + k * kWarps * 32, 16);
    }
    cp_commit();
  };
  // lane (j, partial) of warp w has the (max, sum) of row w + kWarps i: all loads first
  constexpr int kSeries = kMaxJoin / 32, kOwn = R / kWarps;
  float2 ml[kOwn][kSeries];
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll
    for (int j = 0; j < kSeries; ++j) {
      const int row = warp + i * kWarps, p = lane + 32 * j;
      ml[i][j] = make_float2(-INFINITY, 0.f);
      if (p < count && row < rows) ml[i][j] = __ldcg(reinterpret_cast<const float2*>(s.part[p]) + row);
    }
  copy(0);
  bool bad_row = false;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int row = warp + i * kWarps;
    float m = ml[i][0].x;
#pragma unroll
    for (int j = 1; j < kSeries; ++j) m = fmaxf(m, ml[i][j].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float z = m == -INFINITY ? 0.f : m;
    float l = 0.f;
#pragma unroll
    for (int j = 0; j < kSeries; ++j) {
      const float c = ex2(ml[i][j].x - z);
      if (lane + 32 * j < count) s.w[lane + 32 * j][row] = c;
      bad_row |= ml[i][j].y < 0.f;
      l = fmaf(ml[i][j].y, c, l);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (lane == 0) s.out[row] = make_float2(m, l);
  }
  const bool bad = __syncthreads_or(bad_row);
  float4 acc[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < count; p0 += fit) {
    cp_wait<0>();
    __syncthreads();  // the copies of all threads; the weights
    const int n = min(fit, count - p0);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = tid + k * kWarps * 32;
      if (i >= items) break;
      const float4* x = reinterpret_cast<const float4*>(ring) + i;
      const int row = i / (HD / 4);
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float4 v = x[p * items];
        const float c = s.w[p0 + p][row];
        acc[k].x = fmaf(v.x, c, acc[k].x);
        acc[k].y = fmaf(v.y, c, acc[k].y);
        acc[k].z = fmaf(v.z, c, acc[k].z);
        acc[k].w = fmaf(v.w, c, acc[k].w);
      }
    }
    if (p0 + fit < count) {
      __syncthreads();
      copy(p0 + fit);
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int i = tid + k * kWarps * 32;
    if (i >= items) break;
    if (!final) {
      reinterpret_cast<float4*>(s.part[0] + 2 * R)[i] = acc[k];
    } else if (!bad) {
      const float l = s.out[i / (HD / 4)].y, f = l == 0.f ? 0.f : 1.f / (l * scale);
      T* dst = o + i * 4;
      store_as(dst, acc[k].x * f);
      store_as(dst + 1, acc[k].y * f);
      store_as(dst + 2, acc[k].z * f);
      store_as(dst + 3, acc[k].w * f);
    }
  }
  if (tid < rows) {
    const float2 ml = s.out[tid];
    if (!final)
      reinterpret_cast<float2*>(s.part[0])[tid] = make_float2(ml.x, bad ? -1.f : ml.y);
    else if (!bad && lse)
      lse[tid] = fmaf(ml.x, kLn2, logf(ml.y));
  }
}

// Counts this CTA's arrival: its writes before the last barrier are released, and
// what the CTAs released that came before is acquired.
__device__ __forceinline__ unsigned arrive(unsigned* counter) {
  unsigned before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

// A piece of a (request, head block) that other shares hold pieces of too.
struct Piece {
  int r, head0, rows, c0, c1;  // c0..c1: the shares that hold one
  float scale;                 // weight_scale of the request
};


// This CTA's share of the batch's units: thread t counts the units of `per`
// neighbouring requests; a scan gives the total and the request of the share's
// first unit, which goes to s_walk (behind a barrier).  count 0: it has none.
template <int kWarps, int kUnit>
__device__ __forceinline__ Shares find_share(const PagedAttnRows& a, int nv, int cap, int64_t (&s_scan)[kWarps], Walk& s_walk, int64_t* first, int* count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_req + kWarps * 32 - 1) / (kWarps * 32), r_lo = min(tid * per, a.n_req), r_hi = min(r_lo + per, a.n_req);
  int64_t mine = 0;
#pragma unroll 4
  for (int r = r_lo; r < r_hi; ++r) mine += units_of<kUnit>(a.len[r], cap);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += s_scan[i];
    total += s_scan[i];
  }
  total *= nv;
  const Shares shares(total, gridDim.x);
  *count = 0;
  if (total == 0 || (int)blockIdx.x >= shares.n) return shares;
  const int64_t begin = shares.begin(blockIdx.x);
  *first = begin;
  *count = (int)(shares.begin(blockIdx.x + 1) - begin);
  if (begin >= before * nv && begin < (before + mine) * nv) {
    int64_t at = before * nv;
    for (int r = r_lo; r < r_hi; ++r) {
      const int len = a.len[r], units = units_of<kUnit>(len, cap);
      if (begin < at + (int64_t)units * nv) {
        s_walk.r = r;
        s_walk.v = (int)((begin - at) / units);
        s_walk.u = (int)(begin - at - (int64_t)s_walk.v * units);
        s_walk.units = units;
        s_walk.len = len;
        s_walk.next_len = len_at(a, r + 1);
        break;
      }
      at += (int64_t)units * nv;
    }
  }
  __syncthreads();
  return shares;
}

// Rows of requests without units: zeros for a length of 0, an error for one out of range.
template <typename T, int HD, int kThreads>
__device__ __forceinline__ void idle_requests(const PagedAttnRows& a, int cap) {
  const int tid = threadIdx.x;
  for (int r = blockIdx.x; r < a.n_req; r += gridDim.x) {
    const int len = a.len[r];
    if (len == 0) {
      for (int i = tid; i < a.nh * HD; i += kThreads) store_as(static_cast<T*>(a.o) + (int64_t)r * a.o_stride + i, 0.f);
      if (a.lse)
        for (int i = tid; i < a.nh; i += kThreads) a.lse[(int64_t)r * a.nh + i] = -INFINITY;
    } else if ((len < 0 || len > cap) && tid == 0) {
      set_error(a.status, MINFER_ERR_POS_OOB);
    }
  }
}

// Reports a share's partials (complete since the last barrier) and joins what is
// complete with them.  Thread 32 i takes piece i.
template <typename T, int HD, int R, int kWarps>
__device__ __forceinline__ void report_pieces(const PagedAttnRows& a, const Piece (&piece)[2], int (&s_last)[2], int (&s_flag)[2], JoinShared<R>& s_join,
                                              unsigned char* ring, int ring_bytes) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned* counters = static_cast<unsigned*>(a.ws);
  float* ws_part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + kPartOffset);
  const int g = blockIdx.x / kGroup;
  if (lane == 0 && warp < 2) {
    const Piece& p = piece[warp];
    bool last = false;
    if (p.rows) {
      const int all = p.c1 - p.c0 + 1;
      const int lo = max(p.c0, g * kGroup), hi = min(p.c1, g * kGroup + kGroup - 1);
      const int n = all <= kDirect ? all : hi - lo + 1;
      unsigned* counter = counters + (all <= kDirect || p.c0 >= g * kGroup ? p.c0 : kMaxShares + g);
      last = n == 1 || arrive(counter) == (unsigned)n - 1;
      if (last && n > 1) *counter = 0;
    }
    s_last[warp] = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!s_last[i]) continue;
    const Piece p = i ? piece[1] : piece[0];
    T* o_row = static_cast<T*>(a.o) + (int64_t)p.r * a.o_stride + (int64_t)p.head0 * HD;
    float* lse_row = a.lse ? a.lse + (int64_t)p.r * a.nh + p.head0 : nullptr;
    auto slot = [&](int c) { return ws_part + (int64_t)(c * 2 + (c == p.c0 ? 1 : 0)) * part_floats(R, HD); };
    const bool direct = p.c1 - p.c0 + 1 <= kDirect;
    const int lo = direct ? p.c0 : max(p.c0, g * kGroup), hi = direct ? p.c1 : min(p.c1, g * kGroup + kGroup - 1);
    if (hi > lo) {
      if (tid <= hi - lo) s_join.part[tid] = slot(lo + tid);
      __syncthreads();
      join_parts<T, HD, R, kWarps>(s_join, ring, ring_bytes, hi - lo + 1, p.rows, direct, p.scale, o_row, lse_row);
      __syncthreads();
    }
    if (!direct) {
      const int g0 = p.c0 / kGroup, g1 = p.c1 / kGroup;
      if (tid == 0) {
        unsigned* counter = counters + kMaxShares + kMaxShares / kGroup + 1 + p.c0;
        s_flag[0] = arrive(counter) == (unsigned)(g1 - g0);
        if (s_flag[0]) *counter = 0;
      }
      if (tid <= g1 - g0) s_join.part[tid] = slot(max(p.c0, (g0 + tid) * kGroup));
      __syncthreads();
      if (s_flag[0]) join_parts<T, HD, R, kWarps>(s_join, ring, ring_bytes, g1 - g0 + 1, p.rows, true, p.scale, o_row, lse_row);
      __syncthreads();
    }
  }
}

}  // namespace
}  // namespace minfer
