// k_paged_attn.cu -- attention of one new token per request over a paged K/V
// cache, split over the requests' lengths and joined.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  j < len
//
// Work is counted in units of 64 keys of one (request, KV head); the units of
// the whole batch, request by request, are cut into equal shares, one per CTA
// of a grid that fills the GPU once, so ragged batches and single long
// requests load every SM alike, without the host knowing a length.  A CTA
// walks its share as a stream: a (request, KV head) that lies inside it is
// finished there; one that crosses a share's border leaves a partial (max,
// sum, unnormalized output) in the workspace.  The CTA that finishes last among
// the shares of a (request, KV head) joins the partials; where there are more
// than kDirect of them, in a tree of two levels: first the last one of each
// group of neighbouring shares, then the last one of the groups.  Who is last
// decides only who adds, never in what order, so the result does not depend on
// it.  A CTA reports its (at most two) partials after its last unit, so that no
// unit waits for a fence.
//
// Inside a CTA each of four warps takes 16 of a unit's 64 keys, copies their
// K and V rows into its own ring in shared memory (cp.async of 16 bytes, page
// by page; rows behind the request's last are filled with zeros) and runs an
// online softmax of its own: no barrier before the end of the (request, KV
// head).  The products are m16n8 MMAs with the query heads of the KV head as
// the 16 rows.  One query token leaves the rows of a tcgen05 tile (128)
// mostly empty and the bound is the bytes of K and V, so the accumulators stay
// in registers, where the softmax needs them.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;               // keys of a unit that one warp takes
constexpr int kUnit = kWarps * kKeys;   // keys of a unit
constexpr int kRows = 16;               // query heads of one MMA tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kGroup = 16;              // neighbouring shares whose partials are joined first
constexpr int kMaxJoin = 64;            // partials of one join: kDirect, kGroup, or the number of groups
constexpr int kDirect = 32;             // partials that are joined in one step

// R: query heads that a CTA carries through the join (8 where a KV head has no
// more, which leaves room for another stage of the ring).
template <typename T, int HD, int R>
struct Cfg {
  static constexpr int kRowBytes = HD * (int)sizeof(T);
  static constexpr int kChunks = kRowBytes / 16;  // 16-byte chunks of a row
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // K and V rows of one warp
  static constexpr int kQBytes = sizeof(T) == 4 ? 2 * kRows * kRowBytes : 0;  // tf32 hi and lo of Q
  // two CTAs per SM, or one where two stages of the ring do not fit twice; the
  // ring takes what is left of the SM's shared memory
  static constexpr int kCtas = kRowBytes == 512 ? 1 : 2;
  static constexpr int kBudget = kCtas == 1 ? 222000 : R == 8 ? 109400 : 105000;
  static constexpr int kFit = (kBudget - kQBytes) / (kWarps * kStageBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kWarps * kStages * kStageBytes + kQBytes;
  static_assert(kStages >= 2, "a ring has two stages at least");
  static_assert(R * HD * 4 <= kStageBytes, "a warp's output fits the stage it has just used");
};

// The workspace: counters (zero between calls; one per share for a piece that
// starts in it, one per group for a piece that started before it, one per share
// for the groups of a piece), then per share two partials, slot 1 for the piece
// that starts in the share and slot 0 for the one that started before it: kRows
// (max, sum) pairs and kRows x HD.
constexpr int kMaxShares = kGroup * (kMaxJoin - 1);
constexpr int64_t kPartOffset = ((2 * kMaxShares + kMaxShares / kGroup + 1) * 4 + 255) / 256 * 256;  // the same for every call
__host__ __device__ inline int64_t ws_part_floats(int hd) { return (int64_t)kRows * (hd + 2); }

// Units of a request; a length out of range counts as none.
__device__ __forceinline__ int units_of(int len, int cap) {
  return (len < 0 || len > cap) ? 0 : (len + kUnit - 1) / kUnit;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
// x = hi + lo, two tf32 values (11 significant bits each; the rest is below 2^-22 |x|)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t* hi, uint32_t* lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*hi) : "f"(__uint_as_float(x)));
  const float rest = __uint_as_float(x) - __uint_as_float(*hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*lo) : "f"(rest));
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store_as(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Walks the units of the batch: request r, head block v (KV head and group of
// kRows query heads), unit u of it.  The next request's length is read one
// request ahead.
struct Walk {
  int r, v, u, units, len, next_len;
};
__device__ __forceinline__ int len_at(const PagedAttnArgs& a, int r) { return r < a.n_req ? a.len[r] : 0; }
__device__ __forceinline__ void walk_next(Walk& w, const PagedAttnArgs& a, int nv, int cap) {
  if (++w.u < w.units) return;
  w.u = 0;
  if (++w.v < nv) return;
  w.v = 0;
  do {
    ++w.r;
    w.len = w.next_len;
    w.next_len = len_at(a, w.r + 1);
    w.units = units_of(w.len, cap);
  } while (w.units == 0 && w.r < a.n_req);
}

// The units are cut into as many shares as there are CTAs, but no empty ones;
// share c begins at share_begin(c).
__device__ __forceinline__ int share_count(int64_t total, int n_ctas) { return (int)min(total, (int64_t)n_ctas); }
__device__ __forceinline__ int64_t share_begin(int64_t total, int c, int n) { return total * c / n; }

// The share that holds unit x: the largest c with share_begin(c) <= x.
__device__ __forceinline__ int share_of(int64_t x, int64_t total, int n) {
  int c = (int)min((x * n) / total, (int64_t)n - 1);
  while (c + 1 < n && share_begin(total, c + 1, n) <= x) ++c;
  while (share_begin(total, c, n) > x) --c;
  return c;
}

// What the threads of a CTA share while they join partials.
template <int R>
struct JoinShared {
  float* part[kMaxJoin];    // the partials, in the order of their shares
  float2 ml[kMaxJoin][R];   // their (max, sum); then .x the weight
  float2 out[R];            // the joined (max, sum)
  int bad;
};

// Joins `count` partials: weights first, then every thread four dims of a row at
// a time.  final: the result goes to o and lse, else it replaces the first
// partial.  A sum below 0 marks a piece that met a bad page; it spoils the
// whole.  All threads; s.part is written before a barrier of the caller's.
template <typename T, int HD, int R>
__device__ void join_parts(JoinShared<R>& s, int count, int rows, bool final, T* o, float* lse) {
  const int tid = threadIdx.x;
  for (int i = tid; i < count * R; i += kWarps * 32)
    if (i % R < rows) s.ml[i / R][i % R] = __ldcg(reinterpret_cast<const float2*>(s.part[i / R]) + i % R);
  if (tid == 0) s.bad = 0;
  __syncthreads();
  if (tid < rows) {
    float m = -INFINITY;
    for (int i = 0; i < count; ++i) m = fmaxf(m, s.ml[i][tid].x);
    const float z = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    bool bad = false;
    for (int i = 0; i < count; ++i) {
      const float2 ml = s.ml[i][tid];
      const float c = ex2(ml.x - z);
      bad |= ml.y < 0.f;
      l = fmaf(ml.y, c, l);
      s.ml[i][tid].x = c;
    }
    s.out[tid] = make_float2(m, l);
    if (bad) s.bad = 1;
  }
  __syncthreads();
  const bool bad = s.bad != 0;
  for (int i = tid; i < rows * HD / 4; i += kWarps * 32) {
    const int row = i / (HD / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < count; ++p) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(s.part[p] + 2 * kRows) + i);
      const float c = s.ml[p][row].x;
      acc.x = fmaf(x.x, c, acc.x);
      acc.y = fmaf(x.y, c, acc.y);
      acc.z = fmaf(x.z, c, acc.z);
      acc.w = fmaf(x.w, c, acc.w);
    }
    if (!final) {
      reinterpret_cast<float4*>(s.part[0] + 2 * kRows)[i] = acc;  // read by this thread alone
    } else if (!bad) {
      const float l = s.out[row].y, f = l == 0.f ? 0.f : 1.f / l;
      T* dst = o + i * 4;
      store_as(dst, acc.x * f);
      store_as(dst + 1, acc.y * f);
      store_as(dst + 2, acc.z * f);
      store_as(dst + 3, acc.w * f);
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

// A piece of a (request, head block) that other shares hold pieces of too.
struct Piece {
  int r, head0, rows, c0, c1;  // c0..c1: the shares that hold one
};

template <typename T, int HD, int R>
__global__ void __launch_bounds__(kWarps * 32, Cfg<T, HD, R>::kCtas)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, int n_groups, float scale_log2) {
  using C = Cfg<T, HD, R>;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kSteps = C::kChunks / 2;  // MMA steps over the head's dims (two chunks each)
  constexpr int kTiles = HD / 8;          // n8 tiles of the output
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ Walk s_walk;
  __shared__ uint8_t s_bad[kWarps][C::kStages];
  __shared__ int s_segbad[2], s_last[2];
  __shared__ JoinShared<R> s_join;
  __shared__ float2 m_ml[kWarps * R];  // the warps' (max, sum) at the end of a piece
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = a.c.page_size, cap = a.max_pages * P;
  const int G = a.nh / a.c.nkv, nv = a.c.nkv * n_groups;
  unsigned* counters = static_cast<unsigned*>(a.ws);
  float* ws_part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + kPartOffset);

  pdl_trigger();
  pdl_wait();

  // ---- this CTA's share: thread t counts the units of `per` neighbouring
  // requests; a scan gives the total and the request of the share's first unit
  if (tid < 2) s_segbad[tid] = 0;
  const int per = (a.n_req + kWarps * 32 - 1) / (kWarps * 32), r_lo = min(tid * per, a.n_req), r_hi = min(r_lo + per, a.n_req);
  int64_t mine = 0;
#pragma unroll 4
  for (int r = r_lo; r < r_hi; ++r) mine += units_of(a.len[r], cap);
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
  // rows of requests without units: zeros for a length of 0, an error for one out of range
  auto idle_requests = [&] {
    for (int r = blockIdx.x; r < a.n_req; r += gridDim.x) {
      const int len = a.len[r];
      if (len == 0) {
        for (int i = tid; i < a.nh * HD; i += kWarps * 32) store_as(static_cast<T*>(a.o) + (int64_t)r * a.o_stride + i, 0.f);
        if (a.lse)
          for (int i = tid; i < a.nh; i += kWarps * 32) a.lse[(int64_t)r * a.nh + i] = -INFINITY;
      } else if ((len < 0 || len > cap) && tid == 0) {
        set_error(a.status, MINFER_ERR_POS_OOB);
      }
    }
  };
  const int n_shares = share_count(total, gridDim.x);
  if ((int)blockIdx.x >= n_shares) {
    idle_requests();
    return;
  }
  const int64_t begin = share_begin(total, blockIdx.x, n_shares);
  const int count = (int)(share_begin(total, blockIdx.x + 1, n_shares) - begin);
  if (begin >= before * nv && begin < (before + mine) * nv) {
    int64_t at = before * nv;
    for (int r = r_lo; r < r_hi; ++r) {
      const int len = a.len[r], units = units_of(len, cap);
      if (begin < at + (int64_t)units * nv) {
        const int off = (int)(begin - at);
        s_walk.r = r;
        s_walk.v = off / units;
        s_walk.u = off - s_walk.v * units;
        s_walk.units = units;
        s_walk.len = len;
        s_walk.next_len = len_at(a, r + 1);
        break;
      }
      at += (int64_t)units * nv;
    }
  }
  __syncthreads();
  Walk cw = s_walk;  // the unit being computed
  Walk lw = cw;      // the unit being loaded

  // ---- loads: lane l < 16 looks up the page of key l, all lanes copy
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  const bool pow2 = (P & (P - 1)) == 0;
  const int shift = __ffs(P) - 1;
  int page_next = 0;  // page id of this lane's key of unit lw
  auto lookup = [&](const Walk& w) {
    const int key = w.u * kUnit + warp * kKeys + (lane & 15);
    if (key >= w.len) return 0;
    const int i = pow2 ? key >> shift : key / P;
    return a.table[(int64_t)w.r * a.table_stride + i];
  };
  page_next = lookup(lw);
  auto load_unit = [&](int stage) {
    const int key0 = lw.u * kUnit + warp * kKeys;
    const int key = key0 + (lane & 15);
    const int in_page = pow2 ? key & (P - 1) : key % P;
    const bool ok = (unsigned)page_next < (unsigned)a.c.n_pages;
    const bool bad = key < lw.len && !ok;
    int64_t off = 0;
    if (key < lw.len && ok)
      off = (int64_t)page_next * a.c.page_stride + (int64_t)in_page * a.c.row_stride +
            (int64_t)(lw.v / n_groups) * a.c.head_stride;
    const unsigned live = __ballot_sync(0xffffffffu, key < lw.len && ok);
    const bool any_bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) s_bad[warp][stage] = any_bad;
    // per instruction: 32 chunks = 32 / kChunks rows
    constexpr int kRowsPer = 32 / C::kChunks > 0 ? 32 / C::kChunks : 1;
    const int c = lane % C::kChunks;
    const uint32_t kdst = ring + stage * C::kStageBytes, vdst = kdst + kKeys * C::kRowBytes;
#pragma unroll
    for (int j = 0; j < kKeys / kRowsPer; ++j) {
      const int row = j * kRowsPer + lane / C::kChunks;
      const int64_t o = __shfl_sync(0xffffffffu, off, row) * (int64_t)sizeof(T) + c * 16;
      const int bytes = (live >> row) & 1 ? 16 : 0;
      const uint32_t d = (uint32_t)(row * C::kRowBytes + ((c ^ (row & 7)) << 4));
      cp16(kdst + d, static_cast<const unsigned char*>(a.c.k) + o, bytes);
      cp16(vdst + d, static_cast<const unsigned char*>(a.c.v) + o, bytes);
    }
    walk_next(lw, a, nv, cap);
  };

  int issued = 0;
#pragma unroll 1
  for (; issued < C::kStages - 1; ++issued) {
    if (issued < count) {
      load_unit(issued);
      if (issued + 1 < count) page_next = lookup(lw);
    }
    cp_commit();
  }

  // ---- one (request, head block) after another
  unsigned char* qs = smem + kWarps * C::kStages * C::kStageBytes;
  Piece piece[2];  // [1]: the one that starts in this share, [0]: the one that started before
  piece[0].rows = piece[1].rows = 0;
  const int g4 = lane >> 2, t4 = lane & 3;
  int stage = 0, seg = 0;
  for (int done = 0; done < count;) {
    const int r = cw.r, kvh = cw.v / n_groups, grp = cw.v % n_groups;
    const int rows = min(kRows, G - grp * kRows);
    const int head0 = kvh * G + grp * kRows;
    const bool from_start = cw.u == 0;
    const int seg_units = min(cw.units - cw.u, count - done);
    const bool to_end = cw.u + seg_units == cw.units;
    const int seg_len = cw.len;
    const T* qrow = static_cast<const T*>(a.q) + (int64_t)r * a.q_stride + (int64_t)head0 * HD;

    // Q as the A operand: 16-bit types in registers, f32 as tf32 hi/lo in shared memory
    uint32_t qa[kF32 ? 1 : kSteps][4];
    if constexpr (!kF32) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d = s * 16 + t4 * 2;
        const uint32_t* lo = reinterpret_cast<const uint32_t*>(qrow + (int64_t)g4 * HD + d);
        const uint32_t* hi = reinterpret_cast<const uint32_t*>(qrow + (int64_t)(g4 + 8) * HD + d);
        qa[s][0] = g4 < rows ? lo[0] : 0u;
        qa[s][2] = g4 < rows ? lo[4] : 0u;
        qa[s][1] = g4 + 8 < rows ? hi[0] : 0u;
        qa[s][3] = g4 + 8 < rows ? hi[4] : 0u;
      }
    } else {
      // the barrier at the end of the previous segment freed qs
      for (int i = tid; i < kRows * HD; i += kWarps * 32) {
        const int row = i / HD, d = i % HD;
        uint32_t hi = 0, lo = 0;
        if (row < rows) split_tf32(__float_as_uint(reinterpret_cast<const float*>(qrow)[i]), &hi, &lo);
        const uint32_t at = (uint32_t)(row * C::kRowBytes + (((d >> 2) ^ (row & 7)) << 4) + (d & 3) * 4);
        *reinterpret_cast<uint32_t*>(qs + at) = hi;
        *reinterpret_cast<uint32_t*>(qs + kRows * C::kRowBytes + at) = lo;
      }
      __syncthreads();
    }

    float o[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g4, g4 + 8
    bool bad = false;

#pragma unroll 1
    for (int i = 0; i < seg_units; ++i, ++done) {
      // refill the stage that the previous unit freed, then wait for this one
      __syncwarp();
      if (issued < count) {
        int st = stage + C::kStages - 1;
        if (st >= C::kStages) st -= C::kStages;
        load_unit(st);
        ++issued;
        if (issued < count) page_next = lookup(lw);
      }
      cp_commit();
      cp_wait<C::kStages - 1>();
      __syncwarp();
      bad |= s_bad[warp][stage] != 0;
      const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + kKeys * C::kRowBytes;

      // S = Q K^T: two n8 tiles of keys
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
        const uint32_t kaddr = ks + key * C::kRowBytes;
        if constexpr (!kF32) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            uint32_t b[4];
            ldsm4(b, kaddr + (((s * 2 + half) ^ (key & 7)) << 4));
            mma(s0, qa[s], b[0], b[1], T());
            mma(s1, qa[s], b[2], b[3], T());
          }
        } else {
          // three tf32 products of the hi/lo halves; the small ones in sums of
          // their own, so the large sum takes kSteps tensor-core adds
          float e0[4] = {0.f, 0.f, 0.f, 0.f}, e1[4] = {0.f, 0.f, 0.f, 0.f};
          const int qr = lane & 15, qh = lane >> 4;
          const uint32_t qaddr = smem_u32(qs) + qr * C::kRowBytes;
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            uint32_t b[4], bh[4], bl[4], ah[4], al[4];
            ldsm4(b, kaddr + (((s * 2 + half) ^ (key & 7)) << 4));
            const uint32_t qo = qaddr + (((s * 2 + qh) ^ (qr & 7)) << 4);
            ldsm4(ah, qo);
            ldsm4(al, qo + kRows * C::kRowBytes);
#pragma unroll
            for (int j = 0; j < 4; ++j) split_tf32(b[j], &bh[j], &bl[j]);
            mma(s0, ah, bh[0], bh[1], T());
            mma(s1, ah, bh[2], bh[3], T());
            mma(e0, ah, bl[0], bl[1], T());
            mma(e1, ah, bl[2], bl[3], T());
            mma(e0, al, bh[0], bh[1], T());
            mma(e1, al, bh[2], bh[3], T());
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s0[j] += e0[j];
            s1[j] += e1[j];
          }
        }
      }

      // online softmax in log2 units
      const int live = seg_len - ((cw.u + i) * kUnit + warp * kKeys);  // keys of this warp's 16
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = t4 * 2 + (j & 1);
        s0[j] = k < live ? s0[j] * scale_log2 : -INFINITY;
        s1[j] = k + 8 < live ? s1[j] * scale_log2 : -INFINITY;
      }
      float n0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
      float n1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 1));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 1));
      n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2)));
      n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2)));
      // nothing seen so far: any finite reference gives p = 0
      const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
      const float c0 = ex2(m0 - z0), c1 = ex2(m1 - z1);
      m0 = n0;
      m1 = n1;
      s0[0] = ex2(s0[0] - z0);
      s0[1] = ex2(s0[1] - z0);
      s1[0] = ex2(s1[0] - z0);
      s1[1] = ex2(s1[1] - z0);
      s0[2] = ex2(s0[2] - z1);
      s0[3] = ex2(s0[3] - z1);
      s1[2] = ex2(s1[2] - z1);
      s1[3] = ex2(s1[3] - z1);
      // the row sums stay per thread until the end of the segment
      l0 = fmaf(l0, c0, (s0[0] + s0[1]) + (s1[0] + s1[1]));
      l1 = fmaf(l1, c1, (s0[2] + s0[3]) + (s1[2] + s1[3]));

      // O = O * c + P V: every unit's product in a fresh accumulator, added in f32
      if constexpr (!kF32) {
        const uint32_t p[4] = {pack2(s0[0], s0[1], T()), pack2(s0[2], s0[3], T()), pack2(s1[0], s1[1], T()),
                               pack2(s1[2], s1[3], T())};
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
        const uint32_t vaddr = vs + key * C::kRowBytes;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          uint32_t b[4];
          ldsm4t(b, vaddr + (((d * 2 + half) ^ (key & 7)) << 4));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            mma(f, p, b[2 * j], b[2 * j + 1], T());
            float* q = o[2 * d + j];
            q[0] = fmaf(q[0], c0, f[0]);
            q[1] = fmaf(q[1], c0, f[1]);
            q[2] = fmaf(q[2], c1, f[2]);
            q[3] = fmaf(q[3], c1, f[3]);
          }
        }
      } else {
        // the MMA's k index t stands for key 2t, t + 4 for key 2t + 1 of a tile
        // of 8: S's accumulator layout is then P's operand layout
        uint32_t ph[2][4], pl[2][4];
        const float* st[2] = {s0, s1};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          split_tf32(__float_as_uint(st[k][0]), &ph[k][0], &pl[k][0]);
          split_tf32(__float_as_uint(st[k][2]), &ph[k][1], &pl[k][1]);
          split_tf32(__float_as_uint(st[k][1]), &ph[k][2], &pl[k][2]);
          split_tf32(__float_as_uint(st[k][3]), &ph[k][3], &pl[k][3]);
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float f[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = k * 8 + t4 * 2 + j;
              const uint32_t v = lds32(vs + key * C::kRowBytes + (((n * 2 + (g4 >> 2)) ^ (key & 7)) << 4) + (g4 & 3) * 4);
              split_tf32(v, &bh[j], &bl[j]);
            }
            mma(f, ph[k], bh[0], bh[1], T());
            mma(e, ph[k], bl[0], bl[1], T());
            mma(e, pl[k], bh[0], bh[1], T());
          }
          o[n][0] = fmaf(o[n][0], c0, f[0] + e[0]);
          o[n][1] = fmaf(o[n][1], c0, f[1] + e[1]);
          o[n][2] = fmaf(o[n][2], c1, f[2] + e[2]);
          o[n][3] = fmaf(o[n][3], c1, f[3] + e[3]);
        }
      }
      if (++stage == C::kStages) stage = 0;
    }
    // the outputs go to the stage that every warp has just used, which is
    // filled again only after the barriers below
    const int used = (stage == 0 ? C::kStages : stage) - 1;
    float* m_out = reinterpret_cast<float*>(smem + used * C::kStageBytes);  // of warp 0
    constexpr int kNext = C::kStages * C::kStageBytes / 4;                  // to the next warp's

    // ---- join the four warps; write the result or this share's partial
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t4 == 0) {
      m_ml[warp * R + g4] = make_float2(m0, l0);
      if constexpr (R > 8) m_ml[warp * R + g4 + 8] = make_float2(m1, l1);
    }
    float* mo = m_out + warp * kNext;
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int d = n * 8 + t4 * 2;
      if (g4 < rows) *reinterpret_cast<float2*>(mo + g4 * HD + d) = make_float2(o[n][0], o[n][1]);
      if constexpr (R > 8)
        if (g4 + 8 < rows) *reinterpret_cast<float2*>(mo + (g4 + 8) * HD + d) = make_float2(o[n][2], o[n][3]);
    }
    if (bad && lane == 0) s_segbad[seg & 1] = 1;
    __syncthreads();
    const bool seg_bad = s_segbad[seg & 1] != 0;
    const bool whole = from_start && to_end;
    if (seg_bad && tid == 0) set_error(a.status, MINFER_ERR_POS_OOB);
    float* part = ws_part + (int64_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * ws_part_floats(HD);
    for (int i = tid; i < rows * HD; i += kWarps * 32) {
      const int row = i / HD, d = i % HD;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, m_ml[w * R + row].x);
      const float z = m == -INFINITY ? 0.f : m;
      float l = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = m_ml[w * R + row];
        const float c = ex2(ml.x - z);
        l = fmaf(ml.y, c, l);
        acc = fmaf(m_out[w * kNext + i], c, acc);
      }
      if (whole) {
        if (!seg_bad) {
          store_as(static_cast<T*>(a.o) + (int64_t)r * a.o_stride + (int64_t)head0 * HD + i, l == 0.f ? 0.f : acc / l);
          if (d == 0 && a.lse) a.lse[(int64_t)r * a.nh + head0 + row] = fmaf(m, kLn2, logf(l));
        }
      } else {
        if (d == 0) reinterpret_cast<float2*>(part)[row] = make_float2(m, seg_bad ? -1.f : l);
        part[2 * kRows + i] = acc;
      }
    }
    // flag of the next piece, free since the barrier above
    if (tid == 0) s_segbad[(seg + 1) & 1] = 0;
    __syncthreads();
    ++seg;
    if (!whole) {
      const int64_t first = begin + (done - seg_units) - cw.u;
      Piece& p = piece[from_start ? 1 : 0];
      p = Piece{r, head0, rows, share_of(first, total, n_shares), share_of(first + cw.units - 1, total, n_shares)};
    }
    // on to the next (request, head block)
    cw.u = cw.units - 1;
    walk_next(cw, a, nv, cap);
  }

  // ---- report the partials (complete since the last barrier) and join what is
  // complete with them.  Thread 32 i takes piece i.
  const int g = blockIdx.x / kGroup;
  if (lane == 0 && warp < 2) {
    const Piece& p = piece[warp];
    bool last = false;
    if (p.rows) {
      const int all = p.c1 - p.c0 + 1;
      const int lo = max(p.c0, g * kGroup), hi = min(p.c1, g * kGroup + kGroup - 1);
      const int n = all <= kDirect ? all : hi - lo + 1;
      unsigned* counter = counters + (all <= kDirect || p.c0 >= g * kGroup ? p.c0 : kMaxShares + g);
      __threadfence();
      last = n == 1 || atomicAdd(counter, 1u) == (unsigned)n - 1;
      if (last && n > 1) *counter = 0;
      __threadfence();
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
    auto slot = [&](int c) { return ws_part + (int64_t)(c * 2 + (c == p.c0 ? 1 : 0)) * ws_part_floats(HD); };
    const bool direct = p.c1 - p.c0 + 1 <= kDirect;
    const int lo = direct ? p.c0 : max(p.c0, g * kGroup), hi = direct ? p.c1 : min(p.c1, g * kGroup + kGroup - 1);
    if (hi > lo) {
      if (tid <= hi - lo) s_join.part[tid] = slot(lo + tid);
      __syncthreads();
      join_parts<T, HD, R>(s_join, hi - lo + 1, p.rows, direct, o_row, lse_row);
      __syncthreads();
    }
    if (!direct) {
      const int g0 = p.c0 / kGroup, g1 = p.c1 / kGroup;
      if (tid == 0) {
        unsigned* counter = counters + kMaxShares + kMaxShares / kGroup + 1 + p.c0;
        __threadfence();
        s_segbad[0] = atomicAdd(counter, 1u) == (unsigned)(g1 - g0);
        if (s_segbad[0]) *counter = 0;
        __threadfence();
      }
      if (tid <= g1 - g0) s_join.part[tid] = slot(max(p.c0, (g0 + tid) * kGroup));
      __syncthreads();
      if (s_segbad[0]) join_parts<T, HD, R>(s_join, g1 - g0 + 1, p.rows, true, o_row, lse_row);
      __syncthreads();
    }
  }
  idle_requests();
}

int shares(int hd, int type, int num_sms) {
  return std::min(num_sms * (hd * (type == MINFER_F32 ? 4 : 2) == 512 ? 1 : 2), kMaxShares);
}

template <typename T, int HD, int R>
cudaError_t launch(const PagedAttnArgs& a, int n, int n_groups, cudaStream_t st) {
  using C = Cfg<T, HD, R>;
  auto kernel = paged_attn_kernel<T, HD, R>;
  cudaError_t e = allow_smem<paged_attn_kernel<T, HD, R>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)n), dim3(kWarps * 32), C::kSmem, st, a, n_groups, a.scale * kLog2e);
}
template <typename T, int HD>
cudaError_t launch(const PagedAttnArgs& a, int type, int num_sms, cudaStream_t st) {
  const int G = a.nh / a.c.nkv, n_groups = (G + kRows - 1) / kRows, n = shares(HD, type, num_sms);
  return G <= 8 ? launch<T, HD, 8>(a, n, n_groups, st) : launch<T, HD, 16>(a, n, n_groups, st);
}

}  // namespace

int64_t paged_attn_workspace(int hd, int type, int num_sms) {
  const int n = shares(hd, type, num_sms);
  return kPartOffset + (int64_t)n * 2 * ws_part_floats(hd) * 4;
}

cudaError_t paged_attn_launch(const PagedAttnArgs& a, int type, int num_sms, cudaStream_t st) {
  if (type == MINFER_F32)
    return a.c.hd == 64 ? launch<float, 64>(a, type, num_sms, st) : launch<float, 128>(a, type, num_sms, st);
  if (type == MINFER_F16)
    return a.c.hd == 64 ? launch<__half, 64>(a, type, num_sms, st) : launch<__half, 128>(a, type, num_sms, st);
  return a.c.hd == 64 ? launch<__nv_bfloat16, 64>(a, type, num_sms, st)
                      : launch<__nv_bfloat16, 128>(a, type, num_sms, st);
}

}  // namespace minfer
