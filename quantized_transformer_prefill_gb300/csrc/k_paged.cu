// k_paged.cu -- the paged K/V cache's bookkeeping and store: block tables and
// slot maps built from request lengths, and bias + QK-norm + RoPE of fused
// Q|K|V rows with K and V written to their slots.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

// ================================================================ page tables
//
// One thread-block cluster does a step, or one CTA where there is little to write
// (32 requests of one token 3.8 us against 4.5 with eight CTAs, 1,087 tokens 5.2
// against 5.8, 2,164 tokens 6.0 against 5.8; sixteen where there is much: 6,364
// tokens 6.3 with either, 21,500 tokens of 1,023 requests 7.0 against 8.4).  Every
// CTA scans all requests (new tokens, grown pages, returned pages: three exclusive
// prefix sums in its own shared memory), checks its share of the page ids the step
// will use, works out its share of the outputs, and writes it after one cluster
// barrier, at which the CTAs learn whether any of them found an error.  Nothing is
// written before the barrier, so an error leaves everything as it was, and nothing
// that is read is written: the entries that grow, the stack above its old depth and
// the outputs are read by nobody.  What is left is a chain: the lengths (1.2 us),
// the searches and page loads (1.7), the barrier (0.8), the stores.
constexpr int kPtThreads = 1024;
// What a launch gets unasked, 48 KB, less the kernel's static bytes: of that size
// are also the CTAs of a cluster of 16 (3,412 requests).
constexpr int kPtUnaskedSmem = 40 * 1024;

__device__ __forceinline__ uint32_t pt_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t pt_cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void pt_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void pt_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x < a[n]), for Q values
// at once: the same number of steps for all, their loads side by side.
template <int Q>
__device__ __forceinline__ void pt_find(const int* a, int n, const int (&x)[Q], int (&i)[Q]) {
#pragma unroll
  for (int q = 0; q < Q; ++q) i[q] = 0;
  for (int w = 1 << (31 - __clz(n)); w > 0; w >>= 1) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (i[q] + w < n && a[i[q] + w] <= x[q]) i[q] += w;
  }
}
__device__ __forceinline__ int pt_find(const int* a, int n, int x) {
  const int y[1] = {x};
  int i[1];
  pt_find<1>(a, n, y, i);
  return i[0];
}

__global__ void __launch_bounds__(kPtThreads, 1) page_tables_kernel(const PageTablesArgs a) {
  extern __shared__ int pt_smem[];
  int* s_start = pt_smem;                  // [n + 1] new tokens before request r
  int* s_grow = s_start + a.n_req + 1;     // [n + 1] new pages before request r
  int* s_back = s_grow + a.n_req + 1;      // [n + 1] returned pages before request r
  __shared__ int s_warp[3][32];
  __shared__ int s_local, s_err;  // error flags: of this CTA, of the whole cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n_req, P = a.page_size;
  const uint32_t rank = pt_cluster_rank(), nrank = pt_cluster_size();
  // A thread's number for what is written side by side; and its numbers for grown,
  // shared and returned pages, of which there are fewer than threads: every CTA has its
  // share of them, in warps of their own.
  const int gtid = (int)rank * kPtThreads + tid, gn = (int)nrank * kPtThreads;
  auto number = [&](int at) { return at * (int)nrank + (int)rank; };
  const int j0 = number(tid), r0_shared = number((tid + kPtThreads / 2) % kPtThreads), k0 = number(kPtThreads - 1 - tid);
  enum { kBadLen = 1, kTooMany = 2, kNoPages = 4, kBadPage = 8 };

  if (tid == 0) s_local = s_err = 0;
  if (nrank > 1) pt_cluster_arrive();  // waited for before a peer's s_err is touched
  // No early launch of the next kernel: the forward's kernels read positions, which
  // this one writes, before they wait for their predecessor.
  pdl_wait();

  const int cap = a.max_pages * P;
  auto pages = [&](int rows) { return rows == 0 ? 0 : a.div.of(rows - 1) + 1; };
  const int n_free = *a.n_free;
  int err = 0;
  int base0 = 0, base1 = 0, base2 = 0;
  for (int r0 = 0; r0 < n; r0 += kPtThreads) {
    const int r = r0 + tid;
    int v0 = 0, v1 = 0, v2 = 0;
    if (r < n) {
      const int L = a.len[r], T = a.target[r];
      if (L < 0 || T < 0 || L > cap || T > cap) {
        err |= kBadLen;
      } else {
        const int held = pages(L), need = pages(T);
        v0 = max(0, T - L);
        v1 = max(0, need - held);
        v2 = max(0, held - need);
      }
    }
    // inclusive scans; the page sums fit (n_req * max_pages does), the token
    // sum saturates at 2^30, which is past any max_tokens
    int x0 = min(v0, 1 << 30), x1 = v1, x2 = v2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y0 = __shfl_up_sync(0xffffffffu, x0, o), y1 = __shfl_up_sync(0xffffffffu, x1, o),
                y2 = __shfl_up_sync(0xffffffffu, x2, o);
      if (lane >= o) {
        x0 = (int)min((unsigned)x0 + (unsigned)y0, 1u << 30);
        x1 += y1;
        x2 += y2;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = x0;
      s_warp[1][warp] = x1;
      s_warp[2][warp] = x2;
    }
    __syncthreads();
    if (warp == 0) {
      int w0 = s_warp[0][lane], w1 = s_warp[1][lane], w2 = s_warp[2][lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y0 = __shfl_up_sync(0xffffffffu, w0, o), y1 = __shfl_up_sync(0xffffffffu, w1, o),
                  y2 = __shfl_up_sync(0xffffffffu, w2, o);
        if (lane >= o) {
          w0 = (int)min((unsigned)w0 + (unsigned)y0, 1u << 30);
          w1 += y1;
          w2 += y2;
        }
      }
      s_warp[0][lane] = w0;
      s_warp[1][lane] = w1;
      s_warp[2][lane] = w2;
    }
    __syncthreads();
    const unsigned p0 = (unsigned)base0 + (warp ? s_warp[0][warp - 1] : 0);
    const int e0 = (int)min(min(p0, 1u << 30) + (unsigned)x0, 1u << 30);
    const int e1 = base1 + (warp ? s_warp[1][warp - 1] : 0) + x1;
    const int e2 = base2 + (warp ? s_warp[2][warp - 1] : 0) + x2;
    if (r < n) {
      s_start[r + 1] = e0;
      s_grow[r + 1] = e1;
      s_back[r + 1] = e2;
    }
    base0 = (int)min((unsigned)base0 + (unsigned)s_warp[0][31], 1u << 30);
    base1 += s_warp[1][31];
    base2 += s_warp[2][31];
    __syncthreads();  // s_warp is written again
  }
  if (tid == 0) s_start[0] = s_grow[0] = s_back[0] = 0;
  if (err) atomicOr(&s_local, err);
  __syncthreads();  // the prefix arrays and the flags are complete
  err = s_local;    // the same in every CTA: each has seen every request
  const int tokens = base0, grown = base1, back = base2;
  const int64_t depth = (int64_t)n_free + back;
  if (!err) {
    if (tokens > a.max_tokens) err |= kTooMany;
    if (n_free < 0 || n_free > a.n_pages)
      err |= kBadPage;
    else if (depth < grown)
      err |= kNoPages;
    else if (depth - grown > a.n_pages)
      err |= kBadPage;
  }

  // where the k-th returned page is, and the j-th new one: the stack from its top,
  // with the returned pages on it
  auto returned_at = [&](int k) -> const int* {
    const int r = pt_find(s_back, n, k);
    return a.table + (int64_t)r * a.max_pages + pages(a.target[r]) + (k - s_back[r]);
  };
  auto new_at = [&](int j) -> const int* {
    const int64_t i = depth - 1 - j;
    return i < n_free ? a.free_pages + i : returned_at((int)(i - n_free));
  };

  // positions and slots of the tokens t0, t0 + gn, ..; -1 behind the last
  constexpr int Q = 2;
  auto tokens_at = [&](int t0, int (&pos)[Q], int (&slot)[Q]) {
    int t[Q], r[Q], off[Q];
    const int* from[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) t[q] = min(t0 + q * gn, tokens - 1);
    if (t0 < tokens) pt_find<Q>(s_start, n, t, r);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      pos[q] = -1;
      off[q] = 0;
      from[q] = nullptr;
      if (t0 + q * gn >= tokens) continue;
      const int L = a.len[r[q]];
      pos[q] = L + (t[q] - s_start[r[q]]);
      const int p = a.div.of(pos[q]), held = pages(L);
      off[q] = pos[q] - p * P;
      from[q] = p < held ? a.table + (int64_t)r[q] * a.max_pages + p : new_at(s_grow[r[q]] + (p - held));
    }
    int page[Q];  // the loads side by side
#pragma unroll
    for (int q = 0; q < Q; ++q) page[q] = from[q] ? *from[q] : 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) slot[q] = from[q] ? (int)((unsigned)page[q] * (unsigned)P + (unsigned)off[q]) : -1;
  };
  auto put_tokens = [&](int t0, const int (&pos)[Q], const int (&slot)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int at = t0 + q * gn;
      if (at >= a.max_tokens) break;
      a.pos[at] = pos[q];
      a.slot[at] = slot[q];
    }
  };
  auto entry_of = [&](int j) {  // where the j-th new page is entered
    const int r = pt_find(s_grow, n, j);
    return a.table + (int64_t)r * a.max_pages + pages(a.len[r]) + (j - s_grow[r]);
  };

  // A thread's first grown page, returned page and shared page (the one that a
  // request's next row shares with its last one) are checked here, and all that a
  // thread will write first is worked out before the barrier, whose wait hides it
  // (after the barrier, the mixed step took 9.5 us).  Nothing that is read here is
  // written by this step.
  int page0 = 0, back0 = 0, *entry0 = nullptr;
  int pos0[Q], slot0[Q];
  if (!err) {
    const unsigned np = (unsigned)a.n_pages;
    auto shared_page = [&](int r) {  // 0 where there is none
      const int L = a.len[r], p = a.div.of(L);
      return s_start[r + 1] > s_start[r] && L > p * P ? a.table[(int64_t)r * a.max_pages + p] : 0;
    };
    if (k0 < back) back0 = *returned_at(k0);
    const int shared0 = r0_shared < n ? shared_page(r0_shared) : 0;
    if (j0 < grown) {
      page0 = *new_at(j0);
      entry0 = entry_of(j0);
    }
    tokens_at(gtid, pos0, slot0);
    bool bad = (unsigned)page0 >= np || (unsigned)back0 >= np || (unsigned)shared0 >= np;
    for (int j = j0 + gn; j < grown; j += gn) bad |= (unsigned)*new_at(j) >= np;
    for (int k = k0 + gn; k < back; k += gn) bad |= (unsigned)*returned_at(k) >= np;
    for (int r = r0_shared + gn; r < n; r += gn) bad |= (unsigned)shared_page(r) >= np;
    if (__syncthreads_or(bad)) err |= kBadPage;
  }
  if (nrank > 1) {
    pt_cluster_wait();
    if (err && tid < (int)nrank) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(&s_err)), "r"(tid));
      asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(err) : "memory");
    }
    pt_cluster_arrive();
    pt_cluster_wait();
    err = s_err;
  }

  if (err) {
    for (int r = gtid; r <= n; r += gn) a.start[r] = 0;
    for (int t = gtid; t < a.max_tokens; t += gn) {
      a.pos[t] = -1;
      a.slot[t] = -1;
    }
    if (gtid == 0)
      set_error(a.status, (err & kBadLen)    ? MINFER_ERR_POS_OOB
                          : (err & kTooMany) ? MINFER_ERR_TOO_LARGE
                          : (err & kNoPages) ? MINFER_ERR_OOM
                                             : MINFER_ERR_ARG);
    return;
  }

  for (int r = gtid; r <= n; r += gn) a.start[r] = s_start[r];
  put_tokens(gtid, pos0, slot0);
  if (j0 < grown) *entry0 = page0;
  for (int j = j0 + gn; j < grown; j += gn) *entry_of(j) = *new_at(j);
  const int pushed = (int)(depth - grown) - n_free;
  if (k0 < pushed) a.free_pages[n_free + k0] = back0;
  for (int k = k0 + gn; k < pushed; k += gn) a.free_pages[n_free + k] = *returned_at(k);
  for (int t0 = gtid + Q * gn; t0 < a.max_tokens; t0 += Q * gn) {
    tokens_at(t0, pos0, slot0);
    put_tokens(t0, pos0, slot0);
  }
  if (gtid == 0) *a.n_free_out = (int)(depth - grown);
}

// ================================================================ RoPE + paged store

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// E values of T as one vector access (E * sizeof(T) = 4, 8 or 16 bytes).
template <typename T, int E>
struct alignas(E * sizeof(T)) Vec {
  T v[E];
};

// cos and sin of 2 pi * f / 2^64.  The quadrant comes off in integers; the rest,
// at most an eighth of a turn, is taken to 2^-34 of a turn (an angle of 4e-10,
// below f32's step for a sine or cosine), and its sine and cosine are the Taylor
// polynomials to the 9th and 10th degree: the first terms left out, x^11 / 11!
// and x^12 / 12! at pi / 4, are 1.8e-9 and 1.1e-10.
__device__ __forceinline__ void turn_cos_sin(uint64_t f, float* c, float* s) {
  const uint64_t g = f + (1ull << 61);
  const uint32_t quad = (uint32_t)(g >> 62);
  const int32_t rest = (int32_t)((uint32_t)(g >> 30) - 0x80000000u);  // 2^-34 turns
  const float x = (float)rest * (float)(6.283185307179586 / 17179869184.0), q = x * x;
  float sr = fmaf(q, 1.f / 362880, -1.f / 5040);
  sr = fmaf(q, sr, 1.f / 120);
  sr = fmaf(q, sr, -1.f / 6);
  sr = fmaf(q * x, sr, x);
  float cr = fmaf(q, -1.f / 3628800, 1.f / 40320);
  cr = fmaf(q, cr, -1.f / 720);
  cr = fmaf(q, cr, 1.f / 24);
  cr = fmaf(q, cr, -0.5f);
  cr = fmaf(q, cr, 1.f);
  const float cc = (quad & 1) ? sr : cr, ss = (quad & 1) ? cr : sr;
  *c = (quad == 1 || quad == 2) ? -cc : cc;
  *s = (quad >= 2) ? -ss : ss;
}

constexpr int kRpWarps = 8;
constexpr int kRpTokens = 4;     // of a CTA, at most
// CTAs per SM that more tokens per CTA must leave (1: 1,001 rows 9.6 us, 500 rows
// 6.3; 2: 7.3 and 5.2; 4: 8.4 and 5.1)
constexpr int kRpFill = 2;
// Values of the bias that are kept in shared memory; read from global memory for
// every head instead, it made the 4096 rows 30 us.
constexpr int kRpMaxBias = 24576;
constexpr int kRpRing = 8;       // units of a warp on their way or at work

// Bound by HBM: 4096 f32 rows of 36 heads of 128 into a bf16 cache, 113 MB, take
// 20 us (5.7 TB/s, 84% of the measured copy); 1,001 f16 rows with QK-norm 6.0 us, in 501
// CTAs of two tokens, 3.3 per SM: a warp has four units behind two barriers and the
// cosines; 64 rows 2.3 us, a launch.
//
// A CTA takes 1, 2 or 4 tokens.  Its threads work out the tokens' cosines and
// sines, one pair each, while the rows are on the way; then 8, 4 or 2 warps go
// over a token's heads.  A lane takes E neighbouring elements of a head (one
// 16-byte vector of the source type), so a unit of 32 lanes is 32 E / HD heads,
// and the lane's cosines and signed sines are the same for every unit.  The pair
// partner of an element lies in the lane itself (interleaved pairs), in another
// lane at the same place (half a rotation is a multiple of E), or, with rotated
// sizes that are no multiples of E, anywhere, and comes through shared memory.
template <typename TS, typename TD, int HD>
__global__ void __launch_bounds__(kRpWarps * 32) rope_paged_kernel(const __grid_constant__ RopePagedArgs a, int tokens, int swap_floats, int bias_floats) {
  constexpr int E = 16 / sizeof(TS), kLanes = HD / E, kPer = 32 / kLanes;  // lanes of a head, heads of a unit
  using VS = Vec<TS, E>;
  using VD = Vec<TD, E>;
  __shared__ uint64_t s_turn[64];
  __shared__ float s_cos[kRpTokens][64], s_sin[kRpTokens][64];
  // [warp][32 E], only where partners lie anywhere; then the bias (read for every
  // unit: from here, or from global memory where it is too large)
  extern __shared__ __align__(16) float rp_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = kRpWarps / tokens, mine = warp / per, first = warp % per;  // warps of a token, token, first unit
  const int t = blockIdx.x * tokens + mine;
  const int nqk = a.nh + a.c.nkv, heads = nqk + a.c.nkv, units = (heads + kPer - 1) / kPer;
  const int sub = lane / kLanes, d0 = (lane % kLanes) * E;  // head of the unit, first element of the head
  const int rot = a.rope.rot_dim, half = rot >> 1, slots = a.c.n_pages * a.c.page_size;
  const bool inter = a.rope.style == MINFER_ROPE_INTERLEAVED;
  const bool in_lane = inter && rot % E == 0, in_place = !inter && half % E == 0;

  pdl_trigger();
  pdl_wait();
  const TS* row = static_cast<const TS*>(a.qkv) + (int64_t)t * a.row_stride + lane * E;
  // The rows come through a ring in shared memory (a lane copies the vectors that
  // it reads itself): what is on its way takes no registers, so more warps fit.
  __shared__ __align__(16) unsigned char s_ring[kRpWarps][kRpRing][512];
  const uint32_t ring = smem_u32(s_ring[warp]) + lane * 16;
  auto fetch = [&](int u, int stage) {
    if (u * kPer + sub < heads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + stage * 512), "l"(row + u * (32 * E)) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = tid * 4; i < bias_floats; i += kRpWarps * 128)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rp_smem + swap_floats + i)), "l"(a.bias + i) : "memory");
  __shared__ __align__(16) float s_norm[2][HD];
  if (a.q_norm && tid < HD / 2)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&s_norm[0][0] + tid * 4)),
                 "l"((tid < HD / 4 ? a.q_norm : a.k_norm - HD) + tid * 4)
                 : "memory");
  asm volatile("cp.async.commit_group;" ::: "memory");
  int slot = -1, pos = 0;
  if (t < a.n_tokens) {
    slot = a.slot[t];
    pos = a.pos[t];
#pragma unroll
    for (int i = 0; i < kRpRing - 1; ++i) fetch(first + i * per, i);
  } else {
    for (int i = 0; i < kRpRing - 1; ++i) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // (a parameter is read fast at one address per warp, and very slowly at 32)
  static_assert(kRpWarps * 8 == 64, "eight entries per warp");
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_turn[warp * 8 + i] = a.rope.turn[warp * 8 + i];
  }
  {
    const int j = tid >> 6, pair = tid & 63, tj = blockIdx.x * tokens + j;
    const bool there = j < tokens && pair < half && tj < a.n_tokens;
    const int p = there ? a.pos[tj] : 0;
    __syncthreads();
    if (there) {
      float c, s;
      turn_cos_sin((uint64_t)(uint32_t)p * s_turn[pair], &c, &s);
      s_cos[j][pair] = c * a.rope.mscale;
      s_sin[j][pair] = s * a.rope.mscale;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kRpRing - 1) : "memory");  // bias and norm weights, the oldest group
    __syncthreads();
  }
  if (slot < 0 || slot >= slots || pos < 0) {  // padding, or refused
    if (slot >= 0 && first == 0 && lane == 0) set_error(a.status, MINFER_ERR_POS_OOB);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  float cs[E], sn[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = d0 + e, p = d >= rot ? 0 : inter ? d >> 1 : d < half ? d : d - half;
    cs[e] = s_cos[mine][p];
    sn[e] = s_sin[mine][p];
    if (inter ? !(d & 1) : d < half) sn[e] = -sn[e];
  }
  const int from = (d0 < half ? lane + half / E : lane - half / E) & 31;
  const bool turned = d0 < rot;
  float* swap = rp_smem + warp * (32 * E);
  const int page = a.c.div.of(slot);
  const int64_t at = (int64_t)page * a.c.page_stride + (int64_t)(slot - page * a.c.page_size) * a.c.row_stride;
  TD* const qdst = static_cast<TD*>(a.q_out) + (int64_t)t * a.q_stride + d0;
  TD* const kdst = static_cast<TD*>(a.c.k) + (at + d0 - a.nh * a.c.head_stride);
  TD* const vdst = static_cast<TD*>(a.c.v) + (at + d0 - nqk * a.c.head_stride);
  const float* const bias = !a.bias ? nullptr : (bias_floats ? rp_smem + swap_floats : a.bias) + lane * E;

  int stage = 0;
  for (int u = first; u < units; u += per) {
    {
      const int h = u * kPer + sub;
      fetch(u + (kRpRing - 1) * per, (stage + kRpRing - 1) % kRpRing);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRpRing - 1) : "memory");
      VS x;
      {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(ring + stage * 512) : "memory");
        x = *reinterpret_cast<const VS*>(&v);
      }
      stage = (stage + 1) % kRpRing;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = to_f32<TS>(x.v[e]);
      if (bias && h < heads) {
        const float4* b = reinterpret_cast<const float4*>(bias + u * (32 * E));
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
          const float4 f = b[j];
          y[4 * j] += f.x;
          y[4 * j + 1] += f.y;
          y[4 * j + 2] += f.z;
          y[4 * j + 3] += f.w;
        }
      }
      if (u * kPer < nqk) {  // some head of the unit is one of Q or K
        const bool qk = h < nqk;
        if (a.q_norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (qk) {
            const float r = rsqrtf(ss * (1.f / HD) + a.eps);
            const float4* w = reinterpret_cast<const float4*>(s_norm[h < a.nh ? 0 : 1] + d0);
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
              const float4 f = w[j];
              y[4 * j] *= r * f.x;
              y[4 * j + 1] *= r * f.y;
              y[4 * j + 2] *= r * f.z;
              y[4 * j + 3] *= r * f.w;
            }
          }
        }
        float z[E];
        if (in_place) {
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = __shfl_sync(0xffffffffu, y[e], from);
        } else if (in_lane) {
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = y[e ^ 1];
        } else {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < E; ++e) swap[lane * E + e] = y[e];
          __syncwarp();
          if (qk) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int d = d0 + e, p = inter ? d ^ 1 : d < half ? d + half : d - half;
              if (d < rot) y[e] = fmaf(swap[sub * HD + p], sn[e], y[e] * cs[e]);
            }
          }
        }
        if ((in_place || in_lane) && turned && qk) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = fmaf(z[e], sn[e], y[e] * cs[e]);
        }
      }
      if (h < heads) {
        VD out;
#pragma unroll
        for (int e = 0; e < E; ++e) out.v[e] = from_f32<TD>(y[e]);
        TD* dst = h < a.nh ? qdst + h * HD : (h < nqk ? kdst : vdst) + h * a.c.head_stride;
        *reinterpret_cast<VD*>(dst) = out;
      }
    }
  }
}

template <typename TS, typename TD, int HD>
cudaError_t rope_paged_sized(const RopePagedArgs& a, int num_sms, cudaStream_t st) {
  constexpr int E = 16 / sizeof(TS);
  // One token per CTA while that keeps the GPU from being full, for its eight
  // warps finish sooner; else up to four, which share the work before the heads.
  int tokens = 1;
  while (tokens < kRpTokens && a.n_tokens / (2 * tokens) >= num_sms * kRpFill) tokens *= 2;
  const bool swap = a.rope.style == MINFER_ROPE_HALF ? (a.rope.rot_dim / 2) % E != 0 : a.rope.rot_dim % E != 0;
  const int swap_floats = swap ? kRpWarps * 32 * E : 0, width = (a.nh + 2 * a.c.nkv) * HD;
  const int bias_floats = a.bias && width <= kRpMaxBias ? width : 0, smem = (swap_floats + bias_floats) * (int)sizeof(float);
  const cudaError_t e = allow_smem<rope_paged_kernel<TS, TD, HD>>((kRpWarps * 32 * E + kRpMaxBias) * (int)sizeof(float));
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_paged_kernel<TS, TD, HD>, dim3((unsigned)((a.n_tokens - 1) / tokens + 1)), dim3(32 * kRpWarps), smem, st, a, tokens,
                    swap_floats, bias_floats);
}
template <typename TS, typename TD>
cudaError_t rope_paged_typed(const RopePagedArgs& a, int num_sms, cudaStream_t st) {
  return a.c.hd == 64 ? rope_paged_sized<TS, TD, 64>(a, num_sms, st) : rope_paged_sized<TS, TD, 128>(a, num_sms, st);
}

// Whether the current device runs a cluster of sixteen CTAs, more than the portable
// size: asked for once per device.
bool pt_sixteen_fit() {
  constexpr int kMaxDevices = 64;
  static int8_t known[kMaxDevices];  // 0: not asked yet, 1 or -1; every thread writes the same
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return false;
  int8_t fit = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (fit == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kPtThreads);
    cfg.dynamicSmemBytes = kPtUnaskedSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    const bool ok = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&clusters, page_tables_kernel, &cfg) == cudaSuccess && clusters > 0;
    if (!ok) (void)cudaGetLastError();  // a cluster of eight serves
    fit = ok ? 1 : -1;
    __atomic_store_n(&known[dev], fit, __ATOMIC_RELAXED);
  }
  return fit > 0;
}

}  // namespace

cudaError_t page_tables_launch(const PageTablesArgs& a, cudaStream_t stream) {
  const size_t smem = 3 * (size_t)(a.n_req + 1) * sizeof(int);
  if (smem > kPtUnaskedSmem) {
    const cudaError_t e = allow_smem<page_tables_kernel>(3 * (kPageTablesMaxReq + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  unsigned cs = (a.max_tokens > 2048 || a.n_req > 1024) ? 8 : 1;
  if (a.max_tokens > 8192 && smem <= kPtUnaskedSmem && pt_sixteen_fit()) cs = 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs);
  cfg.blockDim = dim3(kPtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, page_tables_kernel, a);
}

cudaError_t rope_paged_launch(const RopePagedArgs& a, int src_type, int cache_type, int num_sms, cudaStream_t st) {
  if (cache_type == MINFER_F32) return rope_paged_typed<float, float>(a, num_sms, st);
  if (cache_type == MINFER_F16)
    return src_type == MINFER_F32 ? rope_paged_typed<float, __half>(a, num_sms, st)
                                  : rope_paged_typed<__half, __half>(a, num_sms, st);
  return src_type == MINFER_F32 ? rope_paged_typed<float, __nv_bfloat16>(a, num_sms, st)
                                : rope_paged_typed<__nv_bfloat16, __nv_bfloat16>(a, num_sms, st);
}

}  // namespace minfer
