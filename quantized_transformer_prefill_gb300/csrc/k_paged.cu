// k_paged.cu -- the paged K/V cache's bookkeeping and store: block tables and
// slot maps built from request lengths, and bias + QK-norm + RoPE of fused
// Q|K|V rows with K and V written to their slots.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace minfer {
namespace {

// ================================================================ page tables
//
// One thread-block cluster does a step.  Every CTA scans all requests (new
// tokens, grown pages, returned pages: three exclusive prefix sums in its own
// shared memory), checks its share of the page ids the step will use, and
// after one cluster barrier, at which the CTAs learn whether any of them found
// an error, writes its share of the outputs.  Nothing is written before the
// barrier, so an error leaves everything as it was, and nothing that another
// CTA still reads is written after it: the entries that grow, the stack above
// its old depth and the outputs are read by nobody.
constexpr int kPtThreads = 1024;
constexpr int kPtCluster = 8;

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
__device__ __forceinline__ void pt_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x < a[n]).
__device__ __forceinline__ int pt_find(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
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
  const int gtid = (int)rank * kPtThreads + tid, gn = (int)nrank * kPtThreads;
  enum { kBadLen = 1, kTooMany = 2, kNoPages = 4, kBadPage = 8 };

  if (tid == 0) s_local = s_err = 0;
  pdl_trigger();
  pdl_wait();
  if (nrank > 1)
    pt_cluster_sync();  // s_err is set in every CTA before a peer may OR into it
  else
    __syncthreads();

  const int cap = a.max_pages * P;
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
        const int held = (int)(((unsigned)L + P - 1) / (unsigned)P);
        const int need = (int)(((unsigned)T + P - 1) / (unsigned)P);
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

  // k-th returned page, and entry i of the stack with the returned pages on top
  auto returned = [&](int k) {
    const int r = pt_find(s_back, n, k);
    const int first = (int)(((unsigned)a.target[r] + P - 1) / (unsigned)P);
    return a.table[(int64_t)r * a.max_pages + first + (k - s_back[r])];
  };
  auto new_page = [&](int j) {
    const int64_t i = depth - 1 - j;
    return i < n_free ? a.free_pages[i] : returned((int)(i - n_free));
  };

  if (!err) {
    const unsigned np = (unsigned)a.n_pages;
    bool bad = false;
    for (int j = gtid; j < grown; j += gn) bad |= (unsigned)new_page(j) >= np;
    for (int k = gtid; k < back; k += gn) bad |= (unsigned)returned(k) >= np;
    for (int r = gtid; r < n; r += gn) {
      // the page that a request's next row shares with its last one
      const int L = a.len[r], p = L / P;
      if (s_start[r + 1] > s_start[r] && L > p * P)
        bad |= (unsigned)a.table[(int64_t)r * a.max_pages + p] >= np;
    }
    if (__syncthreads_or(bad)) err |= kBadPage;
  }
  if (nrank > 1) {
    if (err && tid < (int)nrank) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(&s_err)), "r"(tid));
      asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(err) : "memory");
    }
    pt_cluster_sync();
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
  for (int j = gtid; j < grown; j += gn) {
    const int r = pt_find(s_grow, n, j);
    const int held = (int)(((unsigned)a.len[r] + P - 1) / (unsigned)P);
    a.table[(int64_t)r * a.max_pages + held + (j - s_grow[r])] = new_page(j);
  }
  const int pushed = (int)(depth - grown) - n_free;
  for (int k = gtid; k < pushed; k += gn) a.free_pages[n_free + k] = returned(k);
  for (int t = gtid; t < a.max_tokens; t += gn) {
    int pos = -1, slot = -1;
    if (t < tokens) {
      const int r = pt_find(s_start, n, t);
      const int L = a.len[r];
      pos = L + (t - s_start[r]);
      const int p = (int)((unsigned)pos / (unsigned)P);
      const int held = (int)(((unsigned)L + P - 1) / (unsigned)P);
      const int page = p < held ? a.table[(int64_t)r * a.max_pages + p] : new_page(s_grow[r] + (p - held));
      slot = page * P + (pos - p * P);
    }
    a.pos[t] = pos;
    a.slot[t] = slot;
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

// cos and sin of 2 pi * f / 2^64.  The quadrant comes off in integers, so the
// rest r (in half turns, |r| <= 1/4) keeps its relative precision in f32.
__device__ __forceinline__ void turn_cos_sin(uint64_t f, float* c, float* s) {
  const uint32_t quad = (uint32_t)((f + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(f - ((uint64_t)quad << 62));
  float sr, cr;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &sr, &cr);
  const float cc = (quad & 1) ? sr : cr, ss = (quad & 1) ? cr : sr;
  *c = (quad == 1 || quad == 2) ? -cc : cc;
  *s = (quad >= 2) ? -ss : ss;
}

constexpr int kRpHeads = 4;      // heads of a warp whose loads are in flight together
constexpr int kRpMaxWarps = 16;

// One CTA per token, kRpHeads heads per warp: warp w of n takes heads w, w + n,
// ... of Q, K and V, lane l the head's elements l*E..l*E+E-1.  The row, the
// bias, the position and the slot are all loaded before the first of them is
// looked at.
template <typename TS, typename TD, int HD>
__global__ void __launch_bounds__(kRpMaxWarps * 32, 2) rope_paged_kernel(const __grid_constant__ RopePagedArgs a) {
  constexpr int E = HD / 32;
  using VS = Vec<TS, E>;
  using VD = Vec<TD, E>;
  using VF = Vec<float, E>;
  __shared__ float s_cos[HD / 2], s_sin[HD / 2];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int nqk = a.nh + a.c.nkv, heads = nqk + a.c.nkv;
  const TS* row = static_cast<const TS*>(a.qkv) + (int64_t)t * a.row_stride + lane * E;
  pdl_trigger();
  pdl_wait();
  VS x[kRpHeads];
  VF b[kRpHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kRpHeads; ++i) {
      const int h = h0 + i * warps;
      if (h < heads) x[i] = *reinterpret_cast<const VS*>(row + (int64_t)h * HD);
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < kRpHeads; ++i) {
        const int h = h0 + i * warps;
        if (h < heads) b[i] = *reinterpret_cast<const VF*>(a.bias + (int64_t)h * HD + lane * E);
      }
    }
  };
  const int slot = a.slot[t], pos = a.pos[t];
  load(warp);
  if (slot < 0) return;  // padding
  if (slot >= a.c.n_pages * a.c.page_size || pos < 0) {
    if (tid == 0) set_error(a.status, MINFER_ERR_POS_OOB);
    return;
  }
  const int rot = a.rope.rot_dim, half = rot >> 1;
  const bool inter = a.rope.style == MINFER_ROPE_INTERLEAVED;
  const int page = slot / a.c.page_size;
  const int64_t at = (int64_t)page * a.c.page_stride + (int64_t)(slot - page * a.c.page_size) * a.c.row_stride;
  for (int i = tid; i < half; i += blockDim.x) {
    float c, s;
    turn_cos_sin((uint64_t)(uint32_t)pos * a.rope.turn[i], &c, &s);
    s_cos[i] = c * a.rope.mscale;
    s_sin[i] = s * a.rope.mscale;
  }
  __syncthreads();

  for (int h0 = warp; h0 < heads; h0 += warps * kRpHeads) {
    if (h0 != warp) load(h0);
#pragma unroll
    for (int i = 0; i < kRpHeads; ++i) {
      const int h = h0 + i * warps;
      if (h >= heads) break;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = to_f32<TS>(x[i].v[e]);
      if (a.bias) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] += b[i].v[e];
      }
      if (h < nqk) {
        if (a.q_norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * (1.f / HD) + a.eps);
          const VF w = *reinterpret_cast<const VF*>((h < a.nh ? a.q_norm : a.k_norm) + lane * E);
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = y[e] * r * w.v[e];
        }
        // the pair partner of element i: i ^ 1, or i + half / i - half
        float z[E];
        if (inter) {
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = y[e ^ 1];
        } else if (half % E == 0) {
          const int src = lane * E < half ? lane + half / E : lane - half / E;
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = __shfl_sync(0xffffffffu, y[e], src & 31);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int p = lane * E + e < half ? lane * E + e + half : lane * E + e - half;
            z[e] = 0.f;
#pragma unroll
            for (int g = 0; g < E; ++g) {
              const float w = __shfl_sync(0xffffffffu, y[g], (p / E) & 31);
              if ((p & (E - 1)) == g) z[e] = w;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane * E + e;
          if (d < rot) {
            const int p = inter ? d >> 1 : (d < half ? d : d - half);
            const bool lower = inter ? !(d & 1) : d < half;
            const float s = lower ? -s_sin[p] : s_sin[p];
            y[e] = fmaf(z[e], s, y[e] * s_cos[p]);
          }
        }
      }
      VD out;
#pragma unroll
      for (int e = 0; e < E; ++e) out.v[e] = from_f32<TD>(y[e]);
      TD* dst;
      if (h < a.nh)
        dst = static_cast<TD*>(a.q_out) + (int64_t)t * a.q_stride + (int64_t)h * HD;
      else if (h < nqk)
        dst = static_cast<TD*>(a.c.k) + at + (int64_t)(h - a.nh) * a.c.head_stride;
      else
        dst = static_cast<TD*>(a.c.v) + at + (int64_t)(h - nqk) * a.c.head_stride;
      *reinterpret_cast<VD*>(dst + lane * E) = out;
    }
  }
}

template <typename TS, typename TD>
cudaError_t rope_paged_typed(const RopePagedArgs& a, cudaStream_t st) {
  const int heads = a.nh + 2 * a.c.nkv, warps = (heads + kRpHeads - 1) / kRpHeads;
  const dim3 grid((unsigned)a.n_tokens), block(32 * (unsigned)(warps < kRpMaxWarps ? warps : kRpMaxWarps));
  if (a.c.hd == 64) return launch_pdl(rope_paged_kernel<TS, TD, 64>, grid, block, 0, st, a);
  return launch_pdl(rope_paged_kernel<TS, TD, 128>, grid, block, 0, st, a);
}

}  // namespace

cudaError_t page_tables_launch(const PageTablesArgs& a, cudaStream_t stream) {
  const size_t smem = 3 * (size_t)(a.n_req + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem<page_tables_kernel>(3 * (kPageTablesMaxReq + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  const unsigned cs = (a.max_tokens > 4096 || a.n_req > 1024) ? kPtCluster : 1;
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

cudaError_t rope_paged_launch(const RopePagedArgs& a, int src_type, int cache_type, cudaStream_t st) {
  if (cache_type == MINFER_F32) return rope_paged_typed<float, float>(a, st);
  if (cache_type == MINFER_F16)
    return src_type == MINFER_F32 ? rope_paged_typed<float, __half>(a, st) : rope_paged_typed<__half, __half>(a, st);
  return src_type == MINFER_F32 ? rope_paged_typed<float, __nv_bfloat16>(a, st)
                                : rope_paged_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace minfer
