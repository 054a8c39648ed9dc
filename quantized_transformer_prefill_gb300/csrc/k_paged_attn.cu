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
// Inside a CTA every warp takes 16 keys of a unit, copies their K and V rows
// into its own ring in shared memory (cp.async of 16 bytes, page by page; rows
// behind the request's last are filled with zeros) and runs an online softmax of
// its own: no barrier before the end of the (request, KV head).  The products
// are m16n8 MMAs with the keys (S^T = K Q^T) and the head's dims (O^T = V^T P^T)
// as the 16 rows and 8 query heads as the columns: with up to 8 query heads per
// KV head no column is wasted more than the heads are few, and the accumulators
// of a warp are HD / 2 x 8 / 32 registers.  One query token would leave the 128
// rows of a tcgen05 tile of heads nearly empty, and with the keys as its rows the
// scores would go through TMEM twice for a few flops per byte; the bound is the
// bytes of K and V, so the accumulators stay in registers, where the softmax
// needs them.
//
// 16-bit caches: Q, K and V are exact in an MMA; a weight goes through two of them, as
// the sum of two 16-bit numbers (split2), which costs 1% of a call bound by its bytes,
// 8% of one of many heads (64 of up to 4096, 32/2 heads of 64: 23.7 us against 21.9),
// and keeps 15 bits and more of it instead of 8 (bf16) or 11 (f16).
//
// f32 caches: every operand is split into two tf32 halves and three products are
// taken (what is left out is at most 5 * 2^-22 of a product, of either sign), and
// each unit's P V is added to the running sum as an f32 addition of its own.
//
// Measured on a GB300 (us a call, device; bytes of K and V at the measured copy
// rate of 6.77 TB/s in brackets): 64 requests of up to 4096 rows, 28/4 heads of
// 128, bf16: 53 (44); one of 131,071, 12/2 heads of 128, f16: 31 (20); 33 of up to
// 2048, 14/2 heads of 64, f32: 15.5 (5); one of 513: 6.3.  While units are worked on
// the rows come in at 7.1 TB/s; what is left is the start (lengths, page lookup,
// first rows: 3 us), equal shares ending up to a tenth apart, and the join (report
// 1 us, 2 to 3 us a level).  Small last shares for CTAs that start where one has
// finished early made 64 x 4096 3% and the single long request 15% slower.
#include <algorithm>

#include "paged_attn.cuh"

namespace minfer {
namespace {

constexpr int kKeys = 16;  // keys of a unit that one warp takes

// R: query heads of a head block, one MMA tile of 8, or two where a KV head of a
// 16-bit cache has more than 8 (32/2 heads of 128, 64 requests of up to 4096, with one
// MMA for the weights: 35 us against 40 with two blocks of 8, which read K and V twice,
// the second time for the most part out of L2; with two MMAs 36).  An f32 block of 16 would not fit the registers.
template <typename T, int HD, int R>
struct Cfg {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kRowBytes = HD * (int)sizeof(T);
  static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks of a row
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // K and V rows of one warp
  // As many CTAs per SM as their registers and two stages of the ring allow; the
  // ring takes what is left of the SM's shared memory.  Rows of 512 bytes (f32,
  // head size 128) have CTAs of two warps: three of them hold 6 warps where one
  // CTA of four would fit (64 requests of up to 1024, 16/8 heads: a sixth less time,
  // 63 us now; 4 of up to 2048, 12/2 heads: 13 against 11, for its shares are smaller).
  static constexpr int kWarps = kRowBytes == 512 ? 2 : 4;
  static constexpr int kCtas = kRowBytes == 128 ? 4 : R == 8 ? 3 : 2;
  static constexpr int kUnit = kWarps * kKeys;  // keys of a unit
  static constexpr int kPBytes = kF32 ? kWarps * kKeys * R * 4 : 0;  // softmax weights on their way to the other layout
  static constexpr int kStatic = (int)sizeof(JoinShared<R>) + 512 + kWarps * R * 8 + R * 16;
  static constexpr int kFit = (233472 / kCtas - 1024 - kStatic - kPBytes) / (kWarps * kStageBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kWarps * kStages * kStageBytes + kPBytes;
  static_assert(kStages >= 2, "a ring has two stages at least");
  static_assert(R * HD * 4 <= kStageBytes, "a warp's output fits the stage it has just used");
};

// x = hi + lo: hi is x rounded to tf32 (11 significant bits), ties away from
// zero, in integer arithmetic (the conversion instruction has a quarter of its
// rate), and at most the largest finite tf32 in size, to which the topmost f32 values
// and infinities are cut; lo = x - hi is exact and at most 2^-11 |x| (of the topmost
// values 2^-11 and a step), and the MMA takes its upper 11 bits, which leaves out less
// than 2^-21 |x|.  An infinity or a NaN lies in lo.  (The cut costs 2% of a call of
// ordinary length and 4% of 64 x 1024, 16/8 heads of 128.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t* hi, uint32_t* lo) {
  const uint32_t near = (x + 0x1000u) & 0xFFFFE000u;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=r"(*hi) : "r"(near), "r"(0x7F7FE000u));
  *lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(*hi));
}

// Weights, at most 1, go into the sums of values times this power of two, and results
// are divided by it.  f32 and bf16: 1 over the request's length, so that no sum of the
// largest finite values overflows (a warp's, under its own maximum, may be one of keys
// that weigh nothing in the end).  f16: 2^15, so that weights stand well above 2^-24,
// where f16 ends.
template <typename T>
__device__ __forceinline__ float weight_scale(int len) {
  return __int_as_float((127 - (32 - __clz(len - 1))) << 23);
}
template <>
__device__ __forceinline__ float weight_scale<__half>(int) {
  return 0x1p15f;
}

// Two weights, each times weight_scale the sum of an upper and a lower 16-bit number.
// The upper one is cut off below the weight, equal to it only for a weight of 0, so
// that the lower one is positive as well: an infinite value times the weight is then
// infinite and not 0 * inf.
//  bf16: the upper 16 bits of the f32 before the weight; what is left is at most
//    2^-7 of the weight and rounded to 2^-8 of itself.
//  f16: the upper number is the weight less 2^-12 of it, cut off; what is left, at
//    most 1.25 * 2^-10, is rounded to 2^-11 of itself, or to a step of 2^-24 (2^-39 of
//    the largest weight), which it keeps if the weight has one.
__device__ __forceinline__ void split2(float a, float b, float scale, uint32_t* hi, uint32_t* lo, __nv_bfloat16) {
  a *= scale;
  b *= scale;
  const uint32_t ua = (max(__float_as_uint(a), 1u) - 1) & 0xFFFF0000u, ub = (max(__float_as_uint(b), 1u) - 1) & 0xFFFF0000u;
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(ua), b - __uint_as_float(ub));
  *hi = ua >> 16 | ub;
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split2(float a, float b, float scale, uint32_t* hi, uint32_t* lo, __half) {
  const float below = scale * (1.f - 0x1p-12f);
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(*hi) : "f"(b * below), "f"(a * below));
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(hi));
  constexpr float kStep = 0x1.01p-25f;  // rounds to a step
  const __half2 l = __floats2half2_rn(fmaxf(fmaf(a, scale, -h.x), fminf(a * scale, kStep)), fmaxf(fmaf(b, scale, -h.y), fminf(b * scale, kStep)));
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
template <typename T, int HD, int R>
__global__ void __launch_bounds__(Cfg<T, HD, R>::kWarps * 32, Cfg<T, HD, R>::kCtas)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, int n_groups, float scale_log2) {
  using C = Cfg<T, HD, R>;
  constexpr bool kF32 = C::kF32;
  constexpr int kWarps = C::kWarps, kUnit = C::kUnit;
  constexpr int kSteps = C::kChunks / 2;  // MMA steps over the head's dims (two chunks each)
  constexpr int kTiles = HD / 16;         // m16 tiles of the output
  constexpr int NH = R / 8;               // n8 tiles of query heads
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ Walk s_walk;
  __shared__ uint8_t s_bad[kWarps][C::kStages];
  __shared__ int s_segbad[2], s_last[2];
  __shared__ JoinShared<R> s_join;
  __shared__ float2 m_ml[kWarps * R];  // the warps' (max, sum) at the end of a piece
  __shared__ float4 m_w[R];            // their weights
  static_assert(kWarps <= 4, "a float4 of weights");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = a.c.page_size, cap = a.max_pages * P;
  const int G = a.nh / a.c.nkv, nv = a.c.nkv * n_groups;
  float* ws_part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + kPartOffset);

  pdl_trigger();
  pdl_wait();

  if (tid < 2) s_segbad[tid] = 0;
  int64_t begin;
  int count;
  const Shares shares = find_share<kWarps, kUnit>(a, nv, cap, s_scan, s_walk, &begin, &count);
  if (count == 0) {
    idle_requests<T, HD, kWarps * 32>(a, cap);
    return;
  }
  Walk cw = s_walk;  // the unit being computed
  Walk lw = cw;      // the unit being loaded

  // ---- loads: every lane looks up the page of the first key, or, where 16 keys may
  // lie in several pages, lane l that of key l % 16; then all lanes copy
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  const bool one_page = (P & (kKeys - 1)) == 0;
  int page_next = 0;  // page id that this lane looked up for unit lw
  auto lookup = [&](const Walk& w) {
    const int key = w.u * kUnit + warp * kKeys + (one_page ? 0 : lane & 15);
    if (key >= w.len) return 0;
    return a.table[(int64_t)w.r * a.table_stride + a.c.div.of(key)];
  };
  page_next = lookup(lw);
  constexpr int kRowsPer = 32 / C::kChunks;  // rows of one copy instruction
  const uint64_t policy = stream_policy();
  const int c = lane % C::kChunks, row0 = lane / C::kChunks;
  auto load_unit = [&](int stage) {
    const int key0 = lw.u * kUnit + warp * kKeys;
    const bool ok = (unsigned)page_next < (unsigned)a.c.n_pages;
    const uint32_t kdst = ring + stage * C::kStageBytes, vdst = kdst + kKeys * C::kRowBytes;
    if (one_page) {
      // (no shuffles of addresses: f32 rows of 128 6% less time, 16-bit rows 1%)
      const int in_page = key0 - a.c.div.of(key0) * P;
      const int live = ok ? lw.len - key0 : 0;
      int64_t off = 0;
      if (live > 0)
        off = (int64_t)page_next * a.c.page_stride + (int64_t)(in_page + row0) * a.c.row_stride + (int64_t)(lw.v / n_groups) * a.c.head_stride;
      const unsigned char* kp = static_cast<const unsigned char*>(a.c.k) + off * (int64_t)sizeof(T) + c * 16;
      const unsigned char* vp = static_cast<const unsigned char*>(a.c.v) + off * (int64_t)sizeof(T) + c * 16;
      const int64_t step = kRowsPer * a.c.row_stride * (int64_t)sizeof(T);
      if (lane == 0) s_bad[warp][stage] = key0 < lw.len && !ok;
#pragma unroll
      for (int j = 0; j < kKeys / kRowsPer; ++j) {
        const int row = j * kRowsPer + row0, bytes = row < live ? 16 : 0;
        const uint32_t d = (uint32_t)(row * C::kRowBytes + ((c ^ (row & 7)) << 4));
        cp16_stream(kdst + d, kp, bytes, policy);
        cp16_stream(vdst + d, vp, bytes, policy);
        kp += step;
        vp += step;
      }
    } else {
      const int key = key0 + (lane & 15);
      const int in_page = key - a.c.div.of(key) * P;
      int64_t off = 0;
      if (key < lw.len && ok)
        off = (int64_t)page_next * a.c.page_stride + (int64_t)in_page * a.c.row_stride + (int64_t)(lw.v / n_groups) * a.c.head_stride;
      const unsigned live = __ballot_sync(0xffffffffu, key < lw.len && ok);
      const bool any_bad = __any_sync(0xffffffffu, key < lw.len && !ok);
      if (lane == 0) s_bad[warp][stage] = any_bad;
#pragma unroll
      for (int j = 0; j < kKeys / kRowsPer; ++j) {
        const int row = j * kRowsPer + row0;
        const int64_t o = __shfl_sync(0xffffffffu, off, row) * (int64_t)sizeof(T) + c * 16;
        const int bytes = (live >> row) & 1 ? 16 : 0;
        const uint32_t d = (uint32_t)(row * C::kRowBytes + ((c ^ (row & 7)) << 4));
        cp16_stream(kdst + d, static_cast<const unsigned char*>(a.c.k) + o, bytes, policy);
        cp16_stream(vdst + d, static_cast<const unsigned char*>(a.c.v) + o, bytes, policy);
      }
    }
    walk_next<kUnit>(lw, a, nv, cap);
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
  // f32: this warp's softmax weights [key][query head]
  float* pbuf = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStageBytes) + warp * (kKeys * R);
  Piece piece[2];  // [1]: the one that starts in this share, [0]: the one that started before
  piece[0].rows = piece[1].rows = 0;
  const int g4 = lane >> 2, t4 = lane & 3;
  int stage = 0, seg = 0;
  // Q's words of the (request, head block) that comes next, loaded while the one
  // before is being joined; heads that the block does not have are zeros
  uint32_t qx[NH][kSteps][2];
  auto load_q = [&] {
    const int grp = cw.v % n_groups, rows = min(R, G - grp * R), head0 = cw.v / n_groups * G + grp * R;
    const T* qrow = static_cast<const T*>(a.q) + (int64_t)cw.r * a.q_stride + (int64_t)head0 * HD;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const uint32_t* q32 = reinterpret_cast<const uint32_t*>(qrow + (int64_t)(g4 + 8 * h) * HD);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) qx[h][s][j] = g4 + 8 * h < rows ? q32[s * 8 + j * 4 + t4] : 0u;
    }
  };
  load_q();
  for (int done = 0; done < count;) {
    const int r = cw.r, kvh = cw.v / n_groups, grp = cw.v % n_groups;
    const int rows = min(R, G - grp * R);
    const int head0 = kvh * G + grp * R;
    const bool from_start = cw.u == 0;
    const int seg_units = min(cw.units - cw.u, count - done);
    const bool whole = from_start && cw.u + seg_units == cw.units;
    const int seg_len = cw.len;
    const float wscale = weight_scale<T>(seg_len);
    const int first_unit = cw.u, all_units = cw.units;
    // Q as the B operand: two dims of a head (16-bit types), or a dim's tf32 halves
    uint32_t qb[NH][kSteps][2], ql[kF32 ? NH : 1][kF32 ? kSteps : 1][2];
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (kF32)
            split_tf32(qx[h][s][j], &qb[h][s][j], &ql[h][s][j]);
          else
            qb[h][s][j] = qx[h][s][j];
        }

    // the thread's query heads are 8 h + 2 t4 and the next, its keys g4 and g4 + 8,
    // its dims 16 n + g4 and 16 n + g4 + 8
    float o[kTiles][NH][4], m[NH][2], l[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      m[h][0] = m[h][1] = -INFINITY;
      l[h][0] = l[h][1] = 0.f;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) o[n][h][0] = o[n][h][1] = o[n][h][2] = o[n][h][3] = 0.f;
    }
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

      // S^T = K Q^T, in two chains of accumulators
      float sc[NH][4], se[NH][4];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[h][j] = se[h][j] = 0.f;
      {
        const int key = lane & 15, half = lane >> 4;
        const uint32_t kaddr = ks + key * C::kRowBytes;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t x[4];
          ldsm4(x, kaddr + (((s * 2 + half) ^ (key & 7)) << 4));
          if constexpr (!kF32) {
#pragma unroll
            for (int h = 0; h < NH; ++h) mma(s & 1 ? se[h] : sc[h], x, qb[h][s][0], qb[h][s][1], T());
          } else {
            // the small products in a chain of their own, so the large ones take
            // kSteps tensor-core adds
            uint32_t xh[4], xl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split_tf32(x[j], &xh[j], &xl[j]);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              mma(sc[h], xh, qb[h][s][0], qb[h][s][1], T());
              mma(se[h], xh, ql[h][s][0], ql[h][s][1], T());
              mma(se[h], xl, qb[h][s][0], qb[h][s][1], T());
            }
          }
        }
      }

      // online softmax in log2 units
      const int live = seg_len - ((first_unit + i) * kUnit + warp * kKeys);  // keys of this warp's 16
      float cf[NH][2];
      bool moved = false;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[h][j] = g4 + (j >> 1) * 8 < live ? (sc[h][j] + se[h][j]) * scale_log2 : -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float n = fmaxf(sc[h][j], sc[h][j + 2]);
          n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
          n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
          n = fmaxf(m[h][j], fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16)));
          // nothing seen so far: any finite reference gives p = 0
          const float z = n == -INFINITY ? 0.f : n;
          cf[h][j] = ex2(m[h][j] - z);
          moved |= n != m[h][j];
          m[h][j] = n;
          sc[h][j] = ex2(sc[h][j] - z);
          sc[h][j + 2] = ex2(sc[h][j + 2] - z);
          // the sums stay per thread until the end of the piece
          l[h][j] = fmaf(l[h][j], cf[h][j], sc[h][j] + sc[h][j + 2]);
        }
      }

      // O^T = O^T c + V^T P^T
      if constexpr (!kF32) {
        // Two MMAs, on the upper and on the lower halves of the weights: what is
        // lost of a weight, 2^-15 of it at most, lies far below the result's own
        // rounding, and 16-bit results can take the tensor core's truncating adds
        // in place.
        uint32_t p[NH][2], pl[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            split2(sc[h][2 * j], sc[h][2 * j + 1], wscale, &p[h][j], &pl[h][j], T());
            p[h][j] = transpose8(p[h][j]);
            pl[h][j] = transpose8(pl[h][j]);
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[n][h][j] *= cf[h][j & 1];
        }
        const int key = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
        const uint32_t vaddr = vs + key * C::kRowBytes;
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          uint32_t x[4];
          ldsm4t(x, vaddr + (((n * 2 + half) ^ (key & 7)) << 4));
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            mma(o[n][h], x, p[h][0], p[h][1], T());
            mma(o[n][h], x, pl[h][0], pl[h][1], T());
          }
        }
      } else {
        // The weights change their layout through shared memory.  The MMA's k
        // index t stands for key 2t, t + 4 for key 2t + 1 of eight, which spreads
        // a fragment's V values over the banks.
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float2*>(pbuf + (g4 + 8 * j) * R + 8 * h + 2 * t4) =
                make_float2(sc[h][2 * j] * wscale, sc[h][2 * j + 1] * wscale);
        __syncwarp();
        uint32_t ph[NH][2][2], pl[NH][2][2];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              split_tf32(__float_as_uint(pbuf[(k * 8 + t4 * 2 + j) * R + 8 * h + g4]), &ph[h][k][j], &pl[h][k][j]);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float f[NH][4], e[NH][4];
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) f[h][j] = e[h][j] = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t xh[4], xl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // a0: dim g4, first key; a1: dim g4 + 8; a2, a3: the same of the second key
              const int key = k * 8 + t4 * 2 + (j >> 1), chunk = n * 4 + (j & 1) * 2 + (g4 >> 2);
              split_tf32(lds32(vs + key * C::kRowBytes + ((chunk ^ (key & 7)) << 4) + (g4 & 3) * 4), &xh[j], &xl[j]);
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              mma(f[h], xh, ph[h][k][0], ph[h][k][1], T());
              mma(e[h], xh, pl[h][k][0], pl[h][k][1], T());
              mma(e[h], xl, ph[h][k][0], ph[h][k][1], T());
            }
          }
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][h][j] = fmaf(o[n][h][j], cf[h][j & 1], f[h][j] + e[h][j]);
        }
      }
      if (++stage == C::kStages) stage = 0;
    }
    // on to the next (request, head block)
    cw.u = all_units - 1;
    walk_next<kUnit>(cw, a, nv, cap);
    if (done < count) load_q();

    // the outputs go to the stage that every warp has just used, which is
    // filled again only after the barriers below
    const int used = (stage == 0 ? C::kStages : stage) - 1;
    float* m_out = reinterpret_cast<float*>(smem + used * C::kStageBytes);  // of warp 0
    constexpr int kNext = C::kStages * C::kStageBytes / 4;                  // to the next warp's

    // ---- join the warps; write the result or this share's partial
    float* mo = m_out + warp * kNext;
    __syncwarp();
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[h][j];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int head = 8 * h + 2 * t4 + j;
        if (g4 == 0) m_ml[warp * R + head] = make_float2(m[h][j], sum);
        if (head < rows) {
          // (dims of neighbouring head pairs are swapped in eights, for the banks)
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            mo[head * HD + ((n * 16 + g4) ^ (t4 * 8))] = o[n][h][j];
            mo[head * HD + ((n * 16 + 8 + g4) ^ (t4 * 8))] = o[n][h][j + 2];
          }
        }
      }
    if (bad && lane == 0) s_segbad[seg & 1] = 1;
    __syncthreads();
    const bool seg_bad = s_segbad[seg & 1] != 0;
    float* part = ws_part + (int64_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_floats(R, HD);
    if (tid < rows) {
      // the warps' weights of a row; of a whole piece with 1 / sum in them
      float mx = -INFINITY, sum = 0.f, c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, m_ml[k * R + tid].x);
      const float z = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = m_ml[k * R + tid];
        c[k] = ex2(ml.x - z);
        sum = fmaf(ml.y, c[k], sum);
      }
      if (!whole) {
        reinterpret_cast<float2*>(part)[tid] = make_float2(mx, seg_bad ? -1.f : sum);
      } else {
        const float f = sum == 0.f ? 0.f : 1.f / (sum * wscale);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) c[k] *= f;
        if (!seg_bad && a.lse) a.lse[(int64_t)r * a.nh + head0 + tid] = fmaf(mx, kLn2, logf(sum));
      }
      m_w[tid] = make_float4(c[0], c[1], c[2], c[3]);
    }
    __syncthreads();
    if (seg_bad && tid == 0) set_error(a.status, MINFER_ERR_POS_OOB);
    // four dims of a row at a time
    for (int i = tid; i < rows * HD / 4; i += kWarps * 32) {
      const int row = i / (HD / 4), d = (i - row * (HD / 4)) * 4;
      const float4 w = m_w[row];
      const float c[4] = {w.x, w.y, w.z, w.w};
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(m_out + k * kNext + row * HD + (d ^ (((row >> 1) & 3) * 8)));
        acc.x = fmaf(x.x, c[k], acc.x);
        acc.y = fmaf(x.y, c[k], acc.y);
        acc.z = fmaf(x.z, c[k], acc.z);
        acc.w = fmaf(x.w, c[k], acc.w);
      }
      if (!whole) {
        reinterpret_cast<float4*>(part + 2 * R)[i] = acc;
      } else if (!seg_bad) {
        T* dst = static_cast<T*>(a.o) + (int64_t)r * a.o_stride + (int64_t)head0 * HD + i * 4;
        store_as(dst, acc.x);
        store_as(dst + 1, acc.y);
        store_as(dst + 2, acc.z);
        store_as(dst + 3, acc.w);
      }
    }
    // flag of the next piece, free since the barrier above
    if (tid == 0) s_segbad[(seg + 1) & 1] = 0;
    __syncthreads();
    ++seg;
    if (!whole) {
      const int64_t first = begin + (done - seg_units) - first_unit;
      Piece& p = piece[from_start ? 1 : 0];
      p = Piece{r, head0, rows, shares.of(first), shares.of(first + all_units - 1), wscale};
    }
  }

  report_pieces<T, HD, R, kWarps>(a, piece, s_last, s_segbad, s_join, smem, kWarps * C::kStages * C::kStageBytes);
  idle_requests<T, HD, kWarps * 32>(a, cap);
}

template <typename T, int HD, int R>
int ctas(int num_sms) {
  return std::min(num_sms * Cfg<T, HD, R>::kCtas, kMaxShares);
}

// Runs f with the type, head size and head block of a call.
template <typename F>
auto with_config(int type, int hd, int G, F f) {
  auto sized = [&](auto t) {
    using T = decltype(t);
    if constexpr (sizeof(T) == 2)
      if (G > 8)
        return hd == 64 ? f.template operator()<T, 64, 16>() : f.template operator()<T, 128, 16>();
    return hd == 64 ? f.template operator()<T, 64, 8>() : f.template operator()<T, 128, 8>();
  };
  return type == MINFER_F32 ? sized(float()) : type == MINFER_F16 ? sized(__half()) : sized(__nv_bfloat16());
}

struct Launch {
  const PagedAttnArgs& a;
  int num_sms;
  cudaStream_t st;
  template <typename T, int HD, int R>
  cudaError_t operator()() {
    using C = Cfg<T, HD, R>;
    const int G = a.nh / a.c.nkv, n_groups = (G + R - 1) / R;
    const cudaError_t e = allow_smem<paged_attn_kernel<T, HD, R>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_kernel<T, HD, R>, dim3((unsigned)ctas<T, HD, R>(num_sms)), dim3(C::kWarps * 32), C::kSmem, st, a,
                      n_groups, a.scale * kLog2e);
  }
};
struct Bytes {
  int num_sms;
  template <typename T, int HD, int R>
  int64_t operator()() {
    return kPartOffset + (int64_t)ctas<T, HD, R>(num_sms) * 2 * part_floats(R, HD) * 4;
  }
};

}  // namespace

int64_t paged_attn_workspace(int G, int hd, int type, int num_sms) { return with_config(type, hd, G, Bytes{num_sms}); }

cudaError_t paged_attn_launch(const PagedAttnArgs& a, int type, int num_sms, cudaStream_t st) {
  return with_config(type, a.c.hd, a.nh / a.c.nkv, Launch{a, num_sms, st});
}

}  // namespace minfer
