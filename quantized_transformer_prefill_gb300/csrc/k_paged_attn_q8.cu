// k_paged_attn_q8.cu -- attention of one new token per request over a paged cache
// of Q8_0 rows (32 int8 codes c and one f16 scale d a block).
//
//   s_j = scale sum_b dk_jb sum_(i in b) q_i ck_ji,   p_j = exp(s_j - max),  j < len
//   o_i = sum_j (p_j dv_jb) cv_ji / sum_j p_j
//
// Shares, partials and their join are those of k_paged_attn.cu (paged_attn.cuh), and
// so are a warp's 16 keys at a time, its ring in shared memory and the m16n8 MMAs
// with keys and dims as the rows and 8 query heads as the columns.  What differs:
//
//  - Half the bytes a key, so twice the keys a second: a row is turned into MMA
//    operands in registers, which must cost little.  A code is exact in f16: one logic
//    operation puts two of them under the exponent of 1024, one packed subtraction
//    takes that off again.
//  - Q K^T: the sum over a block is an accumulator of its own, two k16 MMAs of f16;
//    the block's scale comes in as an f32 multiply-add.  Which 16 dims an MMA takes is
//    free as long as Q follows, so a lane reads 8 neighbouring codes of a key.  Q is
//    f16: exact, or times a power of two that brings the head's largest value to between
//    2^14 and 2^15 (bf16, and f32 as the sum of two), so that f16's steps of 2^-24 lose 2^-39 of
//    it at most.
//  - P V: a weight times the row's scale is what the MMAs take, per block of 32 dims, as
//    the sum of two f16 numbers (one would leave 2^-11 of the weight, more than a
//    result's own rounding).  They count in units of 2^-15 of a power of two that no scale
//    of the piece so far exceeds; when a larger one comes, the outputs are scaled down as
//    they are for a new maximum.  So none overflows, and what is lost lies 2^-22 below the
//    weight or 2^-39 below the largest scale (half a step of 2^-24 of these units, which are at
//    most twice that large).  The weights change from the layout of S^T to that
//    of P^T as f32, in two halves of 16 bits (transpose8); V's codes come transposed out
//    of ldmatrix, two neighbouring dims in a 16-bit element.
//  - With 16-bit queries and heads of 128 a warp takes two tiles of 16 keys at a time: two
//    chains of dependent steps instead of one.
//
// Measured: 64 requests of up to 4096 tokens, 28/4 heads of 128, bf16, 144 MB: 39 to 42 us, by
// the lengths (3.4 TB/s; f32 50 where bf16 takes 39: twice the MMAs in Q K^T, one tile at a time,
// sums added up outside the tensor core, 52 bytes of registers spilled); one of 131,071, 12/2 heads of 128, f16, 71 MB: 26 us; 33 of up to 2048, 14/2 heads
// of 64, f32: 13.4 us; one of 513: 7.2 us.  Of the first 13 us are start, uneven ends and
// join; of the rest the loads alone take 15 and the arithmetic alone 22, so issue slots bound
// it: a key and head block of 8 costs the same MMAs and conversions whether 7 or 8 of its
// columns are heads.  Four CTAs an SM with one tile took 51 us (registers spill), branches
// that leave out the masks of whole tiles 44, packed f16 products of weights and scales the
// same 42 and more with heads of 64.
#include <algorithm>
#include <type_traits>

#include "paged_attn.cuh"

namespace minfer {
namespace {

constexpr int R = 8;       // query heads of a head block

// KT: tiles of 16 keys that a warp takes at a time.
template <typename T, int HD, int KT>
struct Cfg {
  static constexpr int kKeys = 16 * KT;  // keys of a unit that one warp takes
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kBlocks = HD / 32;
  static constexpr int kChunks = HD / 16;         // 16-byte chunks of a row's codes
  static constexpr int kScaleBytes = kBlocks * 2;  // of a row
  static constexpr int kCodeBytes = kKeys * HD;    // of K or V of one warp
  static constexpr int kStageBytes = 2 * (kCodeBytes + kKeys * kScaleBytes);
  static constexpr int kWarps = 4;
  static constexpr int kCtas = HD == 64 ? 4 : 3;
  static constexpr int kUnit = kWarps * kKeys;  // keys of a unit
  static constexpr int kStatic = (int)sizeof(JoinShared<R>) + 512 + kWarps * (R * 8 + 4) + R * 16;
  static constexpr int kFit = (233472 / kCtas - 1024 - kStatic) / (kWarps * kStageBytes);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static_assert(kStages >= 2 && R * HD * 4 <= kStageBytes, "a warp's output fits the stage it has just used");
};

// The 16-byte chunk c of row `row` of a warp's K or V codes lies at this offset.
// K: a lane reads 8 bytes, the lanes of 4 rows together; V: ldmatrix reads the same
// chunk of 8 rows.  Either way all banks serve at once.
template <int HD>
__device__ __forceinline__ int k_at(int row, int c) {
  if constexpr (HD == 128) return row * 128 + ((c ^ ((row & 3) << 1)) << 4);
  return (row >> 1) * 128 + ((((row & 1) << 2 | c) ^ (row & 2)) << 4);
}
template <int HD>
__device__ __forceinline__ int v_at(int row, int c) {
  if constexpr (HD == 128) return row * 128 + ((c ^ (row & 7)) << 4);
  return (row >> 1) * 128 + ((((row & 1) << 2 | c) ^ ((row >> 1) & 3)) << 4);
}

// Codes of bytes 0 and 2 of x as two f16 numbers.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
  const uint32_t y = (x & 0x00FF00FFu) ^ 0x64806480u;  // 1024 + (c + 128)
  const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 z = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

template <int HD>
__device__ __forceinline__ void load_scales(float (&d)[HD / 32], uint32_t addr) {
  if constexpr (HD == 128) {
    uint32_t x, y;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr));
    const float2 a = halves(x), b = halves(y);
    d[0] = a.x, d[1] = a.y, d[2] = b.x, d[3] = b.y;
  } else {
    const float2 a = halves(lds32(addr));
    d[0] = a.x, d[1] = a.y;
  }
}
// one row's scales, or zeros
template <int HD>
__device__ __forceinline__ void cp_scales(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(HD / 16), "r"(live ? HD / 16 : 0) : "memory");
}

template <typename T, int HD, int KT>
__global__ void __launch_bounds__(Cfg<T, HD, KT>::kWarps * 32, Cfg<T, HD, KT>::kCtas)
    paged_attn_q8_kernel(const __grid_constant__ PagedAttnQ8Args a, int n_groups, float scale_log2) {
  using C = Cfg<T, HD, KT>;
  constexpr bool kF32 = C::kF32;
  constexpr int kWarps = C::kWarps, kUnit = C::kUnit, kBlocks = C::kBlocks, kKeys = C::kKeys;
  constexpr int kTiles = HD / 16;  // m16 tiles of the output
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ Walk s_walk;
  __shared__ uint8_t s_bad[kWarps][C::kStages];
  __shared__ int s_segbad[2], s_last[2];
  __shared__ JoinShared<R> s_join;
  __shared__ float2 m_ml[kWarps * R];  // the warps' (max, sum) at the end of a piece
  __shared__ float4 m_w[R];            // their weights
  __shared__ float m_unit[kWarps];     // what their outputs are in units of
  static_assert(kWarps == 4, "a float4 of weights");
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

  // ---- loads: lane l looks up the page of key l % kKeys and copies the scales of its rows;
  // then all lanes copy the codes
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  int page_next = 0;  // page id that this lane looked up for unit lw
  auto lookup = [&](const Walk& w) {
    const int key = w.u * kUnit + warp * kKeys + (lane & (kKeys - 1));
    if (key >= w.len) return 0;
    return a.table[(int64_t)w.r * a.table_stride + a.c.div.of(key)];
  };
  page_next = lookup(lw);
  constexpr int kRowsPer = 32 / C::kChunks;  // rows of one copy instruction
  const uint64_t policy = stream_policy();
  const int c = lane % C::kChunks, row0 = lane / C::kChunks;
  const bool whole_tiles = (P & 15) == 0;  // a tile lies in one page
  const int64_t step = kRowsPer * a.c.row_stride, off0 = (int64_t)row0 * a.c.row_stride + c * 16;
  auto load_unit = [&](int stage) {
    const uint32_t kdst = ring + stage * C::kStageBytes, vdst = kdst + C::kCodeBytes, sdst = vdst + C::kCodeBytes;
    const int key0 = lw.u * kUnit + warp * kKeys, key = key0 + (lane & (kKeys - 1));
    const int in_page = key - a.c.div.of(key) * P, head = n_groups == 1 ? lw.v : lw.v / n_groups;
    const bool wanted = key < lw.len, ok = wanted && (unsigned)page_next < (unsigned)a.c.n_pages;
    const bool any_bad = __any_sync(0xffffffffu, wanted && !ok);
    if (lane == 0) s_bad[warp][stage] = any_bad;
    int64_t off = 0, soff = 0;
    if (ok) {
      off = (int64_t)page_next * a.c.page_stride + (int64_t)in_page * a.c.row_stride + (int64_t)head * a.c.head_stride;
      soff = (int64_t)page_next * a.s.page_stride + (int64_t)in_page * a.s.row_stride + (int64_t)head * a.s.head_stride;
    }
    if constexpr (KT == 1) {
      cp_scales<HD>(sdst + lane * C::kScaleBytes, static_cast<const __half*>(lane < 16 ? a.s.k : a.s.v) + soff, ok);
    } else {
      cp_scales<HD>(sdst + lane * C::kScaleBytes, static_cast<const __half*>(a.s.k) + soff, ok);
      cp_scales<HD>(sdst + (kKeys + lane) * C::kScaleBytes, static_cast<const __half*>(a.s.v) + soff, ok);
    }
    const unsigned live = __ballot_sync(0xffffffffu, ok);
    if (whole_tiles) {
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        // the tile's first row, and from there in steps
        const int rows = (live >> (16 * t)) & 1 ? lw.len - key0 - 16 * t : 0;
        int64_t o = __shfl_sync(0xffffffffu, off, 16 * t);
        o = rows > 0 ? o + off0 : 0;
        const unsigned char* kp = static_cast<const unsigned char*>(a.c.k) + o;
        const unsigned char* vp = static_cast<const unsigned char*>(a.c.v) + o;
#pragma unroll
        for (int j = 0; j < 16 / kRowsPer; ++j) {
          const int row = 16 * t + j * kRowsPer + row0, bytes = j * kRowsPer + row0 < rows ? 16 : 0;
          cp16_stream(kdst + k_at<HD>(row, c), kp, bytes, policy);
          cp16_stream(vdst + v_at<HD>(row, c), vp, bytes, policy);
          kp += step;
          vp += step;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kKeys / kRowsPer; ++j) {
        const int row = j * kRowsPer + row0;
        const int64_t o = __shfl_sync(0xffffffffu, off, row) + c * 16;
        const int bytes = (live >> row) & 1 ? 16 : 0;
        cp16_stream(kdst + k_at<HD>(row, c), static_cast<const unsigned char*>(a.c.k) + o, bytes, policy);
        cp16_stream(vdst + v_at<HD>(row, c), static_cast<const unsigned char*>(a.c.v) + o, bytes, policy);
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
  Piece piece[2];  // [1]: the one that starts in this share, [0]: the one that started before
  piece[0].rows = piece[1].rows = 0;
  const int g4 = lane >> 2, t4 = lane & 3;
  int stage = 0, seg = 0;
  // Q's words of the (request, head block) that comes next, loaded while the one
  // before is being joined: of block b the lane's 8 dims 32 b + 8 t4 of head g4; heads
  // that the block does not have are zeros
  constexpr int kWords = 8 * (int)sizeof(T) / 4;
  uint32_t qx[kBlocks][kWords];
  auto load_q = [&] {
    const int grp = cw.v % n_groups, rows = min(R, G - grp * R), head0 = cw.v / n_groups * G + grp * R;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)cw.r * a.q_stride + (int64_t)(head0 + g4) * HD + 8 * t4);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int w = 0; w < kWords / 4; ++w) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (g4 < rows) x = q[b * (32 * (int)sizeof(T) / 16) + w];
        qx[b][4 * w] = x.x, qx[b][4 * w + 1] = x.y, qx[b][4 * w + 2] = x.z, qx[b][4 * w + 3] = x.w;
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
    const int first_unit = cw.u, all_units = cw.units;
    // Q as the B operand: MMA i of block b takes dims 8 t4 + 4 i + {0, 2} and {1, 3}
    uint32_t qb[kBlocks][2][2], ql[kF32 ? kBlocks : 1][2][2];
    float fac[2];  // scale, over the power of two in Q, of the thread's heads
    if constexpr (std::is_same<T, __half>::value) {
      fac[0] = fac[1] = scale_log2;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qb[b][i][0] = __byte_perm(qx[b][2 * i], qx[b][2 * i + 1], 0x5410);
          qb[b][i][1] = __byte_perm(qx[b][2 * i], qx[b][2 * i + 1], 0x7632);
        }
    } else {
      auto value = [&](int b, int i) {  // dim 8 t4 + i of the block
        if constexpr (kF32) return __uint_as_float(qx[b][i]);
        return __uint_as_float(i & 1 ? qx[b][i >> 1] & 0xFFFF0000u : qx[b][i >> 1] << 16);
      };
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(value(b, i)));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // times 2^up: the largest in [2^14, 2^15), if it is a finite number above 2^-110
      const int e = (int)(__float_as_uint(top) >> 23);  // 127 + its exponent
      const int up = e > 16 && e < 255 ? 14 + 127 - e : 0;
      const float mul0 = __uint_as_float((uint32_t)(127 + up / 2) << 23), mul1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = value(b, 4 * i + j) * mul0 * mul1, y = value(b, 4 * i + j + 2) * mul0 * mul1;
            qb[b][i][j] = pack_f16(x, y);
            if constexpr (kF32) {
              const float2 h = halves(qb[b][i][j]);
              ql[b][i][j] = pack_f16(x - h.x, y - h.y);
            }
          }
      const float f = scale_log2 / mul0 / mul1;
      fac[0] = __shfl_sync(0xffffffffu, f, 8 * t4);
      fac[1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
    }

    // the thread's query heads are 2 t4 and the next, its keys of a tile g4 and g4 + 8; its
    // dims of output tile n are 16 n + 2 g4 and the next
    float o[kTiles][4], m[2], l[2];
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    bool bad = false;
    // V's scales so far are at most top_d, a power of two; outputs are in units of top_d 2^-15
    float top_d = 0x1p-24f;

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
      const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + C::kCodeBytes, ss = vs + C::kCodeBytes;

      // S^T = K Q^T, block by block
      float sc[KT][4];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        float d0[kBlocks], d1[kBlocks];
        load_scales<HD>(d0, ss + (16 * t + g4) * C::kScaleBytes);
        load_scales<HD>(d1, ss + (16 * t + g4 + 8) * C::kScaleBytes);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint32_t x[2], y[2];  // 8 codes of key g4, and of key g4 + 8
          const int half = (t4 & 1) * 8;
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(ks + k_at<HD>(16 * t + g4, 2 * b + (t4 >> 1)) + half));
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(y[0]), "=r"(y[1]) : "r"(ks + k_at<HD>(16 * t + g4 + 8, 2 * b + (t4 >> 1)) + half));
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            const uint32_t k4[4] = {codes_f16(x[i2]), codes_f16(y[i2]), codes_f16(x[i2] >> 8), codes_f16(y[i2] >> 8)};
            mma(acc, k4, qb[b][i2][0], qb[b][i2][1], __half());
            if constexpr (kF32) mma(acc, k4, ql[b][i2][0], ql[b][i2][1], __half());
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[t][j] = b == 0 ? acc[j] * (j < 2 ? d0[b] : d1[b]) : fmaf(acc[j], j < 2 ? d0[b] : d1[b], sc[t][j]);
        }
      }

      // online softmax in log2 units
      const int live = seg_len - ((first_unit + i) * kUnit + warp * kKeys);  // keys of this warp's
      float cf[2];
      bool moved = false;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[t][j] = 16 * t + g4 + (j >> 1) * 8 < live ? sc[t][j] * fac[j & 1] : -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float n = fmaxf(sc[0][j], sc[0][j + 2]);
#pragma unroll
        for (int t = 1; t < KT; ++t) n = fmaxf(n, fmaxf(sc[t][j], sc[t][j + 2]));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
        n = fmaxf(m[j], fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16)));
        // nothing seen so far: any finite reference gives p = 0
        const float z = n == -INFINITY ? 0.f : n;
        cf[j] = ex2(m[j] - z);
        moved |= n != m[j];
        m[j] = n;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          sc[t][j] = ex2(sc[t][j] - z);
          sc[t][j + 2] = ex2(sc[t][j + 2] - z);
          sum += sc[t][j] + sc[t][j + 2];
        }
        // the sums stay per thread until the end of the piece
        l[j] = fmaf(l[j], cf[j], sum);
      }

      // V's scales of keys 2 t4, 2 t4 + 1, and 8 further, and the largest of all
      uint32_t vd[KT][4][kBlocks / 2];
      {
        __half2 top = __float2half2_rn(0.f);
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t at = ss + (kKeys + 16 * t + 2 * t4 + (j & 1) + (j >> 1) * 8) * C::kScaleBytes;
            if constexpr (HD == 128)
              asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(vd[t][j][0]), "=r"(vd[t][j][1]) : "r"(at));
            else
              vd[t][j][0] = lds32(at);
#pragma unroll
            for (int b = 0; b < kBlocks / 2; ++b) top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&vd[t][j][b])));
          }
        float d = fmaxf(__low2float(top), __high2float(top));
        d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, 1));
        d = fminf(fmaxf(d, __shfl_xor_sync(0xffffffffu, d, 2)), 65504.f);
        if (d > top_d) {  // (the same for all lanes)
          const float up = __uint_as_float((__float_as_uint(d) + 0x7FFFFFu) & 0xFF800000u);
          cf[0] *= top_d / up;
          cf[1] *= top_d / up;
          top_d = up;
          moved = true;
        }
      }
      if (!kF32 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][j] *= cf[j & 1];
      }
      const float unit = 0x1p15f / top_d;

      // O^T += V^T (P d)^T
      float add[kF32 ? kTiles : 1][4];
      if constexpr (kF32)
#pragma unroll
        for (int n = 0; n < kTiles; ++n) add[n][0] = add[n][1] = add[n][2] = add[n][3] = 0.f;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        // weights of the scales' keys under head g4
        float p[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = __float_as_uint(sc[t][2 * j] * unit), v = __float_as_uint(sc[t][2 * j + 1] * unit);
          const uint32_t hi = transpose8(__byte_perm(u, v, 0x7632)), lo = transpose8(__byte_perm(u, v, 0x5410));
          p[2 * j] = __uint_as_float(__byte_perm(lo, hi, 0x5410));
          p[2 * j + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint32_t w[2][2];  // the upper and the lower numbers
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 d0 = halves(vd[t][2 * j][b >> 1]), d1 = halves(vd[t][2 * j + 1][b >> 1]);
            const float x = p[2 * j] * (b & 1 ? d0.y : d0.x), y = p[2 * j + 1] * (b & 1 ? d1.y : d1.x);
            w[0][j] = pack_f16(x, y);
            const float2 h = halves(w[0][j]);
            w[1][j] = pack_f16(x - h.x, y - h.y);
          }
          // matrices: keys 0-7 and 8-15 of the block's first 16 dims, the same of its others
          uint32_t x[4];
          ldsm4t(x, vs + v_at<HD>(16 * t + (lane & 15), 2 * b + (lane >> 4)));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v4[4] = {codes_f16(x[2 * h]), codes_f16(x[2 * h] >> 8), codes_f16(x[2 * h + 1]), codes_f16(x[2 * h + 1] >> 8)};
            float(&to)[4] = kF32 ? add[kF32 ? 2 * b + h : 0] : o[2 * b + h];
            mma(to, v4, w[1][0], w[1][1], __half());
            mma(to, v4, w[0][0], w[0][1], __half());
          }
        }
      }
      if constexpr (kF32) {  // the tensor core's adds cut off, so f32 sums are added up here
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][j] = fmaf(o[n][j], cf[j & 1], add[n][j]);
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
    for (int j = 0; j < 2; ++j) {
      float sum = l[j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int head = 2 * t4 + j;
      if (g4 == 0) m_ml[warp * R + head] = make_float2(m[j], sum);
      if (head < rows) {
        // (dims of neighbouring head pairs are swapped in sixteens, for the banks)
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
          *reinterpret_cast<float2*>(mo + head * HD + ((n * 16 + 2 * g4) ^ ((t4 & 1) * 16))) = make_float2(o[n][j], o[n][j + 2]);
      }
    }
    if (lane == 0) m_unit[warp] = top_d * 0x1p-15f;
    if (bad && lane == 0) s_segbad[seg & 1] = 1;
    __syncthreads();
    const bool seg_bad = s_segbad[seg & 1] != 0;
    float* part = ws_part + (int64_t)(blockIdx.x * 2 + (from_start ? 1 : 0)) * part_floats(R, HD);
    if (tid < rows) {
      // the warps' weights of a row; of a whole piece with 1 / sum in them
      float mx = -INFINITY, sum = 0.f, w[4];
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, m_ml[k * R + tid].x);
      const float z = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = m_ml[k * R + tid];
        w[k] = ex2(ml.x - z);
        sum = fmaf(ml.y, w[k], sum);
      }
      if (!whole) {
        reinterpret_cast<float2*>(part)[tid] = make_float2(mx, seg_bad ? -1.f : sum);
      } else {
        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) w[k] *= f;
        if (!seg_bad && a.lse) a.lse[(int64_t)r * a.nh + head0 + tid] = fmaf(mx, kLn2, logf(sum));
      }
      m_w[tid] = make_float4(w[0] * m_unit[0], w[1] * m_unit[1], w[2] * m_unit[2], w[3] * m_unit[3]);
    }
    __syncthreads();
    if (seg_bad && tid == 0) set_error(a.status, MINFER_ERR_POS_OOB);
    // four dims of a row at a time
    for (int i = tid; i < rows * HD / 4; i += kWarps * 32) {
      const int row = i / (HD / 4), dim = (i - row * (HD / 4)) * 4;
      const float4 w4 = m_w[row];
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(m_out + k * kNext + row * HD + (dim ^ (((row >> 1) & 1) * 16)));
        acc.x = fmaf(x.x, w[k], acc.x);
        acc.y = fmaf(x.y, w[k], acc.y);
        acc.z = fmaf(x.z, w[k], acc.z);
        acc.w = fmaf(x.w, w[k], acc.w);
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
      p = Piece{r, head0, rows, shares.of(first), shares.of(first + all_units - 1), 1.f};
    }
  }

  report_pieces<T, HD, R, kWarps>(a, piece, s_last, s_segbad, s_join, smem, C::kSmem);
  idle_requests<T, HD, kWarps * 32>(a, cap);
}

template <int HD>
int ctas(int num_sms) {
  static_assert(Cfg<float, HD, 1>::kCtas == Cfg<__half, HD, 2>::kCtas, "the shares of a call are the same for every type");
  return std::min(num_sms * Cfg<float, HD, 1>::kCtas, kMaxShares);
}

template <typename T, int HD, int KT>
cudaError_t launch(const PagedAttnQ8Args& a, int num_sms, cudaStream_t st) {
  using C = Cfg<T, HD, KT>;
  const int G = a.nh / a.c.nkv, n_groups = (G + R - 1) / R;
  const cudaError_t e = allow_smem<paged_attn_q8_kernel<T, HD, KT>>(C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_q8_kernel<T, HD, KT>, dim3((unsigned)ctas<HD>(num_sms)), dim3(C::kWarps * 32), C::kSmem, st, a, n_groups,
                    a.scale * kLog2e);
}
template <typename T, int HD>
cudaError_t launch(const PagedAttnQ8Args& a, int num_sms, cudaStream_t st) {
  // Two tiles at a time, where the registers allow it (64 of up to 4096, 28/4 heads of 128,
  // bf16: 42 us against 48; heads of 64 and f32 the same either way).
  return launch<T, HD, HD == 128 && sizeof(T) == 2 ? 2 : 1>(a, num_sms, st);
}
template <typename T>
cudaError_t launch(const PagedAttnQ8Args& a, int num_sms, cudaStream_t st) {
  return a.c.hd == 64 ? launch<T, 64>(a, num_sms, st) : launch<T, 128>(a, num_sms, st);
}

}  // namespace

int64_t paged_attn_q8_workspace(int hd, int num_sms) {
  return kPartOffset + (int64_t)(hd == 64 ? ctas<64>(num_sms) : ctas<128>(num_sms)) * 2 * part_floats(R, hd) * 4;
}

cudaError_t paged_attn_q8_launch(const PagedAttnQ8Args& a, int type, int num_sms, cudaStream_t st) {
  return type == MINFER_F32 ? launch<float>(a, num_sms, st) : type == MINFER_F16 ? launch<__half>(a, num_sms, st) : launch<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace minfer
