// k_sample_stream.cu -- sampling (k_sample.cu has the definition) for many rows: one pass
// over all logits, then a CTA per row that looks at a few hundred of them again.
//
// The pass is bound by HBM.  A warp takes a block of 128 vectors of 16 bytes and leaves
// the maxima of its four parts and, where a row wants it (top-p without top-k, or no
// filter at all), the sum of its weights, relative to the block's own maximum.  Blocks begin
// at addresses that are multiples of 16: which tokens share one depends on the row's.
//
// A row's CTA finds its maximum and, for top-k, the k-th largest of the parts' maxima:
// at least k tokens reach it and hardly more, for the first k rarely share a part.  The
// parts that reach it are read again and what lies above goes to a list, which is cut,
// sorted and drawn from (finish_list).  Top-p alone takes the first 128 parts, and
// compares the list's weights with the row's.  Without a filter the
// blocks' sums name the block that is drawn from.  Rows that need more (a k past 640, a
// nucleus past the list, weights whose exponents are taken from x - max) are
// left to sample_kernel.
//
// 512 f32 rows of 151,936 (311 MB): greedy 64 us, plain 125, top-k 164, top-k and top-p 221,
// top-p 212, min-p 77, all of them mixed 158, of which the pass takes 70 (4.4 TB/s), the rows
// 30 and those left 52.  (Of the rows with a k an eighth have 1,000, which is left, and an eighth
// all tokens.)
#include <algorithm>

#include "sample.cuh"

namespace minfer {
namespace {

constexpr int kBlock = 128;            // vectors of a block
constexpr int kParts = kBlock / 32;    // its parts
constexpr int kBlockDown = 10;         // of its weights: up to 1,024 of them
constexpr int kMaxParts = 8192;        // of a row: their maxima are kept in shared memory
constexpr int kScanThreads = 256, kScanCopies = 8;
constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;
constexpr int kList = 2048;            // tokens that a CTA sorts
// Past it lists overflow (64 rows of 151,936: k = 500 38 us, left to sample_kernel 60; k =
// 1,000 109 and 61).
constexpr int kLargeK = 640;
constexpr int kGuess = 128;            // of top-p alone: parts whose tokens are looked at
constexpr float kFar = 8300.f;         // exponents of blocks reach a little past those of rows

// Scratch, written before it is read: [rows][parts] keys, [rows][blocks] sums and the
// whole parts of their exponents, the rows that are left and their number.
struct Scratch {
  uint32_t* keys;
  u64* sum;
  int* top;
  SampleLeft* list;
  int* count;
  int blocks;
};
template <typename T>
int blocks_of(int64_t vocab) {
  constexpr int E = Logits<T>::E;
  return (int)(((vocab + 2 * E - 2) / E + kBlock - 1) / kBlock);
}

template <typename T>
__device__ __forceinline__ uint4 load_vector(const T* x, int64_t i0, int64_t vocab) {
  if (Logits<T>::inside(i0, vocab)) return __ldg(reinterpret_cast<const uint4*>(x + i0));
  return Logits<T>::edge(x, i0, vocab);
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads) sample_scan_kernel(const __grid_constant__ SampleArgs a, Scratch w, PageDiv by_blocks) {
  constexpr int E = Logits<T>::E;
  __shared__ uint2 s_table[256 * kScanCopies];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint2* table = s_table + (lane & (kScanCopies - 1));
  pdl_trigger();
  fill_table(s_table, kScanCopies, threadIdx.x, kScanThreads);
  __syncthreads();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.count = 0;
  const int items = (int)a.rows * w.blocks;
  for (int item = blockIdx.x * (kScanThreads / 32) + warp; item < items; item += gridDim.x * (kScanThreads / 32)) {
    const int row = by_blocks.of(item), block = item - row * w.blocks;
    const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
    const int head = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    uint4 q[kParts];
#pragma unroll
    for (int j = 0; j < kParts; ++j) q[j] = load_vector(x, (int64_t)(block * kBlock + j * 32 + lane) * E - head, a.vocab);
    const Settings set = settings_of(a, row);
    uint32_t key[kParts];
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      float y[E];
      Logits<T>::unpack(q[j], y);
      float top = y[0];
#pragma unroll
      for (int e = 1; e < E; ++e) top = max_nan(top, y[e]);
      key[j] = __reduce_max_sync(0xffffffffu, key_of(top));
    }
    if (lane == 0) *reinterpret_cast<uint4*>(w.keys + (int64_t)item * kParts) = make_uint4(key[0], key[1], key[2], key[3]);
    if (set.skip || set.bad) continue;
    const float t = set.whole_row(), m = of_key(max(max(key[0], key[1]), max(key[2], key[3])));
    if (t == 0.f) continue;
    Weigh weigh;
    weigh.at(t, m, kBlockDown, kFar);
    u64 sum = 0;
    if (m > -INFINITY && m < INFINITY && !weigh.apart) {  // (an exponent that far weighs nothing, or the row is left)
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        float y[E];
        Logits<T>::unpack(q[j], y);
#pragma unroll
        for (int e = 0; e < E; ++e) sum += weigh.one<kScanCopies, false>(y[e], table);
      }
      sum = warp_sum(sum);
    }
    if (lane == 0) {
      w.sum[item] = sum;
      w.top[item] = weigh.top;
    }
  }
}

struct RowShared {
  u64 list[kList];
  u64 red[kRowWarps];
  uint2 table[256];
  int parts[kList];
  uint32_t lo[kRowWarps], hi[kRowWarps];
  int n, n_parts;
  int count[2][kRowWarps];
  int block, part;
  u64 target;
  float floor;
};

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 2) sample_rows_kernel(const __grid_constant__ SampleArgs a, Scratch w, int down) {
  constexpr int E = Logits<T>::E;
  extern __shared__ __align__(16) unsigned char smem[];
  RowShared& s = *reinterpret_cast<RowShared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + (sizeof(RowShared) + 15) / 16 * 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int parts = w.blocks * kParts;
  pdl_trigger();
  fill_table(s.table, 1, tid, kRowThreads);
  pdl_wait();
  const Settings set = settings_of(a, row);
  if (set.skip) return;
  if (set.bad) {
    if (tid == 0) set_error(a.status, MINFER_ERR_ARG);
    return;
  }
  const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
  const int head = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  auto load = [&](int v) { return load_vector(x, (int64_t)v * E - head, a.vocab); };
  auto write = [&](int token, float logprob) {
    a.token[row] = token;
    if (a.logprob) a.logprob[row] = logprob;
  };
  auto leave = [&](u64 whole) {
    if (tid == 0) w.list[atomicAdd(w.count, 1)] = SampleLeft{(int)row, whole};
  };

  // ---- the parts' maxima
  uint32_t lo_key = 0xFFFFFFFFu, hi_key = 0;
  for (int i = tid; i < parts / 4; i += kRowThreads) {
    const uint4 k4 = __ldcg(reinterpret_cast<const uint4*>(w.keys + row * parts) + i);
    reinterpret_cast<uint4*>(keys)[i] = k4;
    lo_key = min(min(lo_key, min(k4.x, k4.y)), min(k4.z, k4.w));
    hi_key = max(max(hi_key, max(k4.x, k4.y)), max(k4.z, k4.w));
  }
  lo_key = __reduce_min_sync(0xffffffffu, lo_key);
  hi_key = __reduce_max_sync(0xffffffffu, hi_key);
  if (lane == 0) s.lo[warp] = lo_key, s.hi[warp] = hi_key;
  if (tid == 0) s.block = s.part = 0x7FFFFFFF, s.n = s.n_parts = 0;
  __syncthreads();
  for (int i = 0; i < kRowWarps; ++i) lo_key = min(lo_key, s.lo[i]), hi_key = max(hi_key, s.hi[i]);
  const float m = of_key(hi_key);
  if (!(m < INFINITY)) {  // a NaN or +inf
    if (tid == 0) set_error(a.status, MINFER_ERR_ARG);
    return;
  }
  if (m == -INFINITY) {
    if (tid == 0) write(-1, -INFINITY);
    return;
  }

  // the first part whose maximum is `least` or more, and its first logit of that size
  auto first_of = [&](float least, float* value) {
    const uint32_t k = key_of(least);
    for (int i = tid; i < parts; i += kRowThreads)
      if (keys[i] >= k) {
        atomicMin(&s.part, i);
        break;
      }
    __syncthreads();
    const int i0 = (s.part * 32 + lane) * E - head;  // (every warp does the same)
    float y[E];
    Logits<T>::unpack(load(s.part * 32 + lane), y);
    int id = 0x7FFFFFFF;
    *value = 0.f;
#pragma unroll
    for (int e = E - 1; e >= 0; --e)
      if (y[e] >= least && y[e] > -INFINITY) id = i0 + e, *value = y[e];
    const int best = __reduce_min_sync(0xffffffffu, id);
    *value = __shfl_sync(0xffffffffu, *value, __ffs(__ballot_sync(0xffffffffu, id == best)) - 1);
    return best;
  };
  float value;
  if (set.greedy) {
    const int id = first_of(m, &value);
    if (tid == 0) write(id, 0.f);
    return;
  }

  Weigh wf, wd;
  wf.at(set.sharp, m, down);
  wd.at(set.temp, m, down);
  if (tid == kRowThreads - 32) s.floor = floor_of(set, m);
  const float t = set.whole_row();
  const bool by_p = set.k == 0 && set.top_p < 1.f, plain = t > 0.f && !by_p;
  u64 whole = 0;
  if (t > 0.f) {
    const Weigh& wt = by_p ? wf : wd;
    if (wt.apart) {
      leave(0);
      return;
    }
    const uint32_t none = key_of(fmaxf(wt.lim, kLowest));
    // a block's sum in the row's units, which are larger by `shift` binary places
    auto sum_of = [&](int i, u64* sum, int* shift) {
      *sum = 0;
      *shift = 1;
      if (i >= w.blocks) return (u64)0;
      const uint4 k4 = reinterpret_cast<const uint4*>(keys)[i];
      if (max(max(k4.x, k4.y), max(k4.z, k4.w)) < none) return (u64)0;
      *sum = __ldcg(w.sum + row * w.blocks + i);
      *shift = wt.top - __ldcg(w.top + row * w.blocks + i) + down - kBlockDown;  // (rows are longer than blocks)
      return *shift < 64 ? ((*sum >> (*shift - 1)) + 1) >> 1 : 0;
    };
    u64 sum;
    int shift;
    for (int base = 0; base < w.blocks; base += kRowThreads) {
      u64 v[1] = {sum_of(base + tid, &sum, &shift)};
      whole += scan_all<kRowThreads, 1>(s.red, v);
    }
    if (plain && set.u > 0.f) {
      // the block that is drawn from, and where in its own units
      bool rest;
      const u64 target = times(whole, set.u, &rest);
      u64 before = 0;
      for (int base = 0; base < w.blocks; base += kRowThreads) {
        const u64 own = sum_of(base + tid, &sum, &shift);
        u64 v[1] = {own};
        const u64 all = scan_all<kRowThreads, 1>(s.red, v);
        const u64 from = before + v[0] - own;
        if (from <= target && target < from + own) {
          s.block = base + tid;
          s.target = min((target - from) << shift, sum - 1);
        }
        before += all;
      }
    }
  }

  if (plain) {
    __syncthreads();
    const float floor_x = s.floor;
    if (set.u == 0.f) {
      const int id = first_of(floor_x, &value);
      if (tid == 0) write(id, log_share(wd, set.temp, value, wd.one<1>(value, s.table), whole));
      return;
    }
    // a warp per part of the block; weights in the block's units
    const uint4 k4 = reinterpret_cast<const uint4*>(keys)[s.block];
    Weigh wb;
    wb.at(set.temp, of_key(max(max(k4.x, k4.y), max(k4.z, k4.w))), kBlockDown, kFar);
    const int v = s.block * kBlock + warp * 32 + lane;
    float y[E];
    u64 one[E], sum = 0;
    if (warp < kParts) {
      Logits<T>::unpack(load(v), y);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        one[e] = y[e] >= floor_x ? wb.one<1, false>(y[e], s.table) : 0;
        sum += one[e];
      }
      const u64 all = warp_sum(sum);
      if (lane == 0) s.red[warp] = all;
    }
    __syncthreads();
    if (warp < kParts) {
      u64 total = 0, from = 0;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        if (j < warp) from += s.red[j];
        total += s.red[j];
      }
      const u64 target = min(s.target, total - 1), incl = warp_scan(sum, lane) + from;
      if (incl - sum <= target && target < incl) {
        u64 at = incl - sum;
        bool hit = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          at += one[e];
          if (!hit && target < at) {
            hit = true;
            write(v * E - head + e, log_share(wd, set.temp, y[e], wd.one<1>(y[e], s.table), whole));
          }
        }
      }
    }
    return;
  }

  // ---- the candidates
  // A key that at least `aim` parts reach, and few more: the warps try a threshold each.
  auto bound_of = [&](int aim) {
    uint32_t lo = lo_key, over = hi_key + 1;
    for (int turn = 0; over - lo > 1; turn ^= 1) {
      const uint32_t range = over - lo;
      auto at = [&](int i) { return max(1u, (range >> 4) * i + ((range & 15) * i >> 4)); };  // i / 16 of the way
      const uint32_t mid = lo + at(warp + 1);
      int c = 0;
      for (int i = lane; i < parts / 4; i += 32) {
        const uint4 k4 = reinterpret_cast<const uint4*>(keys)[i];
        c += (k4.x >= mid) + (k4.y >= mid) + (k4.z >= mid) + (k4.w >= mid);
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) s.count[turn][warp] = c;
      __syncthreads();
      c = s.count[turn][lane & (kRowWarps - 1)];
      // how many thresholds are reached by enough parts, and by how many the last of them
      const int n = __popc(__ballot_sync(0xffffffffu, c >= aim) & ((1u << kRowWarps) - 1));
      c = __shfl_sync(0xffffffffu, c, max(n - 1, 0));
      over = n < kRowWarps ? lo + at(n + 1) : over;
      if (n > 0) lo += at(n);
      if (n > 0 && c <= aim + aim / 8 + 2) break;
    }
    return fmaxf(of_key(lo), kLowest);  // -inf is no candidate
  };
  static_assert(kRowWarps == 16, "sixteenths");
  if (set.k > min(parts, kLargeK)) {
    leave(whole);
    return;
  }
  const float b = set.k > 0 || by_p ? bound_of(set.k > 0 ? set.k : min(parts, kGuess)) : kLowest;
  __syncthreads();
  const float floor_x = s.floor;
  const float from = set.k > 0 && set.top_p < 1.f ? b : fmaxf(b, floor_x);
  const uint32_t from_key = key_of(from);
  for (int i = tid; i < parts; i += kRowThreads)
    if (keys[i] >= from_key) {
      const int at = atomicAdd(&s.n_parts, 1);
      if (at < kList) s.parts[at] = i;
    }
  __syncthreads();
  if (s.n_parts > kList) {
    leave(whole);
    return;
  }
  constexpr int kFlight = 4;
  const int last = (head + (int)a.vocab) / (32 * E);  // parts before it, but the first, lie inside the row
  for (int j0 = warp; j0 < s.n_parts; j0 += kRowWarps * kFlight) {
    uint4 q[kFlight];
    int part[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int at = j0 + j * kRowWarps;
      part[j] = at < s.n_parts ? s.parts[at] : -1;
      if (part[j] > 0 && part[j] < last)
        q[j] = __ldg(reinterpret_cast<const uint4*>(x - head) + (part[j] * 32 + lane));
      else if (part[j] >= 0)
        q[j] = load(part[j] * 32 + lane);
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (part[j] < 0) break;
      float y[E];
      Logits<T>::unpack(q[j], y);
      uint32_t hits = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) hits |= (uint32_t)(y[e] >= from) << e;
      if (hits) {  // of a lane or two
        int to = atomicAdd(&s.n, __popc(hits));
        const int i0 = (part[j] * 32 + lane) * E - head;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (hits >> e & 1) {
            if (to < kList) s.list[to] = by_logit(y[e], i0 + e);
            ++to;
          }
      }
    }
  }
  __syncthreads();
  const int n = s.n;
  if (n > kList || !finish_list<kRowThreads, kList, 1>(s.list, s.red, n, set, wf, wd, s.table, floor_x, whole, by_p && from > floor_x && from > kLowest, write))
    leave(whole);
}

template <typename T>
int64_t bytes_of(int64_t rows, int64_t vocab, Scratch* w, unsigned char* base) {
  const int64_t blocks = blocks_of<T>(vocab);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return base + from;
  };
  unsigned char* const keys = take(rows * blocks * kParts * 4);
  unsigned char* const sum = take(rows * blocks * 8);
  unsigned char* const top = take(rows * blocks * 4);
  unsigned char* const list = take(rows * (int64_t)sizeof(SampleLeft));
  unsigned char* const count = take(4);
  if (w)
    *w = Scratch{reinterpret_cast<uint32_t*>(keys), reinterpret_cast<u64*>(sum), reinterpret_cast<int*>(top), reinterpret_cast<SampleLeft*>(list),
                 reinterpret_cast<int*>(count), (int)blocks};
  return at;
}

template <typename T>
cudaError_t stream_typed(const SampleArgs& a, int type, int num_sms, void* scratch, cudaStream_t st) {
  Scratch w;
  bytes_of<T>(a.rows, a.vocab, &w, static_cast<unsigned char*>(scratch));
  const int64_t items = a.rows * w.blocks;
  constexpr int kWarps = kScanThreads / 32;
  const int ctas = (int)std::min<int64_t>((items + kWarps - 1) / kWarps, num_sms * 8);
  cudaError_t e = launch_pdl(sample_scan_kernel<T>, dim3(ctas), dim3(kScanThreads), 0, st, a, w, PageDiv(w.blocks));
  if (e != cudaSuccess) return e;
  int down = 1;
  while ((1ll << down) < a.vocab) ++down;
  constexpr int kFixed = (int)((sizeof(RowShared) + 15) / 16 * 16);
  e = allow_smem<sample_rows_kernel<T>>(kFixed + kMaxParts * 4);
  if (e != cudaSuccess) return e;
  e = launch_pdl(sample_rows_kernel<T>, dim3((unsigned)a.rows), dim3(kRowThreads), kFixed + w.blocks * kParts * 4, st, a, w, down);
  if (e != cudaSuccess) return e;
  return sample_launch(a, type, num_sms, st, w.list, w.count);
}

template <typename F>
auto typed(int type, F f) {
  return type == MINFER_F32 ? f(float()) : type == MINFER_F16 ? f(__half()) : f(__nv_bfloat16());
}

}  // namespace

int64_t sample_stream_bytes(int64_t rows, int64_t vocab, int type, int num_sms) {
  return typed(type, [&](auto t) -> int64_t {
    using T = decltype(t);
    // While the clusters that keep the rows fit the GPU at once, there is nothing to stream
    // (nor for rows that are short): f32, settings of all kinds, device time: 16 rows of
    // 151,936 38 us against 51, 256 161 against 120; 256 of 10,007 66 against 83.
    if (vocab * (int64_t)sizeof(T) < (64 << 10) || rows * sample_cluster(vocab, type) <= 2 * num_sms) return 0;
    if (vocab / 32 > (int64_t)kMaxParts * Logits<T>::E) return 0;
    const int blocks = blocks_of<T>(vocab);
    if (blocks * kParts > kMaxParts || rows * blocks > (1ll << 30)) return 0;
    return bytes_of<T>(rows, vocab, nullptr, nullptr);
  });
}

cudaError_t sample_stream_launch(const SampleArgs& a, int type, int num_sms, void* scratch, cudaStream_t st) {
  return typed(type, [&](auto t) { return stream_typed<decltype(t)>(a, type, num_sms, scratch, st); });
}

}  // namespace minfer
