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
// numbers: 2^t is put together from a table of 2^(j/256) and a quadratic (to 2^-29 of
// itself, see Weigh) and shifted to a fixed point that is the same for the whole row; their
// sums are exact in 64 bits and do not depend on who adds what first.
//
// Many rows are streamed once (k_sample_stream.cu); this file: rows that a thread-block
// cluster keeps.  A CTA copies its slice of the row into shared memory (cp.async, all of it
// on its way at once; a thread reads what it has copied itself), so further passes cost no
// memory traffic.  What lies behind the room in shared memory is read again from L2.
//
// Most rows need two or three exchanges in the cluster: (1) the maximum, and a bound
// under which nothing can be among the first k, from the maxima of half threads; (2) with
// top-p and no top-k, the sum of all weights; (3) what lies above the bound goes to the
// first CTA, which sorts it (a few hundred tokens), cuts it by the three filters, sorts
// what is left by id and draws.  Rows for which that list overflows or does not reach (no
// filter, high temperatures, large k) go the wide way: a histogram brackets the border of a
// filter until a list holds what lies between, and the draw goes segment by segment.
//
// Measured, f32 rows of 151,936: one with top-k and top-p 13 to 17 us, by its settings, four
// with top-p alone 25; of 200,001, which shared memory does not hold, one 28 to 39 us, eight 31
// without a filter, 60 with top-p and 102 with top-k and top-p:
// a chain of memory round trip, barriers of the cluster (1 us each) and a sort.  65 bf16
// rows of 150,001 with top-p alone and temperatures up to 1.3, whose nuclei hold thousands of
// tokens, 93 us (0.2 TB/s): the longest row sets the time.  It weighs all of its tokens, adds
// them to a histogram, weighs those above the border exactly, and again to draw, each 10 to
// 25 us of issue slots with two CTAs an SM, and barriers.
#include <algorithm>

#include "sample.cuh"

namespace minfer {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 512;    // tokens between which a border is looked for, sorted by the first CTA
constexpr int kShort = 2048;  // tokens that a row's only CTA sorts; of a cluster kList, for they come one by one
constexpr int kPicked = 32;   // tokens that a lane picks out of its vectors, at most
constexpr int kGuess = 64;    // of top-p alone: tokens that the first bound aims at
constexpr int kCopies = 4;    // of the table, against bank conflicts
constexpr int kSlots = 5;     // numbers of one exchange
constexpr int kBins = 1024;   // of a histogram: four to a thread
constexpr int kRoom = 76800;  // bytes of a row's slice that a CTA keeps, at most: two CTAs fit an SM

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
__device__ __forceinline__ void get4(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ int peer_get(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct SampleShared {
  uint2 table[256 * kCopies];
  u64 list[kList];
  uint32_t bins[kBins];            // tokens, or their weights as shares of 2^31
  union {
    uint16_t picked[kWarps][kPicked][32];  // where they lie in the segment
    u64 longer[kShort];                // a list of the short way
  };
  u64 ex[2][kSlots][kMaxCluster];  // what the CTAs of the cluster tell, by turns
  u64 red[kWarps][kSlots];
  u64 part[kWarps];                // of one warp's segment
  u64 found;                       // a token that one CTA told all: logit bits, id
  float floor;                     // logits below are out
  int count;                       // entries of list
  int local, base;                 // of what this CTA adds to it: how many, from where on
  int edge[2];                     // bins between which a border lies
  u64 before;                      // tokens in the bins before
  uint32_t keys[2][kWarps];
};

template <typename A>
constexpr int kLength = std::extent<typename std::remove_reference<A>::type>::value;

// What a CTA has of a row.
template <typename T>
struct Slice {
  static constexpr int E = Logits<T>::E;
  int64_t first;      // logit (of the first CTA maybe below 0) at which vector 0 begins
  const uint4* far;   // vector 0 in global memory
  const uint4* near;  // and in shared memory, where the first `kept` and the last lie
  int vectors, kept;
  int seg;            // vectors of a warp, a multiple of 32

  __device__ __forceinline__ void load(int v, float (&y)[E]) const {
    uint4 q;
    if (v < kept)
      q = near[v];
    else
      q = v == vectors - 1 ? near[kept] : __ldg(far + v);
    Logits<T>::unpack(q, y);
  }
  // This warp's vectors, 32 at a time: f(values, id of the first), by all lanes; a lane
  // without a vector has -inf.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, end = min((warp + 1) * seg, vectors);
    for (int b = warp * seg; b < end; b += 32) {
      float y[E];
      if (b + lane < end) {
        load(b + lane, y);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = -INFINITY;
      }
      f(y, (int)first + (b + lane) * E);
    }
  }
  // The same where some lane has a logit of `least` or more.
  template <typename F>
  __device__ __forceinline__ void each_from(float least, F f) const {
    each([&](const float (&y)[E], int i0) {
      float top = y[0];
#pragma unroll
      for (int e = 1; e < E; ++e) top = fmaxf(top, y[e]);
      if (__any_sync(0xffffffffu, top >= least)) f(y, i0);
    });
  }
};

// Adds up (or, of those in kMax, takes the largest of) N numbers of every thread of the
// cluster; before, own: the first of them, of the CTAs before this one and its own.
template <int N, int kMax = 0>
__device__ __forceinline__ void exchange(SampleShared& s, u64 (&v)[N], uint32_t rank, int cluster, int& turn, u64* before = nullptr, u64* own = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (kMax >> i & 1)
      v[i] = __reduce_max_sync(0xffffffffu, (unsigned)v[i]);
    else
      v[i] = warp_sum(v[i]);
    if (lane == 0) s.red[warp][i] = v[i];
  }
  __syncthreads();
  if (tid < N * cluster) {
    const int i = tid % N;
    u64 t = 0;
    for (int w = 0; w < kWarps; ++w) t = kMax >> i & 1 ? max(t, s.red[w][i]) : t + s.red[w][i];
    put(peer(&s.ex[turn][i][rank], tid / N), t);
  }
  cluster_sync();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0;
    if (i == 0 && before) *before = 0;
    for (int c = 0; c < cluster; ++c) {
      const u64 x = s.ex[turn][i][c];
      v[i] = kMax >> i & 1 ? max(v[i], x) : v[i] + x;
      if (i == 0 && before && c < (int)rank) *before += x;
    }
    if (i == 0 && own) *own = s.ex[turn][0][rank];
  }
  turn ^= 1;
}

// A row in the hands of a cluster.
template <typename T>
struct Wide {
  static constexpr int E = Logits<T>::E;
  SampleShared& s;
  const Slice<T> r;
  const uint2* table;
  const uint32_t rank;
  const int cluster;
  int turn;
  float xb;  // kept: what is larger, and of its equals the ids up to idb
  int idb;
  int n_picked, most;  // by this lane, by any of the warp; most below 0: nothing has been picked

  // Every lane picks the logits of `least` and more out of its vectors; sums then go over
  // these.
  __device__ __forceinline__ void pick(float least) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    const int first = (int)r.first + warp * r.seg * E;
    r.each_from(least, [&](const float (&y)[E], int i0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (y[e] >= least) {
          if (n < kPicked) s.picked[warp][n][lane] = (uint16_t)(i0 + e - first);
          ++n;
        }
    });
    const int top = __reduce_max_sync(0xffffffffu, n);
    // (all of the slice is in shared memory, and a segment's places fit 16 bits)
    const bool over = top > kPicked || r.kept < r.vectors || r.seg * E > 65536;
    u64 v[1] = {over};
    exchange<1, 1>(s, v, rank, cluster, turn);
    n_picked = n;
    most = v[0] ? -1 : top;
  }
  // f(logits, ids) for what may be `least` or more, by all lanes; one of them at a time, or, where
  // whole vectors are gone through, E, whose chains of steps overlap
  template <typename F>
  __device__ __forceinline__ void each(float least, F f) const {
    if (most >= 0) {
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      const T* const seg = reinterpret_cast<const T*>(r.near + warp * r.seg);
      const int first = (int)r.first + warp * r.seg * E;
      for (int i = 0; i < most; ++i) {
        float x[1] = {-INFINITY};
        int id[1] = {0};
        if (i < n_picked) {
          const int at = s.picked[warp][i][lane];
          if constexpr (sizeof(T) == 4)
            x[0] = seg[at];
          else if constexpr (std::is_same<T, __half>::value)
            x[0] = __half2float(seg[at]);
          else
            x[0] = __bfloat162float(seg[at]);
          id[0] = first + at;
        }
        f(x, id);
      }
    } else {
      r.each_from(least, [&](const float (&y)[E], int i0) {
        int id[E];
#pragma unroll
        for (int e = 0; e < E; ++e) id[e] = i0 + e;
        f(y, id);
      });
    }
  }

  // (nothing is compared with xb before there is a border: xb is -inf)
  __device__ __forceinline__ bool kept(float x, int id) const { return x >= xb && (x != xb || id <= idb); }

  // The first token, in the order of ids, at which the sum of what weigh(logits, ids, weights)
  // gives exceeds target(whole): to all threads of the cluster, with the whole.  Logits below `least`
  // weigh nothing.
  template <typename W, typename F>
  __device__ __forceinline__ u64 locate(float least, W weigh, F target, u64* whole) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 mine = 0;
    each(least, [&](const auto& y, const auto& id) {
      constexpr int N = kLength<decltype(y)>;
      u64 w[N];
      weigh(y, id, w);
#pragma unroll
      for (int e = 0; e < N; ++e) mine += w[e];
    });
    u64 v[1] = {mine}, before, own;
    exchange<1>(s, v, rank, cluster, turn, &before, &own);
    *whole = v[0];
    const u64 t = target(v[0]);
    if (t >= before && t < before + own) {  // in this CTA: s.red holds its warps' sums
      int at = 0;
      for (; t >= before + s.red[at][0]; ++at) before += s.red[at][0];
      // the warps share the segment of warp `at`, `per` times 32 vectors each
      const int v0 = at * r.seg, end = min(v0 + r.seg, r.vectors), per = (r.seg / 32 + kWarps - 1) / kWarps;
      const int mine0 = v0 + warp * per * 32, mine1 = min(mine0 + per * 32, end);
      auto vector = [&](int b, float (&y)[E], u64 (&w)[E]) {  // of this lane, in the 32 from b on; returns its sum
        int id[E];
        if (b + lane < end) r.load(b + lane, y);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (b + lane >= end) y[e] = -INFINITY;
          id[e] = (int)r.first + (b + lane) * E + e;
        }
        weigh(y, id, w);
        u64 sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) sum += w[e];
        return sum;
      };
      float y[E];
      u64 w[E], sum = 0;
      for (int b = mine0; b < mine1; b += 32) sum += vector(b, y, w);
      sum = warp_sum(sum);
      if (lane == 0) s.part[warp] = sum;
      __syncthreads();
      for (int i = 0; i < warp; ++i) before += s.part[i];
      if (t >= before && t < before + s.part[warp]) {
        for (int b = mine0; b < mine1; b += 32) {
          const u64 own_sum = vector(b, y, w);
          const u64 incl = warp_scan(own_sum, lane) + before;
          if (incl - own_sum <= t && t < incl) {
            u64 sofar = incl - own_sum;
            bool hit = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              sofar += w[e];
              if (!hit && t < sofar) {
                hit = true;
                for (int c = 0; c < cluster; ++c) put(peer(&s.found, c), (u64)__float_as_uint(y[e]) << 32 | (uint32_t)((int)r.first + (b + lane) * E + e));
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
  }

  // Entries for the first CTA's list: a CTA collects its own, in place of the bins (its own
  // list, if there is no other CTA), and hands them over together, for a word of another
  // CTA's is far away.  add: by any thread; hand_over: by all, behind the last add; the
  // entries are there behind the next barrier of the cluster.
  __device__ __forceinline__ u64* own_list(u64* list) const { return cluster == 1 ? list : reinterpret_cast<u64*>(s.bins); }
  __device__ __forceinline__ void add(u64* own, int entries, u64 entry) const {
    const int at = atomicAdd(&s.local, 1);
    if (at < entries) own[at] = entry;
  }
  __device__ __forceinline__ void hand_over(u64* list, int entries) const {
    __syncthreads();
    const int n = s.local;
    if (threadIdx.x == 0) s.base = peer_add(peer(&s.count, 0), n);
    __syncthreads();  // s.base; and all have read s.local
    if (threadIdx.x == 0) s.local = 0;
    if (cluster == 1) return;
    const u64* const own = own_list(list);
    for (int i = threadIdx.x; i < n && s.base + i < entries; i += kThreads) put(peer(&list[s.base + i], 0), own[i]);
  }

  // Logits of `from` and more, to the first CTA's list, in any order; returns how many.
  __device__ __forceinline__ int gather(float from, u64* list, int entries) {
    u64* const own = own_list(list);
    r.each_from(from, [&](const float (&y)[E], int i0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (y[e] >= from) add(own, entries, by_logit(y[e], i0 + e));
    });
    hand_over(list, entries);
    cluster_sync();
    return peer_get(peer(&s.count, 0));
  }

  // The nth token (from 1 on), in the order of ids, that is kept and lies in [lo, hi].  (The
  // rare cases are functions of their own.)
  __device__ __noinline__ u64 nth_of(float lo, float hi, u64 nth) {
    u64 sum;
    return locate(lo,
                  [&](const auto& y, const auto& id, auto& w) {
                    constexpr int N = kLength<decltype(y)>;
#pragma unroll
                    for (int e = 0; e < N; ++e) w[e] = y[e] >= lo && y[e] <= hi && kept(y[e], id[e]);
                  },
                  [&](u64) { return nth - 1; }, &sum);
  }
  __device__ __forceinline__ u64 nth(float lo, float hi, u64 n) {
    Wide w = *this;  // (its address is taken: this one stays in registers)
    const u64 found = w.nth_of(lo, hi, n);
    turn = w.turn;
    return found;
  }

  // What is left of `cut` when the border is one value: of its equals the first ones.
  template <bool kMass>
  __device__ __forceinline__ void cut_equals(float at, u64 rest, const Weigh& wf) {
    const u64 w = kMass ? wf.one<kCopies>(at, table) : 1;
    const u64 found = nth(at, at, (rest + w - 1) / w);
    xb = at;
    idb = (int)(uint32_t)found;
  }

  // The same as `cut` below by halving, on exact sums alone: for borders that a histogram of
  // rounded weights does not place.
  template <bool kMass>
  __device__ __noinline__ void bisect(u64 goal, float m, const Weigh& wf) {
    uint32_t lo = key_of(kLowest), hi = key_of(m) + 1;  // `goal` is reached at lo, not at hi
    u64 f_hi = 0;
    for (bool first = true; first || hi - lo > 1; first = false) {
      const uint32_t mid = first ? lo : lo + (hi - lo) / 2;
      const float t = of_key(mid);
      u64 v[1] = {0};
      each(t, [&](const auto& y, const auto& id) {
        constexpr int N = kLength<decltype(y)>;
        u64 w[N];
        if constexpr (kMass) wf.all<kCopies>(y, w, table);
#pragma unroll
        for (int e = 0; e < N; ++e) v[0] += y[e] >= t && kept(y[e], id[e]) ? (kMass ? w[e] : 1) : 0;
      });
      exchange<1>(s, v, rank, cluster, turn);
      if (v[0] >= goal)
        lo = mid;
      else if (first)
        return;  // all of it is kept
      else
        hi = mid, f_hi = v[0];
    }
    cut_equals<kMass>(of_key(lo), goal - f_hi, wf);
  }

  template <bool kMass>
  __device__ __forceinline__ void by_halves(u64 goal, float m, const Weigh& wf) {
    Wide w = *this;
    const Weigh copy = wf;
    w.template bisect<kMass>(goal, m, copy);
    xb = w.xb;
    idb = w.idb;
    turn = w.turn;
  }

  // Moves the border (xb, idb) to the last token, in descending order, before which less
  // than `goal` is kept: tokens (kMass false) or weights, of which there are `whole`.  It is
  // not expected below `low`; no more than n_in tokens lie above that.
  //
  // A histogram over [lo, hi], first in equal steps of the value, then of its bits, says
  // between which two of its bins the border lies (weights in it are rounded to 2^-31 of all
  // in [lo, hi], so the bins next to the border are taken in too); a second pass adds up
  // exactly what lies above them and collects what lies in them: sorted, if the list holds
  // it, else [lo, hi] closes in on it.
  template <bool kMass>
  __device__ __forceinline__ void cut(u64 goal, u64 whole, float m, float low, u64 n_in, const Weigh& wf) {
    const int tid = threadIdx.x;
    float hi = m, lo = fmaxf(low, kLowest), first = 0.f;
    if constexpr (kMass) {  // the maximum's exponent less wf.top
      float th = 0.f, tl = 0.f;
      if (!wf.apart) wf.exponent<false>(m, 0.f, &th, &tl);
      first = (th - (float)wf.top) + tl;
    }
    u64 above = 0;  // the measure of what is larger than hi
    lo = fmaxf(lo, xb);
    bool by_value = hi - lo > 1e-30f && hi - lo < INFINITY;
    for (int step = 0;; ++step, by_value = false) {
      const float scale = (float)kBins / (hi - lo);
      const uint32_t top_key = key_of(hi);
      const int shift = max(0, 22 - (int)__clz(top_key - key_of(lo)));  // 1,024 steps of 2^shift hold all
      const float unit = kMass ? exp2f((float)(62 - wf.down)) / (float)whole * 0x1p31f : 0.f;
      // of y in [lo, hi] (hi is the maximum while steps are by value); the sum's last bits are
      // the nearest whole number (a conversion has a quarter of an addition's rate)
      auto bin_of = [&](float y) {
        return by_value ? min((int)(__float_as_uint(fmaf(hi - y, scale, 0x1p23f)) & 0x7FFFFFu), kBins - 1) : (int)((top_key - key_of(y)) >> shift);
      };
      auto inside = [&](float y, int id) { return y >= lo && y <= hi && kept(y, id); };
      for (int i = tid; i < kBins; i += kThreads) s.bins[i] = 0;
      __syncthreads();
      each(lo, [&](const auto& y, const auto& id) {
        constexpr int N = kLength<decltype(y)>;
        uint32_t n[N];
        int b[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          n[e] = kMass ? __float2uint_rn(ex2(fmaf(y[e] - m, wf.c, first)) * unit) : 1;
          b[e] = bin_of(y[e]);
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (inside(y[e], id[e])) atomicAdd(&s.bins[b[e]], n[e]);
      });
      cluster_sync();
      // the whole cluster's: four bins of this thread
      u64 v[4] = {0, 0, 0, 0};
      for (int c = 0; c < cluster; ++c) {
        uint32_t n[4];
        get4(peer(&s.bins[4 * tid], c), n);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += n[i];
      }
      if (tid == 0) s.edge[0] = s.edge[1] = kBins - 1;
      const u64 own0 = v[0], all = scan_all<kThreads, 4>(&s.red[0][0], v);
      bool below = false;  // the border lies below lo
      if constexpr (kMass) {
        const float share = (float)(goal - above) / (float)whole * 0x1p31f;
        const float slack = (float)n_in + 16384.f;  // a unit a token, and 2^-17: 62 2^-23 of an exponent and the rest
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = (float)v[i];
          if (w + slack >= share) atomicMin(&s.edge[0], 4 * tid + i);
          if (w - slack >= share) atomicMin(&s.edge[1], 4 * tid + i);
        }
      } else {
        below = above + all < goal;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (above + v[i] >= goal) atomicMin(&s.edge[0], 4 * tid + i), atomicMin(&s.edge[1], 4 * tid + i);
        __syncthreads();
        // the tokens in the bins above the border's are counted already
        const int at = s.edge[0] - 4 * tid;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at == i) s.before = i > 0 ? v[i > 0 ? i - 1 : 0] : v[0] - own0;
      }
      __syncthreads();
      if (below) {
        if (lo == kLowest) return;  // all of it is kept
        above += all;
        hi = of_key(key_of(lo) - 1);
        lo = kLowest;
        cluster_sync();  // the bins have been read
        continue;
      }
      const int b0 = s.edge[0], b1 = s.edge[1];
      u64 x[5] = {0, 0, 0, 0, 0};  // measure above, tokens and measure between, the largest and smallest there
      if constexpr (!kMass) {
        if (rank == 0 && tid == 0) x[0] = s.before;
      }
      if (tid == 0) s.count = 0;
      cluster_sync();  // (the bins have been read as well)
      u64* const own = own_list(s.list);
      // nothing below this can be in the bins up to b1
      const float least_y = by_value ? fmaxf(lo, hi - (float)(b1 + 2) / scale) : fmaxf(lo, of_key(top_key - min(top_key, (uint32_t)((u64)(b1 + 1) << shift))));
      each(least_y, [&](const auto& y, const auto& id) {
        constexpr int N = kLength<decltype(y)>;
        u64 w[N];
        int b[N];
        if constexpr (kMass) wf.all<kCopies>(y, w, table);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          b[e] = y[e] >= least_y && inside(y[e], id[e]) ? bin_of(y[e]) : kBins;
          if constexpr (kMass) x[0] += b[e] < b0 ? w[e] : 0;
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (b[e] >= b0 && b[e] <= b1) {
            x[1] += 1;
            x[2] += kMass ? w[e] : 1;
            x[3] = max(x[3], (u64)key_of(y[e]));
            x[4] = max(x[4], (u64)~key_of(y[e]) & 0xFFFFFFFFull);
            add(own, kList, by_logit(y[e], id[e]));
          }
      });
      hand_over(s.list, kList);
      exchange<5, 24>(s, x, rank, cluster, turn);
      above += x[0];
      if (kMass && (above >= goal || above + x[2] < goal)) return by_halves<kMass>(goal, m, wf);
      const uint32_t top = (uint32_t)x[3], least = ~(uint32_t)x[4];
      const u64 n = x[1];
      if (n <= kList) {
        if (rank == 0) {
          constexpr int kPer = kList / kThreads;
          sort_list<kThreads, kList>(s.list, (int)n);
          u64 w[kPer], one[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) one[i] = w[i] = tid * kPer + i < n ? (kMass ? wf.one<kCopies>(logit_of(s.list[tid * kPer + i]), table) : 1) : 0;
          scan_all<kThreads, kPer>(&s.red[0][0], w);
#pragma unroll
          for (int i = 0; i < kPer; ++i)  // the one whose weight reaches the goal
            if (above + w[i] - one[i] < goal && above + w[i] >= goal && one[i] > 0) {
              const u64 e = s.list[tid * kPer + i];
              for (int c = 0; c < cluster; ++c) put(peer(&s.found, c), (u64)__float_as_uint(logit_of(e)) << 32 | (uint32_t)e);
            }
        }
        cluster_sync();
        xb = __uint_as_float((uint32_t)(s.found >> 32));
        idb = (int)(uint32_t)s.found;
        return;
      }
      if (top == least) return cut_equals<kMass>(of_key(top), goal - above, wf);
      // (a border in the slack between two large bins keeps both)
      if (step >= 8 || (!by_value && of_key(top) == hi && of_key(least) == lo)) return by_halves<kMass>(goal, m, wf);
      hi = of_key(top);
      lo = of_key(least);
      whole = x[2];
      if constexpr (kMass) n_in = n;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int cluster, int64_t slice_vectors, int room_vectors, int down,
                                                                     const SampleLeft* list, const int* count) {
  constexpr int E = Logits<T>::E;
  extern __shared__ __align__(16) unsigned char smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  uint4* slice = reinterpret_cast<uint4*>(smem + (sizeof(SampleShared) + 15) / 16 * 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const uint2* table = s.table + (lane & (kCopies - 1));

  pdl_trigger();
  cluster_arrive();  // waited for before a peer's memory is touched
  fill_table(s.table, kCopies, tid, kThreads);
  pdl_wait();
  cluster_wait();

  int turn = 0;
  const int64_t rows = list ? *count : a.rows;
  for (int64_t i = blockIdx.x / cluster; i < rows; i += gridDim.x / cluster) {
    const int64_t row = list ? list[i].row : i;
    const Settings set = settings_of(a, row);
    if (set.skip) continue;
    if (set.bad) {
      if (rank == 0 && tid == 0) set_error(a.status, MINFER_ERR_ARG);
      continue;
    }

    // ---- the row
    const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
    const int head = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));  // logits of its first vector that are not its own
    const int64_t all = (head + a.vocab + E - 1) / E;
    Slice<T> r;
    r.first = (int64_t)rank * slice_vectors * E - head;
    r.far = reinterpret_cast<const uint4*>(x + r.first);
    r.near = slice;
    r.vectors = (int)max((int64_t)0, min(slice_vectors, all - (int64_t)rank * slice_vectors));
    r.kept = r.vectors <= room_vectors ? r.vectors : room_vectors - 1;
    r.seg = ((r.vectors + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int begin = warp * r.seg + lane, end = min((warp + 1) * r.seg, r.vectors);
    float top[2] = {-INFINITY, -INFINITY};  // of the halves of this thread's vectors
    {
      // all copies at once, in four groups
      const int quarter = max(32, (r.seg / 4 + 31) / 32 * 32);
      int v = begin;
#pragma unroll
      for (int q = 1; q <= 4; ++q) {
        const int stop = q == 4 ? end : min(end, warp * r.seg + q * quarter);
        for (; v < stop; v += 32) {
          const bool last = v == r.vectors - 1;
          if (v >= r.kept && !last) continue;
          uint4* dst = slice + min(v, r.kept);
          if (Logits<T>::inside(r.first + (int64_t)v * E, a.vocab))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(r.far + v) : "memory");
          else
            *dst = Logits<T>::edge(x, r.first + (int64_t)v * E, a.vocab);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (tid == 0) s.count = s.local = 0;
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
          for (int e = 0; e < E; ++e) top[q > 2] = max_nan(top[q > 2], y[e]);
        }
      }
    }
    // ---- the maximum, and the bound
    const uint32_t key0 = key_of(top[0]), key1 = key_of(top[1]);
    // Each CTA finds a logit that its share of the first k reaches, at least: the smallest
    // of these bounds serves.  0: there are more of them than maxima.
    const int first_k = set.greedy ? 0 : set.k > 0 ? set.k : set.top_p < 1.f && !list ? kGuess : 0;
    const int aim = first_k > 0 && (first_k - 1) / cluster < 2 * kThreads ? (first_k - 1) / cluster + 1 : 0;
    uint32_t bound = 0;
    if (aim > 0) {
      const uint32_t hi_w = __reduce_max_sync(0xffffffffu, max(key0, key1)), lo_w = __reduce_min_sync(0xffffffffu, min(key0, key1));
      if (lane == 0) s.keys[0][warp] = lo_w, s.keys[1][warp] = hi_w;
      __syncthreads();
      uint32_t lo = 0xFFFFFFFFu, hi = 0;
      for (int i = 0; i < kWarps; ++i) lo = min(lo, s.keys[0][i]), hi = max(hi, s.keys[1][i]);
      // at least `aim` of the maxima are lo or more, fewer are `over` or more
      for (uint32_t over = hi == 0xFFFFFFFFu ? hi : hi + 1; over - lo > 1;) {
        const uint32_t mid = lo + (over - lo) / 2;
        const int n = __syncthreads_count(key0 >= mid) + __syncthreads_count(key1 >= mid);
        if (n >= aim) {
          lo = mid;
          if (n <= aim + aim / 4 + 2) break;
        } else {
          over = mid;
        }
      }
      bound = lo;
    }
    u64 v2[2] = {max(key0, key1), (uint32_t)~bound};
    exchange<2, 3>(s, v2, rank, cluster, turn);
    v2[1] = (uint32_t)~(uint32_t)v2[1];
    const float m = of_key((uint32_t)v2[0]);
    const float b = v2[1] ? fmaxf(of_key((uint32_t)v2[1]), kLowest) : kLowest;  // -inf is no candidate

    auto write = [&](int token, float logprob) {
      a.token[row] = token;
      if (a.logprob) a.logprob[row] = logprob;
    };
    if (!(m < INFINITY)) {  // a NaN or +inf
      if (rank == 0 && tid == 0) set_error(a.status, MINFER_ERR_ARG);
    } else if (m == -INFINITY) {
      if (rank == 0 && tid == 0) write(-1, -INFINITY);
    } else if (set.greedy) {
      int id = 0x7FFFFFFF;
      r.each([&](const float (&y)[E], int i0) {
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
          if (y[e] == m) id = min(id, i0 + e);
      });
      u64 v1[1] = {0x7FFFFFFFu - (unsigned)id};
      exchange<1, 1>(s, v1, rank, cluster, turn);
      if (rank == 0 && tid == 0) write((int)(0x7FFFFFFFu - (unsigned)v1[0]), 0.f);
    } else {
      // ---- the weights' scale; logits below the floor are out
      if (tid == 0) s.floor = floor_of(set, m);
      Weigh wf, wd;
      wf.at(set.sharp, m, down);
      wd.at(set.temp, m, down);
      u64 whole = list ? list[i].whole : 0;
      bool covered = false;
      if (set.k == 0 && set.top_p < 1.f && whole == 0) {
        u64 v3[2] = {0, 0};
        r.each([&](const float (&y)[E], int) {
          u64 w[E];
          wf.all<kCopies>(y, w, table);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            v3[0] += w[e];
            v3[1] += y[e] >= b ? w[e] : 0;
          }
        });
        exchange<2>(s, v3, rank, cluster, turn);
        whole = v3[0];
        covered = v3[1] >= need_of(whole, set.top_p);
      } else {
        __syncthreads();  // s.floor
      }
      const float floor_x = s.floor;
      Wide<T> row_in{s, r, table, rank, cluster, turn, -INFINITY, 0x7FFFFFFF, 0, -1};

      // ---- the short way
      bool wide = list != nullptr;
      float from = kLowest;
      if (!wide && a.vocab > (cluster == 1 ? kShort : kList)) {
        if (set.k > 0) {
          wide = aim == 0;
          from = set.top_p < 1.f ? b : fmaxf(b, floor_x);
        } else if (set.top_p < 1.f) {
          wide = !covered && floor_x < b;
          from = fmaxf(b, floor_x);
        } else {
          wide = set.min_p == 0.f;
          from = floor_x;
        }
      }
      if (!wide) {
        const int entries = cluster == 1 ? kShort : kList, n = row_in.gather(from, s.longer, entries);
        wide = n > entries;
        if (!wide && rank == 0) finish_list<kThreads, kShort, kCopies>(s.longer, &s.red[0][0], n, set, wf, wd, table, floor_x, whole, false, write);
      }

      // ---- the wide way
      if (wide) {
        if (set.k > 0) {
          row_in.pick(b);
          row_in.template cut<false>((u64)set.k, 0, m, b, 0, wf);
          if (set.top_p < 1.f) {
            u64 v1[1] = {0};
            row_in.each(row_in.xb, [&](const auto& y, const auto& id) {
              constexpr int N = kLength<decltype(y)>;
              u64 w[N];
              wf.all<kCopies>(y, w, table);
#pragma unroll
              for (int e = 0; e < N; ++e) v1[0] += row_in.kept(y[e], id[e]) ? w[e] : 0;
            });
            exchange<1>(s, v1, rank, cluster, row_in.turn);
            whole = v1[0];
          }
        }
        if (set.top_p < 1.f) {
          // All that weighs less than a token's share of what may be left out is left out
          // (2^(63 - down) is more than any weight; the margin is for the logarithm).  A unit
          // less than this share: a weight counts for up to half a unit more than it is, and the
          // whole, if it comes from blocks, for half a unit a token more than their weights'
          // sum.  So what is picked reaches `need`, and nothing else is ever kept.
          const u64 need = need_of(whole, set.top_p);
          const float share = ((float)(whole > need ? whole - need : 0) / (float)a.vocab - 1.f) * exp2f((float)(down - 63));
          const float low = fmaxf(m + set.sharp * (logf(fmaxf(share, 0x1p-62f)) - 0.01f) - fabsf(m) * 0x1p-20f, kLowest);
          if (set.k == 0) row_in.pick(low);
          if (low > row_in.xb) row_in.xb = low, row_in.idb = 0x7FFFFFFF;
          row_in.template cut<true>(need, whole, m, low, (u64)a.vocab, wf);
        }
        from = fmaxf(floor_x, row_in.xb);
        u64 found = row_in.locate(from,
                                  [&](const auto& y, const auto& id, auto& w) {
                                    constexpr int N = kLength<decltype(y)>;
                                    wd.all<kCopies>(y, w, table);
#pragma unroll
                                    for (int e = 0; e < N; ++e)
                                      if (!(y[e] >= from && row_in.kept(y[e], id[e]))) w[e] = 0;
                                  },
                                  [&](u64 n) {
                                    bool rest;
                                    return times(n, set.u, &rest);
                                  },
                                  &whole);
        if (set.u == 0.f) found = row_in.nth(from, m, 1);
        turn = row_in.turn;
        if (rank == 0 && tid == 0) {
          const float y = __uint_as_float((uint32_t)(found >> 32));
          write((int)(uint32_t)found, log_share(wd, set.temp, y, wd.one<kCopies>(y, table), whole));
        }
      }
    }
    cluster_sync();  // the next row's first words
  }
}

template <typename T>
int cluster_of(int64_t vocab) {  // the fewest CTAs that keep a row
  constexpr int E = Logits<T>::E;
  const int64_t all = (vocab + 2 * E - 2) / E;
  int cluster = 1;
  while (cluster < kMaxCluster && (all + cluster - 1) / cluster * 16 > kRoom) cluster *= 2;
  return cluster;
}

template <typename T>
cudaError_t sample_typed(const SampleArgs& a, int num_sms, cudaStream_t st, const SampleLeft* list, const int* count) {
  constexpr int E = Logits<T>::E;
  const int64_t all = (a.vocab + 2 * E - 2) / E;  // vectors of a row, wherever it begins
  // As many CTAs as keep the row; more while they leave SMs idle and have something to do.
  int cluster = cluster_of<T>(a.vocab);
  auto slice = [&] { return (all + cluster - 1) / cluster; };
  while (cluster < kMaxCluster && a.rows * cluster * 2 <= num_sms && slice() * 16 > 8192) cluster *= 2;
  const int room = (int)std::min<int64_t>(slice(), kRoom / 16);
  const int smem = (int)((sizeof(SampleShared) + 15) / 16 * 16) + room * 16;
  const cudaError_t e = allow_smem<sample_kernel<T>>((int)((sizeof(SampleShared) + 15) / 16 * 16) + kRoom);
  if (e != cudaSuccess) return e;
  int down = 1;  // weights of 2^(63 - down) at most: the sum of all fits 64 bits
  while ((1ll << down) < a.vocab) ++down;
  cudaLaunchConfig_t cfg = {};
  // (a list is short as a rule: what fits at once goes over it)
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.rows, list ? 2 * num_sms / cluster : 1 << 24) * cluster));
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, cluster, slice(), room, down, list, count);
}

}  // namespace

int sample_cluster(int64_t vocab, int type) {
  return type == MINFER_F32 ? cluster_of<float>(vocab) : cluster_of<__half>(vocab);
}

cudaError_t sample_launch(const SampleArgs& a, int type, int num_sms, cudaStream_t st, const SampleLeft* list, const int* count) {
  return type == MINFER_F32   ? sample_typed<float>(a, num_sms, st, list, count)
         : type == MINFER_F16 ? sample_typed<__half>(a, num_sms, st, list, count)
                              : sample_typed<__nv_bfloat16>(a, num_sms, st, list, count);
}

}  // namespace minfer
