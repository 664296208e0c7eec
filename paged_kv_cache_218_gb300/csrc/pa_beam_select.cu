// pa_beam_select.cu -- the best continuations of each request of a beam search,
// over its beams and the vocabulary (sm_103a).
//
// Beam w with score s_w and logits x_wv proposes token v with the value
//
//   s_w + x_wv - lse_w,   lse_w = ln sum_u exp x_wu;
//
// an ended beam proposes its end token with the value s_w.  The K best of a
// request are wanted, equal values in the order of (w, v).
//
// What bounds it: HBM, one pass over the logits; at bf16 the exponential unit is
// near behind (11 elements per cycle and SM arrive, 16 exponentials leave).  So
// the pass does as little as it can per element: its exponential for the sum, and
// a maximum.  Behind it comes a chain of short steps on one SM.  64 requests of
// 4 x 131072 in bf16 (67 MB) take 19.6 us, 12.7 of them the pass (6.3 TB/s once it
// runs) and 5.6 the choice; 16 of 16 x 131072 in fp32 (134 MB) 32.4; one of 4 x 32000
// 6.5, a launch and some eight dependent round trips.
//
// A cluster serves a request, its CTAs take a share of every row, a warp 1024 bf16 (512
// fp32) elements at a time, twice 32 bytes a lane; the maxima of such blocks and the rows'
// (maximum, sum) go to the cluster's first CTA.
//
// Selection, in that CTA: with 128 groups of blocks, the (K + 1)-th best group's best
// candidate is a bound that K + 1 candidates reach.  The blocks that reach it, a few
// more than K, are read again (from L2), the candidates that reach it are gathered
// and put in order by counting.  Few blocks, or a beam far above the others, make a finer
// bound of the best in 128 shares of the candidates themselves (109 requests of 20 beams,
// 53 choices of 931 tokens: 24 us instead of 139).  Where more than 256 blocks or
// candidates reach the bound all the same (many equal logits), lists that are kept
// sorted in a warp's registers find first the K + 1 best blocks, equal ones in their
// order, which hold the K + 1 best candidates (each other block's best comes behind
// theirs), then those.
//
// Exactness.  Within a row the logits themselves give the order.  Between rows it
// hangs on lse_w, which the pass knows to a bound: values are kept as sums of two floats
// (48 bits; halved, so that sums of far scores and logits stay within fp32), and where two
// beams' candidates around the choice are nearer than twice that bound (`margin`), those
// rows' sums are taken again, to 1e-9 and 1e-15 for each token: exponentials by table and
// short polynomial (Tang's method), added as whole numbers, so that equal logits in
// whatever order and place give equal sums.  The cluster's CTAs wait for their
// share of that where it is likely (two rows of 131072 in fp32: 14 us more, one CTA 53;
// 103 requests of 6 x 50497, two CTAs each, 58 us, of which 35 without doubts).
//
// NaN and +inf logits count as -inf: no candidates, no part of the sum.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "pa_beam.h"
#include "pa_window_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kVecs = 2;       // 32-byte vectors of a lane in a warp load
constexpr float kMove = 5.5f;  // a lane's reference moves when passed by this much
constexpr int kMaxCtas = 16;   // of a cluster
constexpr int kMaxEntries = 8192;  // block maxima of a request
constexpr float kLog2e = 1.4426950408889634f;
// Values are kept halved (see base_of): the largest finite one, and a number below all.
constexpr float kMost = 0.5f * FLT_MAX, kLowest = -0.75f * FLT_MAX;

__device__ __forceinline__ void ldg32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "l"(reinterpret_cast<uint64_t>(p)));
}

__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

__device__ __forceinline__ void st_remote(uint32_t addr, uint64_t x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(x) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

__device__ __forceinline__ float sane(float x) { return x < INFINITY ? x : -INFINITY; }

// The elements of 32 bytes as floats, and the lowest element in their type.
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 16;
  static __device__ __forceinline__ float2 pair(const uint32_t (&v)[8], int i) {
    return make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ float load(const void* row, int64_t e) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]);
  }
  static __device__ __forceinline__ float max(const uint32_t (&v)[8]) {
    auto two = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&v[i]); };
    const __nv_bfloat162 a = __hmax2(__hmax2(two(0), two(1)), __hmax2(two(2), two(3)));
    const __nv_bfloat162 b = __hmax2(__hmax2(two(4), two(5)), __hmax2(two(6), two(7)));
    const float2 m = __bfloat1622float2(__hmax2(a, b));
    return fmaxf(m.x, m.y);
  }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float2 pair(const uint32_t (&v)[8], int i) {
    return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
  }
  static __device__ __forceinline__ float load(const void* row, int64_t e) {
    return static_cast<const float*>(row)[e];
  }
  static __device__ __forceinline__ float max(const uint32_t (&v)[8]) {
    float m = __uint_as_float(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(v[i]));
    return m;
  }
};

// A beam's logits in vectors of 32 aligned bytes: vector i holds the elements
// [kVec * i - lead, + kVec), as far as the row has them.  Warp load t takes vectors
// [64 t, 64 t + 64), a lane the ones at its own number and 32 behind.
template <typename T>
struct Row {
  using E = Elem<T>;
  static constexpr int kLoad = 32 * kVecs * E::kVec;  // elements
  const T* p;
  int lead;
  __device__ __forceinline__ Row(const BeamSelectArgs& a, int r, int w) {
    p = static_cast<const T*>(a.logits) + r * a.request_stride + w * a.beam_stride;
    lead = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 31) / static_cast<int>(sizeof(T));
  }
  // Loads [first, last) have none but elements of the row.
  __device__ __forceinline__ int first() const { return lead ? 1 : 0; }
  __device__ __forceinline__ int last(int vocab) const { return (lead + vocab) / kLoad; }
};

template <typename T>
__device__ __forceinline__ void load_whole(const T* at, uint32_t (&v)[kVecs][8]) {
#pragma unroll
  for (int u = 0; u < kVecs; ++u) ldg32(at + u * 32 * Elem<T>::kVec, v[u]);
}

// (Rare work is kept out of line and its loops rolled: a CTA runs each step but a few
// times, and fetching instructions decides how long they take.  With everything in line,
// 113 KB of code, finding the bound of a choice took 3.6 us of which 0.1 was work.)

// A vector of a row's first or last elements, -inf where they end.
template <typename T>
__device__ __noinline__ void gather_edge(const T* p, int vocab, int e, uint4* to) {
  T t[Elem<T>::kVec];
#pragma unroll
  for (int j = 0; j < Elem<T>::kVec; ++j)
    t[j] = e + j >= 0 && e + j < vocab ? p[e + j] : static_cast<T>(-INFINITY);
  T* const out = reinterpret_cast<T*>(to);
#pragma unroll
  for (int j = 0; j < Elem<T>::kVec; ++j) out[j] = t[j];
}

// NaN and +inf of a vector become -inf.
template <typename T>
__device__ __noinline__ void clean_vector(uint4* v) {
  T* const t = reinterpret_cast<T*>(v);
#pragma unroll 1
  for (int j = 0; j < Elem<T>::kVec; ++j)
    if (!(static_cast<float>(t[j]) < INFINITY)) t[j] = static_cast<T>(-INFINITY);
}

__device__ __forceinline__ void unpack(const uint4* from, uint32_t (&v)[8]) {
  const uint4 lo = from[0], hi = from[1];
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
  v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}

// Any load, partial vectors through `edges`, the lane's own 32 bytes.
template <typename T>
__device__ __forceinline__ void load_edge(const T* p, int vocab, int e0, uint4* edges,
                                          uint32_t (&v)[kVecs][8]) {
  constexpr int kVec = Elem<T>::kVec;
  constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // (-inf)
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int e = e0 + u * 32 * kVec;
    if (e >= 0 && e <= vocab - kVec) {
      ldg32(p + e, v[u]);
    } else if (e > -kVec && e < vocab) {
      gather_edge(p, vocab, e, edges);
      unpack(edges, v[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = kNone;
    }
  }
}

// A value as a sum of two floats, the second below half a step of the first: one
// 64-bit number in the order of such values, 0 below all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float2 two_sum(float a, float b) {  // (exact)
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
// Half of score - top - ln: the whole may lie past fp32 where it and a logit do not.
__device__ __forceinline__ float2 base_of(float score, float top, float2 ln) {
  const float2 a = two_sum(0.5f * score, -0.5f * top), b = two_sum(a.x, -0.5f * ln.x);
  return two_sum(b.x, (b.y + a.y) - 0.5f * ln.y);
}
__device__ __forceinline__ uint64_t value_key(float2 base, float x) {
  const float2 s = two_sum(base.x, 0.5f * x);
  const float2 v = two_sum(s.x, __fadd_rn(s.y, base.y));
  if (!(fabsf(v.x) <= kMost)) return 0;
  return static_cast<uint64_t>(ordered(v.x)) << 32 | ordered(v.y);
}
// How far one value lies above another.
__device__ __forceinline__ float key_gap(uint64_t a, uint64_t b) {
  return (unordered(static_cast<uint32_t>(a >> 32)) - unordered(static_cast<uint32_t>(b >> 32))) +
         (unordered(static_cast<uint32_t>(a)) - unordered(static_cast<uint32_t>(b)));
}
__device__ __forceinline__ bool better(uint64_t ka, uint32_t ia, uint64_t kb, uint32_t ib) {
  return ka > kb || (ka == kb && ia < ib);
}

// The best 32 * KL (key, index) pairs that a warp has seen, best first: place
// 32 * r + lane in register r.  Empty places have key 0.
template <int KL>
struct WarpList {
  uint64_t key[KL];
  uint32_t idx[KL];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < KL; ++r) {
      key[r] = 0;
      idx[r] = 0xffffffffu;
    }
  }
  // Takes each lane's pair whose key is at least `floor`.
  __device__ __forceinline__ void offer(uint64_t k, uint32_t i, uint64_t floor, int lane) {
    for (unsigned todo = __ballot_sync(0xffffffffu, k != 0 && k >= floor); todo;
         todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const uint64_t nk = __shfl_sync(0xffffffffu, k, from);
      const uint32_t ni = __shfl_sync(0xffffffffu, i, from);
      int place = 0;
#pragma unroll
      for (int r = 0; r < KL; ++r)
        place += __popc(__ballot_sync(0xffffffffu, better(key[r], idx[r], nk, ni)));
      if (place == 32 * KL) continue;
#pragma unroll
      for (int r = KL - 1; r >= 0; --r) {
        uint64_t pk = __shfl_up_sync(0xffffffffu, key[r], 1);
        uint32_t pi = __shfl_up_sync(0xffffffffu, idx[r], 1);
        if (r > 0) {
          const uint64_t ck = __shfl_sync(0xffffffffu, key[r - 1], 31);
          const uint32_t ci = __shfl_sync(0xffffffffu, idx[r - 1], 31);
          if (lane == 0) {
            pk = ck;
            pi = ci;
          }
        }
        const int at = 32 * r + lane;
        key[r] = at < place ? key[r] : (at == place ? nk : pk);
        idx[r] = at < place ? idx[r] : (at == place ? ni : pi);
      }
    }
  }
};

// 2^(j / 64) in units of 2^-31, j < 64: for sums that need more than fp32.
struct ExpTable {
  uint32_t t[64];
};

// A sum in units of 2^-50, whole numbers in two parts: no order of its terms changes it.
struct FixedSum {
  uint64_t hi = 0, lo = 0;  // hi 2^32 + lo
  __device__ __forceinline__ void add(uint64_t t) {
    hi += t >> 32;
    lo += t & 0xffffffffu;
  }
};

// e^(x - m) for x <= m, some 1e-9 of itself off, added to a sum.
__device__ __forceinline__ void add_exp(FixedSum& sum, const ExpTable& tab, float x, float m) {
  const float2 d = two_sum(x, -m);
  if (!(d.x > -36.f)) return;  // (below 2^-51)
  // d log2(e) = n / 64 + f, |f| <= 1 / 128
  constexpr float kL1 = 1.44269502162933349609f, kL2 = 1.92596299112661746887e-8f;
  const float t = d.x * kL1;
  const float tl = __fmaf_rn(d.x, kL1, -t) + (d.x * kL2 + d.y * kL1);
  const float n = rintf(t * 64.f);
  const float f = __fmaf_rn(n, -0.015625f, t) + tl;
  // 2^f - 1 = sum (f ln 2)^k / k!
  const float g = f * 0.69314718055994530942f;
  const float p = g * __fmaf_rn(g, __fmaf_rn(g, __fmaf_rn(g, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
  // in whole numbers from here on, a conversion to 64 bits costs eight of these: p in units
  // of 2^-38 (|p| < 0.006, so 31 bits hold it)
  const int k = static_cast<int>(n);
  const uint32_t e = tab.t[k & 63];
  const int64_t ep = static_cast<int64_t>(e) * __float2int_rn(p * 0x1p38f);
  sum.add(((static_cast<uint64_t>(e) << 19) + (ep >> 19)) >> -(k >> 6));
}

// e^(x - m) as 2^((x - m) log2 e) in fp32, steps (2^-24) of itself that it may be off for each
// unit of |x - m|: the difference is rounded, the product is, and log2 e is 0.22 steps off.
constexpr double kArgSteps = 2.3;

constexpr int kGroups = 128;     // of block maxima, whose best bound the choice
constexpr int kMaxPicked = 256;  // blocks, and candidates, that are gathered unsorted

// Shared memory besides the block maxima.
template <int KL>
struct SelectSmem {
  uint4 edges[kThreads][2];          // of rows, elements on their way to registers
  float2 part[kMaxBeams][kMaxCtas];  // rows' (maximum, sum) of each CTA
  float2 red[kMaxBeams][kWarps];     // and of each warp
  float2 base[kMaxBeams];            // (s - lse) / 2 in two floats
  float group[kThreads / kGroups][kGroups];
  uint32_t group_key[4][kGroups / 4 + 4];  // (quarters in different banks)
  union {
    struct {
      uint64_t key[kMaxPicked];
      uint32_t idx[kMaxPicked];
      uint32_t block[kMaxPicked];
    } pick;
    struct {
      uint64_t key[kWarps][32 * KL];
      uint32_t idx[kWarps][32 * KL];
    } list;
  };
  uint64_t key[kMaxPicked];  // candidates in order
  uint32_t idx[kMaxPicked];
  float bound;        // no candidate below it is chosen
  unsigned doubtful;  // rows whose sums are to be taken again
  int found, blocks, picked;
  ExpTable table;
  // Rows that the whole cluster is to sum again (0: the choice is made), and their maxima, a
  // reference that the order of the logits does not change.  The first CTA writes every CTA's.
  struct Call {
    unsigned rows;
    float top[kMaxBeams];
  } call;
};

// The best `n` of the warps' lists into sm.key / sm.idx, their number into sm.found.
// Called by the whole CTA.
template <int KL>
__device__ __forceinline__ void join_lists(SelectSmem<KL>& sm, const WarpList<KL>& mine, int n,
                                           int warp, int lane) {
#pragma unroll
  for (int r = 0; r < KL; ++r) {
    sm.list.key[warp][32 * r + lane] = mine.key[r];
    sm.list.idx[warp][32 * r + lane] = mine.idx[r];
  }
  if (threadIdx.x == 0) sm.found = 0;
  __syncthreads();
  for (int t = threadIdx.x; t < kWarps * n; t += kThreads) {
    const int w = t / n, at = t - w * n;
    const uint64_t k = sm.list.key[w][at];
    const uint32_t i = sm.list.idx[w][at];
    if (k == 0) continue;
    int rank = at;
#pragma unroll
    for (int o = 1; o < kWarps; ++o) {
      const int l = (w + o) % kWarps;
      int lo = 0, hi = n;  // how many of list l come before
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (better(sm.list.key[l][mid], sm.list.idx[l][mid], k, i))
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank < n) {
      sm.key[rank] = k;
      sm.idx[rank] = i;
      atomicMax(&sm.found, rank + 1);
    }
  }
  __syncthreads();
}

enum BeamState : int { kDead = 0, kLive = 1, kEnded = 2 };

// The beam of entry e of the block maxima.
__device__ __forceinline__ int beam_of(const BeamSelectArgs& a, int e) {
  return a.blocks_per_row == 1 ? e : static_cast<int>(__umulhi(e, a.blocks_inverse));
}

// What the first CTA's threads know of the choice.
template <typename T, int KL>
struct Choice {
  using E = Elem<T>;
  const BeamSelectArgs& a;
  SelectSmem<KL>& sm;
  float* block_max;
  int r;
  unsigned live, ended;
  unsigned exact;  // rows whose base is known to 1e-9
  float bound;     // finite: no candidate below it is chosen
  float slack;     // what sums and roundings are off, besides off() of the row

  // What a row's values may be off in fp32 for its base's size.  (The row's own: beams that
  // are held back by scores of -1e9 leave the others' bound where it is.)
  static __device__ __forceinline__ float off(float base) { return fabsf(base) * 0x1p-20f; }
  // the value of a block's best candidate
  __device__ __forceinline__ uint64_t entry_key(int e) const {
    return value_key(sm.base[beam_of(a, e)], block_max[e]);
  }
  // The lane's elements of load number `part` of block e, a live beam w's.
  __device__ __forceinline__ int fetch(const Row<T>& row, int w, int e, int part, int lane,
                                       uint32_t (&v)[kVecs][8]) const {
    const int t = ((e - w * a.blocks_per_row) << a.block_shift) + part;
    const int e0 = t * Row<T>::kLoad + lane * E::kVec - row.lead;
    if (t >= row.first() && t < row.last(a.vocab))
      load_whole(row.p + e0, v);
    else
      load_edge(row.p, a.vocab, e0, sm.edges[threadIdx.x], v);
    return e0;
  }
  // Best values, at the least, among quarters of them (every fourth pair), in fp32.
  __device__ __forceinline__ void best_of(int e, int part, int lane, float (&best)[4]) const {
    const int w = beam_of(a, e);
    if ((ended >> w) & 1) {
      const float base = sm.base[w].x;
      if (lane == 0 && part == 0) best[0] = fmaxf(best[0], base - off(base));
      return;
    }
    uint32_t v[kVecs][8];
    fetch(Row<T>(a, r, w), w, e, part, lane, v);
    const float base = sm.base[w].x - off(sm.base[w].x);
#pragma unroll
    for (int i = 0; i < kVecs * E::kVec / 2; ++i) {
      const float2 x = E::pair(v[i / (E::kVec / 2)], i % (E::kVec / 2));
      best[i % 4] = fmaxf(best[i % 4], __fmaf_rn(0.5f, fmaxf(sane(x.x), sane(x.y)), base));
    }
  }
  // Load number `part` of block e: f(key, index) for the candidates that may reach the
  // bound, the whole warp together (key 0: this lane has none).
  template <typename F>
  __device__ __forceinline__ void scan(int e, int part, int lane, F f) const {
    const int w = beam_of(a, e);
    const float2 base = sm.base[w];
    const uint32_t index0 = static_cast<uint32_t>(w) * a.vocab;
    if ((ended >> w) & 1) {
      f(lane == 0 && part == 0 ? value_key(base, 0.f) : 0, index0 + a.end_token);
      return;
    }
    const Row<T> row(a, r, w);
    uint32_t v[kVecs][8];
    const int e0 = fetch(row, w, e, part, lane, v);
    unsigned hits = 0;
    const float least = fmaxf(2.f * ((bound - base.x) - (slack + off(base.x))), -FLT_MAX);
#pragma unroll
    for (int i = 0; i < kVecs * E::kVec / 2; ++i) {
      const float2 x = E::pair(v[i / (E::kVec / 2)], i % (E::kVec / 2));
      hits |= (x.x >= least ? 1u : 0u) << (2 * i) | (x.y >= least ? 1u : 0u) << (2 * i + 1);
    }
#pragma unroll 1
    while (__any_sync(0xffffffffu, hits != 0)) {
      uint64_t k = 0;
      int token = 0;
      if (hits) {
        const int j = __ffs(hits) - 1;
        token = e0 + (j / E::kVec) * 32 * E::kVec + j % E::kVec;
        hits &= hits - 1;
        k = value_key(base, sane(E::load(row.p, token)));
      }
      f(k, index0 + token);
      __syncwarp();
    }
  }
  // Load number `part` of block e: the candidates that may reach the bound into sm.pick,
  // their number added to sm.picked; no lane's that are more than sm.pick takes (one at a
  // time, a thousand of them took 35 us).
  __device__ __forceinline__ void gather(int e, int part, int lane) const {
    const int w = beam_of(a, e);
    const float2 base = sm.base[w];
    const uint32_t index0 = static_cast<uint32_t>(w) * a.vocab;
    const bool over = (ended >> w) & 1;
    const Row<T> row(a, r, w);
    unsigned hits = over && lane == 0 && part == 0;
    int e0 = 0;
    if (!over) {
      uint32_t v[kVecs][8];
      e0 = fetch(row, w, e, part, lane, v);
      const float least = fmaxf(2.f * ((bound - base.x) - (slack + off(base.x))), -FLT_MAX);
#pragma unroll
      for (int i = 0; i < kVecs * E::kVec / 2; ++i) {
        const float2 x = E::pair(v[i / (E::kVec / 2)], i % (E::kVec / 2));
        hits |= (x.x >= least && x.x < INFINITY ? 1u : 0u) << (2 * i) |
                (x.y >= least && x.y < INFINITY ? 1u : 0u) << (2 * i + 1);
      }
    }
    if (hits == 0) return;
    int at = atomicAdd(&sm.picked, __popc(hits));
    if (at + __popc(hits) > kMaxPicked) return;
#pragma unroll 1
    for (; hits; hits &= hits - 1, ++at) {
      const int j = __ffs(hits) - 1;
      const int token = over ? a.end_token : e0 + (j / E::kVec) * 32 * E::kVec + j % E::kVec;
      sm.pick.key[at] = value_key(base, over ? 0.f : E::load(row.p, token));
      sm.pick.idx[at] = index0 + token;
    }
  }
  __device__ __forceinline__ void doubt(int w0, int w1) const {
    const unsigned both = 1u << w0 | 1u << w1;
    if (w0 != w1 && (both & ~exact)) atomicOr(&sm.doubtful, both);
  }
};

// The n-th best of 128 groups' best values, of which each thread brings a share of group
// threadIdx.x % 128's, rounded down; -inf where fewer groups have one.  Called by the
// whole CTA.
template <int KL>
__device__ __noinline__ float group_bound(SelectSmem<KL>& sm, float best, int n) {
  constexpr int kQuarter = kGroups / 4;
  static_assert(kThreads / kGroups == 4, "a thread for each quarter");
  sm.group[threadIdx.x / kGroups][threadIdx.x % kGroups] = best;
  if (threadIdx.x == 0) sm.bound = -INFINITY;
  __syncthreads();
  if (threadIdx.x < kGroups) {
#pragma unroll
    for (int i = 1; i < 4; ++i) best = fmaxf(best, sm.group[i][threadIdx.x]);
    // (the last bits tell equal groups apart)
    sm.group_key[threadIdx.x / kQuarter][threadIdx.x % kQuarter] =
        best > -INFINITY ? (ordered(best) & ~(kGroups - 1u)) | threadIdx.x : threadIdx.x;
  }
  __syncthreads();
  // thread 4 g + h: how many of quarter h come before group g
  const int g = threadIdx.x >> 2, h = threadIdx.x & 3;
  const uint32_t mine = sm.group_key[g / kQuarter][g % kQuarter];
  int place = 0;
#pragma unroll 2
  for (int i = 0; i < kQuarter; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(&sm.group_key[h][i]);
    place += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
  }
  place += __shfl_xor_sync(0xffffffffu, place, 1);
  place += __shfl_xor_sync(0xffffffffu, place, 2);
  if (place == n - 1 && h == 0 && mine >= kGroups) sm.bound = unordered(mine & ~(kGroups - 1u));
  __syncthreads();
  return sm.bound;
}

// The K + 1 best by sorted lists: first the blocks, then of these the candidates; and which
// rows' order is in doubt.  Called by the whole CTA.
template <typename T, int KL>
__device__ __noinline__ void choose_by_lists(const Choice<T, KL>& c) {
  SelectSmem<KL>& sm = c.sm;
  const BeamSelectArgs& a = c.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = a.num_choices, L = K + 1, V = a.vocab;
  const int entries = a.num_beams * a.blocks_per_row, sh = a.block_shift;
  uint64_t floor = static_cast<uint64_t>(ordered(c.bound)) << 32;
  WarpList<KL> list;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    list.clear();
    const int chosen = round == 0 ? entries : sm.found << sh;
    if (round == 1) floor = sm.found == L ? sm.key[L - 1] : 0;
#pragma unroll 1
    for (int t = round == 0 ? warp * 32 : warp; t < chosen; t += round == 0 ? kThreads : kWarps) {
      auto offer = [&](uint64_t k, uint32_t i) { list.offer(k, i, floor, lane); };
      if (round == 0)
        offer(t + lane < entries ? c.entry_key(t + lane) : 0, t + lane);
      else
        c.scan(sm.idx[t >> sh], t & ((1 << sh) - 1), lane, offer);
    }
    __syncthreads();  // sm.idx and sm.found have been read
    join_lists(sm, list, L, warp, lane);
  }
  const int found = sm.found;
  for (int i = threadIdx.x; i < K && i + 1 < found; i += kThreads)
    if (key_gap(sm.key[i], sm.key[i + 1]) < a.margin) c.doubt(sm.idx[i] / V, sm.idx[i + 1] / V);
  if (found < L) return;
  const uint64_t last = sm.key[K - 1];
  const int w0 = sm.idx[K - 1] / V;
  if (static_cast<int>(sm.idx[K] / V) != w0 || key_gap(last, sm.key[K]) >= a.margin) return;
  // Another row's candidate next to the last choice, displaced by candidates of that
  // choice's own row?
#pragma unroll 1
  for (int e0 = warp * 32; e0 < entries; e0 += kThreads) {
    const int e = e0 + lane;
    const int w = e < entries ? beam_of(a, e) : w0;
    const uint64_t k = e < entries ? c.entry_key(e) : 0;
    const bool look = w != w0 && ((1u << w0 | 1u << w) & ~c.exact) && k != 0 &&
                      key_gap(last, k) < a.margin;
    if (look && k < last) c.doubt(w0, w);
#pragma unroll 1
    for (unsigned todo = __ballot_sync(0xffffffffu, look && k >= last); todo; todo &= todo - 1) {
      const int from = e0 + __ffs(todo) - 1;
#pragma unroll 1
      for (int part = 0; part < 1 << sh; ++part)
        c.scan(from, part, lane, [&](uint64_t kx, uint32_t i) {
          if (kx != 0 && kx < last && key_gap(last, kx) < a.margin) c.doubt(w0, beam_of(a, from));
        });
    }
  }
}

// A CTA's share of the sums that sm.call names, in whole numbers, to the first CTA's sm.part
// (upper halves) and sm.red, which nothing else needs any more.  Called by the whole CTA.
template <typename T, int KL>
__device__ __noinline__ void sum_share(const BeamSelectArgs& a, SelectSmem<KL>& sm, int r, int rank,
                                       int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = a.vocab, step = ctas * kThreads;
  struct Sums {
    uint64_t hi[kMaxBeams][kWarps], lo[kMaxBeams][kWarps];
  };
  static_assert(sizeof(Sums) <= sizeof(sm.edges), "no load uses it meanwhile");
  static_assert(sizeof(sm.part) == 8 * kMaxBeams * kMaxCtas && sizeof(sm.red) == sizeof(sm.part),
                "a number for each row and CTA");
  Sums& all = *reinterpret_cast<Sums*>(sm.edges);
  if (threadIdx.x < 64)
    sm.table.t[threadIdx.x] = __double2uint_rn(exp2(threadIdx.x / 64.0) * 0x1p31);
  __syncthreads();
#pragma unroll 1
  for (unsigned todo = sm.call.rows; todo; todo &= todo - 1) {
    const int w = __ffs(todo) - 1;
    const Row<T> row(a, r, w);
    const float top = sm.call.top[w];
    FixedSum sum;
    // (eight loads are under way behind the eight at hand)
    auto get = [&](int x0, float (&x)[8]) {  // (a row has up to 2^30 elements)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = x0 + i * step < V ? Elem<T>::load(row.p, x0 + i * step) : -INFINITY;
    };
    float x[8], next[8];
    int x0 = rank * kThreads + threadIdx.x;
    get(x0, next);
#pragma unroll 1
    for (; x0 < V; x0 += 8 * step) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = next[i];
      get(x0 + 8 * step, next);
#pragma unroll
      for (int i = 0; i < 8; ++i) add_exp(sum, sm.table, sane(x[i]), top);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      sum.hi += __shfl_xor_sync(0xffffffffu, sum.hi, off);
      sum.lo += __shfl_xor_sync(0xffffffffu, sum.lo, off);
    }
    if (lane == 0) {
      all.hi[w][warp] = sum.hi;
      all.lo[w][warp] = sum.lo;
    }
  }
  __syncthreads();
  if (threadIdx.x < kMaxBeams && (sm.call.rows >> lane & 1)) {
    FixedSum sum;
#pragma unroll 1
    for (int i = 0; i < kWarps; ++i) {
      sum.hi += all.hi[lane][i];
      sum.lo += all.lo[lane][i];
    }
    st_remote(mapa_shared(smem_u32(&sm.part[lane][rank]), 0), sum.hi);
    st_remote(mapa_shared(smem_u32(&sm.red[lane][rank]), 0), sum.lo);
  }
  __syncwarp();
}

// Every other CTA of the cluster learns of sm.call.  Called by the whole first CTA.
template <int KL>
__device__ __forceinline__ void pass_on_call(SelectSmem<KL>& sm, int ctas) {
  constexpr int kWords = sizeof(sm.call) / 4;
  __syncthreads();
  const float* const word = reinterpret_cast<const float*>(&sm.call);
  for (int t = threadIdx.x; t < kWords * (ctas - 1); t += kThreads)
    st_remote(mapa_shared(smem_u32(word + t % kWords), 1 + t / kWords), word[t % kWords]);
  __syncwarp();
}

// The bases of these rows, to 1e-9, by so many CTAs of the cluster: the first one's part in
// it.  What has been gathered gets its keys anew: it has the choices all the same, since the
// sums move by less than its bound allows for.
template <typename T, int KL>
__device__ __noinline__ void sum_again(const Choice<T, KL>& c, unsigned rows, float score,
                                       int ctas, int picked) {
  SelectSmem<KL>& sm = c.sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NB = c.a.blocks_per_row;
  if (threadIdx.x == 0) sm.call.rows = rows;
#pragma unroll 1
  for (int w = warp; w < c.a.num_beams; w += kWarps) {
    if (!(rows >> w & 1)) continue;
    float top = -INFINITY;
#pragma unroll 1
    for (int b = lane; b < NB; b += 32) top = fmaxf(top, c.block_max[w * NB + b]);
    top = warp_max(top);
    if (lane == 0) sm.call.top[w] = top;
  }
  pass_on_call(sm, ctas);
  if (ctas > 1) cluster_sync();
  sum_share<T, KL>(c.a, sm, c.r, 0, ctas);
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  if (threadIdx.x < kMaxBeams && (rows >> lane & 1)) {
    const uint64_t* const his = reinterpret_cast<const uint64_t*>(sm.part[lane]);
    const uint64_t* const los = reinterpret_cast<const uint64_t*>(sm.red[lane]);
    FixedSum sum;
#pragma unroll 1
    for (int i = 0; i < ctas; ++i) {
      sum.hi += his[i];
      sum.lo += los[i];
    }
    const double ln = log(static_cast<double>(sum.hi) * 0x1p-18 +
                          static_cast<double>(sum.lo) * 0x1p-50);
    const float hi = static_cast<float>(ln);
    sm.base[lane] =
        base_of(score, sm.call.top[lane], make_float2(hi, static_cast<float>(ln - hi)));
  }
  if (threadIdx.x == 0) sm.doubtful = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < picked; i += kThreads) {
    const int w = sm.pick.idx[i] / c.a.vocab;
    const int token = static_cast<int>(sm.pick.idx[i]) - w * c.a.vocab;
    if (rows >> w & 1)
      sm.pick.key[i] = value_key(sm.base[w], Elem<T>::load(Row<T>(c.a, c.r, w).p, token));
  }
  __syncthreads();
}

// (__grid_constant__: the arguments' address goes to functions out of line, and a copy of
// them in local memory cost a fifth of the time.)
template <typename T, int KL>
__global__ void __launch_bounds__(kThreads, 2)
    beam_select_kernel(const __grid_constant__ BeamSelectArgs a) {
  using E = Elem<T>;
  extern __shared__ float block_max[];  // [beams][blocks_per_row], of the first CTA
  __shared__ SelectSmem<KL> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int C = static_cast<int>(ctas);
  const int r = static_cast<int>(blockIdx.x) / C;
  const int W = a.num_beams, V = a.vocab, NB = a.blocks_per_row, sh = a.block_shift;
  // the first CTA clears its shared memory before others write there
  if (rank == 0)
    for (int e = threadIdx.x; e < W * NB; e += kThreads) block_max[e] = -INFINITY;
  for (int e = threadIdx.x; e < W * kWarps; e += kThreads)
    sm.red[e / kWarps][e % kWarps] = make_float2(-FLT_MAX, 0.f);
  if (threadIdx.x == 0) sm.call.rows = 0;
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  griddep_launch_dependents();
  griddep_wait();

  // lane w: state of beam w
  float score = -INFINITY;
  int state = kDead;
  if (lane < W) {
    score = a.scores[static_cast<int64_t>(r) * W + lane];
    const bool ended = a.finished && a.finished[static_cast<int64_t>(r) * W + lane];
    // (a score that is no number, or infinite, ends the beam without a candidate)
    state = !(score > -INFINITY && score < INFINITY) ? kDead : (ended ? kEnded : kLive);
  }
  const unsigned live = __ballot_sync(0xffffffffu, state == kLive);
  const unsigned ended = __ballot_sync(0xffffffffu, state == kEnded);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  // ---- the pass over the logits: the CTA's blocks [b0, b1) of every live beam, one
  // row behind another, in a range of them for each warp
  const uint32_t remote_max = mapa_shared(smem_u32(block_max), 0);
  const int t0 = (NB * rank / C) << sh, t1 = (NB * (rank + 1) / C) << sh;  // loads of a row
  const int per_row = t1 - t0, all = __popc(live) * (per_row >> sh);
  const int first = (all * warp / kWarps) << sh;
  int left = ((all * (warp + 1) / kWarps) << sh) - first;  // to be fetched
  if (left > 0) {
    const int part_mask = (1 << sh) - 1;
    unsigned get_rows = live;  // beams from the one fetched on
    int skip = first;
    for (; skip >= per_row; skip -= per_row) get_rows &= get_rows - 1;
    int get = t0 + skip;       // load fetched next, and the row's whole ones
    int whole0 = 0, whole1 = 0;
    const T* row = nullptr;    // the lane's first element of the row's load 0
    auto begin = [&]() {
      const Row<T> x(a, r, __ffs(get_rows) - 1);
      row = x.p - x.lead + lane * E::kVec;
      whole0 = x.first();
      whole1 = x.last(V);
    };
    begin();
    uint32_t v[kVecs][8];
    auto fetch = [&]() {
      if (get >= whole0 && get < whole1) {
        load_whole(row + static_cast<int64_t>(get) * Row<T>::kLoad, v);
      } else {
        const Row<T> x(a, r, __ffs(get_rows) - 1);
        load_edge(x.p, V, get * Row<T>::kLoad + lane * E::kVec - x.lead, sm.edges[threadIdx.x],
                  v);
      }
      --left;
      if (++get == t1 && left > 0) {
        get = t0;
        get_rows &= get_rows - 1;
        begin();
      }
    };
    unsigned use_rows = get_rows;
    int use = get, todo = left;
    fetch();
    // sum of 2^((x - ref) log2 e) of the lane's elements of this row; ref is finite, and
    // at most kMove below the largest
    float ref = -FLT_MAX, sum = 0.f, block = -INFINITY;
    while (todo > 0) {
      float mx, more;
      bool clean = false;
      while (true) {
        mx = E::max(v[0]);
#pragma unroll
        for (int c = 1; c < kVecs; ++c) mx = fmaxf(mx, E::max(v[c]));
        if (mx > ref + kMove && mx < INFINITY) {
          sum *= fast_exp2((ref - mx) * kLog2e);
          ref = mx;
        }
        const uint64_t nref = f32x2(-ref, -ref), scale = f32x2(kLog2e, kLog2e);
        uint64_t sums[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kVecs * E::kVec / 2; ++i) {
          const float2 x = E::pair(v[i / (E::kVec / 2)], i % (E::kVec / 2));
          const float2 d = f32x2_parts(mul2(add2(f32x2(x.x, x.y), nref), scale));
          sums[i & 1] = add2(sums[i & 1], f32x2(fast_exp2(d.x), fast_exp2(d.y)));
        }
        const float2 two = f32x2_parts(add2(sums[0], sums[1]));
        more = two.x + two.y;
        if (clean || (mx < INFINITY && more == more)) break;
        // NaN or +inf among them: once more without
        clean = true;
        uint4* const edges = sm.edges[threadIdx.x];
#pragma unroll
        for (int c = 0; c < kVecs; ++c) {
          uint32_t (&x)[8] = v[c];
          edges[0] = make_uint4(x[0], x[1], x[2], x[3]);
          edges[1] = make_uint4(x[4], x[5], x[6], x[7]);
          clean_vector<T>(edges);
          unpack(edges, x);
        }
      }
      if (left > 0) fetch();  // (the next one: this one's elements are used up)
      sum += more;
      --todo;
      __syncwarp();
      block = fmaxf(block, warp_max(mx));
      const int w = __ffs(use_rows) - 1;
      if ((use & part_mask) == part_mask) {
        if (lane == 0) st_remote(remote_max + 4 * (w * NB + (use >> sh)), block);
        block = -INFINITY;
      }
      if (++use == t1 || todo == 0) {  // the warp's share of this row is done
        const float top = warp_max(ref);
        sum *= fast_exp2((ref - top) * kLog2e);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) sm.red[w][warp] = make_float2(top, sum);
        ref = -FLT_MAX;
        sum = 0.f;
        use = t0;
        use_rows &= use_rows - 1;
      }
    }
  }
  __syncthreads();
  // a row's share of this CTA, a half warp for each
  {
    static_assert(kThreads / kWarps == kMaxBeams, "rows at once");
    const int w = threadIdx.x / kWarps;
    const float2 x = sm.red[w][threadIdx.x % kWarps];
    float top = x.x;
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = x.y * fast_exp2((x.x - top) * kLog2e);
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (w < W && threadIdx.x % kWarps == 0) {
      const uint32_t at = mapa_shared(smem_u32(&sm.part[w][rank]), 0);
      st_remote(at, top);
      st_remote(at + 4, sum);
    }
  }
  cluster_sync();
  const int hands = a.all_sum ? C : 1;
  if (rank != 0) {  // a hand with rows whose sums are taken again, until the choice is made
    while (a.all_sum) {
      cluster_sync();
      if (sm.call.rows == 0) return;
      sum_share<T, KL>(a, sm, r, rank, C);
      cluster_sync();
    }
    return;
  }

  // ---- the first CTA: (s - lse) / 2 of each row
  for (int w = warp; w < W; w += kWarps) {
    const float mine = __shfl_sync(0xffffffffu, score, w);
    float2 base = make_float2(0.5f * mine, 0.f);
    if ((live >> w) & 1) {
      const float2 x = lane < C ? sm.part[w][lane] : make_float2(-FLT_MAX, 0.f);
      const float top = warp_max(x.x);
      float s = x.y * fast_exp2((x.x - top) * kLog2e);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      // (a row of -inf: no candidates, whatever the base)
      if (s > 0.f) base = base_of(mine, top, make_float2(logf(s), 0.f));
    } else if (((ended >> w) & 1) && lane == 0) {
      const Row<T> row(a, r, w);  // one candidate, in its token's block
      block_max[w * NB + ((a.end_token + row.lead) / Row<T>::kLoad >> sh)] = 0.f;
    }
    if (lane == 0) sm.base[w] = base;
  }
  const int K = a.num_choices, L = K + 1, entries = W * NB;
  Choice<T, KL> c{a, sm, block_max, r, live, ended, ended, 0.f, 0.f};
  __syncthreads();

  // f(entry, value in fp32, what that may be off) for this thread's blocks, those of group
  // threadIdx.x % 128
  auto each_entry = [&](auto f) {
#pragma unroll 4
    for (int e = threadIdx.x; e < entries; e += kThreads) {
      const float base = sm.base[beam_of(a, e)].x;
      f(e, __fmaf_rn(0.5f, block_max[e], base), c.off(base));
    }
  };

  while (true) {
    // ---- a bound: the L-th best of 128 groups' best blocks, each at the least that it may
    // be, less what sums and roundings may be off
    if (threadIdx.x == 0) {
      sm.blocks = sm.picked = sm.found = 0;
      sm.doubtful = 0;
    }
    float best = -INFINITY;
    each_entry([&](int, float v, float off) { best = fmaxf(best, v - off); });
    float least = group_bound(sm, best, L);
    auto set_bound = [&]() {
      c.slack = fabsf(least) * 0x1p-20f + 2 * a.margin;
      // (finite, so that blocks without a candidate, -inf, lie below it)
      c.bound = least > -INFINITY ? fmaxf(least - c.slack, kLowest) : kLowest;
      if (least == -INFINITY) c.slack = INFINITY;
    };
    set_bound();
    // ---- the blocks that reach it (of an ended beam, its token's alone: each is listed
    // once, and so is each candidate), and of them the candidates
    each_entry([&](int e, float v, float off) {
      if (v + off >= c.bound) {
        const int at = atomicAdd(&sm.blocks, 1);
        if (at < kMaxPicked) sm.pick.block[at] = e;
      }
    });
    __syncthreads();
    const int blocks = sm.blocks;
    if (blocks <= kMaxPicked) {
      // where blocks are too few for a bound, or give too low a one (a few beams far above
      // the others have all the candidates): that of the best candidates in quarters of
      // lanes' shares, so that one block fills the 128 groups
      bool lanes = least == -INFINITY;
      while (true) {
        if (lanes) {
          float quarter[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int t = warp; t < blocks << sh; t += kWarps)
            c.best_of(sm.pick.block[t >> sh], t & ((1 << sh) - 1), lane, quarter);
          __syncthreads();  // (no load uses sm.edges any more)
          float* const all = reinterpret_cast<float*>(sm.edges);
#pragma unroll
          for (int q = 0; q < 4; ++q) all[q * kThreads + threadIdx.x] = quarter[q];
          __syncthreads();
          // group 32 q + l: quarter q of lane l, of the next warp's lane l + 8, and so on,
          // since short rows fill but their warps' first lanes
          best = -INFINITY;
          if (warp < 4)
#pragma unroll 4
            for (int w = 0; w < kWarps; ++w)
              best = fmaxf(best, all[warp * kThreads + 32 * w + ((lane + 8 * w) & 31)]);
          least = fmaxf(least, group_bound(sm, best, L));
          set_bound();
        }
#pragma unroll 1
        for (int t = warp; t < blocks << sh; t += kWarps)
          c.gather(sm.pick.block[t >> sh], t & ((1 << sh) - 1), lane);
        __syncthreads();
        const bool enough = lanes || sm.picked <= kMaxPicked;
        __syncthreads();
        if (enough) break;
        lanes = true;
        if (threadIdx.x == 0) sm.picked = 0;
      }
    }
    const int picked = sm.picked;
    const bool few = blocks <= kMaxPicked && picked <= kMaxPicked;
    unsigned again;
    do {
      if (few) {
        // in order: eight lanes compare one with all
#pragma unroll 1
        for (int i0 = 0; i0 < picked; i0 += kThreads / 8) {
          const int i = i0 + threadIdx.x / 8;
          int place = 0;
          if (i < picked) {
            const uint64_t k = sm.pick.key[i];
            const uint32_t id = sm.pick.idx[i];
#pragma unroll 1
            for (int o = threadIdx.x & 7; o < picked; o += 8)
              place += better(sm.pick.key[o], sm.pick.idx[o], k, id);
          }
#pragma unroll
          for (int off = 1; off < 8; off <<= 1) place += __shfl_xor_sync(0xffffffffu, place, off);
          if (i < picked && (threadIdx.x & 7) == 0) {
            sm.key[place] = sm.pick.key[i];
            sm.idx[place] = sm.pick.idx[i];
          }
        }
        if (threadIdx.x == 0) sm.found = picked;
        __syncthreads();
        // order between rows, where their sums may not tell
        if (threadIdx.x < K)
#pragma unroll 1
          for (int i = threadIdx.x, j = i + 1;
               j < picked && key_gap(sm.key[i], sm.key[j]) < a.margin; ++j)
            c.doubt(sm.idx[i] / V, sm.idx[j] / V);
      } else {
        __syncthreads();  // (sm.pick ends here)
        choose_by_lists(c);
      }
      __syncthreads();
      again = sm.doubtful & ~c.exact;
      if (__builtin_expect(!again, 1)) break;
      sum_again(c, again, score, hands, few ? picked : 0);
      c.exact |= again;
    } while (few);
    if (!again) break;
  }
  if (hands > 1) {  // the others may go
    if (c.exact != ended) {
      if (threadIdx.x == 0) sm.call.rows = 0;
      pass_on_call(sm, hands);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }

  // ---- the choices
  for (int i = threadIdx.x; i < K; i += kThreads) {
    const int64_t at = static_cast<int64_t>(r) * K + i;
    int w = -1, token = -1;
    float value = -INFINITY;
    if (i < sm.found && sm.key[i] != 0) {  // (key 0: its value lies past fp32)
      w = sm.idx[i] / V;
      token = sm.idx[i] - static_cast<uint32_t>(w) * V;
      value = 2.f * unordered(static_cast<uint32_t>(sm.key[i] >> 32));
    }
    a.parents[at] = w;
    a.tokens[at] = token;
    a.out_scores[at] = value;
    if (a.out_finished)
      a.out_finished[at] = w >= 0 && (((ended >> w) & 1) || token == a.end_token);
  }
  __syncwarp();
  if (hands > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int KL>
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(int requests, int ctas, int smem, cudaStream_t stream) {
    cfg.gridDim = dim3(static_cast<unsigned>(requests) * static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// The largest cluster, up to *ctas, of which as many as there are requests run at once: a
// cluster lies within one part of the device, and parts differ in size.  (At two CTAs an
// SM 14 clusters of 16 run at once, 19 of 13, 36 of 8, 74 of 4: sixteen requests of
// 16 x 131072 in fp32 took 35.3 us in clusters of 16, of which two began 13 us late, and
// take 32.8 in clusters of 13.)  What the device answers for a size is asked once.
template <typename T, int KL>
cudaError_t fit_cluster(int requests, int* ctas) {
  const auto kernel = beam_select_kernel<T, KL>;
  static std::mutex mu;
  static bool set_for[64] = {};
  static int at_once[64][kMaxCtas + 1] = {};  // 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!set_for[dev]) {  // allow clusters of 16
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxEntries * 4);
    if (e != cudaSuccess) return e;
    set_for[dev] = true;
  }
  for (; *ctas > 1; --*ctas) {
    int& n = at_once[dev][*ctas];
    if (n == 0) {
      const Launch<T, KL> one(1, *ctas, kMaxEntries * 4, nullptr);
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &one.cfg);
      if (e != cudaSuccess) return e;
    }
    if (n >= requests) break;
  }
  return cudaSuccess;
}

template <typename T, int KL>
cudaError_t launch(BeamSelectArgs a, int num_sms, cudaStream_t stream) {
  const int lead = Elem<T>::kVec - 1;  // a row may begin anywhere in its first 32 bytes
  const int elems = 32 * kVecs * (lead + 1);  // of a warp load
  const int64_t steps = (static_cast<int64_t>(a.vocab) + lead + elems - 1) / elems;
  int sh = 0;
  while (((steps + (1 << sh) - 1) >> sh) * a.num_beams > kMaxEntries) ++sh;
  a.block_shift = sh;
  a.blocks_per_row = static_cast<int>((steps + (1 << sh) - 1) >> sh);
  // e / blocks_per_row = e * inverse / 2^32 for e < kMaxEntries
  a.blocks_inverse = static_cast<uint32_t>(((int64_t{1} << 32) - 1) / a.blocks_per_row + 1);
  // As many CTAs per request as run at once, two on an SM; one on an SM where that leaves
  // a warp at most two loads, since a second one delays the choice more than it speeds
  // the pass (us, one / two: 1.6 loads a warp, 100 requests of 4 x 10000 10.2 / 11.2; 1.9,
  // 150 of 5 x 3000 in fp32 12.1 / 13.5; 2.3, 37 of 3 x 50001 10.3 / 9.8; 3.2, 60 of
  // 4 x 32000 12.4 / 11.9; 64 of 4 x 131072 27.0 / 19.3, 16 of 16 x 131072 in fp32
  // 36.6 / 32.8).
  const int64_t loads = (static_cast<int64_t>(a.num_beams) * a.blocks_per_row << sh) *
                        a.num_requests;
  const int64_t most = (loads <= 2ll * kWarps * num_sms ? 1 : 2) * static_cast<int64_t>(num_sms);
  int ctas = static_cast<int>(std::min<int64_t>(std::max<int64_t>(most / a.num_requests, 1),
                                                kMaxCtas));
  if (const cudaError_t e = fit_cluster<T, KL>(a.num_requests, &ctas)) return e;
  // The margin of two rows is twice the error of a row's sum in the pass, relative, all
  // roundings adding up (a step of fp32 is 2^-24): exponentials 4 steps, their arguments
  // kArgSteps |x - m| (a weighted mean of which is at most ln V, and kMove); additions of a
  // lane, 10 and one for each load, a warp, a CTA and a cluster; rescalings by an
  // exponential, 5 and its argument's, once for a lane (a moved reference shrinks what came
  // before) and at each of the three; the logarithm's 2 ln V.
  const int64_t lane_loads =
      (static_cast<int64_t>(a.num_beams) * (a.blocks_per_row / ctas + 1) / kWarps + 1) << sh;
  const double ln_v = log(static_cast<double>(a.vocab));
  const double err =
      0x1p-24 * (4 + kArgSteps * (kMove + ln_v) + 10 + static_cast<double>(lane_loads) + 5 + 4 +
                 4 + 4 * (5 + kArgSteps * kMove) + 2 * ln_v);
  a.margin = static_cast<float>(err);  // (of values that are halved)
  // Where a second sum of two rows is likely (neighbours among the best candidates nearer
  // than the margin: 3 of 100 calls of 16 requests of 16 x 131072, 32 choices; nearly all of
  // 103 of 6 x 50497, 57 choices) or takes long, the cluster stays for it:
  // 0.5 us of every call (64 of 4 x 131072 19.8 / 19.3, 37 of 3 x 50001 10.3 / 9.7),
  // against 53 us of one CTA's time for two rows of 131072 in fp32.
  a.all_sum = static_cast<int64_t>(a.num_requests) * a.num_choices * a.vocab >= 1 << 21;
  const Launch<T, KL> l(a.num_requests, ctas, a.num_beams * a.blocks_per_row * 4, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, beam_select_kernel<T, KL>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectArgs& a, bool fp32, int num_sms,
                               cudaStream_t stream) {
  const bool wide = a.num_choices + 1 > 32;
  if (fp32)
    return wide ? launch<float, 3>(a, num_sms, stream) : launch<float, 1>(a, num_sms, stream);
  return wide ? launch<__nv_bfloat16, 3>(a, num_sms, stream)
              : launch<__nv_bfloat16, 1>(a, num_sms, stream);
}

}  // namespace pa
