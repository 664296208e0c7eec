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
// a maximum.  A cluster serves a request, its CTAs take a share of every row,
// a warp 512 bf16 (256 fp32) elements at a time, 32 bytes a lane; the maxima of
// such blocks and the rows' (maximum, sum) go to the cluster's first CTA.
//
// Selection, in that CTA: the K best candidates lie in the K blocks with the best
// (s_w - lse_w + block maximum), ties to the first: each other block's best
// candidate comes behind K blocks' best.  So K blocks are read again (from L2),
// and of them the candidates that are not below the K-th block's best: a few more
// than K.  Lists are kept sorted in a warp's registers, a lane each.
//
// Exactness.  Within a row the logits themselves give the order.  Between rows it
// hangs on lse_w, which the pass knows to `margin` / 2: values are kept as sums
// of two floats (48 bits), and where two beams' candidates around the choice are
// nearer than `margin`, those rows' sums are taken again, to 1e-9: exponentials by
// table and short polynomial (Tang's method) in two floats, added as whole numbers,
// so that equal logits in whatever order and place give equal sums.
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

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnroll = 4;     // loads a warp has under way
constexpr int kMaxCtas = 16;   // of a cluster
constexpr int kMaxEntries = 8192;  // block maxima of a request
constexpr float kLog2e = 1.4426950408889634f;

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
  static __device__ __forceinline__ void put(uint32_t (&v)[8], int i, float x) {
    const uint32_t b = __float_as_uint(x) >> 16;  // (x is a bf16 value)
    v[i / 2] = (i & 1) ? (v[i / 2] & 0xffffu) | (b << 16) : (v[i / 2] & 0xffff0000u) | b;
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
  static __device__ __forceinline__ void put(uint32_t (&v)[8], int i, float x) {
    v[i] = __float_as_uint(x);
  }
  static __device__ __forceinline__ float max(const uint32_t (&v)[8]) {
    float m = __uint_as_float(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(v[i]));
    return m;
  }
};

// A beam's logits in vectors of 32 aligned bytes: vector i holds the elements
// [kVec * i - lead, + kVec), as far as the row has them.
template <typename T>
struct Row {
  using E = Elem<T>;
  const T* p;
  int lead;
  int vecs;
  int vocab;
  __device__ __forceinline__ Row(const BeamSelectArgs& a, int r, int w) {
    p = static_cast<const T*>(a.logits) + r * a.request_stride + w * a.beam_stride;
    vocab = a.vocab;
    lead = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 31) / static_cast<int>(sizeof(T));
    vecs = (lead + vocab + E::kVec - 1) / E::kVec;
  }
  // Vector i, -inf outside the row.  The first and the last one may be partial: they
  // go through `edges`, 64 bytes of the warp's.
  __device__ __forceinline__ void load(int i, uint32_t (&v)[8], uint4* edges) const {
    const int e = i * E::kVec - lead;
    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // (-inf)
    if (i < vecs && e >= 0 && e <= vocab - E::kVec) {
      ldg32(p + e, v);
    } else if (i < vecs) {
      uint4* const mine = edges + (i == 0 ? 0 : 2);
      T* const t = reinterpret_cast<T*>(mine);
#pragma unroll 1
      for (int j = 0; j < E::kVec; ++j)
        t[j] = e + j >= 0 && e + j < vocab ? p[e + j] : static_cast<T>(-INFINITY);
      const uint4 lo = mine[0], hi = mine[1];
      v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
      v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = none;
    }
  }
  __device__ __forceinline__ int blocks(int shift) const {
    return (((vecs + 31) >> 5) + (1 << shift) - 1) >> shift;
  }
};

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
__device__ __forceinline__ uint64_t value_key(float2 base, float x) {
  const float2 s = two_sum(base.x, x);
  const float2 v = two_sum(s.x, __fadd_rn(s.y, base.y));
  if (!(v.x > -INFINITY && v.x < INFINITY)) return 0;
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

// 2^(j / 64), as a sum of two floats, j < 64: for sums that need more than fp32.
struct ExpTable {
  float2 t[64];
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
  const int k = static_cast<int>(n);
  const float2 b = tab.t[k & 63];
  const float scale = __uint_as_float(static_cast<uint32_t>((k >> 6) + 127 + 50) << 23);
  const float hi = b.x * scale;
  sum.add(static_cast<uint64_t>(__float2ll_rn(hi) + __float2ll_rn(__fmaf_rn(hi, p, b.y * scale))));
}

// Shared memory besides the block maxima.
template <int KL>
struct SelectSmem {
  uint4 edges[kWarps][4];            // of rows, elements on their way to registers
  float2 part[kMaxBeams][kMaxCtas];  // rows' (maximum, sum) of each CTA
  float2 red[kMaxBeams][kWarps];     // and of each warp
  float2 base[kMaxBeams];            // s - lse in two floats
  float top[kMaxBeams];              // rows' maxima
  uint64_t list_key[kWarps][32 * KL];
  uint32_t list_idx[kWarps][32 * KL];
  uint64_t key[32 * KL];  // the lists' best, in order
  uint32_t idx[32 * KL];
  uint64_t floor[kWarps];
  FixedSum sum[kWarps];
  unsigned doubtful;  // rows whose sums are to be taken again
  int found;
  ExpTable table;
};

// The best `n` of the warps' lists into sm.key / sm.idx, their number into sm.found.
// Called by the whole CTA.
template <int KL>
__device__ __forceinline__ void join_lists(SelectSmem<KL>& sm, const WarpList<KL>& mine, int n,
                                           int warp, int lane) {
#pragma unroll
  for (int r = 0; r < KL; ++r) {
    sm.list_key[warp][32 * r + lane] = mine.key[r];
    sm.list_idx[warp][32 * r + lane] = mine.idx[r];
  }
  if (threadIdx.x == 0) sm.found = 0;
  __syncthreads();
  for (int t = threadIdx.x; t < kWarps * n; t += kThreads) {
    const int w = t / n, at = t - w * n;
    const uint64_t k = sm.list_key[w][at];
    const uint32_t i = sm.list_idx[w][at];
    if (k == 0) continue;
    int rank = at;
#pragma unroll
    for (int o = 1; o < kWarps; ++o) {
      const int l = (w + o) % kWarps;
      int lo = 0, hi = n;  // how many of list l come before
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (better(sm.list_key[l][mid], sm.list_idx[l][mid], k, i))
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

template <typename T, int KL>
__global__ void __launch_bounds__(kThreads, 3) beam_select_kernel(const BeamSelectArgs a) {
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
  // the first CTA runs before its shared memory is written
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

  // ---- the pass over the logits
  const uint32_t remote_max = mapa_shared(smem_u32(block_max), 0);
  for (unsigned todo = live; todo; todo &= todo - 1) {
    const int w = __ffs(todo) - 1;
    const Row<T> row(a, r, w);
    const int blocks = row.blocks(sh);
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / C);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / C);
    // this warp's blocks b0 + warp, + kWarps ..., a warp load at a time
    const int mine = b1 - b0 > warp ? ((b1 - b0 - warp + kWarps - 1) / kWarps) << sh : 0;
    float m = -INFINITY, s = 0.f, bm = -INFINITY;
    for (int q0 = 0; q0 < mine; q0 += kUnroll) {
      uint32_t v[kUnroll][8];
      auto step_of = [&](int q) {
        return ((b0 + warp + kWarps * (q >> sh)) << sh) + (q & ((1 << sh) - 1));
      };
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = q0 + u;
        row.load(q < mine ? step_of(q) * 32 + lane : row.vecs, v[u], sm.edges[warp]);
      }
      float mx[kUnroll], total = 0.f, ref = 0.f, m_new = m;
      bool clean = false;
      while (true) {
        m_new = m;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          mx[u] = E::max(v[u]);
          m_new = fmaxf(m_new, mx[u]);
        }
        ref = fmaxf(m_new, -FLT_MAX);  // finite
        const uint64_t nref = f32x2(-ref, -ref), scale = f32x2(kLog2e, kLog2e);
        uint64_t acc = 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < E::kVec / 2; ++i) {
            const float2 x = E::pair(v[u], i);
            const float2 d = f32x2_parts(mul2(add2(f32x2(x.x, x.y), nref), scale));
            sums[i & 1] = add2(sums[i & 1], f32x2(fast_exp2(d.x), fast_exp2(d.y)));
          }
          acc = add2(acc, add2(sums[0], sums[1]));
        }
        const float2 two = f32x2_parts(acc);
        total = two.x + two.y;
        // NaN or +inf among them: once more without
        if (clean || (m_new < INFINITY && total == total)) break;
        clean = true;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
          for (int i = 0; i < E::kVec / 2; ++i) {
            const float2 x = E::pair(v[u], i);
            E::put(v[u], 2 * i, sane(x.x));
            E::put(v[u], 2 * i + 1, sane(x.y));
          }
      }
      s = s * fast_exp2((m - ref) * kLog2e) + total;  // (s is 0 where m is -inf)
      m = m_new;
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = q0 + u;
        bm = fmaxf(bm, warp_max(mx[u]));
        if (q < mine && ((q + 1) & ((1 << sh) - 1)) == 0) {
          if (lane == 0)
            st_remote(remote_max + 4 * (w * NB + b0 + warp + kWarps * (q >> sh)), bm);
          bm = -INFINITY;
        }
      }
    }
    const float top = warp_max(m);
    s *= fast_exp2((m - fmaxf(top, -FLT_MAX)) * kLog2e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) sm.red[w][warp] = make_float2(top, s);
  }
  __syncthreads();
  if (threadIdx.x < W && ((live >> threadIdx.x) & 1)) {
    const int w = threadIdx.x;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sm.red[w][i].x);
    float s[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
      s[i] = sm.red[w][i].y * fast_exp2((sm.red[w][i].x - fmaxf(top, -FLT_MAX)) * kLog2e);
#pragma unroll
    for (int h = kWarps / 2; h > 0; h >>= 1)
#pragma unroll
      for (int i = 0; i < h; ++i) s[i] += s[i + h];
    const uint32_t at = mapa_shared(smem_u32(&sm.part[w][rank]), 0);
    st_remote(at, top);
    st_remote(at + 4, s[0]);
  }
  cluster_sync();
  if (rank != 0) return;

  // ---- the first CTA: s - lse of each row
  for (int w = warp; w < W; w += kWarps) {
    if (!((live >> w) & 1)) continue;
    const float2 x = lane < C ? sm.part[w][lane] : make_float2(-INFINITY, 0.f);
    const float top = warp_max(x.x);
    float s = x.y * fast_exp2((x.x - fmaxf(top, -FLT_MAX)) * kLog2e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mine = __shfl_sync(0xffffffffu, score, w);
    if (lane == 0) {
      // (a row of -inf: no candidates, whatever the base)
      const double b = s > 0.f ? (mine - static_cast<double>(top)) - log(static_cast<double>(s))
                               : 0.0;
      const float hi = static_cast<float>(b);
      sm.base[w] = make_float2(hi, static_cast<float>(b - hi));
      sm.top[w] = top;
    }
  }
  if (warp == 0 && state == kEnded) sm.base[lane] = make_float2(score, 0.f);
  const int K = a.num_choices, L = K + 1;
  unsigned exact = ended;  // rows whose base is known to 1e-9
  __syncthreads();

  // the value of a row's block's best candidate
  auto entry_key = [&](int w, int b) -> uint64_t {
    if ((live >> w) & 1) {
      const Row<T> row(a, r, w);
      return b < row.blocks(sh) ? value_key(sm.base[w], block_max[w * NB + b]) : 0;
    }
    if ((ended >> w) & 1) {
      const Row<T> row(a, r, w);
      return b == (((a.end_token + row.lead) / E::kVec) >> 5) >> sh
                 ? value_key(sm.base[w], 0.f)
                 : 0;
    }
    return 0;
  };

  while (true) {
    WarpList<KL> list;
    // ---- the L best blocks
    const int entries = W * NB;
    uint64_t best = 0;
    for (int e = threadIdx.x; e < entries; e += kThreads) {
      const uint64_t k = entry_key(e / NB, e % NB);
      best = k > best ? k : best;
    }
    uint64_t floor = 0;
    if (L <= 32) {
      // L lanes of a warp have a block that is as good as its L-th lane's
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int off = size / 2; off > 0; off >>= 1) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
          const bool up = ((lane & off) == 0) == ((lane & size) == 0 || size == 32);
          best = (o > best) == up ? o : best;
        }
      if (lane == L - 1) sm.floor[warp] = best;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; ++i) floor = sm.floor[i] > floor ? sm.floor[i] : floor;
    }
    list.clear();
    for (int e0 = warp * 32; e0 < entries; e0 += kThreads) {
      const int e = e0 + lane;
      list.offer(e < entries ? entry_key(e / NB, e % NB) : 0, e, floor, lane);
    }
    join_lists(sm, list, L, warp, lane);
    // ---- the L best candidates of these blocks
    const int chosen = sm.found;
    floor = chosen == L ? sm.key[L - 1] : 0;
    const float floor_value = floor ? unordered(static_cast<uint32_t>(floor >> 32)) : -FLT_MAX;
    list.clear();
    for (int t = warp; t < chosen << sh; t += kWarps) {
      const int e = sm.idx[t >> sh];
      const int w = e / NB, b = e % NB;
      const float2 base = sm.base[w];
      if ((ended >> w) & 1) {
        if ((t & ((1 << sh) - 1)) == 0)
          list.offer(lane == 0 ? value_key(base, 0.f) : 0,
                     static_cast<uint32_t>(w) * V + a.end_token, floor, lane);
        continue;
      }
      const Row<T> row(a, r, w);
      const int i = ((b << sh) + (t & ((1 << sh) - 1))) * 32 + lane;
      uint32_t v[8];
      row.load(i, v, sm.edges[warp]);
      // logits from here on may reach the floor (two roundings of the sums)
      const float slack = (fabsf(floor_value) + fabsf(base.x)) * 0x1p-21f;
      const float least = (floor_value - base.x) - slack;
      unsigned hits = 0;
#pragma unroll
      for (int j = 0; j < E::kVec / 2; ++j) {
        const float2 x = E::pair(v, j);
        hits |= (x.x >= least ? 1u : 0u) << (2 * j) | (x.y >= least ? 1u : 0u) << (2 * j + 1);
      }
      while (__any_sync(0xffffffffu, hits != 0)) {
        uint64_t k = 0;
        uint32_t id = 0;
        if (hits) {
          const int x = i * E::kVec - row.lead + __ffs(hits) - 1;
          hits &= hits - 1;
          if (x >= 0 && x < V) {
            k = value_key(base, sane(E::load(row.p, x)));
            id = static_cast<uint32_t>(w) * V + x;
          }
        }
        __syncwarp();
        list.offer(k, id, floor, lane);
      }
    }
    __syncthreads();  // sm.idx has been read
    join_lists(sm, list, L, warp, lane);
    // ---- order between rows, where their sums may not tell
    if (threadIdx.x == 0) sm.doubtful = 0;
    __syncthreads();
    const int found = sm.found;
    for (int i = threadIdx.x; i < K && i + 1 < found; i += kThreads) {
      const int w0 = sm.idx[i] / V, w1 = sm.idx[i + 1] / V;
      const unsigned both = 1u << w0 | 1u << w1;
      if (w0 != w1 && (both & ~exact) && key_gap(sm.key[i], sm.key[i + 1]) < a.margin)
        atomicOr(&sm.doubtful, both);
    }
    if (found == L) {
      // Another row's candidate next to the last choice, displaced by candidates of
      // that choice's own row?
      const uint64_t last = sm.key[K - 1];
      const int w0 = sm.idx[K - 1] / V;
      if (static_cast<int>(sm.idx[K] / V) == w0 && key_gap(last, sm.key[K]) < a.margin) {
        for (int e = threadIdx.x; e < entries; e += kThreads) {
          const int w = e / NB, b = e % NB;
          const unsigned both = 1u << w0 | 1u << w;
          if (w == w0 || !(both & ~exact)) continue;
          const uint64_t k = entry_key(w, b);
          if (k == 0 || key_gap(last, k) >= a.margin) continue;
          bool near = k < last;
          if (!near && ((live >> w) & 1)) {
            const Row<T> row(a, r, w);
            const int x0 = ((b << sh) * 32) * E::kVec - row.lead;
            const int x1 = min(V, x0 + (32 << sh) * E::kVec);
            for (int x = max(0, x0); x < x1 && !near; ++x) {
              const uint64_t kx = value_key(sm.base[w], sane(E::load(row.p, x)));
              near = kx != 0 && kx < last && key_gap(last, kx) < a.margin;
            }
          }
          if (near) atomicOr(&sm.doubtful, both);
        }
      }
    }
    __syncthreads();
    const unsigned again = sm.doubtful & ~exact;
    if (!again) break;
    // ---- those rows' sums once more
    if (threadIdx.x < 64) {
      const double t = exp2(threadIdx.x / 64.0);
      const float hi = static_cast<float>(t);
      sm.table.t[threadIdx.x] = make_float2(hi, static_cast<float>(t - hi));
    }
    __syncthreads();
    for (unsigned todo = again; todo; todo &= todo - 1) {
      const int w = __ffs(todo) - 1;
      const Row<T> row(a, r, w);
      const float top = sm.top[w];
      FixedSum sum;
      for (int x = threadIdx.x; x < V; x += kThreads)
        add_exp(sum, sm.table, sane(E::load(row.p, x)), top);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        sum.hi += __shfl_xor_sync(0xffffffffu, sum.hi, off);
        sum.lo += __shfl_xor_sync(0xffffffffu, sum.lo, off);
      }
      if (lane == 0) sm.sum[warp] = sum;
      __syncthreads();
      const float mine = __shfl_sync(0xffffffffu, score, w);
      if (threadIdx.x == 0) {
        for (int i = 1; i < kWarps; ++i) {
          sum.hi += sm.sum[i].hi;
          sum.lo += sm.sum[i].lo;
        }
        const double s = static_cast<double>(sum.hi) * 0x1p-18 +
                         static_cast<double>(sum.lo) * 0x1p-50;
        const double b = (mine - static_cast<double>(top)) - log(s);
        const float hi = static_cast<float>(b);
        sm.base[w] = make_float2(hi, static_cast<float>(b - hi));
      }
      __syncthreads();
    }
    exact |= again;
  }

  // ---- the choices
  for (int i = threadIdx.x; i < K; i += kThreads) {
    const int64_t at = static_cast<int64_t>(r) * K + i;
    int w = -1, token = -1;
    float value = -INFINITY;
    if (i < sm.found) {
      w = sm.idx[i] / V;
      token = sm.idx[i] - static_cast<uint32_t>(w) * V;
      value = unordered(static_cast<uint32_t>(sm.key[i] >> 32));
    }
    a.parents[at] = w;
    a.tokens[at] = token;
    a.out_scores[at] = value;
    if (a.out_finished)
      a.out_finished[at] = w >= 0 && (((ended >> w) & 1) || token == a.end_token);
  }
}

template <typename T, int KL>
cudaError_t launch(const BeamSelectArgs& a, int ctas, cudaStream_t stream) {
  const int smem = a.num_beams * a.blocks_per_row * 4;
  {  // allow clusters of 16, once per device
    static std::mutex mu;
    static bool set_for[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!set_for[dev]) {
      e = cudaFuncSetAttribute(beam_select_kernel<T, KL>,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(beam_select_kernel<T, KL>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxEntries * 4);
      if (e != cudaSuccess) return e;
      set_for[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_requests) * static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, beam_select_kernel<T, KL>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(BeamSelectArgs a, bool fp32, int num_sms, cudaStream_t stream) {
  const int elems = 32 * (fp32 ? 8 : 16);  // of a warp load
  // a row may begin anywhere in its first 32 bytes
  const int64_t steps = (static_cast<int64_t>(a.vocab) + elems / 32 - 1 + elems - 1) / elems;
  int sh = 0;
  while (((steps + (1 << sh) - 1) >> sh) * a.num_beams > kMaxEntries) ++sh;
  a.block_shift = sh;
  a.blocks_per_row = static_cast<int>((steps + (1 << sh) - 1) >> sh);
  const int ctas = kMaxCtas / 2;
  // Twice the error of a row's sum in the pass, relative, all roundings adding up:
  // exponentials 2^-22, their arguments 1.3 * 2^-24 |x - m| (a weighted mean of which is
  // at most ln V), the additions of a lane (9 in a step of 4 loads, 3 more for each step),
  // a warp, the CTA and the cluster, a rescaling by an exponential at each of the three.
  const double chain = 9 + static_cast<double>((steps + ctas * kWarps * kUnroll - 1) /
                                               (ctas * kWarps * kUnroll)) * 3 + 5 + 3 + 5;
  const double err = 0x1p-22 * 4 + 1.3 * 0x1p-24 * (4 + log(static_cast<double>(a.vocab))) +
                     chain * 0x1p-24;
  a.margin = static_cast<float>(2 * err);
  const bool wide = a.num_choices + 1 > 32;
  if (fp32) return wide ? launch<float, 3>(a, ctas, stream) : launch<float, 1>(a, ctas, stream);
  return wide ? launch<__nv_bfloat16, 3>(a, ctas, stream)
              : launch<__nv_bfloat16, 1>(a, ctas, stream);
}

}  // namespace pa
