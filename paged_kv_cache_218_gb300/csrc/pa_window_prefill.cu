// pa_window_prefill.cu -- causal paged prefill chunks under a sliding window
// and a few first tokens that stay visible, on tcgen05 tensor cores (sm_103a).
//
// A query at position p sees the keys j <= p with j < sinks or p - j < window.
// The tensor-core pipeline of a tile is pa_prefill_body.cuh's: CTA pairs
// (cta_group::2) on two consecutive query tiles of a kv head, K and V halves
// loaded by each CTA, three score buffers in tensor memory, online softmax
// with P written back over its scores.  What a window changes:
//
//  * Key tiles run over a list of blocks, not over positions: the sinks'
//    blocks [0, nsb), then the blocks from the one that holds the first key
//    of the pair's first row's window on.  A list index is a "virtual" block;
//    virtual key = key - shift behind the sinks, where shift is 16 times the
//    blocks left out.  So a few sinks cost a few rows of the first tile, and
//    blocks that no row sees are neither loaded nor looked up.
//  * A row's mask over a 64-column half of a tile is
//    vk <= hi && (vk < sinks || vk >= lo): one 64-bit mask per row and half,
//    built from three counts; halves that all rows of a warp see whole skip
//    it.
//  * V rows that no row of the pair may see (ends of the sinks' and of the
//    window's first block, slots behind the last key) are zeroed in shared
//    memory before the product: they may hold anything, and 0 * NaN is NaN.
//  * Work per query tile is short (window / 128 key tiles), so setting up and
//    draining a pipeline per tile would cost as much as the tile.  The launch
//    is persistent: one CTA pair per two SMs walks (chunk, query tile, kv head)
//    items; barriers, rings and phases run on across items, and Q has two
//    buffers.  A pair's items are every pairs-th of the list; the K loader finds
//    them with a warp-wide scan over the chunks' lengths (so ragged chunks leave
//    no empty items) and publishes them, one ahead of its loads, in a ring that
//    the other roles read.  Block ids of the next item are fetched while the
//    last one's tiles load, and the softmax writes P of an item's first tile
//    before it turns to the output of the item before, whose last product is
//    then done.  Outputs are turned around in shared memory, so that a store
//    instruction covers whole 128-byte lines (written straight from the
//    registers, a row per lane, they took 1.6 us per item; as a tensor store
//    per warp, 0.8, half of it the proxy fence and the issue).
//
// Weights enter the second product rounded to bf16, as tensor memory holds them for
// it, each within 2^-8 of itself (the normalizer sums them unrounded): the output is
// within 0.0023 of 64 bits (root mean square, relative) where rounding only at the
// end gives 0.0017.  The low halves in a product of their own, as in the decode
// kernel, would take this kernel's bound, the tensor pipe, half as long again.
//
// What bounds it.  In long windows the tensor pipe and its hand-overs: 0.75 us per
// pair and key tile (8192 queries, windows of 2048 and 4096), 1.70 PFLOP/s over the
// device at 1.93 GHz, where cuBLAS reaches 1.92 in a burst and the products alone
// would take 0.53 us; 8192 queries x 4096 keys take 390 us in a graph (1.45 PFLOP/s
// of the products that the masks leave), 405 to 414 called one by one.  In
// short ones instruction fetches: the roles' loops go through 50 KB of code per
// item, more than an SM caches, and the cache behind it serves a whole GPC.  So
// each role is one loop with one copy of each step, the masks are a loop over
// tensor memory in front of a tile's only softmax, waits share their slow path,
// and divisions by the group are shifts.  With 124 KB of code (a first tile and
// masked tiles of their own, three searches for the next item) that cache was at
// 78 % of its request rate, SMs of full GPCs took 20 % longer than others, and an
// item's ends took 3.9 us; now 2.7.  Only the products stay unrolled: their
// issue is on the critical path (a tile rolled by two took 0.16 us more).
// Every mbarrier wait is bounded, as in pa_prefill_body.cuh.
#include <mutex>

#include "pa_prefill_body.cuh"
#include "pa_window.h"
#include "pa_window_ptx.cuh"

namespace pa {
namespace pre {
namespace {

constexpr uint64_t kSettleNs = 1000000;  // far longer than any copy takes
// Reference maximum (log2 units) of a row that saw nothing yet: next to the lowest
// fp32, so that no visible score lies below it; hidden scores (-inf) weigh 0.
constexpr float kFloor = -0x1.fffff0p127f;
constexpr float kFarScore = 0x1p31f;  // (log2 units)

// Shared memory of one CTA of a pair: two Q tiles, four K and three V half
// tiles, an output tile, block ids of both loaders, the softmax's exchange, barriers.
struct WPlan {
  static constexpr int kNK = 4, kNV = 3;
  static constexpr int kKSlot = kHalf, kVSlot = kHalf;
  static constexpr int kQOff = 0;  // [2][2 * kHalf]
  static constexpr int kKOff = kQOff + 4 * kHalf;
  static constexpr int kVOff = kKOff + kNK * kKSlot;
  static constexpr int kOutOff = kVOff + kNV * kVSlot;  // [2 halves][128 rows][64 columns]
  static constexpr int kIdsOff = kOutOff + 2 * kHalf;
  static constexpr int kRedOff = kIdsOff + 2 * kIdRing * 8 * 4;
  static constexpr int kRedOff2 = kRedOff + 2 * 2 * 128 * 4;
  static constexpr int kBarOff = kRedOff2 + 2 * 128 * 4;
  static constexpr int kItemsOff = kBarOff + 448;  // [kItemRing]
  static constexpr int kSmemBytes = kItemsOff + 8 * 64;
};
static_assert(WPlan::kSmemBytes + 1024 <= 227 * 1024, "shared memory of one CTA");

// One work item of a pair: query tiles 2 mg, 2 mg + 1 of a chunk, one kv head.
struct Item {
  int nkt;          // key tiles; 0 ends the list
  int c, kvh;
  int q0, qlen, p0; // the chunk's rows and first position
  int tc0;          // first query token of the pair
  int kmax;         // keys [0, kmax) are visible to some row, window and sinks aside
  int lo;           // first key of the first row's window
  int nsb, b_first; // the sinks' blocks; first block behind them
  int nvb;          // virtual blocks
  int edge[3];      // tiles with rows that no row of the pair sees, or -1
};
// Blocks of an item's key tile j: eight, fewer in the last one.
__device__ __forceinline__ int tile_blocks(int nvb, int j) { return min(8, nvb - 8 * j); }

constexpr int kItemRing = 8;
static_assert(sizeof(Item) <= 64, "ring slot");

// Walks a pair's items: every `stride`-th of the list.
struct Cursor {
  int want;    // list index of the next item
  int before;  // items of the chunks before `chunk`
  int chunk;
};

static_assert(kBlockSize == 16, "shifts below");
__device__ __forceinline__ int blocks_of(int keys) { return (keys + 15) >> 4; }

// Rows of virtual blocks that no row of the pair sees: at most three ranges.
struct Hidden {
  int vb[3], r0[3], r1[3];  // rows [r0, r1) of block vb; vb < 0: none
  __device__ __forceinline__ Hidden(const Item& it, int sinks) {
#pragma unroll
    for (int e = 0; e < 3; ++e) vb[e] = -1;
    auto set = [&](int e, int b, int from, int to) {
      if (from < to) {
        vb[e] = b;
        r0[e] = from;
        r1[e] = to;
      }
    };
    // between the sinks and the window, in the sinks' last block
    if (it.nsb > 0) {
      const int base = (it.nsb - 1) * kBlockSize;
      set(0, it.nsb - 1, min(sinks, it.kmax) - base, min(kBlockSize, it.lo - base));
    }
    // before the window, in its first block
    if (it.lo >> 4 >= it.nsb) set(1, it.nsb, 0, it.lo & 15);
    // behind the last key
    if (it.kmax & 15) set(2, it.nvb - 1, it.kmax & 15, kBlockSize);
  }
};

// The next item (nkt 0 at the end of the list).  Called by a whole warp.  The
// caller that passes flag = true reports chunks with inconsistent metadata.
__device__ __forceinline__ Item next_item(const WindowPrefillArgs& a, Cursor& cur, int stride,
                                          int lane, bool flag) {
  Item it;
  it.nkt = 0;
  const int rs = 9 - __ffs(a.group);  // log2 of the query tokens per item (a group divides 128)
  const int rows = 1 << rs;
  while (cur.chunk < a.num_chunks) {
    // items of 32 chunks at a time, and their inclusive sums
    const int c = cur.chunk + lane;
    int items = 0, q0 = 0, q1 = 0, p0 = 0;
    if (c < a.num_chunks) {
      q0 = a.cu_q_lens[c];
      q1 = a.cu_q_lens[c + 1];
      p0 = a.q_start_pos[c];
      if (chunk_ok(q0, q1, p0, a.seq_lens[c], a.total_q, a.max_blocks))
        items = ((q1 - q0 + rows - 1) >> rs) * a.num_kv_heads;
      else if (flag)
        atomicOr(a.err, PA_DEVERR_CHUNK);
    }
    int sum = items;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, cur.before + sum > cur.want);
    if (past == 0) {
      cur.before += __shfl_sync(0xffffffffu, sum, 31);
      cur.chunk += 32;
      continue;
    }
    const int w = __ffs(past) - 1;
    cur.before += __shfl_sync(0xffffffffu, sum - items, w);
    const int at = cur.want - cur.before;
    cur.chunk += w;
    cur.want += stride;
    it.c = cur.chunk;
    it.q0 = __shfl_sync(0xffffffffu, q0, w);
    it.qlen = __shfl_sync(0xffffffffu, q1 - q0, w);
    it.p0 = __shfl_sync(0xffffffffu, p0, w);
    const int tile = at / a.num_kv_heads;
    it.kvh = at - tile * a.num_kv_heads;
    // last query tiles first: where the window has not closed they are longest
    it.tc0 = (((it.qlen + rows - 1) >> rs) - 1 - tile) << rs;
    it.kmax = it.p0 + min(it.qlen, it.tc0 + rows);
    it.lo = max(0, it.p0 + it.tc0 - (a.window - 1));
    const int ns = min(a.sinks, it.kmax);
    it.nsb = blocks_of(ns);
    it.b_first = max(it.lo >> 4, it.nsb);
    it.nvb = it.nsb + max(0, blocks_of(it.kmax) - it.b_first);
    it.nkt = (it.nvb + 7) >> 3;
    const Hidden hid(it, a.sinks);
#pragma unroll
    for (int e = 0; e < 3; ++e) it.edge[e] = hid.vb[e] >> 3;  // (-1 stays)
    break;
  }
  return it;
}

// The waits of pa_prefill_body.cuh with one copy of what follows a first
// attempt: code size decides how long an item's ends take.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort,
                                     unsigned int* err, uint64_t limit_ns) {
  if (*abort) return false;
  if (mbar_wait(bar, parity, limit_ns)) return true;
  *abort = 1;
  atomicOr(err, PA_DEVERR_TIMEOUT);
  return false;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                     const WindowPrefillArgs& a) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, a.err, a.wait_ns);
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          const WindowPrefillArgs& a) {
  bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  if (!ok) {
    ok = wait_on(bar, parity, abort, a.err, a.wait_ns);
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// Ids of an item's virtual blocks [8 t_first, + 8 kIdBatch) into a loader's
// ring, where the ids of the warp's tile T are at slot T % kIdRing and `base` is
// the number of the item's tile 0.  A slot is rewritten only when its tile's
// loads have been issued.  Ids past the list are -1, a box outside the pool,
// which reads as zeros.  Called by a whole warp.
__device__ __noinline__ void fetch_ids(const int32_t* table, int64_t num_blocks, unsigned int* err,
                                       int* ids, int nsb, int b_first, int nvb, int t_first,
                                       unsigned base) {
  const int lane = threadIdx.x & 31;
  int v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int vb = t_first * 8 + lane + 32 * i;
    v[i] = vb < nvb ? table[vb < nsb ? vb : vb - nsb + b_first] : -1;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int vb = t_first * 8 + lane + 32 * i;
    if (vb < nvb && (v[i] < 0 || v[i] >= num_blocks)) {
      atomicOr(err, PA_DEVERR_BLOCK_ID);
      v[i] = -1;
    }
    ids[(base * 8 + vb) % (kIdRing * 8)] = v[i];
  }
  __syncwarp();
}

// Bits [0, k) of 64.
__device__ __forceinline__ uint64_t low_bits(int k) {
  return k <= 0 ? 0ull : (k >= 64 ? ~0ull : (1ull << k) - 1);
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_window_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const WindowPrefillArgs a) {
  using P = WPlan;
  constexpr int kNK = P::kNK, kNV = P::kNV;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_q = sbase + P::kBarOff;         // [2]: Q of the pair landed
  const uint32_t bar_q_empty = bar_q + 16;           // [2]: its score products are done
  const uint32_t bar_k_full = bar_q_empty + 16;      // [kNK]
  const uint32_t bar_k_empty = bar_k_full + 8 * kNK;
  const uint32_t bar_v_full = bar_k_empty + 8 * kNK;   // [kNV]: this CTA's V landed (edge tiles)
  const uint32_t bar_v_ready = bar_v_full + 8 * kNV;   // [kNV]: V of the pair ready
  const uint32_t bar_s_full = bar_v_ready + 8 * kNV;   // [kNS]: scores of a tile
  const uint32_t bar_p_full = bar_s_full + 8 * kNS;    // [kNS]: softmax done
  const uint32_t bar_o_done = bar_p_full + 8 * kNS;    // [kNS]: PV done, and so V slot free
  const uint32_t bar_item = bar_o_done + 8 * kNS;      // [kItemRing]: item published
  static_assert(32 + 8 * (2 * kNK + 2 * kNV + 3 * kNS + kItemRing) <= 336, "barrier area");
  static_assert(kNV == kNS, "V slot of a tile = its score buffer");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + P::kBarOff + 336);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::kBarOff + 340);
  volatile int* go_flag = reinterpret_cast<volatile int*>(smem + P::kBarOff + 352);
  auto ring_item = [&](unsigned k) {
    return reinterpret_cast<Item*>(smem + P::kItemsOff + 64 * (k % kItemRing));
  };
  int* ids_smem = reinterpret_cast<int*>(smem + P::kIdsOff) +
                  ((threadIdx.x >> 5) == kLoadVWarp ? kIdRing * 8 : 0);
  float* red_max = reinterpret_cast<float*>(smem + P::kRedOff);
  float* red_sum = reinterpret_cast<float*>(smem + P::kRedOff2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, gs = __ffs(G) - 1;  // (a group divides 128)
  const int tpt = kTileKeys >> gs;
  const int rank = static_cast<int>(blockIdx.x) & 1;
  const bool issuer = rank == 0;

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar_q + 8 * k, 1);
      mbar_init(bar_q_empty + 8 * k, 1);
    }
    for (int k = 0; k < kNK; ++k) {
      mbar_init(bar_k_full + 8 * k, 1);
      mbar_init(bar_k_empty + 8 * k, 1);
    }
    for (int k = 0; k < kNV; ++k) {
      mbar_init(bar_v_full + 8 * k, 1);
      mbar_init(bar_v_ready + 8 * k, 2);
    }
    for (int k = 0; k < kNS; ++k) {
      mbar_init(bar_s_full + 8 * k, 1);
      mbar_init(bar_p_full + 8 * k, kSoftmaxWarps * 2);
      mbar_init(bar_o_done + 8 * k, 1);
    }
    for (int k = 0; k < kItemRing; ++k) mbar_init(bar_item + 8 * k, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc<2>(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before either reports to the other
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == kLoadKWarp || warp == kLoadVWarp) {
    // ------------------------------------------------------------ loaders
    const uint64_t pol = l2_policy_evict_last();
    unsigned total = 0;  // tiles loaded by this warp, over all items
    // after a timeout: let the copies in flight land before the CTA may exit
    auto settle = [&]() {
      if (!*abort_flag) return;
      const uint64_t t = global_ns();
      while (global_ns() - t < kSettleNs) __nanosleep(1000);
    };
    if (warp == kLoadKWarp) {
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
      }
      Cursor cur{static_cast<int>(blockIdx.x >> 1), 0, 0};
      unsigned published = 0;
      auto publish = [&]() {
        const Item x = next_item(a, cur, static_cast<int>(gridDim.x >> 1), lane, blockIdx.x == 0);
        if (lane == 0) {
          *ring_item(published) = x;
          mbar_arrive(bar_item + 8 * (published % kItemRing));
        }
        ++published;
        return x;
      };
      // (One place for each step: the code of all roles has to stay small.)
      Item it, next;
      it.nkt = 0;
      int jf = 0, jk = 0;  // tiles of `it` with ids, and loaded
      int lead = 0;        // tiles of `it` to load before the next item is looked for
      bool next_ids = true;
      unsigned qi = 0;     // items begun
      while (true) {
        if (jk == lead) {
          next = publish();
          if (a.stall_loads) break;  // a stalled test launch issues no load
          next_ids = next.nkt == 0;
          lead = -1;
        }
        const bool more = jf < it.nkt && jk + kIdBatch / 2 >= jf;
        if (more || (!next_ids && jf >= it.nkt && it.nkt - jk <= kIdBatch)) {
          const Item& x = more ? it : next;
          fetch_ids(a.block_tables + static_cast<int64_t>(x.c) * a.max_blocks, a.num_blocks, a.err,
                    ids_smem, x.nsb, x.b_first, x.nvb, more ? jf : 0,
                    total - jk + (more ? 0 : it.nkt));
          if (more)
            jf += kIdBatch;
          else
            next_ids = true;
        }
        if (jk == it.nkt) {  // on to the next item
          if (next.nkt == 0) break;
          it = next;
          jf = kIdBatch;
          jk = 0;
          const unsigned qb = qi & 1;
          if (qi >= 2 &&
              !wait_warp(bar_q_empty + 8 * qb, ((qi >> 1) - 1) & 1, abort_flag, a))
            break;
          lead = qi == 0 ? min(it.nkt, kNK) : 0;
          ++qi;
          if (lane < 2) {  // a half each
            const uint32_t bar = bar_q + 8 * qb;
            if (issuer && lane == 0) mbar_arrive_expect_tx(bar, 4 * kHalf);  // the pair's Q tiles
            const uint32_t dst = sbase + P::kQOff + (2 * qb + lane) * kHalf;
            const int row = it.q0 + it.tc0 + rank * tpt;
            if (issuer)
              tma_load_3d(dst, &tm_q, lane * 64, it.kvh * G, row, bar, pol);
            else
              tma_load_3d_pair(dst, &tm_q, lane * 64, it.kvh * G, row, mapa_shared(bar, 0), pol);
          }
          __syncwarp();
          if (lead == 0) continue;
        }
        const unsigned slot = total % kNK;
        if (total >= kNK &&
            !wait_warp(bar_k_empty + 8 * slot, ((total / kNK) - 1) & 1, abort_flag, a))
          break;
        const uint32_t bar = bar_k_full + 8 * slot;
        // each CTA takes half of the tile's blocks, their number made even (an
        // id past the list loads zeros)
        const int half = (tile_blocks(it.nvb, jk) + 1) / 2;
        if (lane == 0 && issuer) mbar_arrive_expect_tx(bar, half * 4 * kBlockBytes);
        __syncwarp();
        if (lane < half) {
          const int id = ids_smem[(total % kIdRing) * 8 + half * rank + lane];
          const uint32_t dst = sbase + P::kKOff + slot * P::kKSlot + lane * 2 * kBlockBytes;
          if (issuer)
            tma_load_4d(dst, &tm_k, 0, 0, 2 * it.kvh, 2 * id, bar, pol);
          else
            tma_load_4d_pair(dst, &tm_k, 0, 0, 2 * it.kvh, 2 * id, mapa_shared(bar, 0), pol);
        }
        __syncwarp();
        ++jk;
        ++total;
      }
      // every load's slot has been released, and so has landed, before exit
      if (lane == 0) {
        for (unsigned b = 0; b < 2 && b < qi; ++b)
          wait(bar_q_empty + 8 * b, ((qi - 1 - b) >> 1) & 1, abort_flag, a);
        for (unsigned sl = 0; sl < kNK && sl < total; ++sl)
          wait(bar_k_empty + 8 * sl, ((total - 1 - sl) / kNK) & 1, abort_flag, a);
      }
      settle();
    } else {
      if (lane == 0) tma_prefetch_desc(&tm_v);
      Item it;
      it.nkt = 0;
      int jf = 0, jv = 0;  // tiles of `it` with ids, and loaded
      bool next_ids = false;
      unsigned k = 0;           // items begun
      unsigned full_phase = 0;  // bit s: parity of v_full[s]'s next use
      int edge_slot = -1;       // slot of the edge tile whose rows are still to be zeroed
      while (!a.stall_loads) {
        if (edge_slot >= 0) {
          if (!wait_warp(bar_v_full + 8 * edge_slot, (full_phase >> edge_slot) & 1, abort_flag, a))
            break;
          const uint32_t vt = sbase + P::kVOff + edge_slot * P::kVSlot;
          const Hidden hid(it, a.sinks);
#pragma unroll
          for (int h = 0; h < 3; ++h) {
            if (it.edge[h] != jv - 1) continue;
            const uint32_t blk = vt + (hid.vb[h] & 7) * kBlockBytes;
#pragma unroll 1
            for (int e = lane + 8 * hid.r0[h]; e < 8 * hid.r1[h]; e += 32)
              st_shared_zero16(blk + e * 16);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!issuer)
              mbar_arrive_remote_release(mapa_shared(bar_v_ready + 8 * edge_slot, 0));
            else
              mbar_arrive(bar_v_ready + 8 * edge_slot);
          }
          full_phase ^= 1u << edge_slot;
          edge_slot = -1;
        }
        const bool more = jf < it.nkt && jv + kIdBatch / 2 >= jf;
        bool fetch = more;
        if (!more && !next_ids && jf >= it.nkt && it.nkt - jv <= kIdBatch) {
          // the next item: waited for at the end of this one, taken before if it is there
          const uint32_t bar = bar_item + 8 * (k % kItemRing), parity = (k / kItemRing) & 1;
          if (jv == it.nkt) {
            if (!wait_warp(bar, parity, abort_flag, a)) break;
            fetch = true;
          } else {
            fetch = __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
          }
        }
        if (fetch) {
          const Item* x = ring_item(more ? k - 1 : k);
          if (x->nkt)
            fetch_ids(a.block_tables + static_cast<int64_t>(x->c) * a.max_blocks, a.num_blocks,
                      a.err, ids_smem, x->nsb, x->b_first, x->nvb, more ? jf : 0,
                      total - jv + (more ? 0 : it.nkt));
          if (more)
            jf += kIdBatch;
          else
            next_ids = true;
        }
        if (jv == it.nkt) {  // on to the next item
          it = *ring_item(k++);
          if (it.nkt == 0) break;
          jf = kIdBatch;
          jv = 0;
          next_ids = false;
        }
        const unsigned slot = total % kNV;
        if (total >= kNV &&
            !wait_warp(bar_o_done + 8 * slot, ((total / kNV) - 1) & 1, abort_flag, a))
          break;
        const bool edge = jv == it.edge[0] || jv == it.edge[1] || jv == it.edge[2];
        const bool remote = !issuer && !edge;
        const uint32_t bar = edge ? bar_v_full + 8 * slot
                                  : (remote ? mapa_shared(bar_v_ready + 8 * slot, 0)
                                            : bar_v_ready + 8 * slot);
        const int blocks = tile_blocks(it.nvb, jv);
        if (lane == 0) {
          if (remote)
            mbar_arrive_expect_tx_remote(bar, blocks * kBlockBytes);
          else
            mbar_arrive_expect_tx(bar, blocks * kBlockBytes);
        }
        __syncwarp();
        if (lane < blocks) {  // CTA r takes columns 64 r .. 64 r + 63 of every key
          const int id = ids_smem[(total % kIdRing) * 8 + lane];
          const uint32_t dst = sbase + P::kVOff + slot * P::kVSlot + lane * kBlockBytes;
          const int x = it.kvh * 128 + rank * 64, y = id * kBlockSize;
          if (remote)
            tma_load_2d_pair(dst, &tm_v, x, y, bar, pol);
          else
            tma_load_2d(dst, &tm_v, x, y, bar, pol);
        }
        __syncwarp();
        if (edge) edge_slot = slot;
        ++jv;
        ++total;
      }
      if (lane == 0)
        for (unsigned sl = 0; sl < kNV && sl < total; ++sl)
          wait(bar_o_done + 8 * sl, ((total - 1 - sl) / kNV) & 1, abort_flag, a);
      settle();
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ------------------------------------------------------------ tensor-core issue
    // Two threads of the even CTA, as in pa_prefill_body.cuh.
    if (lane == 0 && issuer) {
      bool ok = true;
      if (warp == kMmaWarp) {
        const uint32_t idesc_s = instr_desc(0, 256) & ~(0x3fu << 17);  // (columns / 8 left out)
        const uint64_t dk0 = smem_desc(sbase + P::kKOff, 16, kKGroupStride);
        const uint64_t dq0 = smem_desc(sbase + P::kQOff, 16, 1024);
        int s_buf = 0, s_round = 0, s_kslot = 0, s_kphase = 0;
        for (unsigned k = 0; ok; ++k) {
          ok = wait(bar_item + 8 * (k % kItemRing), (k / kItemRing) & 1, abort_flag, a);
          const int nkt = ok ? ring_item(k)->nkt : 0;
          if (nkt == 0) break;
          const int nvb = ring_item(k)->nvb;
          const uint64_t dq = dq0 + static_cast<uint64_t>(((k & 1) * 2 * kHalf) >> 4);
          ok = wait(bar_q + 8 * (k & 1), (k >> 1) & 1, abort_flag, a);
          int js = 0;
          while (ok && js < nkt) {
            const uint64_t dk = dk0 + static_cast<uint64_t>((s_kslot * P::kKSlot) >> 4);
            const uint32_t dst = tmem + s_buf * 128;
            // 32 columns for every two blocks
            const uint32_t idesc = idesc_s | (((tile_blocks(nvb, js) + 1) / 2 * 4) << 17);
            ok = wait(bar_k_full + 8 * s_kslot, s_kphase, abort_flag, a) &&
                 (s_round == 0 || wait(bar_o_done + 8 * s_buf, (s_round + 1) & 1, abort_flag, a));
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc_mma_f16<2>(dst, dq + (((ks >> 2) * kHalf + (ks & 3) * 32) >> 4),
                              dk + (((ks >> 2) * kKHalfOffset + (ks & 3) * 32) >> 4), idesc,
                              ks > 0);
              tc_commit_pair(bar_s_full + 8 * s_buf);
              tc_commit_pair(bar_k_empty + 8 * s_kslot);
              ++js;
              if (++s_buf == kNS) {
                s_buf = 0;
                ++s_round;
              }
              if (++s_kslot == kNK) {
                s_kslot = 0;
                s_kphase ^= 1;
              }
            }
          }
          if (ok) tc_commit_pair(bar_q_empty + 8 * (k & 1));
        }
      } else {
        const uint32_t idesc_o = instr_desc(1, 256);
        const uint64_t dv0 = smem_desc(sbase + P::kVOff, kHalf, 1024);
        int p_buf = 0, p_phase = 0, p_vslot = 0, p_vphase = 0;
        for (unsigned k = 0; ok; ++k) {
          ok = wait(bar_item + 8 * (k % kItemRing), (k / kItemRing) & 1, abort_flag, a);
          const int nkt = ok ? ring_item(k)->nkt : 0;
          if (nkt == 0) break;
          const int e0 = ring_item(k)->edge[0], e1 = ring_item(k)->edge[1],
                    e2 = ring_item(k)->edge[2];
          const int nvb = ring_item(k)->nvb;
          int jp = 0;
          while (ok && jp < nkt) {
            const uint64_t dv = dv0 + static_cast<uint64_t>((p_vslot * P::kVSlot) >> 4);
            const uint32_t ta = tmem + p_buf * 128;
            const int blocks = tile_blocks(nvb, jp);
            const bool zeroed = jp == e0 || jp == e1 || jp == e2;
            ok = wait(bar_v_ready + 8 * p_vslot, p_vphase, abort_flag, a) &&
                 wait(bar_p_full + 8 * p_buf, p_phase, abort_flag, a);
            if (ok) {
              if (zeroed) fence_acq_rel_cluster();  // the peer's zeroed rows
              tc_fence_after();
              if (blocks == 8) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                  tc_mma_f16_tmem_a<2>(tmem + kTmemO, ta + (ks >> 2) * 64 + (ks & 3) * 8,
                                       dv + ((ks * kBlockBytes) >> 4), idesc_o,
                                       (jp > 0 || ks > 0) ? 1u : 0u);
              } else {
#pragma unroll 1
                for (int ks = 0; ks < blocks; ++ks)
                  tc_mma_f16_tmem_a<2>(tmem + kTmemO, ta + (ks >> 2) * 64 + (ks & 3) * 8,
                                       dv + ((ks * kBlockBytes) >> 4), idesc_o,
                                       (jp > 0 || ks > 0) ? 1u : 0u);
              }
              tc_commit_pair(bar_o_done + 8 * p_buf);
              ++jp;
              if (++p_buf == kNS) {
                p_buf = 0;
                p_phase ^= 1;
              }
              if (++p_vslot == kNV) {
                p_vslot = 0;
                p_vphase ^= 1;
              }
            }
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps
    const int qd = warp & 3, hc = warp >> 2;
    const int r = qd * 32 + lane;  // query row = tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>(qd * 32) << 16;
    const float sl = a.scale_log2;
    const float sl_pow2 = __uint_as_float(__float_as_uint(sl) & 0x7f800000u);  // in (sl / 2, sl]
    const float floor_score = sl > 1.f ? kFloor / sl : kFloor, floor2 = floor_score * sl;
    const float floor_n = fabsf(floor2) >= kFarScore ? floor_score * sl_pow2 : floor2;
    const uint32_t ocol = tmem + lane_off + kTmemO + hc * 64;
    uint32_t v[64];
    int jt = 0;                // tiles, over all items
    int b3 = 0, s_phase = 0;   // score buffer of tile jt and its parity

    // The output of an item, written once its last PV is done: O / l -> bf16,
    // and lse.  The next item's first PV, which overwrites O, waits for this
    // warp's arrival on p_full behind these loads of O.  The barrier in it also
    // hands over the key tiles of the item after the one at hand (go_flag 0 ..
    // 7; -1: not published yet).
    const int tok = r >> gs, warp_toks = 32 >> gs;
    const uint32_t stage = sbase + P::kOutOff + hc * kHalf + qd * 32 * 128;
    bool pending = false;
    int64_t out_row = 0;            // of the pending item: the warp's first row, [token][head],
    int out_toks = 0;               // and how many of its tokens exist (<= 0: none)
    float out_m = 0.f, out_l = 0.f;
    uint32_t out_bar = 0, out_phase = 0;  // PV of its last tile
    auto write_out = [&](unsigned k) {
      volatile int* go = go_flag + (k & 1) * 4 + qd;
      if (hc == 0 && lane == 0)
        *go = mbar_test_wait(bar_item + 8 * (k % kItemRing), (k / kItemRing) & 1)
                  ? ring_item(k)->nkt
                  : -1;
      wait_warp(out_bar, out_phase, abort_flag, a);
      tc_fence_after();
      red_sum[hc * 128 + r] = out_l;
      named_barrier(1 + qd, 64);
      const float l_tot = out_l + red_sum[(hc ^ 1) * 128 + r];
      const float inv = l_tot == 0.f ? 0.f : 1.f / l_tot;  // a NaN sum stays visible
      const uint64_t inv2 = f32x2(inv, inv);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t (&w)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
        tmem_ld32(ocol + 32 * c, w);
        // 16-byte column q of row `lane` goes to q ^ (lane & 7)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 8 * q + 2 * i;
            const float2 x =
                f32x2_parts(mul2(f32x2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), inv2));
            pk[i] = pack_bf16x2(x.x, x.y);
          }
          sts128(stage + lane * 128 + (((4 * c + q) ^ (lane & 7)) << 4),
                 make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
      }
      __syncwarp();
      const bool good = !warp_flag(abort_flag);
      // four rows at a time, eight lanes on the 128 bytes of each
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + lane / 8, t = row >> gs;
        const uint4 x = lds128(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        if (good && t < out_toks)
          *reinterpret_cast<uint4*>(
              a.out + (out_row + static_cast<int64_t>(t) * a.num_q_heads + (row & (G - 1))) * 128 +
              hc * 64 + (lane & 7) * 8) = x;
      }
      if (good && hc == 0 && a.out_lse && lane >> gs < out_toks)
        a.out_lse[out_row + static_cast<int64_t>(lane >> gs) * a.num_q_heads + (lane & (G - 1))] =
            l_tot == 0.f ? -INFINITY : (out_m + __log2f(l_tot)) * kLn2;
      __syncwarp();  // the staging rows may be written again
      return *go;
    };

    // Both warps of a quadrant act on what the first one found of the next
    // item: they meet at a named barrier for every tile, also after a timeout
    // (when the waits are skipped and what they compute is not stored).
    int nkt = -1;
    for (unsigned k = 0;; ++k) {
      const uint32_t item_bar = bar_item + 8 * (k % kItemRing);
      if (nkt < 0) {
        volatile int* go = go_flag + 8 + (k & 1) * 4 + qd;
        if (hc == 0) {
          const bool got = wait_warp(item_bar, (k / kItemRing) & 1, abort_flag, a);
          if (lane == 0) *go = got ? ring_item(k)->nkt : 0;
        }
        named_barrier(1 + qd, 64);
        nkt = *go;
      }
      const bool last = nkt == 0;  // the list's end: the pending output only
      if (last && !pending) break;
      int next_nkt = -1;
      const Item& it = *ring_item(k);
      const int kmax = it.kmax, p0 = it.p0, t0 = it.tc0 + rank * tpt;
      const int shift = (it.b_first - it.nsb) * kBlockSize;
      const int pos = p0 + t0 + tok;
      const int tv = min(it.qlen - t0, tpt);  // tokens of this tile (<= 0: none)
      const int first_tok = t0 + qd * warp_toks;  // of this warp
      const int64_t row =
          static_cast<int64_t>(it.q0 + first_tok) * a.num_q_heads + it.kvh * G;
      // last and first visible virtual key of the row's window
      const int hi = min(pos, kmax - 1) - shift;
      const int lo = max(0, pos - (a.window - 1)) - shift;
      // reference maximum: a score, in log2 units, and as the softmax subtracts it
      float m_run = floor_score, m_run2 = floor2, n_run = floor_n;
      float l_run = 0.f;
#pragma unroll 1
      for (int j = 0; j < nkt || last; ++j) {
        const bool first = j == 0;
        if (!last) {
          const int b = jt & 1;
          wait_warp(bar_s_full + 8 * b3, s_phase, abort_flag, a);
          tc_fence_after();
          const int kb = j * kTileKeys + hc * 64;
          const bool whole = hi >= kb + 63 && (lo <= kb || a.sinks >= kb + 64);
          float mloc;
          const uint32_t sc = tmem + lane_off + b3 * 128 + hc * 64;
          if (!__all_sync(0xffffffffu, whole)) {
            // hidden scores, whatever they hold, become -inf in tensor memory
            const uint64_t seen =
                low_bits(hi - kb + 1) &
                (low_bits(a.sinks > kb ? min(a.sinks - kb, 64) : 0) | ~low_bits(lo - kb));
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              const uint32_t m = static_cast<uint32_t>(seen >> (32 * c));
              if (__all_sync(0xffffffffu, m == 0xffffffffu)) continue;
              uint32_t (&w)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
              tmem_ld32(sc + 32 * c, w);
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i] = ((m >> i) & 1u) ? w[i] : 0xff800000u;
              tmem_st32(sc + 32 * c, w);
            }
          }
          tmem_ld64_max(sc, v, mloc);
          red_max[(b * 2 + hc) * 128 + r] = mloc;
          named_barrier(1 + qd, 64);
          // (scale > 0 keeps the order of scores)
          const float m_new = fmaxf(m_run, fmaxf(mloc, red_max[(b * 2 + (hc ^ 1)) * 128 + r]));
          const float m_new2 = m_new * sl;
          const bool move = m_new2 > m_run2 + kRescaleThreshold;
          const float alpha = move ? fast_exp2(m_run2 - m_new2) : 1.f;
          // x = s sl - m sl by one fused multiply-add, whose product is exact and so
          // differs from m_run2, which is rounded, by up to half a step of it: a
          // common factor of a row's weights, within 2^64 below kFarScore.  From there
          // on the factor leaves fp32, and neighbouring scores are 2^7 apart: any
          // multiplier near sl tells them apart, and a power of two is exact.  (m_new2
          // is far where m_run2 is: they differ by less than that step, or it moves.)
          const bool far = fabsf(m_new2) >= kFarScore;
          const float slx = far ? sl_pow2 : sl, n_new = far ? m_new * sl_pow2 : m_new2;
          m_run = move ? m_new : m_run;
          m_run2 = move ? m_new2 : m_run2;
          n_run = move ? n_new : n_run;
          uint64_t rsp[2] = {0, 0};
          uint32_t pk[32];
          const uint64_t sl2 = f32x2(slx, slx), nm2 = f32x2(-n_run, -n_run);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            // -inf (hidden) gives exactly 0: n_run is finite
            const uint64_t s2 = f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            const float2 x = f32x2_parts(fma2(s2, sl2, nm2));
            const float e0 = fast_exp2(x.x), e1 = fast_exp2(x.y);
            rsp[(i >> 1) & 1] = add2(rsp[(i >> 1) & 1], f32x2(e0, e1));
            pk[i / 2] = pack_bf16x2(e0, e1);
          }
          const float2 rs = f32x2_parts(add2(rsp[0], rsp[1]));
          l_run = l_run * alpha + (rs.x + rs.y);
          // O is rescaled only when a row maximum moved; PV of the previous
          // tile must have landed first (tile 0's PV overwrites O)
          if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
            const int pb = b3 == 0 ? kNS - 1 : b3 - 1;
            wait_warp(bar_o_done + 8 * pb, b3 == 0 ? s_phase ^ 1 : s_phase, abort_flag, a);
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {
              uint32_t (&w)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
              tmem_ld32(ocol + 32 * cc, w);
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
              tmem_st32(ocol + 32 * cc, w);
            }
          }
          tmem_st32(sc, pk);
        }
        if (first && pending) next_nkt = write_out(k + 1);
        if (last) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!issuer)
            mbar_arrive_remote(mapa_shared(bar_p_full + 8 * b3, 0));
          else
            mbar_arrive(bar_p_full + 8 * b3);
        }
        if (++b3 == kNS) {
          b3 = 0;
          s_phase ^= 1;
        }
        ++jt;
      }
      if (last) break;
      out_bar = bar_o_done + 8 * (b3 == 0 ? kNS - 1 : b3 - 1);
      out_phase = b3 == 0 ? s_phase ^ 1 : s_phase;
      pending = true;
      out_row = row;
      out_toks = tv - qd * warp_toks;
      out_m = m_run2;
      out_l = l_run;
      nkt = next_nkt;
    }
  }
  tc_fence_before();
  // Neither CTA leaves while the other may still report to it.  No data changes
  // hands here, so outputs need not have landed: a release would wait for them
  // (0.6 us).
  cluster_sync_relaxed();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<2>(tmem, kTmemCols);
}

}  // namespace
}  // namespace pre

using namespace pre;

cudaError_t launch_prefill_window(const WindowPrefillArgs& args, const CUtensorMap* tm_q,
                                  const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                  int64_t max_items, int num_sms, cudaStream_t stream) {
  WindowPrefillArgs a = args;
  if (a.wait_ns == 0) a.wait_ns = kWaitLimitNs;
  constexpr int smem = WPlan::kSmemBytes + 1024;
  static std::mutex mu;
  static bool set_for[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set_for[dev]) {
      e = cudaFuncSetAttribute(prefill_window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               smem);
      if (e != cudaSuccess) return e;
      set_for[dev] = true;
    }
  }
  const int pairs = num_sms / 2 < 1 ? 1 : num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(max_items < pairs ? max_items : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, prefill_window_kernel, *tm_q, *tm_k, *tm_v, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
