// pa_shared_prefix.cu -- attention of the sequences of a group over the prefix that
// they share, read once for all of them, on tcgen05 tensor cores (sm_103a).
//
// The queries of a group's members, G heads a kv head, are the rows of one dense
// product with the prefix's keys: no mask but the members' lengths.  What is left
// of each sequence is decoded by pa_window_decode.cu beside it; a third kernel, below,
// joins both.
//
// The tensor-core pipeline of a key tile (128 keys) is that of the windowed prefill:
// K and V tiles by TMA, three score buffers in tensor memory, online softmax with P
// written back over its scores, bounded waits.  What differs:
//
//  * Groups of up to 128 query rows a kv head are a lone CTA's (cta_group::1), larger ones
//    a pair's, 256 rows at a time (cta_group::2, K and V halves loaded by each CTA): 128
//    rows fill but half of a pair's products, and those of a tile would then take as
//    long as its bytes.
//  * Work is cut along the keys, so that a single long prefix fills the device: teams
//    of workers (CTAs or pairs), one for each kv head, take equal ranges of all key tiles.
//    The workers of a team read the same blocks at the same time, each its own head's 256
//    bytes of a token's row; together they read whole rows, which memory serves faster.
//  * A piece (a unit's key tiles in a team's range) leaves its reference maximum, sum
//    and weighted values, in fp32 and undivided, for the join behind.
//  * Warps whose 32 rows no member fills wait for scores and pass them on unread.
//  * P is the sum of two bf16 numbers (to 2^-16 of itself), as in the decode of the own
//    parts, so that the output does not depend on which of both reads a key.  One bf16
//    took 78 / 57 / 81 us in the cases below, and 0.79 a tile of 256 rows.  Of groups of up
//    to 16 rows the lower parts are rows of their own beside the upper ones, multiplied at
//    no cost, and their lanes take half of the exponentials (with two products instead 90
//    us for 82).
//
// What bounds it: HBM.  In the steady state lone CTAs read 7.3 TB/s (0.65 us for every
// 72 tiles of 64 KB); pairs take 1.14 us a tile for 256 rows, 1.6 PFLOP/s of their three
// products (of 1.88 that a library product reaches).
// The first 8 us go to round trips: offsets, lengths, block ids, keys.
// With 32 query and 8 kv heads of 128: 64 groups of 4 sequences behind 256 to 2048 tokens
// (392 MB with their own parts) 82 us, 4.8 TB/s; 32 sequences behind 65536 (273 MB) 59 us;
// 256 behind 8192 (322 MB, of which 294 are own parts) 88 us.
#include <limits.h>

#include <mutex>

#include "pa_prefill_body.cuh"
#include "pa_shared.h"
#include "pa_window_ptx.cuh"

namespace pa {
namespace pre {
namespace {

constexpr uint64_t kSettleNs = 1000000;  // far longer than any copy takes
// Reference maximum (log2 units) of a row that saw nothing yet: next to the lowest
// fp32, so that no visible score lies below it; hidden scores (-inf) weigh 0.
constexpr float kFloor = -0x1.fffff0p127f;
constexpr float kFarScore = 0x1p31f;  // (log2 units)
// Weights, each the sum of two bf16 numbers, lie over their scores: of 64 columns the upper
// parts of 64 keys take the first 32, the lower ones the others.
constexpr uint32_t kLowCols = 32;

// Shared memory of one CTA: Q tiles, K and V tiles (a pair's CTAs hold half of each), block
// ids of both loaders, the softmax's exchange, barriers.  Small groups (kQRows > 0: at most
// so many query rows), of which a worker has many short items, have the next item's Q
// tile beside; an operand tile has 128 rows, and the second one lies kQRows behind the
// first, whose other rows no member has.  Otherwise an item's Q waits for the scores of
// the one before.  (What is left of an SM holds CTAs of the decode of the sequences' own
// parts.)
template <int CG, int kQRows>
struct SPlan {
  static constexpr int kNQ = kQRows > 0 ? 2 : 1;
  static constexpr int kNK = 2, kNV = CG == 2 ? 3 : 2;
  static constexpr int kKSlot = 2 * kHalf / CG, kVSlot = 2 * kHalf / CG;
  static constexpr int kQNext = kQRows * 128;           // to the next Q tile
  static constexpr int kQHalf = kQNext + kHalf;         // to the other 64 columns
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kQHalf;
  static constexpr int kVOff = kKOff + kNK * kKSlot;
  static constexpr int kIdsOff = kVOff + kNV * kVSlot;
  static constexpr int kRedOff = kIdsOff + 2 * kIdRing * 8 * 4;
  static constexpr int kRedOff2 = kRedOff + 2 * 2 * 128 * 4;
  static constexpr int kBarOff = kRedOff2 + 2 * 128 * 4;
  static constexpr int kItemsOff = kBarOff + 512;  // [kItemRing]
  static constexpr int kSmemBytes = kItemsOff + 8 * 64;
  static_assert(kSmemBytes + 1024 <= 227 * 1024, "shared memory of one CTA");
  static_assert(kQNext % 1024 == 0, "swizzle atoms");
};

// One work item of a worker (a CTA, or a pair of them): a piece of a unit's key tiles,
// one kv head.
struct Item {
  int nkt;         // key tiles; 0 ends the list
  int row;         // table row that names the prefix's blocks: the first member's
  int kvh;
  int q0, tokens;  // the unit's first member, and how many
  int block0;      // first block of the piece
  int nvb;         // blocks to load, one at least
  int ids;         // and how many of them some member sees: no other table entry is read
  int keys;        // keys [0, keys) of the sequence are the prefix
  int hidden;      // rows of the last block from this one on are seen by no member; or 16
  int slot;        // of the results
  int whole;       // every member sees the whole prefix
};
// Blocks of an item's key tile j: eight, fewer in the last one.
__device__ __forceinline__ int tile_blocks(int nvb, int j) { return min(8, nvb - 8 * j); }

constexpr int kItemRing = 8;
static_assert(sizeof(Item) <= 64, "ring slot");
static_assert(kBlockSize == 16, "shifts below");

// Units and key tiles of 32 groups at a time, a lane each, and their sums, with
// `before` units in front of them.  Groups that overlap could make more units than
// there are slots: what is too many is left out.
struct Groups {
  SharedGroup g;
  int units, tiles;          // of the lane's group
  int units_sum, tiles_sum;  // up to and with it
  __device__ __forceinline__ Groups(const SharedArgs& a, int g0, int before, int lane) {
    g = SharedGroup{0, 0, 0, true};
    if (g0 + lane < a.num_groups) g = shared_group(a, g0 + lane);
    const int rows = a.lay.unit_tokens;
    units = g.blocks > 0 ? (g.members + rows - 1) / rows : 0;
    units_sum = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, units_sum, off);
      if (lane >= off) units_sum = min(units_sum + u, 1 << 30);
    }
    if (__any_sync(0xffffffffu, before + units_sum > a.lay.max_units)) {
      const int room = max(a.lay.max_units - before, 0);
      const int start = units_sum - units;
      if (units_sum > room) {
        units = 0;
        g.sound = false;
      }
      units_sum = __reduce_max_sync(0xffffffffu, start + units <= room ? start + units : 0);
      units_sum = min(start + units, units_sum);
    }
    tiles = units * ((g.blocks + 7) >> 3);
    tiles_sum = tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, tiles_sum, off);
      if (lane >= off) tiles_sum += t;
    }
  }
};

// Walks a worker's pieces.
struct Cursor {
  int pos, end;      // key tiles of the team's range that are left
  int group0;        // groups at hand, 32 at a time,
  int units, tiles;  // and units and key tiles before them
  int team, kvh;
};

// The next item (nkt 0 at the end of the list); x: the groups at hand.  Called by a
// whole warp.
__device__ __forceinline__ Item next_item(const SharedArgs& a, Cursor& cur, Groups& x, int lane) {
  Item it;
  it.nkt = 0;
  while (cur.pos < cur.end && cur.group0 < a.num_groups) {
    const unsigned past = __ballot_sync(0xffffffffu, cur.tiles + x.tiles_sum > cur.pos);
    if (past == 0) {
      cur.units += __shfl_sync(0xffffffffu, x.units_sum, 31);
      cur.tiles += __shfl_sync(0xffffffffu, x.tiles_sum, 31);
      cur.group0 += 32;
      x = Groups(a, cur.group0, cur.units, lane);
      continue;
    }
    const int w = __ffs(past) - 1;
    const int at = cur.pos - cur.tiles - __shfl_sync(0xffffffffu, x.tiles_sum - x.tiles, w);
    const int unit0 = cur.units + __shfl_sync(0xffffffffu, x.units_sum - x.units, w);
    const int first = __shfl_sync(0xffffffffu, x.g.first, w);
    const int members = __shfl_sync(0xffffffffu, x.g.members, w);
    const int blocks = __shfl_sync(0xffffffffu, x.g.blocks, w);
    const int nkt = (blocks + 7) >> 3;
    const int u = at / nkt, tile0 = at - u * nkt;
    const int n = min(nkt - tile0, cur.end - cur.pos);
    cur.pos += n;
    const int rows = a.lay.unit_tokens;
    it.row = first;
    it.kvh = cur.kvh;
    it.q0 = first + u * rows;
    it.tokens = min(members - u * rows, rows);
    it.block0 = 8 * tile0;
    it.slot = (cur.team + unit0 + u) * a.num_kv_heads + cur.kvh;
    it.keys = blocks * kBlockSize;
    // the last key that some member sees, and whether all see the last one
    int seen = 0, least = INT_MAX;
    for (int i = lane; i < it.tokens; i += 32) {
      const int n = __ldcg(a.seq_lens + it.q0 + i);
      seen = max(seen, n);
      least = min(least, n);
    }
    seen = min(__reduce_max_sync(0xffffffffu, seen), it.keys);
    it.whole = __reduce_min_sync(0xffffffffu, least) >= it.keys;
    // (one block at least, so that there are scores)
    const int left = ((seen + 15) >> 4) - it.block0;
    it.ids = min(max(left, 0), min(8 * n, blocks - it.block0));
    it.nvb = max(it.ids, 1);
    it.nkt = (it.nvb + 7) >> 3;
    it.hidden = min(max(seen - (it.block0 + it.nvb - 1) * kBlockSize, 0), kBlockSize);
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
                                     const SharedArgs& a) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, a.err, a.wait_ns);
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          const SharedArgs& a) {
  bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  if (!ok) {
    ok = wait_on(bar, parity, abort, a.err, a.wait_ns);
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// Ids of an item's blocks [8 t_first, + 8 kIdBatch) into a loader's
// ring, where the ids of the warp's tile T are at slot T % kIdRing and `base` is
// the number of the item's tile 0.  A slot is rewritten only when its tile's
// loads have been issued.  Ids past the list (nid of them) are -1, a box outside the pool,
// which reads as zeros.  Called by a whole warp.
__device__ __noinline__ void fetch_ids(const int32_t* table, int64_t num_blocks, unsigned int* err,
                                       int* ids, int nid, int t_first, unsigned base) {
  const int lane = threadIdx.x & 31;
  int v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int vb = t_first * 8 + lane + 32 * i;
    v[i] = vb < nid ? __ldcg(table + vb) : -1;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int vb = t_first * 8 + lane + 32 * i;
    if (vb < nid && (v[i] < 0 || v[i] >= num_blocks)) {
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

// 32 bytes to memory.
__device__ __forceinline__ void stg32(float* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                   reinterpret_cast<uint64_t>(p)),
               "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]),
               "r"(x[7])
               : "memory");
}

// CG: CTAs of a worker.  Two of them (a tcgen05 pair) take 256 query rows, one 128.
// (The bound of 512 threads is one of 128 registers: three warps of this kernel on a
// quarter of an SM then leave room for one of the decode's beside it.)
template <int CG, int kQRows>
__global__ void __launch_bounds__(512, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const SharedArgs a) {
  using P = SPlan<CG, kQRows>;
  constexpr int kNK = P::kNK, kNV = P::kNV, kNQ = P::kNQ;
  // Up to 16 query rows: the lower parts of row r's weights are row r + 16, so that one
  // product takes both, and that row's lane computes half of the weights.
  constexpr bool kFold = kQRows > 0;
  static_assert(kQRows <= 16, "rows of a half warp");
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
  const uint32_t bar_o_done = bar_p_full + 8 * kNS;    // [kNS]: PV done
  const uint32_t bar_item = bar_o_done + 8 * kNS;      // [kItemRing]: item published
  const uint32_t bar_v_empty = bar_item + 8 * kItemRing;  // [kNV]: PV done, slot free
  static_assert(32 + 8 * (2 * kNK + 3 * kNV + 3 * kNS + kItemRing) <= 384, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + P::kBarOff + 384);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P::kBarOff + 388);
  volatile int* go_flag = reinterpret_cast<volatile int*>(smem + P::kBarOff + 400);
  auto ring_item = [&](unsigned k) {
    return reinterpret_cast<Item*>(smem + P::kItemsOff + 64 * (k % kItemRing));
  };
  int* ids_smem = reinterpret_cast<int*>(smem + P::kIdsOff) +
                  ((threadIdx.x >> 5) == kLoadVWarp ? kIdRing * 8 : 0);
  float* red_max = reinterpret_cast<float*>(smem + P::kRedOff);
  float* red_sum = reinterpret_cast<float*>(smem + P::kRedOff2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, tpt = a.lay.tile_tokens;
  const int rank = CG == 2 ? static_cast<int>(blockIdx.x) & 1 : 0;
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
      mbar_init(bar_v_ready + 8 * k, CG);
      mbar_init(bar_v_empty + 8 * k, 1);
    }
    for (int k = 0; k < kNS; ++k) {
      mbar_init(bar_s_full + 8 * k, 1);
      mbar_init(bar_p_full + 8 * k, kSoftmaxWarps * CG);
      mbar_init(bar_o_done + 8 * k, 1);
    }
    for (int k = 0; k < kItemRing; ++k) mbar_init(bar_item + 8 * k, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc<CG>(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync();  // both CTAs' barriers exist before either reports to the other
  else
    __syncthreads();
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
      // all key tiles, and where each group's begin (the first pair writes it down)
      int units = 0, tiles = 0;
      const Groups head(a, 0, 0, lane);
      for (int g0 = 0; g0 < a.num_groups; g0 += 32) {
        const Groups x = g0 == 0 ? head : Groups(a, g0, units, lane);
        if (blockIdx.x == 0 && g0 + lane < a.num_groups) {
          a.lay.info[g0 + lane] =
              make_int4(units + x.units_sum - x.units, tiles + x.tiles_sum - x.tiles,
                        x.units > 0 ? (x.g.blocks + 7) >> 3 : 0, x.g.first);
          if (!x.g.sound) atomicOr(a.err, PA_DEVERR_GROUP);
        }
        units += __shfl_sync(0xffffffffu, x.units_sum, 31);
        tiles += __shfl_sync(0xffffffffu, x.tiles_sum, 31);
      }
      if (blockIdx.x == 0 && lane == 0) a.lay.info[a.num_groups] = make_int4(units, tiles, 0, 0);
      const int worker = static_cast<int>(blockIdx.x) / CG;
      const int team = worker / a.lay.team_workers;
      const int teams = shared_teams(a.lay, tiles);
      const int from =
          team < teams ? static_cast<int>(static_cast<int64_t>(tiles) * team / teams) : 0;
      const int to =
          team < teams ? static_cast<int>(static_cast<int64_t>(tiles) * (team + 1) / teams) : 0;
      Cursor cur{from, to, 0, 0, 0, team, worker - team * a.lay.team_workers};
      Groups at_hand = head;
      unsigned published = 0;
      auto publish = [&]() {
        if (cur.pos == cur.end && cur.kvh + a.lay.team_workers < a.num_kv_heads) {
          cur = Cursor{from, to, 0, 0, 0, team, cur.kvh + a.lay.team_workers};
          if (a.num_groups > 32) at_hand = Groups(a, 0, 0, lane);
        }
        const Item x = next_item(a, cur, at_hand, lane);
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
          fetch_ids(a.block_tables + static_cast<int64_t>(x.row) * a.max_blocks + x.block0,
                    a.num_blocks, a.err, ids_smem, x.ids, more ? jf : 0,
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
          const unsigned qb = qi % kNQ;
          if (qi >= kNQ &&
              !wait_warp(bar_q_empty + 8 * qb, ((qi / kNQ) - 1) & 1, abort_flag, a))
            break;
          lead = qi == 0 ? min(it.nkt, kNK) : 0;
          ++qi;
          if (lane < 2) {  // a half each
            const uint32_t bar = bar_q + 8 * qb;
            // (the CTAs' query tiles, two halves of box_tokens tokens of G heads)
            if (issuer && lane == 0)
              mbar_arrive_expect_tx(bar, CG * 2 * a.lay.box_tokens * G * 128);
            const uint32_t dst = sbase + P::kQOff + qb * P::kQNext + lane * P::kQHalf;
            const int row = it.q0 + rank * tpt;
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
        // each CTA takes its share of the tile's blocks, their number made even (an
        // id past the list loads zeros)
        const int half = (tile_blocks(it.nvb, jk) + 1) / 2;
        const int mine = half * 2 / CG;
        if (lane == 0 && issuer) mbar_arrive_expect_tx(bar, half * 4 * kBlockBytes);
        __syncwarp();
        if (lane < mine) {
          const int id = ids_smem[(total % kIdRing) * 8 + mine * rank + lane];
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
        for (unsigned b = 0; b < kNQ && b < qi; ++b)
          wait(bar_q_empty + 8 * b, ((qi - 1 - b) / kNQ) & 1, abort_flag, a);
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
          const uint32_t blk = vt + ((it.nvb - 1) & 7) * kBlockBytes;
#pragma unroll 1
          for (int e = lane + 8 * it.hidden; e < 8 * kBlockSize; e += 32) {
            st_shared_zero16(blk + e * 16);
            if constexpr (CG == 1) st_shared_zero16(blk + kHalf + e * 16);
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
            fetch_ids(a.block_tables + static_cast<int64_t>(x->row) * a.max_blocks + x->block0,
                      a.num_blocks, a.err, ids_smem, x->ids, more ? jf : 0,
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
            !wait_warp(bar_v_empty + 8 * slot, ((total / kNV) - 1) & 1, abort_flag, a))
          break;
        const bool edge = jv == it.nkt - 1 && it.hidden < kBlockSize;
        const bool remote = !issuer && !edge;
        const uint32_t bar = edge ? bar_v_full + 8 * slot
                                  : (remote ? mapa_shared(bar_v_ready + 8 * slot, 0)
                                            : bar_v_ready + 8 * slot);
        const int blocks = tile_blocks(it.nvb, jv);
        if (lane == 0) {
          if (remote)
            mbar_arrive_expect_tx_remote(bar, blocks * kBlockBytes);
          else
            mbar_arrive_expect_tx(bar, blocks * kBlockBytes * (2 / CG));
        }
        __syncwarp();
        // 64 columns of a block each: CTA r of a pair takes columns 64 r .. 64 r + 63 of
        // every key, a lone CTA both halves
        const int blk = lane & 7, h = CG == 2 ? rank : lane >> 3;
        if (lane < 16 / CG && blk < blocks) {
          const int id = ids_smem[(total % kIdRing) * 8 + blk];
          const uint32_t dst = sbase + P::kVOff + slot * P::kVSlot + blk * kBlockBytes +
                               (CG == 1 ? h * kHalf : 0);
          const int x = it.kvh * 128 + h * 64, y = id * kBlockSize;
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
          wait(bar_v_empty + 8 * sl, ((total - 1 - sl) / kNV) & 1, abort_flag, a);
      settle();
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ------------------------------------------------------------ tensor-core issue
    // Two threads of the even CTA, as in pa_prefill_body.cuh.
    if (lane == 0 && issuer) {
      bool ok = true;
      auto commit = [&](uint32_t bar) {
        if constexpr (CG == 2)
          tc_commit_pair(bar);
        else
          tc_commit<1>(bar);
      };
      if (warp == kMmaWarp) {
        // (columns / 8 left out)
        const uint32_t idesc_s = instr_desc(0, 128 * CG) & ~(0x3fu << 17);
        const uint64_t dk0 = smem_desc(sbase + P::kKOff, 16, kKGroupStride);
        const uint64_t dq0 = smem_desc(sbase + P::kQOff, 16, 1024);
        int s_buf = 0, s_round = 0, s_kslot = 0, s_kphase = 0;
        for (unsigned k = 0; ok; ++k) {
          ok = wait(bar_item + 8 * (k % kItemRing), (k / kItemRing) & 1, abort_flag, a);
          const int nkt = ok ? ring_item(k)->nkt : 0;
          if (nkt == 0) break;
          const int nvb = ring_item(k)->nvb;
          const uint64_t dq = dq0 + static_cast<uint64_t>(((k % kNQ) * P::kQNext) >> 4);
          ok = wait(bar_q + 8 * (k % kNQ), (k / kNQ) & 1, abort_flag, a);
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
                tc_mma_f16<CG>(dst, dq + (((ks >> 2) * P::kQHalf + (ks & 3) * 32) >> 4),
                              dk + (((ks >> 2) * kKHalfOffset + (ks & 3) * 32) >> 4), idesc,
                              ks > 0);
              commit(bar_s_full + 8 * s_buf);
              commit(bar_k_empty + 8 * s_kslot);
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
          if (ok) commit(bar_q_empty + 8 * (k % kNQ));
        }
      } else {
        const uint32_t idesc_o = instr_desc(1, 128 * CG);
        const uint64_t dv0 = smem_desc(sbase + P::kVOff, kHalf, 1024);
        int p_buf = 0, p_phase = 0, p_vslot = 0, p_vphase = 0;
        for (unsigned k = 0; ok; ++k) {
          ok = wait(bar_item + 8 * (k % kItemRing), (k / kItemRing) & 1, abort_flag, a);
          const int nkt = ok ? ring_item(k)->nkt : 0;
          if (nkt == 0) break;
          const bool hides = ring_item(k)->hidden < kBlockSize;
          const int nvb = ring_item(k)->nvb;
          int jp = 0;
          while (ok && jp < nkt) {
            const uint64_t dv = dv0 + static_cast<uint64_t>((p_vslot * P::kVSlot) >> 4);
            const uint32_t ta = tmem + p_buf * 128;
            const int blocks = tile_blocks(nvb, jp);
            const bool zeroed = hides && jp == nkt - 1;
            ok = wait(bar_v_ready + 8 * p_vslot, p_vphase, abort_flag, a) &&
                 wait(bar_p_full + 8 * p_buf, p_phase, abort_flag, a);
            if (ok) {
              if (zeroed) fence_acq_rel_cluster();  // the peer's zeroed rows
              tc_fence_after();
              // (upper parts, then lower ones; where those are other rows, all at once)
#pragma unroll 1
              for (int part = 0; part < (kFold ? 1 : 2); ++part) {
                const uint32_t tp = ta + part * kLowCols;
                const bool more = jp > 0 || part > 0;
                if (blocks == 8) {
#pragma unroll
                  for (int ks = 0; ks < 8; ++ks)
                    tc_mma_f16_tmem_a<CG>(tmem + kTmemO, tp + (ks >> 2) * 64 + (ks & 3) * 8,
                                         dv + ((ks * kBlockBytes) >> 4), idesc_o,
                                         (more || ks > 0) ? 1u : 0u);
                } else {
#pragma unroll 1
                  for (int ks = 0; ks < blocks; ++ks)
                    tc_mma_f16_tmem_a<CG>(tmem + kTmemO, tp + (ks >> 2) * 64 + (ks & 3) * 8,
                                         dv + ((ks * kBlockBytes) >> 4), idesc_o,
                                         (more || ks > 0) ? 1u : 0u);
                }
              }
              commit(bar_o_done + 8 * p_buf);
              commit(bar_v_empty + 8 * p_vslot);
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

    // The results of an item, written once its last PV is done: O undivided, maximum and
    // sum.  The next item's first PV, which overwrites O, waits for this
    // warp's arrival on p_full behind these loads of O.  The barrier in it also
    // hands over the key tiles of the item after the one at hand (go_flag 0 ..
    // 7; -1: not published yet).
    const int tok = r / G;
    bool pending = false;
    int64_t out_row = 0;            // of the pending item: this lane's row of the results,
    bool out_here = false;          // and whether a member has it
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
      if constexpr (kFold) out_l += __shfl_xor_sync(0xffffffffu, out_l, 16);
      red_sum[hc * 128 + r] = out_l;
      named_barrier(1 + qd, 64);
      const float l_tot = out_l + red_sum[(hc ^ 1) * 128 + r];
      const bool sound = !warp_flag(abort_flag);  // (asked by the whole warp)
      const bool good = sound && out_here;
      float* const to = a.lay.part_o + out_row * 128 + hc * 64;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t (&w)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
        tmem_ld32(ocol + 32 * c, w);
        if constexpr (kFold) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            w[i] = __float_as_uint(__uint_as_float(w[i]) +
                                   __shfl_xor_sync(0xffffffffu, __uint_as_float(w[i]), 16));
        }
        if (good) {
#pragma unroll
          for (int q = 0; q < 4; ++q) stg32(to + 32 * c + 8 * q, &w[8 * q]);
        }
        __syncwarp();
      }
      if (good && hc == 0) a.lay.part_ml[out_row] = make_float2(out_m, l_tot);
      __syncwarp();
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
      const int mine = rank * tpt + tok;  // member of the unit
      const bool here = !last && tok < tpt && mine < it.tokens;
      const bool active = __any_sync(0xffffffffu, here);
      // last key of the piece that the row sees (a length below zero, which the decode of
      // the own parts reports, is none)
      int hi = -1;
      if (here)
        hi = (it.whole ? it.keys : max(min(__ldcg(a.seq_lens + it.q0 + mine), it.keys), 0)) -
             1 - it.block0 * kBlockSize;
      const int64_t row =
          static_cast<int64_t>(it.slot) * a.lay.slot_rows + rank * tpt * G + r;
      // reference maximum: a score, in log2 units, and as the softmax subtracts it
      float m_run = floor_score, m_run2 = floor2, n_run = floor_n;
      float l_run = 0.f;
#pragma unroll 1
      for (int j = 0; j < nkt || last; ++j) {
        const bool first = j == 0;
        if (!last) wait_warp(bar_s_full + 8 * b3, s_phase, abort_flag, a);
        if (active) {
          const int b = jt & 1;
          tc_fence_after();
          const int kb = j * kTileKeys + hc * 64;
          const bool whole = !here || hi >= kb + 63;  // (rows of no member hold anything)
          float mloc;
          const uint32_t sc = tmem + lane_off + b3 * 128 + hc * 64;
          if (!__all_sync(0xffffffffu, whole)) {
            // hidden scores, whatever they hold, become -inf in tensor memory
            const uint64_t seen = low_bits(hi - kb + 1);
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
          if constexpr (kFold) mloc = __shfl_sync(0xffffffffu, mloc, lane & 15);
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
          uint32_t pk[32], low[32];
          const uint64_t sl2 = f32x2(slx, slx), nm2 = f32x2(-n_run, -n_run);
          // weights of two keys, their upper and their lower parts
          auto weigh = [&](uint32_t s0, uint32_t s1, int at, uint32_t& hi, uint32_t& lo) {
            // -inf (hidden) gives exactly 0: n_run is finite
            const uint64_t s2 = f32x2(__uint_as_float(s0), __uint_as_float(s1));
            const float2 x = f32x2_parts(fma2(s2, sl2, nm2));
            const float e0 = fast_exp2(x.x), e1 = fast_exp2(x.y);
            rsp[at] = add2(rsp[at], f32x2(e0, e1));
            hi = pack_bf16x2(e0, e1);
            lo = pack_bf16x2(e0 - __uint_as_float(hi << 16),
                             e1 - __uint_as_float(hi & 0xffff0000u));
          };
          if constexpr (kFold) {
            const bool lower = lane >= 16;  // lower parts, and the second 32 keys
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint32_t theirs = __shfl_sync(0xffffffffu, v[32 + i], lane & 15);
              v[i] = lower ? theirs : v[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t hi, lo;
              weigh(v[2 * i], v[2 * i + 1], i & 1, hi, lo);
              const uint32_t theirs = __shfl_xor_sync(0xffffffffu, lower ? hi : lo, 16);
              pk[i] = lower ? theirs : hi;
              pk[16 + i] = lower ? lo : theirs;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              weigh(v[2 * i], v[2 * i + 1], i & 1, pk[i], low[i]);
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
          if constexpr (!kFold) tmem_st32(sc + kLowCols, low);
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
      pending = active;
      out_row = row;
      out_here = here;
      out_m = m_run2;
      out_l = l_run;
      nkt = next_nkt;
    }
  }
  tc_fence_before();
  // Neither CTA leaves while the other may still report to it.  No data changes
  // hands here, so outputs need not have landed: a release would wait for them
  // (0.6 us).
  if constexpr (CG == 2)
    cluster_sync_relaxed();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<CG>(tmem, kTmemCols);
}

}  // namespace
}  // namespace pre

using namespace pre;

namespace {

template <int CG, int kQRows>
cudaError_t launch_workers(const SharedArgs& a, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                           const CUtensorMap* tm_v, cudaStream_t stream) {
  constexpr int smem = SPlan<CG, kQRows>::kSmemBytes + 1024;
  const auto kernel = shared_prefix_kernel<CG, kQRows>;
  static std::mutex mu;
  static bool set_for[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set_for[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
      set_for[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CG * static_cast<unsigned>(a.lay.teams * a.lay.team_workers));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, *tm_q, *tm_k, *tm_v, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_prefix(const SharedArgs& args, const CUtensorMap* tm_q,
                                 const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                 cudaStream_t stream) {
  SharedArgs a = args;
  if (a.wait_ns == 0) a.wait_ns = kWaitLimitNs;
  if (a.lay.worker_ctas == 2) return launch_workers<2, 0>(a, tm_q, tm_k, tm_v, stream);
  // Up to 16 query rows: the next item's Q tile in front of its turn, and the weights' lower
  // parts as rows of their own.  (us with 4 query heads a kv head, with / without: 200
  // groups of 4 sequences behind 256 tokens 82.0 / 90.4, 64 of 4 behind 1024 61.3 / 68.5,
  // 12 of 4 behind 2048 28.6 / 31.2.  A Q tile ahead for up to 64 rows gained nothing: 40
  // groups of 8 behind 256 28.8 / 27.9, 20 of 8 behind 2048 42.3 / 41.2, when weights were
  // one bf16.)
  if (a.lay.box_tokens * a.group <= 16) return launch_workers<1, 16>(a, tm_q, tm_k, tm_v, stream);
  return launch_workers<1, 0>(a, tm_q, tm_k, tm_v, stream);
}

namespace {

constexpr int kJoinWarps = 8;

// What a warp has of a row: four columns a lane, the maximum and the sum.
struct Joined {
  float4 o;
  float m, l;
  __device__ __forceinline__ void move(float top) {
    const float f = fast_exp2(m - top);
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    l *= f;
    m = top;
  }
  __device__ __forceinline__ void add(float4 x, float2 ml) {  // (m is not below ml.x)
    const float f = fast_exp2(ml.x - m);
    o.x += f * x.x;
    o.y += f * x.y;
    o.z += f * x.z;
    o.w += f * x.w;
    l += f * ml.y;
  }
};

// kRowWarps warps for each (sequence, head): the own part and the prefix's pieces,
// weighted by their sums, always in the same order.
template <int kRowWarps>
__global__ void __launch_bounds__(32 * kJoinWarps, 7)
    shared_join_kernel(const SharedArgs a, __nv_bfloat16* out, float* out_lse) {
  constexpr int kRows = kJoinWarps / kRowWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part_of = warp % kRowWarps;
  // (rows fit 31 bits, as the call checks)
  const int all = a.num_seqs * a.num_q_heads;
  const int at = static_cast<int>(blockIdx.x) * kRows + warp / kRowWarps;
  const int row = at < all ? at : all - 1;
  const int s = row / a.num_q_heads;
  const int head = row - s * a.num_q_heads;
  const int kvh = head / a.group, h = head - kvh * a.group;
  const SharedLayout& lay = a.lay;
  griddep_launch_dependents();
  griddep_wait();
  const int4 member = lay.member[s];
  const int4 info = lay.info[max(member.x, 0)];  // (of any group where there is none)
  const int tiles = lay.info[a.num_groups].y;
  Joined x{make_float4(0.f, 0.f, 0.f, 0.f), kFloor, 0.f};
  if (part_of == 0) {
    x.o = reinterpret_cast<const float4*>(lay.own_o)[static_cast<int64_t>(row) * 32 + lane];
    const float2 ml = lay.own_ml[row];
    x.m = ml.x;
    x.l = ml.y;
  }
  if (member.x >= 0 && info.z > 0) {
    const int rows = lay.unit_tokens;
    const int u = member.y / rows;
    const int t0 = info.y + u * info.z;
    const int teams = shared_teams(lay, tiles);
    const int j0 = shared_team(t0, tiles, teams);
    const int parts = shared_team(t0 + info.z - 1, tiles, teams) - j0 + 1;
    const int64_t span = static_cast<int64_t>(a.num_kv_heads) * lay.slot_rows;
    const int64_t first =
        (static_cast<int64_t>(j0 + info.x + u) * a.num_kv_heads + kvh) * lay.slot_rows +
        (member.y - u * rows) * a.group + h;
    // (a few at a time: their loads are under way together)
    constexpr int kAhead = 2;
#pragma unroll 1
    for (int p0 = part_of; p0 < parts; p0 += kAhead * kRowWarps) {
      float2 ml[kAhead];
      float4 o[kAhead];
      float top = x.m;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = first + min(p0 + i * kRowWarps, parts - 1) * span;
        ml[i] = lay.part_ml[r];
        o[i] = reinterpret_cast<const float4*>(lay.part_o + r * 128)[lane];
        top = fmaxf(top, ml[i].x);
      }
      x.move(top);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (p0 + i * kRowWarps < parts) x.add(o[i], ml[i]);
    }
  }
  if constexpr (kRowWarps > 1) {
    __shared__ float4 others[kJoinWarps][32];
    __shared__ float2 others_ml[kJoinWarps];
    others[warp][lane] = x.o;
    if (lane == 0) others_ml[warp] = make_float2(x.m, x.l);
    __syncthreads();
    if (part_of != 0) return;
    float top = x.m;
#pragma unroll
    for (int i = 1; i < kRowWarps; ++i) top = fmaxf(top, others_ml[warp + i].x);
    x.move(top);
#pragma unroll
    for (int i = 1; i < kRowWarps; ++i) x.add(others[warp + i][lane], others_ml[warp + i]);
  }
  if (at >= all) return;
  const bool none = x.l == 0.f;
  uint2 o;
  o.x = none ? 0u : pack_bf16x2(x.o.x / x.l, x.o.y / x.l);
  o.y = none ? 0u : pack_bf16x2(x.o.z / x.l, x.o.w / x.l);
  reinterpret_cast<uint2*>(out)[static_cast<int64_t>(row) * 32 + lane] = o;
  if (lane == 0 && out_lse) out_lse[row] = none ? -INFINITY : (x.m + log2f(x.l)) * kLn2;
}

template <int kRowWarps>
cudaError_t launch_join(const SharedArgs& a, __nv_bfloat16* out, float* out_lse,
                        cudaStream_t stream) {
  constexpr int kRows = kJoinWarps / kRowWarps;
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kRows - 1) / kRows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_join_kernel<kRowWarps>, a, out, out_lse);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_join(const SharedArgs& a, __nv_bfloat16* out, float* out_lse,
                               cudaStream_t stream) {
  // Few rows behind a long prefix have a piece from every team: four warps on each.  (us
  // of a call, four warps / one: 512 rows behind 16384 tokens 26.9 / 27.9, 608 behind
  // 32768 38.4 / 39.6; 5120 rows behind 2048 31.7 / 29.3, 8192 behind 4096 44.1 / 39.2, 3200
  // the same.)
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
  return rows <= 2048 ? launch_join<4>(a, out, out_lse, stream)
                      : launch_join<1>(a, out, out_lse, stream);
}

}  // namespace pa
