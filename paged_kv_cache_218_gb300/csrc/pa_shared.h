// pa_shared.h -- launch parameters of the shared-prefix decode (pa_decode_shared),
// shared between the C-ABI front end (pa_api.cu) and its kernels.  Not part of the
// public ABI.
#pragma once

#include "pa_window.h"

namespace pa {

// The prefix pass cuts its work into teams of workers (CTAs, or pairs of them), one worker
// for each kv head.  Units are (group, rows of a worker's query tiles), in order; a team
// takes a range of the units' key tiles, all units behind one another, and leaves a
// partial result (maximum, sum, weighted values) for each unit that it meets: that of
// team j and unit u in slot (j + u) * kv heads + kv head, so that a unit's slots are
// neighbours.
struct SharedLayout {
  int worker_ctas;   // 1, or 2 for groups of more than 128 query rows per kv head
  int teams;
  int team_workers;  // of a team; a worker takes every team_workers-th kv head
  int tile_tokens;   // members (query tokens) of a query tile, 128 / group
  int unit_tokens;   // and of a unit, worker_ctas tiles
  int box_tokens;    // and of a load of one: no group has more
  int slot_rows;    // query rows of a slot
  int max_units;    // that the slots have room for
  float* part_o;    // [slots][slot_rows][128], not divided by the sum
  float2* part_ml;  // [slots][slot_rows]: reference maximum (log2 units), sum
  // [num_groups + 1]: a group's first unit, its first key tile, key tiles of each of its
  // units, first member; last entry: .y all key tiles.  Written by the prefix pass.
  int4* info;
  // Of the decode of each sequence's own part: [num_seqs] its group (-1: none), its number
  // in it, its prefix's blocks; [num_seqs][q heads][128] weighted values, and [num_seqs]
  // [q heads] maximum and sum, as above.
  int4* member;
  float* own_o;
  float2* own_ml;
};

struct SharedArgs {
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* group_offsets;  // [num_groups + 1]
  const int32_t* shared_blocks;  // [num_groups]
  unsigned int* err;
  int64_t num_blocks;
  int max_blocks;
  int num_seqs;
  int num_groups;
  int max_group;  // members that a group may have
  int num_q_heads;
  int num_kv_heads;
  int group;  // q heads per kv head
  float scale_log2;
  uint64_t wait_ns;  // limit of every mbarrier wait (0: the default)
  int stall_loads;   // test launch: the loaders issue no load, every wait runs out
  SharedLayout lay;
};

// What a group's metadata say, as far as they are sound.
struct SharedGroup {
  int first, members, blocks;
  bool sound;
};
__device__ __forceinline__ SharedGroup shared_group(const SharedArgs& a, int g) {
  SharedGroup x;
  const int f = __ldcg(a.group_offsets + g), e = __ldcg(a.group_offsets + g + 1);
  const int b = __ldcg(a.shared_blocks + g);
  x.first = min(max(f, 0), a.num_seqs);
  x.members = min(min(max(e, x.first), a.num_seqs) - x.first, a.max_group);
  x.blocks = min(max(b, 0), a.max_blocks);
  x.sound = f == x.first && e == f + x.members && b == x.blocks;
  return x;
}

// The group of sequence s (-1: none), s's number in it, its prefix's blocks.  Called by a
// whole warp.
__device__ __forceinline__ int4 find_group(const SharedArgs& a, int s, int lane) {
  if (a.num_groups == 0) return make_int4(-1, 0, 0, 0);
  // offsets rise: 32 of them at a time narrow the range [lo, hi) whose group holds s
  int lo = 0, hi = a.num_groups;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && __ldcg(a.group_offsets + at) <= s;
    // (at least the first one: sequences before every group have none, seen below)
    const int n = max(__popc(__ballot_sync(0xffffffffu, below)), 1);
    const int next = lo + (n - 1) * step;
    hi = min(hi, next + step);
    lo = next;
  }
  const SharedGroup g = shared_group(a, lo);
  if (s < g.first || s >= g.first + g.members) return make_int4(-1, 0, 0, 0);
  return make_int4(lo, s - g.first, g.blocks, 0);
}

// Teams that take part: with at least four key tiles each where there are as many (the
// others' SMs are free for the sequences' own parts meanwhile: nine ragged groups of up
// to 37 blocks 31.6 us, with one tile 34.4, with eight 37.1).  None has an empty range.
__device__ __forceinline__ int shared_teams(const SharedLayout& lay, int tiles) {
  return min(lay.teams, max((tiles + 3) / 4, 1));
}

// The team that takes key tile t of `tiles`: the last one whose first tile
// j * tiles / teams is not behind t.
__device__ __forceinline__ int shared_team(int t, int tiles, int teams) {
  // (a 64-bit division takes as long as a load)
  if (tiles < 1 << 20)  // (teams <= SMs)
    return static_cast<int>((static_cast<unsigned>(t + 1) * teams - 1) /
                            static_cast<unsigned>(tiles));
  return static_cast<int>(((static_cast<int64_t>(t) + 1) * teams - 1) / tiles);
}

// Decode over each sequence's own blocks.
struct SharedDecodeArgs : WindowDecodeArgs {
  SharedArgs shared;
};

cudaError_t launch_shared_prefix(const SharedArgs& a, const CUtensorMap* tm_q,
                                 const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                 cudaStream_t stream);
cudaError_t launch_shared_decode(const SharedDecodeArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_shared_join(const SharedArgs& a, __nv_bfloat16* out, float* out_lse,
                               cudaStream_t stream);

}  // namespace pa
