// pa_beam_reorder.cu -- block tables, lengths and partly filled blocks of a
// paged cache after a beam selection (sm_103a).
//
// New beam i of a request continues old beam p = parents[i], of n tokens: the
// blocks [0, n / 16) of its table are history, which beams share, and block
// n / 16 and those behind it are a beam's own (the next tokens go there).
// Of a parent's children the first keeps the parent's own blocks; every other
// one takes those of a childless beam, the n % 16 tokens already in the block
// copied over in every layer.  A childless beam's blocks are no child's
// source, so all copies of a request run at once, in any order, in place.
// There are as many childless beams as beams in want of blocks, since each
// beam with children gives up one of W and takes one of W.
//
// What bounds it: HBM, by the bytes copied: 64 requests of 4 beams in 32 layers of 8 heads
// of 128 (84 MB, read and written) take 31.3 us, 5.4 TB/s, 81 % of what a plain copy
// reaches; one request 4.5 us, a launch and four dependent round trips.  A beam's filled
// slots of one layer are contiguous in each pool, so a copy is a run of up to 15 token
// rows; a warp reads its share of a run, 16 bytes a lane and eight of them
// under way, before it writes.  The mapping is a few ballots of a warp, which
// every warp makes for itself rather than wait for another.
#include <algorithm>

#include "../../include/pa.h"
#include "pa_beam.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // 16-byte vectors a thread has under way

__device__ __forceinline__ unsigned low_lanes(int n) { return n >= 32 ? ~0u : (1u << n) - 1; }

// Place of the k-th set bit (from 0) of a mask that has one.
__device__ __forceinline__ int nth_bit(unsigned mask, int k) {
  for (; k > 0; --k) mask &= mask - 1;
  return __ffs(mask) - 1;
}

__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const BeamReorderArgs a) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x, W = a.num_beams;
  griddep_launch_dependents();
  griddep_wait();

  // ---- lane i: old beam i, and new beam i
  const int64_t row = static_cast<int64_t>(r) * W + lane;
  const bool here = lane < W;
  int parent = here ? a.parents[row] : -1;
  int len = here ? a.lens[row] : 0;
  const bool reports = blockIdx.y == 0 && threadIdx.x < 32;
  if (parent < -1 || parent >= W) {
    if (reports) atomicOr(a.err, PA_DEVERR_BEAM);
    parent = -1;
  }
  const int cap = a.max_blocks * kBlockSize;
  if (len < 0 || len > cap) {
    if (reports) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    len = len < 0 ? 0 : cap;
  }
  // ---- the beam's first own block, and whether another beam has the same (rows of a fork
  // do until their last blocks are copied): nobody's to give away
  const int32_t* const tables = a.tables + static_cast<int64_t>(r) * W * a.max_blocks;
  const int own_col = len / kBlockSize;
  const int own = here && own_col < a.max_blocks
                      ? tables[static_cast<int64_t>(lane) * a.max_blocks + own_col]
                      : -1;
  const unsigned like = __match_any_sync(0xffffffffu, own);
  const int taken = own >= 0 && (like & (like - 1)) != 0;
  const unsigned before = (1u << lane) - 1;
  const unsigned siblings = __match_any_sync(0xffffffffu, parent);
  const bool child = here && parent >= 0;
  const bool first = child && (siblings & before) == 0;
  const unsigned chosen = __reduce_or_sync(0xffffffffu, child ? 1u << parent : 0u);
  const unsigned idle = low_lanes(W) & ~chosen;
  const unsigned extra = __ballot_sync(0xffffffffu, child && !first);
  const unsigned orphan = __ballot_sync(0xffffffffu, here && !child);
  int owner = parent;  // whose own blocks this beam takes
  if (here && !first)
    owner = nth_bit(idle, child ? __popc(extra & before)
                                : __popc(extra) + __popc(orphan & before));
  if (!here) owner = 0;
  const int from = parent < 0 ? 0 : parent;
  const int parent_len = __shfl_sync(0xffffffffu, len, from);
  const int owner_len = __shfl_sync(0xffffffffu, len, owner);
  const int new_len = child ? parent_len : 0;
  const int keep = new_len / kBlockSize;         // blocks of history
  const int shift = owner_len / kBlockSize - keep;  // own block of column c: the owner's c + shift
  if (reports && here) a.out_lens[row] = new_len;

  // ---- copies: lane i's source and destination block, and vectors to copy
  int32_t* const out = a.out_tables + static_cast<int64_t>(r) * W * a.max_blocks;
  const int filled = new_len % kBlockSize;
  const int src = __shfl_sync(0xffffffffu, own, from);
  const int dst = __shfl_sync(0xffffffffu, own, owner);
  const bool begun = child && !first && filled > 0;
  bool copy = begun && a.num_layers > 0;
  if ((__shfl_sync(0xffffffffu, taken, owner) && begun) ||
      (copy && (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks))) {
    if (reports) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
    copy = false;
  }
  // what every thread needs of each beam
  __shared__ int4 row_of[kMaxBeams];  // history's row, own row, history's blocks, shift
  __shared__ int2 copy_of[kMaxBeams];
  __shared__ int filled_of[kMaxBeams];
  const unsigned copies = __ballot_sync(0xffffffffu, copy);
  if (threadIdx.x < 32) {
    row_of[lane] = make_int4(from, owner, keep, shift);
    if (copy) {
      const int at = __popc(copies & before);
      copy_of[at] = make_int2(src, dst);
      filled_of[at] = filled;
    }
  }
  __syncthreads();

  // ---- tables: the request's CTAs take entries in turn
  const int entries = W * a.max_blocks, step = gridDim.y * kThreads;
  for (int e = blockIdx.y * kThreads + threadIdx.x; e < entries; e += step) {
    const int i = e / a.max_blocks, c = e - i * a.max_blocks;
    const int4 x = row_of[i];
    int id = -1;
    if (c < x.z)
      id = tables[static_cast<int64_t>(x.x) * a.max_blocks + c];
    else if (c + x.w < a.max_blocks)
      id = tables[static_cast<int64_t>(x.y) * a.max_blocks + c + x.w];
    out[e] = id;
  }

  // ---- units of the copies: beam, layer, pool, part of the run of filled slots; a warp
  // each, so that a CTA has eight on their way
  const int64_t block_bytes = a.token_bytes * kBlockSize;
  const int runs = 2 * a.num_layers * a.parts;
  const int64_t units = static_cast<int64_t>(__popc(copies)) * runs;
  const int warps = gridDim.y * (kThreads / 32);
  for (int64_t u = blockIdx.y * (kThreads / 32) + threadIdx.x / 32; u < units; u += warps) {
    const int at = static_cast<int>(u / runs), run = static_cast<int>(u - at * runs);
    const int pool_run = run / a.parts, part = run - pool_run * a.parts;
    char* const pool = ((pool_run & 1) ? a.v : a.k) + (pool_run >> 1) * a.layer_bytes;
    const int2 ids = copy_of[at];
    const uint4* const s = reinterpret_cast<const uint4*>(pool + ids.x * block_bytes);
    uint4* const d = reinterpret_cast<uint4*>(pool + ids.y * block_bytes);
    const int64_t vecs = filled_of[at] * a.token_bytes / 16;
    const int64_t end = vecs * (part + 1) / a.parts;
    for (int64_t v = vecs * part / a.parts + lane; v < end; v += 32 * kVecs) {
      uint4 x[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (v + j * 32 < end) x[j] = s[v + j * 32];
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (v + j * 32 < end) d[v + j * 32] = x[j];
    }
  }
}

}  // namespace

cudaError_t launch_beam_reorder(BeamReorderArgs a, int num_sms, cudaStream_t stream) {
  // A run of one layer's pool is up to 15 token rows; four warps share one of 2 KB rows.
  // CTAs of eight warps: for every run of all beams but one, at most as many as fit the
  // device, eight on an SM.
  a.parts = static_cast<int>(std::min<int64_t>(std::max<int64_t>(a.token_bytes / 512, 1), 8));
  const int64_t want = (8ll * num_sms + a.num_requests - 1) / a.num_requests;
  const int64_t runs = (2ll * a.num_layers * a.parts * std::max(1, a.num_beams - 1) + 7) / 8;
  const int64_t columns =
      (static_cast<int64_t>(a.num_beams) * a.max_blocks + kThreads - 1) / kThreads;
  const int64_t units = std::max(runs, columns);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_requests),
                     static_cast<unsigned>(std::max<int64_t>(1, std::min(units, want))));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, beam_reorder_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
