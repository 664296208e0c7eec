// pa_window_decode.cu -- paged decode attention over a sliding window and a
// few first tokens that stay visible (sm_103a).
//
// One query per sequence, GQA group G <= 8.  With n = seq_len, window W and S
// sinks, query head h sees the keys j < n with j < S or j >= n - W:
//
//   out = sum_j 2^(c x_j - m) v_j / sum_j 2^(c x_j - m),  x_j = <q, k_j>,
//   c = scale * log2(e), m a running reference maximum.
//
// What bounds it: HBM.  Every visible K/V row is read once (4 D bytes per key
// and kv head against 4 D G multiply-adds), so the kernel's job is to keep
// enough bytes in flight, in requests that memory likes.  A warp owns one kv
// head and walks 16-token blocks (8 KB of K and V at head_dim 128) through a
// ring of three in shared memory, filled by asynchronous copies: a copy
// instruction takes whole rows (two of 256 bytes), so each 128-byte line is
// asked for once.  The ring is the warp's own, so the warp alone waits for it,
// and 192 KB per SM are on their way.  At 256 sequences x 4096 keys this reads
// 7.1 TB/s (measured copy rate: 6.8).  What it replaced, at the same case: rows
// loaded straight into the MMA's registers, 16 bytes a lane and so 64 of a K
// row at a time, 688 us; 32 bytes a lane 645; lane-private copies of 16 bytes
// through shared memory, again 64 of a row at a time, 742; this 590 to 613.
//
//   scores  S^T (16 keys x 8 heads) = K (A, 16 keys x 16 d) Q^T (B)
//           lane (g, t) = (lane / 4, lane % 4) holds keys g and g + 8, columns
//           [8 (4 j + t), + 8) for j < D / 32, as it reads them (16 bytes):
//           the order of a contraction is free, and the query operand is
//           permuted the same way;
//   output  O^T (16 d x 8 heads) = V^T (A, 16 d x 16 keys) P^T (B)
//           lane (g, t) holds keys 2t, 2t + 1, 2t + 8, 2t + 9, columns
//           [8 (8 h + g), + 8) for h < D / 64; byte permutes pair two keys of
//           one column into an A register.
//
// In the ring, 16-byte column c of row r sits at c ^ 4 (r & 1) for K and at
// c ^ (r & 6) for V, which spreads both read patterns over all banks.
//
// P enters the tensor core as a sum of two bf16 numbers (p = hi + lo, relative
// error 2^-17), so that the output is rounded to bf16 once, at the end; the
// second product costs 8 of 24 MMAs of a block that waits for memory anyway.
// Scores, statistics and accumulators are fp32.
//
// Split over the key axis: the warps of a CTA, and the CTAs of a cluster, take
// a sequence's blocks in turn; their (m, l, O) are joined in shared memory,
// then across the cluster through distributed shared memory, always in the same
// order: the call needs no workspace, and its bits do not depend on timing.
//
// A prefill call of few query tokens comes here too, a token as a sequence of
// its own that ends with it, and finds its chunk with one more round trip.
//
// So does the decode of sequences that share prefixes, for what is each one's own:
// the blocks behind its group's prefix.  It runs beside the prefix pass, whose CTAs leave
// room on each SM for the rings of two warps (beside a lone CTA) or four (beside one of a
// pair), and reads nothing of it; a third kernel joins both (pa_shared_prefix.cu).  Alone
// it reads 294 MB of 256 sequences in 54 us.  Beside the pass a CTA of one warp lives 20 us
// for 17 blocks, 9 for 4 or 5: 5 us for its chain of round trips, 0.9 a block.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "../../include/pa.h"
#include "pa_shared.h"
#include "pa_window_ptx.cuh"

namespace pa {
namespace {

// Lowest reference maximum (log2 units), the lowest finite fp32: a row whose
// scores are all -inf keeps it, so its weights are 0 rather than NaN.
constexpr float kFloor = -FLT_MAX;
// The reference maximum moves only when a score passes it by this much (log2
// units): p stays below 2^8 and most blocks need no cross-lane maximum.
constexpr float kMoveThreshold = 8.f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float bf16_round(float x) {
  return __bfloat162float(__float2bfloat16(x));
}

// Blocks in flight per warp; two where two warps have a unit behind a shared prefix, so
// that both fit beside a lone CTA of the prefix pass.
template <int W, int M>
constexpr int kStages = 3;
template <>
constexpr int kStages<2, 2> = 2;

// Shared memory: the warps' rings [W][kStages][K, V][16 rows][D]; once a warp
// has read its last block its outputs [8 heads][D] (fp32) take the front of its
// ring, and those of the whole CTA the next part of warp 0's; maxima and sums
// [W][8], and the CTA's [8], behind the rings.
template <int D, int W, int M>
struct DecodePlan {
  static constexpr int kStage = 2 * kBlockSize * D * 2;
  static constexpr int kRing = kStages<W, M> * kStage;
  static constexpr int kStatOff = W * kRing;
  static constexpr int kBytes = kStatOff + (W + 1) * 16 * 4;
  static_assert(2 * 8 * D * 4 <= kRing, "outputs in the ring");
};

// The chunk that holds query token s: its table's row, and the number of keys
// up to the token's own; -1 where no consistent chunk does.  Called by a whole
// warp.
__device__ __forceinline__ int find_chunk(const WindowDecodeArgs& a, int s, int lane, int& n) {
  for (int c0 = 0; c0 < a.num_chunks; c0 += 32) {
    const int c = c0 + lane;
    int q0 = 0, q1 = 0, p0 = 0;
    bool mine = false;
    if (c < a.num_chunks) {
      q0 = a.cu_q_lens[c];
      q1 = a.cu_q_lens[c + 1];
      p0 = a.q_start_pos[c];
      mine = q0 <= s && s < q1 && chunk_ok(q0, q1, p0, a.seq_lens[c], a.num_seqs, a.max_blocks);
    }
    const unsigned at = __ballot_sync(0xffffffffu, mine);
    if (at == 0) continue;
    n = __shfl_sync(0xffffffffu, p0 + s - q0 + 1, __ffs(at) - 1);
    return c0 + __ffs(at) - 1;
  }
  return -1;
}

// What the queries are: a sequence's last token each, those of chunks (see
// WindowDecodeArgs), or a sequence's last token behind a shared prefix.
enum DecodeKind : int { kSequences = 0, kChunks = 1, kShared = 2 };

template <int M>
struct KindArgs {
  using type = WindowDecodeArgs;
};
template <>
struct KindArgs<kShared> {
  using type = SharedDecodeArgs;
};

// (Behind a shared prefix at most 128 registers: what three warps of the prefix pass leave
// of a quarter of an SM.)
template <int D, int W, int M>
__global__ void __launch_bounds__(32 * W, M == kShared ? 16 / W : 0)
    decode_window_kernel(const typename KindArgs<M>::type a) {
  constexpr bool C = M == kChunks;
  using P = DecodePlan<D, W, M>;
  constexpr int kStages = pa::kStages<W, M>;
  constexpr int KJ = D / 32;  // 16-byte pieces of a K row per lane
  constexpr int VH = D / 64;  // 16-byte pieces of a V row per lane
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kPart = P::kRing / 4;  // floats from one warp's outputs to the next
  float* const sm_o = reinterpret_cast<float*>(smem);
  float* const sm_m = reinterpret_cast<float*>(smem + P::kStatOff);
  float* const sm_l = sm_m + W * 8;
  float* const cta_o = sm_o + 8 * D;
  float* const cta_m = sm_l + W * 8;
  float* const cta_l = cta_m + 8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int splits = a.splits;
  const int rank = static_cast<int>(blockIdx.x) % splits;
  const int unit = static_cast<int>(blockIdx.x) / splits;
  const int kvh = unit % a.num_kv_heads;
  const int s = unit / a.num_kv_heads;
  const int G = a.group;

  griddep_launch_dependents();
  // (beside the prefix pass: what that waited for before it let this kernel start is
  // there, and read past L1)
  if constexpr (M != kShared) griddep_wait();

  // q: head g of the group, the columns of this lane's K pieces
  uint4 qf[KJ];
  const __nv_bfloat16* qrow =
      a.q + (static_cast<int64_t>(s) * a.num_q_heads + kvh * G + (g < G ? g : 0)) * D;
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    const uint4* const at = reinterpret_cast<const uint4*>(qrow + 8 * (4 * j + t));
    qf[j] = M == kShared ? __ldcg(at) : *at;
    if (g >= G) qf[j] = make_uint4(0, 0, 0, 0);
  }

  int n, table_row = s;
  if constexpr (C) {
    if (blockIdx.x == 0 && warp == 0)
      for (int c = lane; c < a.num_chunks; c += 32)
        if (!chunk_ok(a.cu_q_lens[c], a.cu_q_lens[c + 1], a.q_start_pos[c], a.seq_lens[c],
                      a.num_seqs, a.max_blocks))
          atomicOr(a.err, PA_DEVERR_CHUNK);
    table_row = find_chunk(a, s, lane, n);
    if (table_row < 0) return;  // (every CTA of the cluster) a row of no chunk stays
  } else {
    n = M == kShared ? __ldcg(a.seq_lens + s) : a.seq_lens[s];
    const int cap = a.max_blocks * kBlockSize;
    if (n < 0 || n > cap) {
      if (threadIdx.x == 0 && rank == 0 && kvh == 0) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
      n = n < 0 ? 0 : cap;
    }
  }
  int lo = n > a.window ? n - a.window : 0;        // first key of the window
  int ns = a.sinks < n ? a.sinks : n;              // visible sinks
  if constexpr (M == kShared) {
    const int4 member = find_group(a.shared, s, lane);
    if (kvh == 0 && threadIdx.x == 0) a.shared.lay.member[s] = member;
    lo = member.z * kBlockSize;                    // first key of the sequence's own
    ns = 0;
  }
  const int nsb = (ns + kBlockSize - 1) / kBlockSize;
  const int b_first = max(lo / kBlockSize, nsb);   // first block behind the sinks'
  const int nb = (n + kBlockSize - 1) / kBlockSize;
  const int nv = nsb + (nb > b_first ? nb - b_first : 0);  // visible blocks
  const int stride = splits * W;
  const int first = rank * W + warp;

  const int64_t tok_bytes = static_cast<int64_t>(a.num_kv_heads) * D * 2;
  const int head_bytes = kvh * (D * 2) + (lane % (D / 8)) * 16;
  const char* const kbase = reinterpret_cast<const char*>(a.k) + head_bytes;
  const char* const vbase = reinterpret_cast<const char*>(a.v) + head_bytes;
  const int32_t* const table = a.block_tables + static_cast<int64_t>(table_row) * a.max_blocks;

  float o[4 * VH][4];
#pragma unroll
  for (int i = 0; i < 4 * VH; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float m0 = kFloor, m1 = kFloor, l0 = 0.f, l1 = 0.f;  // heads 2t, 2t + 1

  // The block of visible index vb; its id, read 32 of this warp's blocks at a
  // time (lane i holds the id of its block first + i * stride).
  auto real_block = [&](int vb) { return vb < nsb ? vb : vb - nsb + b_first; };
  int ids = 0;
  auto read_ids = [&](int vb) {
    const int mine = vb + lane * stride;
    ids = 0;
    if (mine < nv) {
      ids = M == kShared ? __ldcg(table + real_block(mine)) : table[real_block(mine)];
      if (ids < 0 || ids >= a.num_blocks) {
        atomicOr(a.err, PA_DEVERR_BLOCK_ID);
        ids = -1;  // reads as zeros
      }
    }
  };
  // Copies of this warp's next block into stage `st` (an empty group past its
  // last one, so that the count of groups runs on).
  const uint32_t ring = smem_u32(smem) + warp * P::kRing;
  constexpr int kRowBytes = D * 2, kChunks = D / 8, kRowsPerCopy = 32 / kChunks;
  const int crow = lane / kChunks, cchunk = lane % kChunks;
  int load_vb = first, load_it = 0;
  auto issue = [&](int st) {
    if (load_vb < nv) {
      if (load_it == 32) {
        read_ids(load_vb);
        load_it = 0;
      }
      const int id = __shfl_sync(0xffffffffu, ids, load_it++);
      load_vb += stride;
      const int bytes = id < 0 ? 0 : 16;
      const int64_t off = (static_cast<int64_t>(id < 0 ? 0 : id) * kBlockSize + crow) * tok_bytes;
      const char* pk = kbase + off;
      const char* pv = vbase + off;
      const uint32_t dst = ring + st * P::kStage;
#pragma unroll
      for (int i = 0; i < kBlockSize / kRowsPerCopy; ++i) {
        const int row = kRowsPerCopy * i + crow;
        cp_async_16_zfill(dst + row * kRowBytes + ((cchunk ^ ((row & 1) << 2)) << 4),
                          pk + i * kRowsPerCopy * tok_bytes, bytes);
      }
#pragma unroll
      for (int i = 0; i < kBlockSize / kRowsPerCopy; ++i) {
        const int row = kRowsPerCopy * i + crow;
        cp_async_16_zfill(
            dst + (kBlockSize + row) * kRowBytes + ((cchunk ^ (row & 6)) << 4),
            pv + i * kRowsPerCopy * tok_bytes, bytes);
      }
    }
    cp_async_commit();
  };
  if (first < nv) read_ids(first);
#pragma unroll
  for (int st = 0; st < kStages; ++st) issue(st);

  int stage = 0;
  for (int vb = first; vb < nv; vb += stride) {
    const int j0 = real_block(vb) * kBlockSize;
    cp_async_wait_group<kStages - 1>();
    __syncwarp();
    const uint32_t src = ring + stage * P::kStage + g * kRowBytes;
    const uint32_t srcv = ring + stage * P::kStage + (kBlockSize + 2 * t) * kRowBytes;
    // ---- scores of 16 keys x 8 heads
    float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const uint32_t at = ((4 * j + t) ^ ((g & 1) << 2)) << 4;
      const uint4 k0 = lds128(src + at), k1 = lds128(src + 8 * kRowBytes + at);
      const uint32_t a0[4] = {k0.x, k1.x, k0.y, k1.y};
      mma_bf16_16816(sc, a0, qf[j].x, qf[j].y);
      const uint32_t a1[4] = {k0.z, k1.z, k0.w, k1.w};
      mma_bf16_16816(sd, a1, qf[j].z, qf[j].w);
    }
    uint4 vr[4][VH];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int h = 0; h < VH; ++h)
        vr[r][h] = lds128(srcv + ((r & 1) + (r >> 1) * 8) * kRowBytes +
                          (((8 * h + g) ^ (2 * t)) << 4));
    // ---- mask (first or last block of the window, last block of the sinks):
    // hidden keys get weight 0 and their V rows, which may hold anything, 0
    const bool edge = !(j0 + kBlockSize <= n && (j0 >= lo || j0 + kBlockSize <= ns));
    float x0 = (sc[0] + sd[0]) * a.scale_log2, x1 = (sc[1] + sd[1]) * a.scale_log2;
    float x2 = (sc[2] + sd[2]) * a.scale_log2, x3 = (sc[3] + sd[3]) * a.scale_log2;
    if (edge) {
      auto seen = [&](int j) { return j < n && (j >= lo || j < ns); };
      if (!seen(j0 + g)) x0 = x1 = -INFINITY;
      if (!seen(j0 + g + 8)) x2 = x3 = -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!seen(j0 + 2 * t + (r & 1) + (r >> 1) * 8))
#pragma unroll
          for (int h = 0; h < VH; ++h) vr[r][h] = make_uint4(0, 0, 0, 0);
    }
    // ---- reference maximum
    float b0 = fmaxf(x0, x2), b1 = fmaxf(x1, x3);
    if (__any_sync(0xffffffffu, b0 > m0 + kMoveThreshold || b1 > m1 + kMoveThreshold)) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, off));
        b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, off));
      }
      b0 = fmaxf(b0, m0);
      b1 = fmaxf(b1, m1);
      const float s0 = fast_exp2(m0 - b0), s1 = fast_exp2(m1 - b1);
      m0 = b0;
      m1 = b1;
      l0 *= s0;
      l1 *= s1;
#pragma unroll
      for (int i = 0; i < 4 * VH; ++i) {
        o[i][0] *= s0;
        o[i][1] *= s1;
        o[i][2] *= s0;
        o[i][3] *= s1;
      }
    }
    const float p0 = fast_exp2(x0 - m0), p1 = fast_exp2(x1 - m1);
    const float p2 = fast_exp2(x2 - m0), p3 = fast_exp2(x3 - m1);
    l0 += p0 + p2;
    l1 += p1 + p3;
    // P^T as the B operand: keys 2t, 2t + 1 (and + 8) of head g
    const uint32_t hi0 = movmatrix_trans(pack_bf16x2(p0, p1));
    const uint32_t hi1 = movmatrix_trans(pack_bf16x2(p2, p3));
    const uint32_t lo0 = movmatrix_trans(pack_bf16x2(p0 - bf16_round(p0), p1 - bf16_round(p1)));
    const uint32_t lo1 = movmatrix_trans(pack_bf16x2(p2 - bf16_round(p2), p3 - bf16_round(p3)));
#pragma unroll
    for (int h = 0; h < VH; ++h) {
      const uint32_t r0[4] = {vr[0][h].x, vr[0][h].y, vr[0][h].z, vr[0][h].w};
      const uint32_t r1[4] = {vr[1][h].x, vr[1][h].y, vr[1][h].z, vr[1][h].w};
      const uint32_t r2[4] = {vr[2][h].x, vr[2][h].y, vr[2][h].z, vr[2][h].w};
      const uint32_t r3[4] = {vr[3][h].x, vr[3][h].y, vr[3][h].z, vr[3][h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t av[4] = {prmt(r0[i], r1[i], 0x5410), prmt(r0[i], r1[i], 0x7632),
                                prmt(r2[i], r3[i], 0x5410), prmt(r2[i], r3[i], 0x7632)};
        mma_bf16_16816(o[4 * h + i], av, hi0, hi1);
        mma_bf16_16816(o[4 * h + i], av, lo0, lo1);
      }
    }
    // ---- the stage's next block (what was read from it is in registers)
    __syncwarp();
    issue(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }

  // ---- join the CTA's warps
  cp_async_wait_all();
  __syncwarp();
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, off);
    l1 += __shfl_xor_sync(0xffffffffu, l1, off);
  }
  if (g == 0) {
    sm_m[warp * 8 + 2 * t] = m0;
    sm_m[warp * 8 + 2 * t + 1] = m1;
    sm_l[warp * 8 + 2 * t] = l0;
    sm_l[warp * 8 + 2 * t + 1] = l1;
  }
#pragma unroll
  for (int h = 0; h < VH; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows g, g + 8 of the tile are columns 8 (8 h + g) + 2 i, + 1
      const int d = 8 * (8 * h + g) + 2 * i;
      float2* dst = reinterpret_cast<float2*>(sm_o + warp * kPart + 2 * t * D + d);
      dst[0] = make_float2(o[4 * h + i][0], o[4 * h + i][2]);
      dst[D / 2] = make_float2(o[4 * h + i][1], o[4 * h + i][3]);
    }
  __syncthreads();
  if constexpr (M == kShared) {
    // four columns of a head, left undivided
    for (int e = 4 * threadIdx.x; e < G * D; e += 4 * 32 * W) {
      const int h = e / D, d = e % D;
      float m = kFloor;
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * 8 + h]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
      auto add = [&](float f, float4 x, float sum) {
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
        l += f * sum;
      };
#pragma unroll
      for (int w = 0; w < W; ++w)
        add(fast_exp2(sm_m[w * 8 + h] - m),
            *reinterpret_cast<const float4*>(sm_o + w * kPart + h * D + d), sm_l[w * 8 + h]);
      const int64_t row = static_cast<int64_t>(s) * a.num_q_heads + kvh * G + h;
      *reinterpret_cast<float4*>(a.shared.lay.own_o + row * D + d) = acc;
      if (d == 0) a.shared.lay.own_ml[row] = make_float2(m, l);
    }
    // (who waits for this kernel waits for the prefix pass, too)
    if (blockIdx.x == 0) griddep_wait();
  } else {
    for (int e = threadIdx.x; e < G * D; e += 32 * W) {
      const int h = e / D, d = e % D;
      float m = kFloor;
  #pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * 8 + h]);
      float acc = 0.f, l = 0.f;
  #pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = fast_exp2(sm_m[w * 8 + h] - m);
        acc += f * sm_o[w * kPart + h * D + d];
        l += f * sm_l[w * 8 + h];
      }
      if (splits == 1) {
        const int64_t row = static_cast<int64_t>(s) * a.num_q_heads + kvh * G + h;
        a.out[row * D + d] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
        if (d == 0 && a.out_lse) a.out_lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        cta_o[e] = acc;
        if (d == 0) {
          cta_m[h] = m;
          cta_l[h] = l;
        }
      }
    }
    if (splits == 1) return;

    // ---- join the cluster's CTAs: CTA r writes every splits-th element
    cluster_sync();
    const uint32_t ro = smem_u32(cta_o), rm = smem_u32(cta_m), rl = smem_u32(cta_l);
    for (int e = rank * 32 * W + threadIdx.x; e < G * D; e += splits * 32 * W) {
      const int h = e / D, d = e % D;
      float m = kFloor;
      for (int c = 0; c < splits; ++c) m = fmaxf(m, ld_dsmem(mapa_shared(rm + 4 * h, c)));
      float acc = 0.f, l = 0.f;
      for (int c = 0; c < splits; ++c) {
        const float f = fast_exp2(ld_dsmem(mapa_shared(rm + 4 * h, c)) - m);
        acc += f * ld_dsmem(mapa_shared(ro + 4 * e, c));
        l += f * ld_dsmem(mapa_shared(rl + 4 * h, c));
      }
      const int64_t row = static_cast<int64_t>(s) * a.num_q_heads + kvh * G + h;
      a.out[row * D + d] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
      if (d == 0 && a.out_lse) a.out_lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while another may still read its shared memory
  }
}

template <int D, int W, int M>
cudaError_t launch(const typename KindArgs<M>::type& a, cudaStream_t stream) {
  {  // raise the kernel's shared-memory limit once per device
    static std::mutex mu;
    static bool set_for[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!set_for[dev]) {
      e = cudaFuncSetAttribute(decode_window_kernel<D, W, M>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               DecodePlan<D, W, M>::kBytes);
      if (e != cudaSuccess) return e;
      if (M == kShared) {
        // (an SM keeps its split of memory while a CTA runs: the prefix pass's, so that
        // CTAs of both share SMs)
        e = cudaFuncSetAttribute(decode_window_kernel<D, W, M>,
                                 cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
      }
      set_for[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                                           a.splits));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = DecodePlan<D, W, M>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_window_kernel<D, W, M>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// How many clusters of 1, 2, 4, 8 and 16 eight-warp CTAs the device runs at
// once (the last is not portable: 0 where the device or a partition of it
// cannot); asked once per device.
struct Residency {
  bool ready = false;
  int clusters[5] = {};
};
static_assert(kMaxWindowSplit == 1 << 4, "cluster sizes");

template <int D, int M>
cudaError_t residency(int num_sms, Residency* out) {
  static std::mutex mu;
  static Residency by_device[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  Residency& r = by_device[dev];
  if (!r.ready) {
    constexpr int smem = DecodePlan<D, 8, M>::kBytes;
    const auto kernel = decode_window_kernel<D, 8, M>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int ctas = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, 32 * 8, smem);
    if (e != cudaSuccess) return e;
    r.clusters[0] = ctas * num_sms;
    const bool wide = cudaFuncSetAttribute(
                          kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int k = 1; k < 5; ++k) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << k);
      cfg.blockDim = dim3(32 * 8);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1 << k;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if ((k == 4 && !wide) || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess)
        n = 0;
      r.clusters[k] = n;
    }
    cudaGetLastError();  // (a size that the device refuses is no error here)
    r.ready = true;
  }
  *out = r;
  return cudaSuccess;
}

template <int D, int M>
cudaError_t choose(WindowDecodeArgs a, int num_sms, cudaStream_t stream) {
  Residency res;
  const cudaError_t e = residency<D, M>(num_sms, &res);
  if (e != cudaSuccess) return e;
  // Blocks that a sequence can attend at most.
  const int64_t visible = std::min<int64_t>(
      a.max_blocks, (static_cast<int64_t>(a.sinks) + kBlockSize - 1) / kBlockSize +
                        (static_cast<int64_t>(a.window) + kBlockSize - 1) / kBlockSize + 1);
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  a.splits = 1;
  if (units <= res.clusters[0]) {
    // Few units: eight warps each, and as large clusters of such CTAs as all run
    // at once and find a block for every warp; none for a few blocks, whose
    // joining costs more (us, at 8 / 16 / 32 / 64 units: 17 blocks 4.7 / 4.8 /
    // 4.8 / 4.8 with one CTA, 4.8 to 5.7 with clusters; 66 blocks 8.6 / 9.0 /
    // 8.9 / 9.8 with one, 5.8 / 6.2 / 6.4 / 9.3 with clusters of 8, 4, 4, 2).
    if (visible > 24)
      for (int k = 1; k < 5; ++k)
        if (units <= res.clusters[k] && (8 << k) <= visible) a.splits = 1 << k;
    return launch<D, 8, M>(a, stream);
  }
  if constexpr (M == kChunks) return launch<D, 4, M>(a, stream);
  // Many units: few warps on each keep more units at once and hide what a unit
  // costs before its first block arrives; many warps spread units of different
  // lengths.  The number with the least estimated time (us; fewer only where that
  // saves a percent): units come in rounds of as many as run at once; a round's
  // blocks share the memory's 7.1 TB/s, a block takes a warp 0.4 us at least, a
  // further round costs 2, and a quarter of a block's time on each of a warp's
  // blocks stands for lengths that differ.  Over 160 to 1760 units of 14 to 108 blocks, head_dim 64 and 128, its
  // choices take 3.3 % longer than the best one's for equal lengths and 6 % for
  // lengths from nothing on, on average; eight warps always 16 and 15, four 7 and
  // 9, two 12 and 41, one 21 and 83.  (us, with 1 / 2 / 4 / 8 warps: 1024 units
  // of 66 blocks, some shorter, 76.3 / 71.5 / 69.3 / 69.5; 2048 of 258 629 / 609 /
  // 605 / 600.)
  const double slots = static_cast<double>(res.clusters[0]) * 8;  // warps at once
  const double block_us = slots * (2 * kBlockSize * D * 2) / 7.1e6;
  int w = 8;
  double least = 0;
  for (int k = 8; k > 0; k /= 2) {
    const int64_t at_once = static_cast<int64_t>(slots) / k;
    const int64_t full = units / at_once, rest = units % at_once;
    const double blocks = static_cast<double>(visible) / k;
    double us = blocks * (0.25 + full * block_us) + 2.0 * (full + (rest > 0 ? 1 : 0));
    if (rest > 0) us += blocks * std::max(0.4, block_us * rest / at_once);
    if (k == 8 || us < 0.99 * least) {
      w = k;
      least = us;
    }
  }
  switch (w) {
    case 1: return launch<D, 1, kSequences>(a, stream);
    case 2: return launch<D, 2, kSequences>(a, stream);
    case 4: return launch<D, 4, kSequences>(a, stream);
    default: return launch<D, 8, kSequences>(a, stream);
  }
}

}  // namespace

cudaError_t launch_decode_window_chunks(const WindowDecodeArgs& a, int num_sms,
                                        cudaStream_t stream) {
  return choose<128, kChunks>(a, num_sms, stream);
}

cudaError_t launch_decode_window(const WindowDecodeArgs& a, int head_dim, int num_sms,
                                 cudaStream_t stream) {
  return head_dim == 128 ? choose<128, kSequences>(a, num_sms, stream)
                         : choose<64, kSequences>(a, num_sms, stream);
}

cudaError_t launch_shared_decode(const SharedDecodeArgs& args, int num_sms, cudaStream_t stream) {
  SharedDecodeArgs a = args;
  a.splits = 1;
  // How long a sequence's own part is, the host does not know.  Eight warps on each up to
  // one on every SM; above, as many as run at once, and few enough to start beside the
  // prefix pass.  (us of a call behind 8192 shared tokens, 8 kv heads, with 8 / 4 / 2 / 1
  // warps: 16 sequences of 1 to 64 tokens of their own 20.2 / 19.6 / 19.8 / 19.9, to 1200
  // 27.1 / 30.2 / 37.6 / 45.5, to 5000 49 / 66 / 102 / 135; 64 to 64 34.1 / 27.1 / 25.8 /
  // 25.2, to 1200 55.1 / 48.8 / 57.6 / 55.8, to 5000 139 / 137 / 162 / 164; 110 to 300 55.2 /
  // 43.6 / 45.6 / 45.5; 256 to 40 88.8 / 64.7 / 61.9 / 57.5.)
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  if (units <= num_sms) return launch<128, 8, kShared>(a, stream);
  if (units <= 6 * num_sms) return launch<128, 2, kShared>(a, stream);
  return launch<128, 1, kShared>(a, stream);
}

}  // namespace pa
