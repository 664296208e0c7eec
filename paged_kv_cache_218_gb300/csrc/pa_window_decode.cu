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
// enough bytes in flight.  A warp owns one kv head and walks 16-token blocks;
// the block's K and V rows go from global memory straight into registers (64
// registers = 8 KB per warp in flight at head_dim 128), with the next block's
// K loads issued as soon as this block's scores are done and its V loads as
// soon as its P V is.  There is no shared-memory staging, because the
// contraction order of a dot product is free: a lane hands the tensor core the
// pieces it loaded, and the query operand is permuted the same way.  Loads are
// 32 bytes a lane, so that each covers whole 128-byte lines: with 16 bytes (64
// of a K row at a time) 256 sequences x 4096 keys took 675 us instead of 645
// (6.77 TB/s, the measured copy rate).  A ring of asynchronous copies in shared
// memory, 192 KB in flight per SM instead of at most 128, took 742.
//
//   scores  S^T (16 keys x 8 heads) = K (A, 16 keys x 16 d) Q^T (B)
//           lane (g, t) = (lane / 4, lane % 4) holds keys g and g + 8, columns
//           [16 (4 j + t), + 16) for j < D / 64;
//   output  O^T (16 d x 8 heads) = V^T (A, 16 d x 16 keys) P^T (B)
//           lane (g, t) holds keys 2t, 2t + 1, 2t + 8, 2t + 9, columns
//           [g D / 8, + D / 8); byte permutes pair two keys of one column into
//           an A register.
//
// P enters the tensor core as a sum of two bf16 numbers (p = hi + lo, relative
// error 2^-17), so that the output is rounded to bf16 once, at the end; the
// second product costs 8 of 24 MMAs of a block that waits for memory anyway.
// Scores, statistics and accumulators are fp32.
//
// Split over the key axis: the warps of a CTA, and the CTAs of a cluster (up
// to kMaxWindowSplit), take a sequence's blocks in turn; their (m, l, O) are joined
// in shared memory, then across the cluster through distributed shared memory.
// So the call needs no workspace, and its result does not depend on timing.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "../../include/pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

// Lowest reference maximum (log2 units): a row whose scores are all -inf keeps
// it, so its weights are 0 rather than NaN.
constexpr float kFloor = -1e30f;
// The reference maximum moves only when a score passes it by this much (log2
// units): p stays below 2^8 and most blocks need no cross-lane maximum.
constexpr float kMoveThreshold = 8.f;
constexpr float kLn2 = 0.6931471805599453f;

struct Piece32 {
  uint32_t w[8];
};

__device__ __forceinline__ Piece32 ld_stream32(const void* p) {
  Piece32 v;
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
                 "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}

__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float bf16_round(float x) {
  return __bfloat162float(__float2bfloat16(x));
}

// Shared memory: the warps' partial outputs [warps][8 heads][D], their maxima
// and sums [warps][8] each, then the CTA's joined output [8][D], maxima [8]
// and sums [8] (read by the cluster's other CTAs).
template <int D>
__host__ __device__ constexpr int window_smem_floats(int warps) {
  return warps * (8 * D + 16) + 8 * D + 16;
}

template <int D, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) decode_window_kernel(const WindowDecodeArgs a) {
  constexpr int KJ = D / 64;  // 32-byte pieces of a K row per lane
  constexpr int VW = D / 16;  // 32-bit words of a V row per lane
  extern __shared__ __align__(16) float sm[];
  float* const sm_o = sm;
  float* const sm_m = sm_o + W * 8 * D;
  float* const sm_l = sm_m + W * 8;
  float* const cta_o = sm_l + W * 8;
  float* const cta_m = cta_o + 8 * D;
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
  griddep_wait();

  // q: head g of the group, the columns of this lane's K pieces
  uint4 qf[KJ][2];
  const __nv_bfloat16* qrow =
      a.q + (static_cast<int64_t>(s) * a.num_q_heads + kvh * G + (g < G ? g : 0)) * D;
#pragma unroll
  for (int j = 0; j < KJ; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qf[j][e] = *reinterpret_cast<const uint4*>(qrow + 16 * (4 * j + t) + 8 * e);
      if (g >= G) qf[j][e] = make_uint4(0, 0, 0, 0);
    }

  int n = a.seq_lens[s];
  const int cap = a.max_blocks * kBlockSize;
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && rank == 0 && kvh == 0) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    n = n < 0 ? 0 : cap;
  }
  const int lo = n > a.window ? n - a.window : 0;  // first key of the window
  const int ns = a.sinks < n ? a.sinks : n;        // visible sinks
  const int nsb = (ns + kBlockSize - 1) / kBlockSize;
  const int b_first = max(lo / kBlockSize, nsb);   // first block behind the sinks'
  const int nb = (n + kBlockSize - 1) / kBlockSize;
  const int nv = nsb + (nb > b_first ? nb - b_first : 0);  // visible blocks
  const int stride = splits * W;
  const int first = rank * W + warp;

  const int64_t tok_bytes = static_cast<int64_t>(a.num_kv_heads) * D * 2;
  const char* const kbase = reinterpret_cast<const char*>(a.k) + kvh * (D * 2) + t * 32;
  const char* const vbase = reinterpret_cast<const char*>(a.v) + kvh * (D * 2) + g * (D / 4);
  const int32_t* const table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks;

  float o[VW][4];
#pragma unroll
  for (int i = 0; i < VW; ++i)
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
      ids = table[real_block(mine)];
      if (ids < 0 || ids >= a.num_blocks) {
        atomicOr(a.err, PA_DEVERR_BLOCK_ID);
        ids = -1;  // reads as zeros
      }
    }
  };
  Piece32 kr[2][KJ];
  uint32_t vr[4][VW];
  auto load_k = [&](int id) {
    const char* p = kbase + (static_cast<int64_t>(id) * kBlockSize + g) * tok_bytes;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        if (id < 0)
          kr[r][j] = Piece32{};
        else
          kr[r][j] = ld_stream32(p + r * 8 * tok_bytes + j * 128);
      }
  };
  auto load_v = [&](int id) {
    const char* p = vbase + (static_cast<int64_t>(id) * kBlockSize + 2 * t) * tok_bytes;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const char* row = p + ((r & 1) + (r >> 1) * 8) * tok_bytes;
      if constexpr (D == 128) {
        const Piece32 x = id < 0 ? Piece32{} : ld_stream32(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) vr[r][i] = x.w[i];
      } else {
        const uint4 x = id < 0 ? make_uint4(0, 0, 0, 0) : ld_stream(row);
        vr[r][0] = x.x;
        vr[r][1] = x.y;
        vr[r][2] = x.z;
        vr[r][3] = x.w;
      }
    }
  };

  if (first < nv) {
    read_ids(first);
    int id = __shfl_sync(0xffffffffu, ids, 0);
    load_k(id);
    load_v(id);
  }
  int it = 0;  // position of this block's id in the batch of 32
  for (int vb = first; vb < nv; vb += stride) {
    const int j0 = real_block(vb) * kBlockSize;
    // ---- scores of 16 keys x 8 heads
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t(&x)[8] = kr[0][j].w;
        const uint32_t(&y)[8] = kr[1][j].w;
        const uint32_t a0[4] = {x[4 * e], y[4 * e], x[4 * e + 1], y[4 * e + 1]};
        mma_bf16_16816(sc, a0, qf[j][e].x, qf[j][e].y);
        const uint32_t a1[4] = {x[4 * e + 2], y[4 * e + 2], x[4 * e + 3], y[4 * e + 3]};
        mma_bf16_16816(sc, a1, qf[j][e].z, qf[j][e].w);
      }
    // ---- the next block's K
    const int next = vb + stride;
    int id = 0;
    if (next < nv) {
      if (++it == 32) {
        read_ids(next);
        it = 0;
      }
      id = __shfl_sync(0xffffffffu, ids, it);
      load_k(id);
    }
    // ---- mask (first or last block of the window, last block of the sinks):
    // hidden keys get weight 0 and their V rows, which may hold anything, 0
    const bool edge = !(j0 + kBlockSize <= n && (j0 >= lo || j0 + kBlockSize <= ns));
    float x0 = sc[0] * a.scale_log2, x1 = sc[1] * a.scale_log2;
    float x2 = sc[2] * a.scale_log2, x3 = sc[3] * a.scale_log2;
    if (edge) {
      auto seen = [&](int j) { return j < n && (j >= lo || j < ns); };
      if (!seen(j0 + g)) x0 = x1 = -INFINITY;
      if (!seen(j0 + g + 8)) x2 = x3 = -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!seen(j0 + 2 * t + (r & 1) + (r >> 1) * 8))
#pragma unroll
          for (int i = 0; i < VW; ++i) vr[r][i] = 0;
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
      for (int i = 0; i < VW; ++i) {
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
    for (int i = 0; i < VW; ++i) {
      const uint32_t av[4] = {prmt(vr[0][i], vr[1][i], 0x5410), prmt(vr[0][i], vr[1][i], 0x7632),
                              prmt(vr[2][i], vr[3][i], 0x5410), prmt(vr[2][i], vr[3][i], 0x7632)};
      mma_bf16_16816(o[i], av, hi0, hi1);
      mma_bf16_16816(o[i], av, lo0, lo1);
    }
    // ---- the next block's V
    if (next < nv) load_v(id);
  }

  // ---- join the CTA's warps
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
  for (int i = 0; i < VW; ++i) {
    // rows g, g + 8 of the tile are columns (D / 8) g + 2 i, + 1
    const int d = D / 8 * g + 2 * i;
    float2* dst = reinterpret_cast<float2*>(sm_o + (warp * 8 + 2 * t) * D + d);
    dst[0] = make_float2(o[i][0], o[i][2]);
    dst[D / 2] = make_float2(o[i][1], o[i][3]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < G * D; e += 32 * W) {
    const int h = e / D, d = e % D;
    float m = kFloor;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * 8 + h]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2(sm_m[w * 8 + h] - m);
      acc += f * sm_o[(w * 8 + h) * D + d];
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

template <int D, int W>
cudaError_t launch(const WindowDecodeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                                           a.splits));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = window_smem_floats<D>(W) * sizeof(float);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_window_kernel<D, W>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Opts the eight-warp kernel into clusters of 16; whether one would fit.
template <int D>
bool allow_16() {
  if (cudaFuncSetAttribute(decode_window_kernel<D, 8>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                           1) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(32 * 8);
  cfg.dynamicSmemBytes = window_smem_floats<D>(8) * sizeof(float);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  return cudaOccupancyMaxActiveClusters(&clusters, decode_window_kernel<D, 8>, &cfg) ==
             cudaSuccess &&
         clusters > 0;
}

}  // namespace

cudaError_t launch_decode_window(WindowDecodeArgs a, int head_dim, int num_sms,
                                 cudaStream_t stream) {
  // Largest cluster that this device runs: 16, if the kernels that use it have
  // opted in and a cluster fits; else the portable 8.  Asked once per device.
  static std::mutex mu;
  static int most_for[64] = {};
  int dev = 0, most_split = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (most_for[dev] == 0) {
      const bool ok = allow_16<128>() && allow_16<64>();
      cudaGetLastError();
      most_for[dev] = ok ? kMaxWindowSplit : 8;
    }
    most_split = most_for[dev];
  }
  // Blocks that a sequence can attend at most.
  const int64_t visible = std::min<int64_t>(
      a.max_blocks, (static_cast<int64_t>(a.sinks) + kBlockSize - 1) / kBlockSize +
                        (static_cast<int64_t>(a.window) + kBlockSize - 1) / kBlockSize + 1);
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int64_t slots = static_cast<int64_t>(num_sms) * 16;  // warps, at 128 registers a thread
  int w = 8;
  a.splits = 1;
  if (units * 16 > slots - 64) {
    // Many units: as many warps each as let all of them run at once, for a unit
    // costs 4 us before its first block arrives (256 sequences x 8 heads x 1024
    // keys: 163 us with one warp per unit, 176 with two, 189 with eight; 64
    // sequences: 94, 70, 49 with four, 53 with eight).  Windows of many blocks
    // pay that less, and lengths that differ spread further over them: eight
    // (256 x 4096: one warp 617 us, eight 648; with lengths from 300 on, 446 and
    // 343).
    if (visible <= 160)
      while (w > 1 && (units * w > slots || w >= 2 * visible)) w /= 2;
  } else {
    // Few units: clusters of CTAs, as many warps as there are slots or blocks,
    // in small CTAs while 16 warps do (148 units of 64 blocks: 4 x 4 warps 6.4
    // us, 2 x 8 6.9, 1 x 8 8.0; 32 units of 2050 blocks: 8 x 8 88 us, 4 x 8 130).
    // Clusters of 16 where one CTA per SM suffices and eight CTAs' warps would
    // have four blocks or more each (8 units of 2050 blocks: 40 us, with 8 CTAs
    // 61; but 16 units 77 and 70, and 8 units of 66 blocks 8.0 and 6.9).
    const int64_t warps = std::min<int64_t>(visible, slots / units);
    w = warps > 16 ? 8 : 4;
    while (a.splits * w < visible && 2 * a.splits * w * units <= slots &&
           (a.splits < 8 || (a.splits < most_split && 2 * a.splits * units <= num_sms &&
                             4 * a.splits * w <= visible)))
      a.splits *= 2;
  }
  switch (w) {
    case 1: return head_dim == 128 ? launch<128, 1>(a, stream) : launch<64, 1>(a, stream);
    case 2: return head_dim == 128 ? launch<128, 2>(a, stream) : launch<64, 2>(a, stream);
    case 4: return head_dim == 128 ? launch<128, 4>(a, stream) : launch<64, 4>(a, stream);
    default: return head_dim == 128 ? launch<128, 8>(a, stream) : launch<64, 8>(a, stream);
  }
}

}  // namespace pa
