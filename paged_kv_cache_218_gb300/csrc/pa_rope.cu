// pa_rope.cu -- norms of queries and keys for each head, the position
// rotation, and the slot scatter of keys and values, in one pass (sm_103a).
//
// For a row x (one head of one token, head_dim D, rotary width R):
//
//   y = x * rsqrt(mean(x^2) + eps) * w              (norm; w null: y = x)
//   pair (a, b) of y, pair index i < R / 2, angle  u = position * freq_i:
//   a' = f (a cos u - b sin u),  b' = f (b cos u + a sin u),  f the rope factor
//
// pairs being (i, i + R/2), or (2i, 2i + 1) when interleaved; columns from R
// on pass through.  Everything is fp32 and rounded once, on the way out.
//
// Angles.  A frequency comes as a 64-bit fixed-point number of turns per
// position, so that position * increment mod 2^64 is the exact phase: one
// integer multiply, with no loss at far positions (in fp32, position 10^6
// would be off by 0.06 rad).  The top 32 bits, as a signed number of half
// turns, go to sincospif.
//
// What bounds it: HBM at large batches (each element is read and written
// once), latency at a decode step's.  A warp takes one token and a run of its
// rows; each lane keeps 8 columns (16 bytes) and the sines and cosines of its
// columns, which all heads of the token share, in registers.  Rows of a head
// take 8, 16 or 32 lanes (head_dim to 64, 128, 256), so the sum of squares is
// a few shuffles and the partner of a half-layout pair another one.
#include <math.h>

#include "../../include/pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRows = 4;  // rows in flight per lane

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// E4M3(x / scale), the division in IEEE fp32: the codes of pa_reshape_and_cache_fp8.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
  uint32_t r[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t a = f32x2_to_e4m3x2(__fdiv_rn(x[4 * k], scale), __fdiv_rn(x[4 * k + 1], scale));
    const uint32_t b =
        f32x2_to_e4m3x2(__fdiv_rn(x[4 * k + 2], scale), __fdiv_rn(x[4 * k + 3], scale));
    r[k] = a | (b << 16);
  }
  return make_uint2(r[0], r[1]);
}

// LPR lanes per row; IL: interleaved pairs; F8: E4M3 pools.
template <int LPR, bool IL, bool F8>
__global__ void __launch_bounds__(128) norm_rope_kernel(const RopeArgs a) {
  constexpr int HW = 32 / LPR;  // heads a warp takes at once
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t tok = wid / a.slices;
  if (tok >= a.num_tokens) return;
  const int slice = static_cast<int>(wid % a.slices);

  const int sub = lane / LPR, c = lane % LPR;  // head within the step, 16-byte column piece
  const int D = a.head_dim, half = a.rot_dim / 2;
  const bool live = c * 8 < D;
  const bool rot = c * 8 < a.rot_dim;
  const int64_t pos = a.rot_dim > 0 ? a.positions[tok] : 0;
  // the lane's angles: half layout, its 8 columns' (sine negated in the lower
  // half, whose partner is c + half / 8; the upper half's is c - half / 8);
  // interleaved, its 4 pairs'
  constexpr int NA = IL ? 4 : 8;
  float cs[NA], sn[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  int partner = lane;
  if (rot) {
    const bool lower = c * 8 < half;
    if (!IL) partner = lower ? lane + half / 8 : lane - half / 8;
    const int i0 = IL ? c * 4 : (lower ? c * 8 : c * 8 - half);
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const uint64_t phase = static_cast<uint64_t>(pos) * static_cast<uint64_t>(a.increments[i0 + i]);
      const float turns2 = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      float sv, cv;
      sincospif(turns2, &sv, &cv);
      cs[i] = cv * a.rope_factor;
      sn[i] = (!IL && lower ? -sv : sv) * a.rope_factor;
    }
  }
  const int64_t slot = a.k_cache ? a.slots[tok] : -1;
  bool cached = slot >= 0;
  if (cached && slot >= a.num_slots) {
    if (slice == 0 && lane == 0) atomicOr(a.err, PA_DEVERR_SLOT);
    cached = false;
  }

  // row groups of HW heads: queries, keys, values
  const int gq = (a.num_q_heads + HW - 1) / HW, gk = (a.num_kv_heads + HW - 1) / HW;
  const int groups = gq + gk + (a.k_cache ? gk : 0);
  const int per = (groups + a.slices - 1) / a.slices;
  const int g1 = min(groups, (slice + 1) * per);
  const float inv_d = 1.f / static_cast<float>(D);

  for (int g0 = slice * per; g0 < g1; g0 += kRows) {
    uint4 raw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int g = g0 + r;
      const int kind = g < gq ? 0 : (g < gq + gk ? 1 : 2);
      const int h = (g - (kind == 0 ? 0 : (kind == 1 ? gq : gq + gk))) * HW + sub;
      const __nv_bfloat16* src = kind == 0 ? a.q + tok * a.q_stride
                                           : (kind == 1 ? a.k + tok * a.k_stride
                                                        : a.v + tok * a.v_stride);
      raw[r] = make_uint4(0, 0, 0, 0);
      if (g < g1 && live && h < (kind == 0 ? a.num_q_heads : a.num_kv_heads))
        raw[r] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h) * D + c * 8);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int g = g0 + r;
      if (g >= g1) break;
      const int kind = g < gq ? 0 : (g < gq + gk ? 1 : 2);
      const int h = (g - (kind == 0 ? 0 : (kind == 1 ? gq : gq + gk))) * HW + sub;
      const bool mine = live && h < (kind == 0 ? a.num_q_heads : a.num_kv_heads);
      float x[8];
      unpack8(raw[r], x);
      if (kind < 2) {
        const float* w = kind == 0 ? a.q_weight : a.k_weight;
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float rs = rsqrtf(fmaf(ss, inv_d, a.eps));
          if (live) {
            const float4 w0 = *reinterpret_cast<const float4*>(w + c * 8);
            const float4 w1 = *reinterpret_cast<const float4*>(w + c * 8 + 4);
            x[0] *= rs * w0.x;
            x[1] *= rs * w0.y;
            x[2] *= rs * w0.z;
            x[3] *= rs * w0.w;
            x[4] *= rs * w1.x;
            x[5] *= rs * w1.y;
            x[6] *= rs * w1.z;
            x[7] *= rs * w1.w;
          }
        }
        if constexpr (IL) {
          if (rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = x[2 * i], q = x[2 * i + 1];
              x[2 * i] = p * cs[i] - q * sn[i];
              x[2 * i + 1] = q * cs[i] + p * sn[i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, x[i], partner);
            if (rot) x[i] = x[i] * cs[i] + o * sn[i];
          }
        }
      }
      if (!mine) continue;
      const int64_t col = static_cast<int64_t>(h) * D + c * 8;
      if (kind == 0) {
        *reinterpret_cast<uint4*>(a.q_out + tok * a.num_q_heads * D + col) = pack8(x);
        continue;
      }
      if (kind == 1 && a.k_out)
        *reinterpret_cast<uint4*>(a.k_out + tok * a.num_kv_heads * D + col) = pack8(x);
      if (!cached) continue;
      const int64_t at = slot * a.num_kv_heads * D + col;
      void* pool = kind == 1 ? a.k_cache : a.v_cache;
      if constexpr (F8)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) =
            quant8(x, (kind == 1 ? a.k_scales : a.v_scales)[h]);
      else
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + at) =
            kind == 1 ? pack8(x) : raw[r];
    }
  }
}

template <int LPR, bool IL, bool F8>
cudaError_t launch(RopeArgs a, int num_sms, cudaStream_t stream) {
  constexpr int HW = 32 / LPR;
  const int gk = (a.num_kv_heads + HW - 1) / HW;
  const int groups = (a.num_q_heads + HW - 1) / HW + gk + (a.k_cache ? gk : 0);
  // few tokens: a token's rows go to several warps, kRows row groups each at
  // least, until the SMs hold about 16 warps each
  const int64_t want = static_cast<int64_t>(num_sms) * 16 / a.num_tokens;
  const int most = (groups + kRows - 1) / kRows;
  a.slices = want < 1 ? 1 : (want > most ? most : static_cast<int>(want));
  const int64_t warps = static_cast<int64_t>(a.num_tokens) * a.slices;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_rope_kernel<LPR, IL, F8>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int LPR>
cudaError_t pick(const RopeArgs& a, bool interleaved, bool f8, int num_sms, cudaStream_t st) {
  if (interleaved)
    return f8 ? launch<LPR, true, true>(a, num_sms, st) : launch<LPR, true, false>(a, num_sms, st);
  return f8 ? launch<LPR, false, true>(a, num_sms, st) : launch<LPR, false, false>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, bool interleaved, bool kv_fp8, int num_sms,
                             cudaStream_t stream) {
  if (a.head_dim <= 64) return pick<8>(a, interleaved, kv_fp8, num_sms, stream);
  if (a.head_dim <= 128) return pick<16>(a, interleaved, kv_fp8, num_sms, stream);
  return pick<32>(a, interleaved, kv_fp8, num_sms, stream);
}

}  // namespace pa

using namespace pa;

extern "C" int pa_rope_increments(int64_t* increments, float* rope_factor, int rot_dim, double base,
                                  int scaling, double factor, double original_context,
                                  double param0, double param1) {
  if (!increments || !rope_factor) return PA_ERR_INVALID;
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !isfinite(base)) return PA_ERR_INVALID;
  if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_WAVELENGTH) return PA_ERR_INVALID;
  if (scaling != PA_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return PA_ERR_INVALID;
  const bool by_parts = scaling == PA_ROPE_YARN || scaling == PA_ROPE_WAVELENGTH;
  if (by_parts && (!(original_context >= 1.0) || !isfinite(original_context) || !(param0 > 0.0) ||
                   !(param1 > 0.0) || !isfinite(param0) || !isfinite(param1)))
    return PA_ERR_INVALID;
  if (scaling == PA_ROPE_YARN && !(param0 > param1)) return PA_ERR_INVALID;
  if (scaling == PA_ROPE_WAVELENGTH && !(param1 > param0)) return PA_ERR_INVALID;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double b = base;
  if (scaling == PA_ROPE_NTK) b = base * pow(factor, rot_dim / (rot_dim - 2.0));
  double low = 0.0, high = 0.0;
  if (scaling == PA_ROPE_YARN) {
    // the pair index that makes param0 (param1) turns over the original context
    auto index = [&](double turns) {
      return rot_dim * log(original_context / (turns * kTwoPi)) / (2.0 * log(base));
    };
    low = fmax(floor(index(param0)), 0.0);
    high = fmin(ceil(index(param1)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(b, -2.0 * i / rot_dim);
    if (scaling == PA_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == PA_ROPE_YARN) {
      const double ramp = fmin(1.0, fmax(0.0, (i - low) / fmax(high - low, 0.001)));
      f = f / factor * ramp + f * (1.0 - ramp);
    } else if (scaling == PA_ROPE_WAVELENGTH) {
      const double turns = original_context * f / kTwoPi;  // over the original context
      const double keep = fmin(1.0, fmax(0.0, (turns - param0) / (param1 - param0)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    // f <= 1 rad per position: below a sixth of a turn, 2^62
    increments[i] = static_cast<int64_t>(rint(f / kTwoPi * 18446744073709551616.0));
  }
  *rope_factor = scaling == PA_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  return PA_OK;
}
