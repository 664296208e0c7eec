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
// position, so that position * increment mod 2^64 is its phase: one integer
// multiply, and at far positions no error but the frequency's own (in fp32,
// position 10^6 would be off by 0.06 rad).  The top 32 bits become an fp32
// angle in [-pi, pi], within 6e-7, and the special-function unit's sine and
// cosine are within 2^-21.4 there: together under 2^-20, a 4000th of the half
// step of bf16 of a value of the pair's size.
//
// What bounds it: HBM at large batches (each element is read and written
// once), latency at a decode step's.  A warp takes one token and a few steps
// of 32 / LPR rows of one kind (queries, keys or values), all of whose loads
// it issues at once.  A lane keeps 16 columns of a row, as two 16-byte pieces
// that hold both members of its eight pairs (half layout: columns [8 i, + 8)
// and [R / 2 + 8 i, + 8); otherwise 16 columns in a row), so a rotation needs
// no other lane.  A row takes LPR = 4, 8 or 16 lanes (head_dim to 64, 128,
// 256); the lanes with the same columns share the work on the angles.  Norm
// weights and sines are multiplied together once per warp, and the arithmetic
// runs on pairs of fp32 values.  8192 tokens of 32 + 8 heads of 128 take 33.4 us
// (6.04 TB/s, 89 % of the measured copy rate; the same loads and stores without
// arithmetic 30.7), 64 tokens 2.3.
#include <math.h>

#include "../../include/pa.h"
#include "pa_window.h"
#include "pa_window_ptx.cuh"

namespace pa {
namespace {

constexpr float kPiOver2to31 = 3.14159265358979f / 2147483648.f;

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A lane's two pieces of a row as the members (a, b) of its pairs: as loaded,
// or, interleaved, with the even columns in the first piece and the odd ones
// in the second.  The same exchange puts a result's pieces back.
__device__ __forceinline__ void deinterleave(uint4& u, uint4& v) {
  const uint4 p = u, q = v;
  u = make_uint4(prmt(p.x, p.y, 0x5410), prmt(p.z, p.w, 0x5410), prmt(q.x, q.y, 0x5410),
                 prmt(q.z, q.w, 0x5410));
  v = make_uint4(prmt(p.x, p.y, 0x7632), prmt(p.z, p.w, 0x7632), prmt(q.x, q.y, 0x7632),
                 prmt(q.z, q.w, 0x7632));
}

__device__ __forceinline__ void interleave(uint4& u, uint4& v) {
  const uint4 p = u, q = v;
  u = make_uint4(prmt(p.x, q.x, 0x5410), prmt(p.x, q.x, 0x7632), prmt(p.y, q.y, 0x5410),
                 prmt(p.y, q.y, 0x7632));
  v = make_uint4(prmt(p.z, q.z, 0x5410), prmt(p.z, q.z, 0x7632), prmt(p.w, q.w, 0x5410),
                 prmt(p.w, q.w, 0x7632));
}

// Bytes of E4M3 codes: 8 columns a piece, the same exchange.
__device__ __forceinline__ void interleave(uint2& u, uint2& v) {
  const uint2 p = u, q = v;
  u = make_uint2(prmt(p.x, q.x, 0x5140), prmt(p.x, q.x, 0x7362));
  v = make_uint2(prmt(p.y, q.y, 0x5140), prmt(p.y, q.y, 0x7362));
}

// Eight bf16 columns as four pairs of fp32, and back.
__device__ __forceinline__ void unpack(const uint4& u, uint64_t (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f32x2(lo_f32(w[i]), hi_f32(w[i]));
}

__device__ __forceinline__ uint4 pack(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f32x2_parts(x[i]);
    w[i] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 fp32 weights at w + c0 and w + c1, split the same way.
__device__ __forceinline__ void load_weights(const float* w, int c0, int c1, bool interleaved,
                                             uint64_t (&a)[4], uint64_t (&b)[4]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 u = *reinterpret_cast<const float4*>(w + c0 + 4 * e);
    const float4 t = *reinterpret_cast<const float4*>(w + c1 + 4 * e);
    if (interleaved) {
      a[e] = f32x2(u.x, u.z);
      b[e] = f32x2(u.y, u.w);
      a[2 + e] = f32x2(t.x, t.z);
      b[2 + e] = f32x2(t.y, t.w);
    } else {
      a[2 * e] = f32x2(u.x, u.y);
      a[2 * e + 1] = f32x2(u.z, u.w);
      b[2 * e] = f32x2(t.x, t.y);
      b[2 * e + 1] = f32x2(t.z, t.w);
    }
  }
}

// E4M3(x / scale) of 8 columns, the division in IEEE fp32: the codes of
// pa_reshape_and_cache_fp8.  The product with the reciprocal is within 2^-22
// of that quotient, and rounding to E4M3 is monotone: where the codes of the
// product a little lower and a little higher agree, they are the quotient's
// code, and the division (eight times the work) is left out.  `inv` 0: a
// scale whose reciprocal is not a normal number; divide.
__device__ __forceinline__ uint2 quant(const uint64_t (&x)[4], float scale, float inv) {
  uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
  const uint64_t inv_lo = f32x2(inv * (1.f - 0x1p-21f), inv * (1.f - 0x1p-21f));
  const uint64_t inv_hi = f32x2(inv * (1.f + 0x1p-21f), inv * (1.f + 0x1p-21f));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 l = f32x2_parts(mul2(x[i], inv_lo)), h = f32x2_parts(mul2(x[i], inv_hi));
    lo[i / 2] |= static_cast<uint32_t>(f32x2_to_e4m3x2(l.x, l.y)) << (16 * (i & 1));
    hi[i / 2] |= static_cast<uint32_t>(f32x2_to_e4m3x2(h.x, h.y)) << (16 * (i & 1));
  }
  if (lo[0] != hi[0] || lo[1] != hi[1] || inv == 0.f) {
    lo[0] = lo[1] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f32x2_parts(x[i]);
      lo[i / 2] |= static_cast<uint32_t>(
                       f32x2_to_e4m3x2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale)))
                   << (16 * (i & 1));
    }
  }
  return make_uint2(lo[0], lo[1]);
}

__device__ __forceinline__ float reciprocal(float scale) {
  return scale >= 0x1p-100f && scale <= 0x1p100f ? __frcp_rn(scale) : 0.f;
}

// LPR lanes per row; R: steps of 32 / LPR rows per warp; F8: E4M3 pools; NORM:
// at least one of the norms; EVEN: rows fill their lanes (head_dim = 16 LPR)
// and heads fill their steps.  Registers for six CTAs per SM; five for E4M3,
// whose codes' arithmetic would spill (2048 tokens: 13.4 us at six, 12.4 at
// five, 13.3 at four).
template <int LPR, int R, bool F8, bool NORM, bool EVEN>
__global__ void __launch_bounds__(128, F8 ? 5 : 6) norm_rope_kernel(const RopeArgs a) {
  constexpr int HW = 32 / LPR;  // rows of a step
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (tok >= a.num_tokens) return;
  const int sub = lane / LPR, i = lane % LPR;  // row of the step, lane of the row
  const int D = EVEN ? 16 * LPR : a.head_dim;
  const bool live = EVEN || i * 16 < D;
  const bool rot = i * 16 < a.rot_dim;
  const bool split = !a.interleaved && rot;  // the pieces are half a rotary width apart
  const int c0 = split ? i * 8 : i * 16;
  const int c1 = split ? i * 8 + a.rot_dim / 2 : i * 16 + 8;

  // blockIdx.y: the queries' warps of a token, the keys', the values'
  constexpr int per = HW * R;  // rows of a warp
  const int uq = (a.num_q_heads + per - 1) / per, uk = (a.num_kv_heads + per - 1) / per;
  const int u = blockIdx.y;
  const int kind = u < uq ? 0 : (u < uq + uk ? 1 : 2);
  const int h0 = (kind == 0 ? u : (kind == 1 ? u - uq : u - uq - uk)) * per;
  const int heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
  const int steps = min(R, (heads - h0 + HW - 1) / HW);  // >= 1
  auto mine = [&](int r) { return EVEN || (live && h0 + r * HW + sub < heads); };
  const __nv_bfloat16* const src = (kind == 0 ? a.q + tok * a.q_stride
                                              : (kind == 1 ? a.k + tok * a.k_stride
                                                           : a.v + tok * a.v_stride)) +
                                   (h0 + sub) * D;
  uint4 raw[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    raw[r][0] = raw[r][1] = make_uint4(0, 0, 0, 0);
    if (r < steps && mine(r)) {
      raw[r][0] = *reinterpret_cast<const uint4*>(src + r * HW * D + c0);
      raw[r][1] = *reinterpret_cast<const uint4*>(src + r * HW * D + c1);
    }
  }
  float scale[R];  // of this lane's rows in E4M3 pools
#pragma unroll
  for (int r = 0; F8 && r < R; ++r)
    scale[r] = kind > 0 && r < steps && mine(r)
                   ? (kind == 1 ? a.k_scales : a.v_scales)[h0 + r * HW + sub]
                   : 1.f;
  int64_t slot = -1;
  if (kind > 0 && a.k_cache) {
    slot = a.slots[tok];
    if (slot >= a.num_slots) {
      if (lane == 0 && u == uq) atomicOr(a.err, PA_DEVERR_SLOT);
      slot = -1;
    }
  }
  // where this lane's first row goes: bf16 outputs y0 and (bf16 pools) y1, codes z
  const int64_t in_cache = slot * a.num_kv_heads * D + (h0 + sub) * D;
  void* const pool = kind == 1 ? a.k_cache : a.v_cache;
  __nv_bfloat16* y0 = kind == 0 ? a.q_out : (kind == 1 ? a.k_out : nullptr);
  if (y0) y0 += (tok * heads + h0 + sub) * D;
  __nv_bfloat16* const y1 =
      !F8 && slot >= 0 ? static_cast<__nv_bfloat16*>(pool) + in_cache : nullptr;
  uint8_t* const z = F8 && slot >= 0 ? static_cast<uint8_t*>(pool) + in_cache : nullptr;

  if constexpr (!F8) {
    if (kind == 2) {  // values pass through
      if (!y1) return;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < steps && mine(r)) {
          *reinterpret_cast<uint4*>(y1 + r * HW * D + c0) = raw[r][0];
          *reinterpret_cast<uint4*>(y1 + r * HW * D + c1) = raw[r][1];
        }
      return;
    }
  }

  // Coefficients of this lane's pairs: a' = rs (ac a + bs b), b' = rs (bc b + as a),
  // with rs = 1 / rms, ac = wa cos, bs = -wb sin, bc = wb cos, as = wa sin.
  uint64_t ac[4], as[4], bc[4], bs[4];
  const float* const w = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : nullptr);
#pragma unroll
  for (int e = 0; e < 4; ++e) ac[e] = bc[e] = f32x2(1.f, 1.f);
  const bool turn = rot && kind < 2;
  if (NORM && w && live) load_weights(w, c0, c1, a.interleaved && turn, ac, bc);
  if (kind < 2 && a.rot_dim > 0) {
    // the HW lanes with the same columns compute 8 / HW angles each
    const int64_t pos = a.positions[tok];
    constexpr int NA = HW >= 8 ? 1 : 8 / HW;
    float c[NA], s[NA];
#pragma unroll
    for (int e = 0; e < NA; ++e) {
      const int64_t inc = rot ? a.increments[i * 8 + (sub * NA + e) % 8] : 0;
      const uint64_t phase = static_cast<uint64_t>(pos) * static_cast<uint64_t>(inc);
      __sincosf(static_cast<float>(static_cast<int32_t>(phase >> 32)) * kPiOver2to31, &s[e], &c[e]);
      c[e] *= a.rope_factor;
      s[e] *= a.rope_factor;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float cc[2], ss[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int from = (2 * e + f) / NA * LPR + i;
        cc[f] = __shfl_sync(0xffffffffu, c[(2 * e + f) % NA], from);
        ss[f] = __shfl_sync(0xffffffffu, s[(2 * e + f) % NA], from);
      }
      as[e] = mul2(ac[e], f32x2(ss[0], ss[1]));
      bs[e] = mul2(bc[e], f32x2(-ss[0], -ss[1]));
      if (rot) {
        ac[e] = mul2(ac[e], f32x2(cc[0], cc[1]));
        bc[e] = mul2(bc[e], f32x2(cc[0], cc[1]));
      }
    }
  }
  const float inv_d = 1.f / static_cast<float>(D);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= steps) break;
    if (a.interleaved && turn) deinterleave(raw[r][0], raw[r][1]);
    uint64_t xa[4], xb[4];
    unpack(raw[r][0], xa);
    unpack(raw[r][1], xb);
    if (NORM && (!F8 || w)) {
      uint64_t s2 = mul2(xa[0], xa[0]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e) s2 = fma2(xa[e], xa[e], s2);
        s2 = fma2(xb[e], xb[e], s2);
      }
      const float2 sp = f32x2_parts(s2);
      float ss = sp.x + sp.y;
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float rs = F8 || w ? rsqrtf(fmaf(ss, inv_d, a.eps)) : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xa[e] = mul2(xa[e], f32x2(rs, rs));
        xb[e] = mul2(xb[e], f32x2(rs, rs));
      }
    }
    if (turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t p = xa[e];
        xa[e] = fma2(ac[e], p, mul2(bs[e], xb[e]));
        xb[e] = fma2(bc[e], xb[e], mul2(as[e], p));
      }
    } else if (NORM && (!F8 || w)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xa[e] = mul2(xa[e], ac[e]);
        xb[e] = mul2(xb[e], bc[e]);
      }
    }
    if (!mine(r)) continue;
    if (!F8 || y0) {
      uint4 p = pack(xa), q = pack(xb);
      if (a.interleaved && turn) interleave(p, q);
      if (y0) {
        *reinterpret_cast<uint4*>(y0 + r * HW * D + c0) = p;
        *reinterpret_cast<uint4*>(y0 + r * HW * D + c1) = q;
      }
      if (y1) {
        *reinterpret_cast<uint4*>(y1 + r * HW * D + c0) = p;
        *reinterpret_cast<uint4*>(y1 + r * HW * D + c1) = q;
      }
    }
    if (F8 && z) {
      const float inv = reciprocal(scale[r]);
      uint2 p = quant(xa, scale[r], inv), q = quant(xb, scale[r], inv);
      if (a.interleaved && turn) interleave(p, q);
      *reinterpret_cast<uint2*>(z + r * HW * D + c0) = p;
      *reinterpret_cast<uint2*>(z + r * HW * D + c1) = q;
    }
  }
}

template <int LPR, int R, bool F8, bool NORM, bool EVEN>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  constexpr int per = 32 / LPR * R;
  const int uk = (a.num_kv_heads + per - 1) / per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.num_tokens) + 3) / 4),
                     (a.num_q_heads + per - 1) / per + uk + (a.k_cache ? uk : 0));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_rope_kernel<LPR, R, F8, NORM, EVEN>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int LPR, bool F8, bool NORM>
cudaError_t pick_steps(const RopeArgs& a, int num_sms, cudaStream_t st) {
  constexpr int HW = 32 / LPR;
  const bool even = a.head_dim == 16 * LPR && a.num_q_heads % HW == 0 && a.num_kv_heads % HW == 0;
  if (!even) return launch<LPR, 2, F8, NORM, false>(a, st);
  // four steps per warp share the angles' cost; two, where four would leave
  // the SMs' schedulers with fewer than two warps each
  constexpr int per = HW * 4;
  const int64_t warps = static_cast<int64_t>(a.num_tokens) *
                        ((a.num_q_heads + per - 1) / per + 2 * ((a.num_kv_heads + per - 1) / per));
  return warps >= num_sms * 8 ? launch<LPR, 4, F8, NORM, true>(a, st)
                              : launch<LPR, 2, F8, NORM, true>(a, st);
}

template <int LPR>
cudaError_t pick(const RopeArgs& a, bool f8, int num_sms, cudaStream_t st) {
  const bool norm = a.q_weight || a.k_weight;
  if (norm)
    return f8 ? pick_steps<LPR, true, true>(a, num_sms, st)
              : pick_steps<LPR, false, true>(a, num_sms, st);
  return f8 ? pick_steps<LPR, true, false>(a, num_sms, st)
            : pick_steps<LPR, false, false>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, bool kv_fp8, int num_sms, cudaStream_t stream) {
  if (a.head_dim <= 64) return pick<4>(a, kv_fp8, num_sms, stream);
  if (a.head_dim <= 128) return pick<8>(a, kv_fp8, num_sms, stream);
  return pick<16>(a, kv_fp8, num_sms, stream);
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
