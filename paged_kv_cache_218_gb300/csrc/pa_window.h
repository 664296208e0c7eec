// pa_window.h -- launch parameters of the windowed attention and of the norm,
// rotation and scatter pass, shared between the C-ABI front end (pa_api.cu) and
// their kernels.  Not part of the public ABI.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kMaxWindowSplit = 16;  // decode: most CTAs that share a unit's blocks

// Decode over a sliding window and sinks (pa_decode_window).
struct WindowDecodeArgs {
  __nv_bfloat16* out;           // [S, Hq, D]
  const __nv_bfloat16* q;       // [S, Hq, D]
  const __nv_bfloat16* k;       // pools
  const __nv_bfloat16* v;
  const int32_t* block_tables;  // [S, max_blocks]
  const int32_t* seq_lens;      // [S]
  float* out_lse;               // [S, Hq] or null
  unsigned int* err;
  int64_t num_blocks;
  int max_blocks;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int group;
  int window;  // keys [len - window, len) are visible,
  int sinks;   // and keys [0, sinks)
  float scale_log2;
  int splits;  // CTAs (a cluster) per (sequence, kv head); set by the launcher
  // Chunks of queries (pa_prefill_window's few tokens): a "sequence" is a query
  // token, and num_seqs the number of tokens; tables and lengths are the chunks'.
  const int32_t* cu_q_lens;    // [num_chunks + 1]
  const int32_t* q_start_pos;  // [num_chunks]
  int num_chunks;
};

// Whether a chunk's query rows [q0, q1), first position and length agree with
// one another and with the call.
__device__ __forceinline__ bool chunk_ok(int q0, int q1, int p0, int n, int total_q,
                                         int max_blocks) {
  return q0 >= 0 && q1 <= total_q && q1 >= q0 && p0 >= 0 && n >= 0 && q1 - q0 <= n &&
         p0 <= n - (q1 - q0) && n <= max_blocks * kBlockSize;
}

// Norms, position rotation and slot scatter (pa_qk_norm_rope_cache).
struct RopeArgs {
  __nv_bfloat16* q_out;      // [T, Hq, D]
  __nv_bfloat16* k_out;      // [T, Hkv, D] or null
  const __nv_bfloat16* q;    // rows at token strides (elements)
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  const float* q_weight;     // [D] or null (no norm)
  const float* k_weight;
  const int64_t* positions;  // [T]
  const int64_t* increments; // [rot_dim / 2], 2^-64 turns per position
  const int64_t* slots;      // [T]
  void* k_cache;             // pools, or both null
  void* v_cache;
  const float* k_scales;     // E4M3 pools: [Hkv]
  const float* v_scales;
  unsigned int* err;
  int64_t num_slots;
  float eps;
  float rope_factor;
  int num_tokens;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  int rot_dim;
  int interleaved;
};

// Prefill chunks under a sliding window and sinks (pa_prefill_window).
struct WindowPrefillArgs : PrefillArgs {
  int window;  // a query at p sees keys (p - window, p]
  int sinks;   // and keys [0, sinks)
};

// Kernel launchers (return cudaError_t of the launch).
cudaError_t launch_norm_rope(const RopeArgs& a, bool kv_fp8, int num_sms, cudaStream_t stream);
cudaError_t launch_decode_window(const WindowDecodeArgs& a, int head_dim, int num_sms,
                                 cudaStream_t stream);
cudaError_t launch_decode_window_chunks(const WindowDecodeArgs& a, int num_sms,
                                        cudaStream_t stream);  // head_dim 128
cudaError_t launch_prefill_window(const WindowPrefillArgs& a, const CUtensorMap* tm_q,
                                  const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                  int64_t max_items, int num_sms, cudaStream_t stream);

}  // namespace pa
