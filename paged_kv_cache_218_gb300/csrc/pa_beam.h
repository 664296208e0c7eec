// pa_beam.h -- launch parameters of the beam-search calls, shared between the
// C-ABI front end (pa_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kMaxBeams = 32;    // beams of a request: a lane each
constexpr int kMaxChoices = 64;  // choices of a request

// The best continuations of each request (pa_beam_select).
struct BeamSelectArgs {
  int32_t* parents;  // [R, K]
  int32_t* tokens;   // [R, K]
  float* out_scores; // [R, K]
  uint8_t* out_finished;    // [R, K] or null
  const void* logits;       // row (r, w) at r * request_stride + w * beam_stride (elements)
  const float* scores;      // [R, W]
  const uint8_t* finished;  // [R, W] or null
  int64_t request_stride;
  int64_t beam_stride;
  int end_token;
  int num_requests;
  int num_beams;
  int num_choices;
  int vocab;
  // set by the launcher
  int block_shift;     // log2 of the warp loads per block of a row
  int blocks_per_row;  // entries of the block maxima for each beam
  uint32_t blocks_inverse;  // 2^32 / blocks_per_row, rounded up
  int all_sum;         // the whole cluster takes sums again
  float margin;        // (halved) values nearer than this are compared again, more exactly
};

// Tables, lengths and partly filled blocks after a selection (pa_beam_reorder).
struct BeamReorderArgs {
  int32_t* out_tables;   // [R * W, max_blocks]
  int32_t* out_lens;     // [R * W]
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* parents;  // [R, W]
  char* k;                 // pools, layer l at + l * layer_bytes
  char* v;
  unsigned int* err;
  int64_t num_blocks;
  int64_t layer_bytes;
  int64_t token_bytes;     // of one token's row of one pool
  int num_requests;
  int num_beams;
  int max_blocks;
  int num_layers;
  int parts;  // CTAs that share one layer's copies of a request; set by the launcher
};

// Kernel launchers (return cudaError_t of the launch).
cudaError_t launch_beam_select(const BeamSelectArgs& a, bool fp32, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_beam_reorder(BeamReorderArgs a, int num_sms, cudaStream_t stream);

}  // namespace pa
