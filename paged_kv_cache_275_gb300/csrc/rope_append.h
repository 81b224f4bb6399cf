// Internal interface of the rotary append kernel (rope_append.cu), used by capi.cu.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Rotation and append of a batch of tokens (rope_append.cu).
constexpr int kMaxPositionAxes = 4;
struct RopeAppendParams {
  const void* q;  // rows of [heads][head_dim] bf16, `stride` 16-byte chunks apart
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int64_t* positions;  // [num_axes][num_tokens], axes axis_stride apart
  int64_t axis_stride;
  const float* cos_sin;      // fp32 [max_position][head_dim]
  int64_t max_position;
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  unsigned* err;
  int64_t num_tokens;
  int64_t num_slots;  // 16 * num_blocks
  int num_q_heads;
  int num_kv_heads;
  int num_axes;
  int parts;  // warps that share a token's rows
  uint8_t freq_axis[64];  // position axis of each of the head_dim / 2 frequencies
};

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, int num_sms, cudaStream_t stream);

}  // namespace pkv
