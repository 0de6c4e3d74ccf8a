// rope_append.h -- the launch of the rotary append (rope_append.cu), shared with the entry
// points (abi.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace pa {

constexpr int kErrAxis = 128;

constexpr int kMaxRopeAxes = 8;
struct RopeArgs {
  const void* q;               // rows of num_q_heads * head_dim elements, q_stride apart; null: none
  void* q_out;                 // the same, q_out_stride apart (may be q itself)
  const void* key;             // rows of num_kv_heads * head_dim; null: nothing to append
  const void* value;
  void* k_cache;
  void* v_cache;
  const int64_t* slot_mapping; // [num_tokens]
  const int64_t* positions;    // [num_axes][num_tokens]
  const float* inv_freq;       // [rotary_dim / 2]
  const int32_t* pair_axis;    // [rotary_dim / 2], or null: every pair on axis 0
  int num_axes;
  int rotary_dim;              // a multiple of 16, at most head_dim
  float rot_scale;
  long long q_stride, key_stride, value_stride, q_out_stride;  // elements between tokens
  long long num_tokens;
  int num_q_heads, num_kv_heads, head_dim, block_size;
  long long num_slots;
  int32_t* err_flag;
  int tokens_per_cta;          // (set by the launcher)
  int units_per_slice;
};
cudaError_t launch_rope_append(RopeArgs a, int elem_bytes, bool adjacent, int num_sms,
                               cudaStream_t stream);

}  // namespace pa
