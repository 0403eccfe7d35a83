// delta_internal.h -- launch interface between the gated delta rule's entry
// points (delta.cu) and its kernels (delta.cu, delta_chunk.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

struct DeltaArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float *g, *beta;
  const int32_t* cu;     // packed sequences: [batch + 1] first rows, or null
  const int32_t* index;  // decode: state of each row, or null
  const float* state_in;
  __nv_bfloat16* out;
  float* state_out;
  int64_t batch, L, H, G, dk, dv, num_states;
  int64_t q_tok, q_seq, k_tok, k_seq, v_tok, v_seq, o_tok, o_seq, gb_tok, gb_seq;
  float scale;
  int l2norm;
  uint32_t two16;  // 65536, a value the compiler does not know
  int* err;
};

constexpr int kDeltaChunk = 64;  // tokens of a chunk

// Heads of 64 channels: two that share their keys fill the 128 rows of a walk.
inline bool delta_pairs(int64_t H, int64_t G, int64_t dv) { return dv == 64 && H / G % 2 == 0; }
// Walks of a sequence: its heads times the slices of 128 channels, or pairs of heads.
inline int64_t delta_walkers(int64_t H, int64_t G, int64_t dv) {
  return delta_pairs(H, G, dv) ? H / 2 : H * ((dv + 127) / 128);
}

// SMs of the current device.
int device_sms();

// 64 tokens at a time on the tensor cores; a.L > 0.
cudaError_t launch_delta_chunk(const DeltaArgs& a, void* ws, cudaStream_t st);
size_t delta_chunk_workspace(int64_t batch, int64_t L, int64_t H, int64_t G, int64_t dk, int64_t dv, bool packed);

constexpr float kL2Eps = 1e-6f;

}  // namespace ssm
