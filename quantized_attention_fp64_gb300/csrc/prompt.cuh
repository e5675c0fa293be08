// What the operators on prompts share: arguments, checked on the host.
#pragma once

#include "common.cuh"

namespace sage {

struct RotaryArgs {
  Bf16In q, k;
  Out q_out, k_out;
  int64_t B, T;
  int32_t H, Hkv;
  int32_t pairs;             // rotary_dim / 2, a multiple of 8
  const uint64_t* turns;     // [pairs] turns of a position, in 2^-64
  const int32_t* positions;
  int64_t pos_b, pos_t;
  float magnitude;
  bool interleaved, inverse;
};
cudaError_t launch_rotary(const RotaryArgs& a, int64_t D, cudaStream_t stream);

struct PromptArgs {
  Bf16In q, k, v;            // (rows, heads, D): sb is not used
  Out out;
  int64_t N, M;              // rows of q and out, of k and v
  int32_t H, Hkv, B;
  const int32_t* offsets;    // [B + 1]
  const int32_t* kv_offsets; // [B + 1]
  float* lse;                // [H][N] or null
  void* workspace;
  bool causal, zero_rest;
  float sm_log2;             // sm_scale * log2(e)
  int* dev_err;
};
cudaError_t launch_prompt_attention(const PromptArgs& a, int64_t D, cudaStream_t stream);
size_t prompt_attention_workspace_bytes(int64_t N, int64_t M, int64_t H, int64_t Hkv, int64_t D, int64_t B);

}  // namespace sage
