// prompt.cuh -- launch entry points of the attention over whole packed prompts.
#pragma once
#include "common.cuh"

namespace pgqa {

// Strides in elements; q, k, v and out are bf16 or (f16) f16.
struct PromptArgs {
  const uint16_t* q;       // [T, Hq, 256]
  const uint16_t* k;       // [T, Hkv, 256]
  const uint16_t* v;
  uint16_t* out;           // [T, Hq, 256]
  float* lse;              // [T, Hq] or null
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh, lse_st, lse_sh;
  const int32_t* qsl;      // [num_seqs + 1]
  int num_seqs, T, Hq, Hkv, G, f16;
  float score_scale_log2;  // softmax_scale * log2(e)
  uint32_t* err;
};

// Warp-level MMA (mma.sync) kernel, a CTA per 64 rows (prompt_mma.cu).
cudaError_t launch_prompt_mma(const PromptArgs& a, cudaStream_t stream);

}  // namespace pgqa
