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
  uint32_t stall_test_ns;  // failure-path test, as in Problem
  uint32_t* err;
};

// Workspace of the tcgen05 kernel: for each cluster two slots (a piece that continues a block, one that begins
// one) of both CTAs' rows, and the counters of the blocks whose first piece has the slot.
struct PromptScratch {
  float* part_o;                // [2 clusters][2][64][128][4]: columns 4 c .. 4 c + 3 of each row, normalised, fp32 (V
                                // may be beyond f16)
  float* part_lse;              // [2 clusters][2][128], log2 units
  unsigned long long* counters; // [2 clusters][2] (tag << 16) | pieces arrived (see ClassPlan::counters)
  unsigned long long* epoch;
  uint32_t call_tag;
};
// tcgen05 kernel (prompt_tc.cu) on `clusters` pairs of CTAs: 1 if launched, 0 if the strides are beyond what it
// handles, -1 on a launch error (tc_last_error()). captured: the call is being captured into a graph.
int launch_prompt_tc(const PromptArgs& a, const PromptScratch& ws, int clusters, bool captured, cudaStream_t stream);
int prompt_clusters(long long T, int num_seqs, int Hkv, int G, int sms);

// Warp-level MMA (mma.sync) kernel, a CTA per 64 rows (prompt_mma.cu).
cudaError_t launch_prompt_mma(const PromptArgs& a, cudaStream_t stream);

}  // namespace pgqa
