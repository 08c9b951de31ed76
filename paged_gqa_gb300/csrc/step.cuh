// step.cuh -- launch entry points of what surrounds the attention in a serving step: block tables,
// tree masks, keeping accepted tokens.
#pragma once
#include "common.cuh"

namespace pgqa {

// Most 32-bit words of a token's mask (new tokens of a sequence: 32 a word).
constexpr int kMaxMaskWords = 32;

// Most requests of a step's block tables.
constexpr int kMaxRequests = 8192;

// Block tables and slot maps (tables.cu); strides in elements.
struct TableArgs {
  const int32_t* q_lens;     // [S]
  const int32_t* ctx_lens;   // [S]
  const int32_t* rows;       // [S]
  int32_t* pages;            // [R, Wp]
  long long pages_st;
  const int32_t* counts;     // [R]
  int32_t* free_pages;       // [F]
  const int32_t* num_free;   // [1]
  int32_t* table;            // [S, W]
  long long table_st;
  int32_t* seq_lens;         // [S]
  int32_t* qsl;              // [S + 1]
  int32_t* slots;            // [T]
  int32_t* counts_out;       // [R]
  int32_t* num_free_out;     // [1]
  int S, R, Wp, F, W, T, P, p_shift;
  uint32_t* err;
};
cudaError_t launch_build_tables(const TableArgs& a, cudaStream_t stream);

// Masks and positions of token trees (tree.cu).
struct TreeMaskArgs {
  const int32_t* parents;    // [T]
  const int32_t* seq_lens;   // [S]
  const int32_t* qsl;        // [S + 1]
  int32_t* masks;            // [T, words]
  long long masks_st;
  int32_t* positions;        // [axes, T]
  long long positions_sa;
  int S, T, words, axes;
  uint32_t* err;
};
cudaError_t launch_tree_masks(const TreeMaskArgs& a, cudaStream_t stream);

// Accepted tokens' K and V into their final places (tree.cu).
struct KeepArgs {
  uint8_t* cache[2];                        // K, V
  long long sb[2], sp[2], sh[2];            // bytes
  const int32_t* bt;
  long long bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;
  const int32_t* kept;                      // [S, D]
  long long kept_st;
  const int32_t* num_kept;                  // [S]
  int32_t* lens_out;                        // [S]
  int S, Hkv, D, P, p_shift, W, NB;
  int row_bytes;                            // 256 (e4m3) or 512 (bf16)
  uint32_t* err;
};
cudaError_t launch_cache_keep(const KeepArgs& a, cudaStream_t stream);

}  // namespace pgqa
