// fp4_merge.cuh -- joins the pieces of a split row of the 4-bit attention kernels.
#pragma once
#include <cstdint>

#include "device_util.cuh"
#include "tc_util.cuh"

namespace pgqa {

// acc += w times the eight f16 of h.
__device__ __forceinline__ void merge_add(float (&acc)[8], const uint4& h, float w) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 o = unpack_f16x2(hw[k]);
    acc[2 * k] += w * o.x;
    acc[2 * k + 1] += w * o.y;
  }
}

// One row of a split block by one warp: with M the largest log2-sum-exp of its pieces and
// w_i = 2^(lse_i - M), the lane's 8 columns of sum_i w_i o_i in acc; returns sum_i w_i. lse and part point at
// the row in the block's first piece, the others follow at the given pitches (elements). The lanes read
// the sums of 32 pieces at once and the partials kBatch pieces ahead (4 registers each): read one
// after the other, each costs a round trip to L2 (16384 keys of one sequence, 16 heads: 39.5 us, now 24.3).
template <int kBatch>
__device__ __forceinline__ float merge_row(const float* lse, int lse_pitch, const uint16_t* part, int part_pitch, int pieces,
                                           int lane, float (&acc)[8]) {
  const float first = lane < pieces ? __ldcg(lse + (size_t)lane * lse_pitch) : -INFINITY;
  float M = first;
  for (int i = lane + 32; i < pieces; i += 32) M = fmaxf(M, __ldcg(lse + (size_t)i * lse_pitch));
  M = tc::warp_max(M);
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float sum = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < pieces; i0 += 32) {
    const int n = min(32, pieces - i0);
    const float x = i0 == 0 ? first : lane < n ? __ldcg(lse + (size_t)(i0 + lane) * lse_pitch) : -INFINITY;
    const float w = tc::ex2(x - M);  // (0 beyond the pieces)
    sum += w;
    const uint16_t* src = part + (size_t)i0 * part_pitch + lane * 8;
#pragma unroll 1
    for (int i = 0; i < n; i += kBatch) {
      uint4 h[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        h[b] = i + b < n ? __ldcg(reinterpret_cast<const uint4*>(src + (size_t)(i + b) * part_pitch)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) merge_add(acc, h[b], __shfl_sync(0xffffffffu, w, i + b));
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

}  // namespace pgqa
