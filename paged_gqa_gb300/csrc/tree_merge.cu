// tree_merge.cu -- joins the pieces of split row blocks of tree attention, after the attention kernels.
//
// The causal calls let a block's last piece merge it, on the one SM that it runs on. Trees have few sequences and
// many rows: one sequence of 32,000 keys is cut into 40 and more pieces of each block, 1.4 MB of partials to
// be read through one SM, and merging took longer than attending. So tree calls leave every piece's partial in the
// workspace, and this kernel joins them row by row over all SMs:
//     M = max_i lse_i,  w_i = 2^(lse_i - M) / sum_j 2^(lse_j - M),  out = v_descale * sum_i w_i o_i
// a warp per row, a lane per eight columns, four pieces in flight, in the pieces' order. Bound by latency: a
// row's block record, its log-sums, its partials. One sequence of 32,000 keys and 8 tokens: 104 us with the merge by the
// last piece, 34 with this one; 60 tokens on 16,000 keys 266 and 39. Of 32 sequences of 33 to 60 tokens it takes 16 us cold
// (15.5 MB, 12 % of HBM), mostly behind the attention kernel's last CTAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "device_util.cuh"
#include "plan.cuh"
#include "tc_kernels.cuh"

namespace pgqa {

namespace {
constexpr int kWarps = 8;
constexpr int kAtOnce = 4, kCtasPerSm = 4;

__device__ __forceinline__ void merge_row(const Problem& p, const Pointers& ptr, const ClassPlan& cp, const RowBlock& b,
                                          int row, int lane) {
  const int ns = b.nsplit;
  const uint16_t* part = slot_o(cp, b.slot_base) + (size_t)row * kHeadDim + lane * 8;
  const size_t step = (size_t)cp.slot_rows * kHeadDim;
  uint4 h[kAtOnce];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) h[i] = __ldcg(reinterpret_cast<const uint4*>(part + min(i0 + i, ns - 1) * step));
  };
  fetch(0);  // on their way while the weights are worked out
  // the largest log-sum, then the sum: pieces by lanes, but added in the pieces' order where they are few
  auto lse_of = [&](int i) { return i < ns ? __ldcg(slot_lse(cp, b.slot_base + i) + row) : -INFINITY; };
  const float mine = lse_of(lane);
  float M = mine;
  for (int i = lane + 32; i < ns; i += 32) M = fmaxf(M, lse_of(i));
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  auto weight = [&](float lse) { return lse == -INFINITY ? 0.f : exp2f(lse - M); };
  float w = weight(mine), sum = 0.f;  // the weights of pieces 0 .. 31
  if (ns <= 32) {
    for (int i = 0; i < ns; ++i) sum += __shfl_sync(0xffffffffu, w, i);
  } else {
    for (int i = lane; i < ns; i += 32) sum += weight(lse_of(i));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float inv = sum > 0.f ? p.out_scale / sum : 0.f;
  float acc[8] = {};
  for (int i0 = 0; i0 < ns; i0 += kAtOnce) {
    if (i0 > 0) fetch(i0);
    if (i0 > 0 && (i0 & 31) == 0) w = weight(lse_of(i0 + lane));
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31) * inv;
      if (i0 + i >= ns) break;
      const uint32_t x[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 o = unpack_f16x2(x[k]);
        acc[2 * k] += wi * o.x;
        acc[2 * k + 1] += wi * o.y;
      }
    }
  }
  const RowMap m = map_row(b.row0 + row, p.G, b.kvh);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(ptr.out) + (size_t)(ptr.qsl[b.seq] + m.t) * p.o_st +
                                        (size_t)m.h * p.o_sh + lane * 8);
  *dst = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                    pack_bf16x2(acc[6], acc[7]));
}

}  // namespace

__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) tree_merge_kernel(Problem p, Pointers ptr, ClassPlan c0, ClassPlan c1,
                                                                 int classes) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long first = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int warps = gridDim.x * kWarps;
#pragma unroll 1
  for (int c = 0; c < kNumClasses; ++c) {
    if (!(classes >> c & 1)) continue;
    const ClassPlan& cp = c ? c1 : c0;
    constexpr int kVShift = 6, kPShift = 7;
    static_assert(1 << kVShift == kVerifyRows && 1 << kPShift == kPrefillRows, "rows of a block");
    const int shift = c ? kPShift : kVShift;
    const long long n = (long long)min(*cp.n_blocks, cp.max_blocks) << shift;  // (may pass 2^31)
    for (long long u = first; u < n; u += warps) {
      const RowBlock& b = cp.blocks[u >> shift];
      const int row = (int)u & ((1 << shift) - 1);
      if (b.nsplit <= 1 || row >= b.nrows) continue;
      // (the plan's own bounds: a record that is none must not lead anywhere)
      if (b.slot_base < 0 || b.slot_base + b.nsplit > cp.max_slots || b.seq < 0 || b.seq >= p.num_seqs || b.kvh < 0 || b.kvh >= p.Hkv)
        continue;
      merge_row(p, ptr, cp, b, row, lane);
    }
  }
}

cudaError_t launch_tree_merge(const Problem& p, const Pointers& ptr, const ClassPlan& c0, const ClassPlan& c1, int classes,
                              bool dependent, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(dependent, tree_merge_kernel, kCtasPerSm * c0.num_ctas, kWarps * 32, 0, stream, p, ptr, c0, c1, classes);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pgqa
