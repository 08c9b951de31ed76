// prompt_mma.cu -- causal attention over whole packed prompts in its simplest form: warp-level
// mma.sync, one CTA per 64 rows (row r of a prompt and kv head: token r / G, head r % G), every
// block by itself. It serves calls whose strides no tensor map can say (a token or head stride of q, k or v
// that is not positive, or of 2^38 elements and more; tokens that share their K, for example), and runs under
// paged_gqa_set_path(1), where the tests compare the tcgen05 kernel with it.
//
// A warp holds 16 rows: their Q as MMA fragments (64 registers), their O in fp32 (128). K and V
// come 32 keys at a time into shared memory; S = Q K^T, the running maximum and sum of the
// softmax in fp32, P rounded to the inputs' type, O += P V. The accumulator layout of S is the
// A operand's layout of P V, so P stays in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "device_util.cuh"
#include "prompt.cuh"

namespace pgqa {

namespace {

constexpr int kRowsOf = 64, kKeys = 32, kWarps = 4, kThreads = kWarps * 32;
constexpr int kPitch = kHeadDim + 8;  // elements: rows 16 bytes apart modulo 128, no bank conflicts

template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  return kF16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

}  // namespace

template <bool kF16>
__global__ void __launch_bounds__(kThreads) prompt_mma_kernel(PromptArgs a) {
  __shared__ __align__(16) uint16_t ks[kKeys * kPitch];
  __shared__ __align__(16) uint16_t vs[kKeys * kPitch];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int kvh = blockIdx.y;
  // the sequence that holds row block blockIdx.x of this kv head; the first CTA goes through all of them, to flag bad ones
  const bool flags = blockIdx.x == 0 && kvh == 0;
  int seq = -1, block = 0, q0 = 0, qn = 0;
  long long pre = 0;
  for (int s0 = 0; s0 < a.num_seqs && (seq < 0 || flags); s0 += 32) {
    const int s = s0 + lane;
    int start = 0, n = 0;
    if (s < a.num_seqs) {
      start = a.qsl[s];
      const int end = a.qsl[s + 1];
      n = end - start;
      if (start < 0 || end < start || end > a.T) {
        if (flags && warp == 0) atomicOr(a.err, kErrBounds);
        n = 0;
      }
    }
    const int blocks = (int)(((long long)n * a.G + kRowsOf - 1) / kRowsOf);
    int x = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const bool mine = blockIdx.x >= pre + x - blocks && blockIdx.x < pre + x;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int j = __ffs(who) - 1;
      seq = s0 + j;
      block = __shfl_sync(0xffffffffu, (int)(blockIdx.x - (pre + x - blocks)), j);
      q0 = __shfl_sync(0xffffffffu, start, j);
      qn = __shfl_sync(0xffffffffu, n, j);
    }
    pre += __shfl_sync(0xffffffffu, x, 31);
  }
  if (seq < 0) return;
  const int row0 = block * kRowsOf, rows = qn * a.G;  // (blocks of a prompt cover its rows: below 2^31)
  const int end = min(row0 + kRowsOf - 1, rows - 1) / a.G + 1;  // keys [0, end) are seen by the block
  int tok[2], head[2];
  bool real[2];
  uint32_t qf[kHeadDim / 16][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + warp * 16 + g + 8 * i;
    real[i] = r < rows;
    tok[i] = real[i] ? r / a.G : -1;
    head[i] = kvh * a.G + (real[i] ? r - tok[i] * a.G : 0);
    const uint16_t* q = a.q + (long long)(q0 + (real[i] ? tok[i] : 0)) * a.q_st + (long long)head[i] * a.q_sh + 2 * tq;
#pragma unroll
    for (int kk = 0; kk < kHeadDim / 16; ++kk) {
      qf[kk][i] = real[i] ? *reinterpret_cast<const uint32_t*>(q + kk * 16) : 0u;
      qf[kk][i + 2] = real[i] ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 8) : 0u;
    }
  }
  float o[kHeadDim / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int k0 = 0; k0 < end; k0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * kHeadDim / 8; i += kThreads) {
      const int key = i / (kHeadDim / 8), d = i % (kHeadDim / 8) * 8;
      uint4 k = make_uint4(0, 0, 0, 0), v = k;  // keys past the block's: their V must not be NaN
      if (k0 + key < end) {
        const long long t = q0 + k0 + key;
        k = *reinterpret_cast<const uint4*>(a.k + t * a.k_st + kvh * a.k_sh + d);
        v = *reinterpret_cast<const uint4*>(a.v + t * a.v_st + kvh * a.v_sh + d);
      }
      *reinterpret_cast<uint4*>(ks + key * kPitch + d) = k;
      *reinterpret_cast<uint4*>(vs + key * kPitch + d) = v;
    }
    __syncthreads();
    float s[kKeys / 8][4] = {};
#pragma unroll
    for (int kk = 0; kk < kHeadDim / 16; ++kk)
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n) {
        const uint16_t* b = ks + (n * 8 + g) * kPitch + kk * 16 + 2 * tq;
        mma16<kF16>(s[n], qf[kk], *reinterpret_cast<const uint32_t*>(b), *reinterpret_cast<const uint32_t*>(b + 8));
      }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = k0 + n * 8 + 2 * tq + (e & 1);
        s[n][e] = key <= tok[e >> 1] ? s[n][e] * a.score_scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
      mx[i] = fmaxf(m[i], fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2)));
      const float alpha = mx[i] == -INFINITY ? 1.f : exp2f(m[i] - mx[i]);
      m[i] = mx[i];
      l[i] *= alpha;
#pragma unroll
      for (int d = 0; d < kHeadDim / 8; ++d) {
        o[d][2 * i] *= alpha;
        o[d][2 * i + 1] *= alpha;
      }
    }
    uint32_t pf[kKeys / 16][4];
#pragma unroll
    for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = m[i] == -INFINITY ? 0.f : m[i];
        const float x = exp2f(s[n][2 * i] - ref), y = exp2f(s[n][2 * i + 1] - ref);
        l[i] += x + y;
        pf[n >> 1][(n & 1) * 2 + i] = pack<kF16>(x, y);
      }
#pragma unroll
    for (int kk = 0; kk < kKeys / 16; ++kk)
#pragma unroll
      for (int d = 0; d < kHeadDim / 16; ++d) {
        // V's 16 x 16 block, transposed by the load: two B operands of 8 columns each
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(vs + (kk * 16 + (lane & 15)) * kPitch + d * 16 + (lane >> 4) * 8);
        uint32_t b[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(at)
                     : "memory");
        mma16<kF16>(o[2 * d], pf[kk], b[0], b[1]);
        mma16<kF16>(o[2 * d + 1], pf[kk], b[2], b[3]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (!real[i]) continue;
    const float inv = 1.f / l[i];  // a token sees itself: l > 0
    uint16_t* dst = a.out + (long long)(q0 + tok[i]) * a.o_st + (long long)head[i] * a.o_sh + 2 * tq;
#pragma unroll
    for (int d = 0; d < kHeadDim / 8; ++d)
      *reinterpret_cast<uint32_t*>(dst + d * 8) = pack<kF16>(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
    if (a.lse && tq == 0)
      a.lse[(long long)(q0 + tok[i]) * a.lse_st + (long long)head[i] * a.lse_sh] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
  }
}

cudaError_t launch_prompt_mma(const PromptArgs& a, cudaStream_t stream) {
  const long long blocks = ((long long)a.T * a.G + kRowsOf - 1) / kRowsOf + a.num_seqs;
  const dim3 grid((unsigned)blocks, (unsigned)a.Hkv);
  if (a.f16) prompt_mma_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else prompt_mma_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pgqa
