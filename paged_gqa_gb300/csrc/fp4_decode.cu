// fp4_decode.cu -- warp-level attention kernel over a 4-bit paged KV cache (fp4.cuh), bf16 Q, for
// batches of single tokens of at most 8 heads per kv head: the verify class's blocks, 8 rows at a time.
//
// With so few rows the tcgen05 kernel (fp4_tc.cu) spends most of its instructions on handing widened
// tiles from warp to warp. Here no tile changes hands: each of the CTA's 16 warps takes every
// 16th 16-key block of the item, copies it into its own ring of shared-memory stages (one bulk copy of
// 2304 bytes each for K and V), widens it straight into the A fragments of mma.sync m16n8k16, and
// keeps its own running maxima, sums and O^T; the warps meet once per item. What bounds it is widening:
// a block takes 128 conversions, 64 permutes and 128 products in f16x2, of which the first two
// share a pipe at 2.07 cycles a warp instruction (measured): ~1000 cycles per 128 keys and SM, below the
// ~1600 that those keys take to arrive from HBM; ~2250 are measured, the rest waiting (four warps
// per scheduler hide only part of the chain load, convert, multiply, MMA).
// Time (graph replays, 8 heads): 14.5 us for one sequence of 600 keys, 36.2 for 32 of 9000 (12.2 at the
// HBM rate), 150 for 256 of 8192 (89). The tcgen05 kernel: 17.0, 43.7, 189. With 8 warps of twice the registers
// this kernel took twice as long per key; with 16 rows a pass (12 warps, O^T of 128 registers, spills) 65 us
// against the tcgen05 kernel's 44 at 32 x 9000 keys, so groups of more than 8 heads go there.
//
//   S^T[16 keys, rows] = K Q^T    A = K: lane (g, t) = (lane / 4, lane % 4) holds fragment rows g and
//       g + 8 and widens 32 code bytes of each of those two keys: k-step s takes bytes 32t + 2s, 2s + 1, so
//       the four lanes of a row share its d evenly and Q's fragments are laid out to match.
//   O^T[256 d, rows] += V^T P^T   A = V^T: fragment m covers code bytes 8m + g (d = 2 byte in row g,
//       2 byte + 1 in row g + 8); one word of a V block is 4 tokens of a byte, and makes a whole
//       fragment when the block's tokens are ordered 4t, 4t + 1 | 4t + 2, 4t + 3 along k. K's fragment
//       rows take the same order, so P^T only needs its 8 x 8 blocks transposed (movmatrix).
// Everything is exact as in fp4_tc.cu: widened values in f16, Q in f16 with a power of two per row,
// P = 2^(s - m + 4) rounded to f16 and a split piece's O (2^-11 each, the output's rounding is 2^-8), fp32 sums. A warp's reference m moves when one of its scores
// exceeds it by more than 2^4.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdio>

#include "common.cuh"
#include "device_util.cuh"
#include "fp4.cuh"
#include "fp4_merge.cuh"
#include "self_plan.cuh"
#include "tc_kernels.cuh"
#include "tc_util.cuh"

namespace pgqa {

namespace {

using namespace tc;

constexpr uint32_t kDStage = 2 * kFp4BlockBytes;  // a 16-key block of K, then of V
constexpr int kDRows = 8;                         // rows of a pass
constexpr float kDTau = 4.f, kDSigma = 4.f, kDMInit = -3.0e38f;
// A staged Q row: its 16-byte chunk (t, j) of d 64 t + 8 j .. + 7 at 64 j + 16 t, so that the four lanes of
// a fragment row read 64 contiguous bytes; the pitch puts the next row in the other 16 banks.
constexpr uint32_t kQPitch = kHeadDim * 2 + 64;

// Two stages: a warp's next block is in flight while it works on one (16 x 2 x 4608 bytes in all).
constexpr int kDWarps = 16, kDThreads = kDWarps * 32, kDStages = 2;
constexpr uint32_t kOffQ = kDWarps * kDStages * kDStage;
constexpr uint32_t kOffMisc = kOffQ + kDRows * kQPitch;
static_assert(kDWarps * 16 * 32 * sizeof(float4) <= kOffQ, "the warps' O^T meets in the stages");
static_assert(sizeof(self_plan::Scratch) <= kOffQ, "the self-plan scratch fits the stages");

template <bool kFused>
struct DMisc {
  alignas(16) float m[kDWarps][kDRows];
  alignas(16) float l[kDWarps][kDRows];
  alignas(16) float cs[kDRows];
  alignas(16) int lim[kDRows];
  alignas(16) long long out_off[kDRows];
  alignas(8) uint64_t full[kDWarps][kDStages];
  uint64_t never;
  int abort_flag, merge_flag, fcount;
  int4 fitem[kFused ? kFusedMaxBlocks : 1];
  int4 fseq[kFused ? kFusedMaxBlocks : 1];
};

struct DItem {
  int block, seq, kvh, nrows, nsplit, split, slot_base, key0, kv_hi, q0, qn, L;
};

template <bool kFused>
__device__ __forceinline__ DItem load_ditem(const Problem& p, const ClassPlan& cp, const Pointers& ptr,
                                            const DMisc<kFused>& ms, int it) {
  DItem r;
  if (kFused) {
    const self_plan::Piece f = self_plan::unpack(p, ms.fitem[it]);
    const int4 sq = ms.fseq[it];
    r.block = f.block;
    r.seq = f.seq;
    r.kvh = f.kvh;
    r.nsplit = f.nsplit;
    r.split = f.split;
    r.slot_base = f.slot_base;
    r.q0 = sq.x;
    r.qn = sq.y;
    r.L = sq.z;
    r.nrows = r.qn * p.G;
    r.key0 = f.tile_begin * kTileKeys;
    r.kv_hi = min((f.tile_begin + f.ntiles) * kTileKeys, r.L);
  } else {
    const WorkItem w = cp.items[it];
    const RowBlock b = cp.blocks[w.block];
    r.block = w.block;
    r.seq = b.seq;
    r.kvh = b.kvh;
    r.nrows = b.nrows;
    r.nsplit = b.nsplit;
    r.split = w.split;
    r.slot_base = b.slot_base;
    r.key0 = w.tile_begin * kTileKeys;
    r.kv_hi = min(w.tile_end * kTileKeys, b.kv_end);
    r.q0 = ptr.qsl[b.seq];
    r.qn = ptr.qsl[b.seq + 1] - r.q0;
    r.L = ptr.seq_lens[b.seq];
  }
  return r;
}

__device__ __forceinline__ void mma_f16_sync(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

}  // namespace

template <bool kFused>
__global__ void __launch_bounds__(kDThreads, 1) fp4_decode_kernel(Problem p, Pointers ptr, ClassPlan cp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  DMisc<kFused>& ms = *reinterpret_cast<DMisc<kFused>*>(smem + kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = &ms.abort_flag;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int item_begin = 0, item_end = 0;
  if (kFused) {
    self_plan::Scratch& fs = *reinterpret_cast<self_plan::Scratch*>(smem);
    self_plan::load(p, ptr, fs);
    if (p.unplanned && blockIdx.x == 0) self_plan::flag_invalid(p, ptr, fs);
    __syncthreads();
    if (warp == 1) self_plan::plan_warp(p, fs, cp.num_ctas, lane, ms.fitem, ms.fseq, &ms.fcount);
  } else {
    item_begin = cp.cta_item_begin[blockIdx.x];
    item_end = cp.cta_item_begin[blockIdx.x + 1];
  }
  if (threadIdx.x == 0) {
    for (int w = 0; w < kDWarps; ++w)
      for (int s = 0; s < kDStages; ++s) mbar_init(smem_u32(&ms.full[w][s]), 1);
    mbar_init(smem_u32(&ms.never), 1);
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  fence_proxy_async_smem();  // the plan's scratch lies where the copies go
  __syncthreads();
  if (kFused) item_end = ms.fcount;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Failure-path test: a bounded wait on a barrier nothing arrives on; no copy is in flight yet.
  if (p.stall_test_ns && !mbar_wait(smem_u32(&ms.never), 0, abort_flag, ptr.err, p.stall_test_ns)) return;

  uint8_t* ring = smem + warp * kDStages * kDStage;
  const uint32_t full0 = smem_u32(&ms.full[warp][0]);
  const uint64_t policy = policy_evict_first();
  const unsigned long long ctag = threadIdx.x == 0 ? split_tag(p, cp) : 0ull;
  uint32_t used = 0;  // stages this warp has filled so far: stage used % kDStages is next
  const int tok0 = 4 * (g >> 1) + (g & 1);  // token of K's fragment row g; row g + 8 has tok0 + 2

  for (int it = item_begin; it < item_end; ++it) {
    const DItem I = load_ditem<kFused>(p, cp, ptr, ms, it);
    const int nblk = (I.kv_hi - I.key0 + kFp4Block - 1) / kFp4Block;  // 16-key blocks of the piece
    const int mine = nblk > warp ? (nblk - warp + kDWarps - 1) / kDWarps : 0;
    const int32_t* bt_row = ptr.block_table + (size_t)I.seq * p.bt_stride;
    const uint8_t* khead = static_cast<const uint8_t*>(ptr.k) + (long long)I.kvh * p.k_sh;
    const uint8_t* vhead = static_cast<const uint8_t*>(ptr.v) + (long long)I.kvh * p.v_sh;
    for (int row0 = 0; row0 < I.nrows; row0 += kDRows) {
      const int rows = min(kDRows, I.nrows - row0);
      // ---- copies: this warp's i-th block of the piece goes to stage (used + i) % kDStages. Lane
      // (i % 32) holds its page, the next 32 are read when these run out.
      int page = -1, window = -1;
      auto issue = [&](int i) {
        if (i / 32 != window) {
          window = i / 32;
          const int key = I.key0 + ((window * 32 + lane) * kDWarps + warp) * kFp4Block;
          page = key < I.kv_hi ? bt_row[key / p.P] : 0;
          if (page < 0 || page >= p.NB) {
            atomicOr(ptr.err, kErrPage);
            page = 0;
          }
        }
        const int pg = __shfl_sync(0xffffffffu, page, i & 31);
        if (lane == 0) {
          const uint32_t st = (used + i) % kDStages, b = full0 + 8 * st;
          const int key = I.key0 + (i * kDWarps + warp) * kFp4Block;
          const long long in = (long long)(key % p.P) * kFp4Row;
          const uint32_t dst = smem_u32(ring) + st * kDStage;
          mbar_expect_tx(b, kDStage);
          bulk_load_hint(dst, khead + (long long)pg * p.k_sb + in, kFp4BlockBytes, b, policy);
          bulk_load_hint(dst + kFp4BlockBytes, vhead + (long long)pg * p.v_sb + in, kFp4BlockBytes, b, policy);
        }
        __syncwarp();
      };
      for (int i = 0; i < min(mine, kDStages); ++i) issue(i);

      // ---- Q rows to shared memory in f16, each times a power of two (to [2^14, 2^15))
      for (int r = warp; r < kDRows; r += kDWarps) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const RowMap m = map_row(row0 + r, p.G, I.kvh);
        if (r < rows)
          v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(ptr.q) + (long long)(I.q0 + m.t) * p.q_st +
                                              (long long)m.h * p.q_sh + lane * 8);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
        const int e = max((int)(top >> 7), 14);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
        *reinterpret_cast<uint4*>(smem + kOffQ + r * kQPitch + (lane & 7) * 64 + (lane >> 3) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) {
          ms.cs[r] = p.score_scale_log2 * __uint_as_float(e > 14 ? (uint32_t)(e - 14) << 23 : 0x00400000u);
          ms.lim[r] = r < rows ? I.L - I.qn + m.t : -1;
          ms.out_off[r] = r < rows ? (long long)(I.q0 + m.t) * p.o_st + (long long)m.h * p.o_sh : 0;
        }
      }
      __syncthreads();

      // ---- this lane's rows 2t, 2t + 1
      float c[2], ref[2], sum[2];
      int lim[2];
      const int min_lim = I.L - I.qn + map_row(row0, p.G, I.kvh).t;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        c[b] = ms.cs[2 * t + b];
        lim[b] = ms.lim[2 * t + b];
        ref[b] = 2 * t + b < rows ? kDMInit : 0.f;  // padding rows never ask for a new one
        sum[b] = 0.f;
      }
      float o[16][4];
#pragma unroll
      for (int m = 0; m < 16; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;

#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        const uint32_t st = (used + i) % kDStages;
        // (a drain: the copy is this warp's own and lands whatever happened elsewhere)
        mbar_drain(full0 + 8 * st, ((used + i) / kDStages) & 1, abort_flag, ptr.err);
        __syncwarp();
        const uint8_t* kb = ring + st * kDStage;
        const uint8_t* vb = kb + kFp4BlockBytes;
        const int key0 = I.key0 + (i * kDWarps + warp) * kFp4Block;
        // S^T = K Q^T
        float s[4], s1[4];  // two chains of products, added up after
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = s1[e] = 0.f;
        const uint32_t sc0 = *reinterpret_cast<const uint32_t*>(kb + tok0 * kFp4Row + kFp4Codes + 4 * t);
        const uint32_t sc1 = *reinterpret_cast<const uint32_t*>(kb + (tok0 + 2) * kFp4Row + kFp4Codes + 4 * t);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 16 of this lane's code bytes: 8 k-steps
          const uint4 x0 = *reinterpret_cast<const uint4*>(kb + tok0 * kFp4Row + 32 * t + 16 * h);
          const uint4 x1 = *reinterpret_cast<const uint4*>(kb + (tok0 + 2) * kFp4Row + 32 * t + 16 * h);
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
          const uint32_t f0 = fp4::scales2(h ? sc0 >> 16 : sc0), f1 = fp4::scales2(h ? sc1 >> 16 : sc1);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // a word of codes: two k-steps
            uint32_t h0[4], h1[4];
            fp4::codes4(w0[k], h0);
            fp4::codes4(w1[k], h1);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              h0[b] = k < 2 ? fp4::mul_f16x2_lo(h0[b], f0) : fp4::mul_f16x2_hi(h0[b], f0);
              h1[b] = k < 2 ? fp4::mul_f16x2_lo(h1[b], f1) : fp4::mul_f16x2_hi(h1[b], f1);
            }
            const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
            // d = 64 t + 32 h + 8 k + 0 .. 7 of row g
            const uint4 q = *reinterpret_cast<const uint4*>(smem + kOffQ + g * kQPitch + (4 * h + k) * 64 + t * 16);
            mma_f16_sync(s, a0, q.x, q.y);
            mma_f16_sync(s1, a1, q.z, q.w);
          }
        }
        // x = s c - m + sigma; keys of this lane: tok0 (s[0], s[1]) and tok0 + 2
        const int ka = key0 + tok0, kc = ka + 2;
        const bool need_mask = key0 + kFp4Block > I.kv_hi || key0 + kFp4Block - 1 > min_lim;
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // rounded before anything is taken from it, as the references are: fused with that, a score of
          // 2^30 would be off from its own maximum by up to 64
          s[b] = __fmul_rn(s[b] + s1[b], c[b]);
          s[2 + b] = __fmul_rn(s[2 + b] + s1[2 + b], c[b]);
          if (need_mask) {
            if (ka >= I.kv_hi || ka > lim[b]) s[b] = -INFINITY;
            if (kc >= I.kv_hi || kc > lim[b]) s[2 + b] = -INFINITY;
          }
          top = max3f(top, s[b] - ref[b], s[2 + b] - ref[b]);
        }
        if (__any_sync(0xffffffffu, top > kDTau)) {
          // new references: the exact maxima of this block's scores
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float mx = fmaxf(s[b], s[2 + b]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(ref[b], mx);
            const float alpha = ex2(ref[b] - mn);
            ref[b] = mn;
            sum[b] *= alpha;
#pragma unroll
            for (int m = 0; m < 16; ++m) {
              o[m][b] *= alpha;
              o[m][2 + b] *= alpha;
            }
          }
        }
        uint32_t pb[2];
        float e[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          e[b] = ex2(s[b] - ref[b & 1] + kDSigma);
          sum[b & 1] += e[b];
        }
        pb[0] = transpose8(pack_f16x2(e[0], e[1]));
        pb[1] = transpose8(pack_f16x2(e[2], e[3]));
        // O^T += V^T P^T; tokens past the piece's end (stale slots) get zero scales
        const uint32_t live = 4 * t + 4 <= I.kv_hi - key0 ? 0xffffffffu
                              : 4 * t >= I.kv_hi - key0   ? 0u
                                                          : (1u << (8 * (I.kv_hi - key0 - 4 * t))) - 1u;
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(vb + (8 * m + g) * kFp4Block + 4 * t);
          const uint32_t sw = *reinterpret_cast<const uint32_t*>(vb + kFp4BlockScales + m * kFp4Block + 4 * t) & live;
          uint32_t h[4];
          fp4::codes4(w, h);
          const uint32_t s01 = fp4::scales2(sw), s23 = fp4::scales2(sw >> 16);
          const uint32_t a[4] = {fp4::mul_f16x2(__byte_perm(h[0], h[1], 0x5410), s01),
                                 fp4::mul_f16x2(__byte_perm(h[0], h[1], 0x7632), s01),
                                 fp4::mul_f16x2(__byte_perm(h[2], h[3], 0x5410), s23),
                                 fp4::mul_f16x2(__byte_perm(h[2], h[3], 0x7632), s23)};
          mma_f16_sync(o[m], a, pb[0], pb[1]);
        }
        __syncwarp();  // every lane has read the stage
        if (i + kDStages < mine) issue(i + kDStages);
      }
      used += mine;

      // ---- the warps meet: references, sums, O^T
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float l = sum[b];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (g == 0) {
          ms.m[warp][2 * t + b] = ref[b];
          ms.l[warp][2 * t + b] = l;
        }
      }
      __syncthreads();  // (also: every warp's stages are consumed)
      const bool split = I.nsplit > 1;
      const int slot = I.slot_base + I.split;
      float mine_w[2], inv[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = 2 * t + b;
        float M = kDMInit, L = 0.f;
#pragma unroll
        for (int w = 0; w < kDWarps; ++w) M = fmaxf(M, ms.m[w][r]);
#pragma unroll
        for (int w = 0; w < kDWarps; ++w) L += ms.l[w][r] * ex2(ms.m[w][r] - M);
        mine_w[b] = ex2(ref[b] - M);
        inv[b] = L > 0.f ? __fdividef(split ? 1.f : p.out_scale, L) : L == 0.f ? 0.f : L;  // NaN stays
        if (split && warp == 0 && g == 0) {
          const float lse = L > 0.f ? M - kDSigma + log2f(L) : L == 0.f ? -INFINITY : L;
          if (r < rows) slot_lse(cp, slot)[row0 + r] = lse;
        }
      }
      // Through shared memory: warp m adds up fragment m of all warps.
      static_assert(kDWarps == 16, "a warp to each fragment of O^T");
      float4* meet = reinterpret_cast<float4*>(smem) + lane;  // [warp][fragment][32 lanes]
#pragma unroll
      for (int m = 0; m < 16; ++m)
        meet[(warp * 16 + m) * 32] =
            make_float4(o[m][0] * mine_w[0], o[m][1] * mine_w[1], o[m][2] * mine_w[0], o[m][3] * mine_w[1]);
      __syncthreads();
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDWarps; ++w) {
        const float4 x = meet[(w * 16 + warp) * 32];
        acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
      }
      const int byte = 8 * warp + g;  // d = 2 byte (acc[0], acc[1]) and 2 byte + 1
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = 2 * t + b;
        if (r < rows) {
          if (split)
            reinterpret_cast<uint32_t*>(slot_o(cp, slot))[(row0 + r) * (kHeadDim / 2) + byte] =
                pack_f16x2(acc[b] * inv[b], acc[2 + b] * inv[b]);
          else
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(ptr.out) + ms.out_off[r] + 2 * byte) =
                pack_bf16x2(acc[b] * inv[b], acc[2 + b] * inv[b]);
        }
      }
      fence_proxy_async_smem();  // the stages were written by these threads: the next copies come after
      __syncthreads();
    }
    if (I.nsplit > 1) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        fence_acq_rel_gpu();
        ms.merge_flag = split_arrive(cp.counters + I.block, I.nsplit, ctag);
        fence_acq_rel_gpu();
      }
      __syncthreads();
      if (ms.merge_flag) {
        // The block's last piece joins all of them. A warp takes whole rows, 16 bytes a lane.
        __threadfence();
        const float* lse = slot_lse(cp, I.slot_base);
        const uint16_t* part = slot_o(cp, I.slot_base);
        for (int r = warp; r < I.nrows; r += kDWarps) {
          float acc[8];
          const float k = p.out_scale /
                          merge_row<8>(lse + r, kVerifyRows, part + r * kHeadDim, kVerifyRows * kHeadDim, I.nsplit, lane, acc);
          const RowMap m = map_row(r, p.G, I.kvh);
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(ptr.out) + (long long)(I.q0 + m.t) * p.o_st +
                                    (long long)m.h * p.o_sh + lane * 8) =
              make_uint4(pack_bf16x2(acc[0] * k, acc[1] * k), pack_bf16x2(acc[2] * k, acc[3] * k),
                         pack_bf16x2(acc[4] * k, acc[5] * k), pack_bf16x2(acc[6] * k, acc[7] * k));
        }
      }
      __syncthreads();  // merge_flag is used again
    }
  }
}

namespace {

template <bool kFused>
int launch(const Problem& p, const Pointers& ptr, const ClassPlan& cp, cudaStream_t stream) {
  auto kern = fp4_decode_kernel<kFused>;
  constexpr size_t smem = kOffMisc + sizeof(DMisc<kFused>) + 128;
  static_assert(smem <= 232448, "shared memory of one CTA");
  static bool done[64] = {};  // one per instance of this template
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  if (e == cudaSuccess) e = launch_pdl(false, kern, cp.num_ctas, kDThreads, smem, stream, p, ptr, cp);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    char buf[160];
    snprintf(buf, sizeof buf, "4-bit decode kernel launch: %s", cudaGetErrorString(e));
    set_tc_error(buf);
    return -1;
  }
  return 1;
}

}  // namespace

int launch_fp4_decode(const Problem& p, const Pointers& ptr, const ClassPlan& cp, cudaStream_t stream) {
  return p.fused_verify ? launch<true>(p, ptr, cp, stream) : launch<false>(p, ptr, cp, stream);
}

}  // namespace pgqa
