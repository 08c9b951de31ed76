// prompt_tc.cu -- tcgen05 (TMEM, TMA) kernel of causal attention over whole packed prompts.
//
// The formula: out = softmax(scale q K^T + causal) V per (token, head), head_dim 256, grouped heads;
// 4 * 256 flops per visible (row, key) pair, K and V re-read from L2 by every block of rows. It is bound by
// the matrix products, and next by L2: 128 rows against 1024 bytes of K and V per key are 128 flops a byte,
// which at 2 PFLOP/s would be 16 TB/s. So two SMs share a block:
//
//   * a cluster of two CTAs (cta_group::2) serves 256 rows of a prompt and kv head. A CTA holds 128 / G tokens,
//     row t * G + g of its half being token t, head g (one TMA box per 128-byte d-quarter of Q). Each CTA
//     loads half of every tile of 128 keys: 64 keys of K, half of d of V; the instruction reads both
//     halves. That halves the bytes from L2 and the shared memory a tile takes (Q 64 KB, two stages of K
//     and of V of 32 KB each per CTA);
//   * S = Q K^T: M = 256, N = 128, 16 instructions of K = 16 per tile; O += P V: M = 256, N = 256, 8
//     instructions, P (the inputs' type) from TMEM. S takes 128 columns, P two buffers of 64, O 256: all 512;
//   * S(g + 1) is issued once the softmax has loaded S(g), and P(g) is written once P.V(g - 2) is done, so the
//     tensor pipe always has the next product queued: a tile's softmax (8 warps, two threads per
//     row) has the time of two products;
//   * online softmax, fp32, one row per TMEM lane; the reference of a row moves, and its O is rescaled, only
//     when a score exceeds it by 2^8;
//   * the even CTA issues the products. The odd CTA's copies complete on its barriers, the
//     softmax warps of both arrive on them, and its commits arrive in both CTAs;
//   * an item's epilogue has a warpgroup of its own, O leaves TMEM at once (part to the stage, part to registers), and
//     the next item's first S is issued before this one's last P.V, so items follow each other without a gap;
//   * the work is cut into equal ranges over the clusters, worked out by each CTA for itself: block b of a
//     prompt costs a fixed part and (b + 1) tokens' worth of keys, a closed form whose prefix sums need no pass
//     over blocks. A block cut across clusters is merged by its last piece (fp32 partials, counters
//     tagged per call).
//
// Measured (GB300, bf16, back to back, L2 warm): 16384 tokens, 16/2 heads 1100 us, 2000 TFLOP/s of visible pairs (a
// cuBLAS bf16 product in a burst: 1930; under a power cap held for seconds 1250 us); 8192 tokens, 8/1 164 us, 1670;
// 2048 tokens 33; 173 tokens 17 (latency: set-up 5, one item's chain of cold steps). Under ncu the tensor pipe is
// busy 78 % of the cycles at 8192 tokens, DRAM 4 %, L2 hits 88 %. The other 22 % are the ends of ranges (tiles
// on the diagonal, of which half is masked) and the softmax where it takes longer than two products.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdio>
#include <type_traits>

#include "common.cuh"
#include "device_util.cuh"
#include "prompt.cuh"
#include "tc_kernels.cuh"
#include "tc_util.cuh"

namespace pgqa {

namespace {

using namespace tc;

constexpr int kRows = 128;                   // rows of a CTA
constexpr int kKeys = 128;                   // keys of a tile
// Warps 0-3: K and V copies, items and Q, products or (odd CTA) tails; 4-11: softmax; 12-15: epilogue. The kernel starts with
// 128 registers a thread, which the warpgroups then share out among themselves (setmaxnreg).
constexpr int kSoftWarp0 = 4, kSoftWarps = 8, kSoftThreads = kSoftWarps * 32;
constexpr int kEpiWarp0 = kSoftWarp0 + kSoftWarps, kEpiWarps = 4, kEpiThreads = kEpiWarps * 32;
constexpr int kThreads = kEpiWarp0 * 32 + kEpiThreads;
constexpr int kLaunchRegs = 128, kSoftRegs = 144, kEpiRegs = 160, kOtherRegs = 64;
static_assert(kThreads * kLaunchRegs == 65536 && 256 * kSoftRegs + 128 * kEpiRegs + 128 * kOtherRegs == 65536, "register split");
constexpr int kStages = 2;                   // of K, and of V
constexpr int kRing = 3;                     // items known at a time: one in its epilogue, one at work, the next
constexpr float kTau = 8.f;                  // a row's reference moves when a score exceeds it by this (log2)
constexpr float kMInit = -3.0e38f;          // reference of a row before its first key

constexpr uint32_t kQQuarter = kRows * 128;  // [128 rows][64 d]
constexpr uint32_t kKQuarter = 64 * 128;     // [64 keys][64 d], four of them
constexpr uint32_t kVQuarter = kKeys * 128;  // [128 keys][64 d], two of them
constexpr uint32_t kTile = 32768;            // a CTA's half of a tile of K or V
constexpr uint32_t kOffQ = 0, kOffK = 4 * kQQuarter, kOffV = kOffK + kStages * kTile, kOffMisc = kOffV + kStages * kTile;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColP = 128, kPBufCols = 64, kColO = 256;

// The cut, in keys: what a block costs a cluster beyond its keys (Q, first and last softmax), and the least of a
// range. A piece has at least kMinPiece tiles: writing and merging partials costs a cluster about what six tiles do.
// There are as many ranges as blocks where those are small.
constexpr int kFixed = 384, kMinPiece = 8, kMinRange = kFixed + kMinPiece * kKeys;

struct Item {
  int q0, n;             // first token of the prompt, its length
  int tok0;              // the block's first token in the prompt
  int kvh, kv_end;       // keys [0, kv_end) are seen by the block's last token
  int t0, t1;            // tiles of this piece
  int split, nsplit;
  int slot, slot0, slot1;  // partial slots: this piece's, the first piece's, the second's (the others follow it by 2)
};

struct Misc {
  alignas(16) float red[2][2][kRows];  // [tile parity][key half][row] partial maxima
  alignas(16) float stat_l[kRing][2][kRows];  // a finished item's row sums (of each key half) and references
  alignas(16) float stat_m[kRing][kRows];
  alignas(16) Item item[kRing];
  alignas(8) uint64_t item_full[kRing], item_empty[kRing], stat_full[kRing];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full, q_empty, s_full, s_free, p_full[2][2], pv_done[2], o_ready, o_free, drain, never;
  // A piece's last tile where it passes the block's keys, of stage g % kStages. Odd CTA: V has landed; even CTA: and its
  // tail is zeroed.
  uint64_t tail_v[kStages], tail_full[kStages];
  long long scan[2][kThreads / 32];  // units, blocks
  long long start_off;   // units before the prompt the range starts in
  int start_seq;
  uint32_t tmem_base;
  int abort_flag, merge_flag;
};
// The epilogue's stage: 96 columns of each row, rows 13 chunks of 16 bytes apart (an odd number: no bank conflicts).
constexpr int kStageCols = 96, kStagePitch = 208;
constexpr uint32_t kOffStage = kOffMisc + (uint32_t)((sizeof(Misc) + 127) / 128 * 128);
constexpr size_t kSmemBytes = kOffStage + kRows * kStagePitch + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// ------------------------------------------------------------------ cluster-wide instructions --
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// The address of a shared variable of the cluster's CTA 0.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// The order between the CTAs of a pair. P, S and O lie in TMEM: the tcgen05 fences on both sides of a relaxed arrival
// order them. The odd CTA's copies of Q, K and V complete on the leader's barriers themselves (.cta_group::2). What
// threads write, the zeros of a tail, takes a release and an acquire at cluster scope; a release costs its thread 1040 cycles
// (an acquire next to nothing), so the odd CTA's warp 3, which has nothing else to do, writes them and releases early. (As
// releases of the softmax warps they cost a call 2-5 %; a relay of landed copies by releases 14-18 %.)
__device__ __forceinline__ void release_to_leader(uint32_t leader_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar) : "memory");
}
__device__ __forceinline__ void signal_leader(uint32_t leader_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar) : "memory");
}
// mbar_wait that acquires at cluster scope.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (try_wait_cluster(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) break;
    }
  }
  atomicOr(err, kErrTimeout);
  *abort_flag = 1;
  return false;
}
__device__ __forceinline__ void alloc2(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc2(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` in both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// `bar`: of either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
// The odd CTA's copies complete where it cannot wait for them. The leader, which can, does before either CTA leaves; only
// after an abort may it not have counted on all of them. They take microseconds: then a millisecond goes by.
__device__ __forceinline__ void outlast_copies() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 1000000ull) __nanosleep(10000);
}

__device__ __forceinline__ void tma_prefetch_3d(const void* tmap, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// ------------------------------------------------------------------------------------ the cut --
// Range c of C begins at unit floor(c U / C) = c q + floor(c r / C), U = q C + r: one 64-bit division a CTA. (By one
// thread, the scheduler's divisions and a binary search took a small prompt 4900 cycles.)
struct Cut {
  long long U, q;
  int C, r;
  __device__ __forceinline__ long long begin(int c) const { return c * q + c * r / C; }
  // the range that holds unit u, from an estimate
  __device__ __forceinline__ int of(long long u) const {
    int c = min(max((int)((float)u * (float)C / (float)U), 0), C - 1);
    while (c > 0 && begin(c) > u) --c;
    while (c + 1 < C && begin(c + 1) <= u) ++c;
    return c;
  }
};
__device__ __forceinline__ int blocks_of(int n, int tb) { return (n + tb - 1) / tb; }
// Units of a prompt's first b blocks (of one kv head).
__device__ __forceinline__ long long units(long long b, int tb) { return b * kFixed + tb * (b * (b + 1) / 2); }

// The last of n blocks that begins at or before unit `off` of its prompt and kv head: the quadratic's root, corrected.
__device__ __forceinline__ int block_at(long long off, int n, int tb) {
  const float h = kFixed + 0.5f * tb;
  int b = (int)((sqrtf(h * h + 2.f * tb * (float)off) - h) / tb);
  b = min(max(b, 0), n - 1);
  while (b > 0 && units(b, tb) > off) --b;
  while (b + 1 < n && units(b + 1, tb) <= off) ++b;
  return b;
}

// Length of prompt s; one that does not lie in [0, T) has none and is flagged by the first CTA.
__device__ __forceinline__ int prompt_len(const PromptArgs& a, int s, int* q0) {
  const int x = a.qsl[s], y = a.qsl[s + 1];
  *q0 = x;
  if (x < 0 || y < x || y > a.T) {
    if (blockIdx.x == 0) atomicOr(a.err, kErrBounds);
    return 0;
  }
  return y - x;
}

// First tile of the range that begins at unit x of a block's span (x < 0: the whole block is later).
__device__ __forceinline__ int cut_tile(long long x, int tiles) {
  if (x <= kFixed) return 0;
  const long long t = (x - kFixed + kKeys / 2) / kKeys;
  return t < kMinPiece ? 0 : t > tiles - kMinPiece ? tiles : (int)t;
}

}  // namespace

template <bool kF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, PromptArgs a, PromptScratch ws) {
  constexpr float kSigma = kF16 ? 4.f : 0.f;  // P is stored times 2^kSigma (f16 has few small values; at most 2^12)
  constexpr uint32_t kIdescS = kF16 ? idesc_f16(256, 128, false, false) : idesc_bf16(256, 128, false, false);
  constexpr uint32_t kIdescO = kF16 ? idesc_f16(256, 256, false, true) : idesc_bf16(256, 256, false, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cta_rank(), cluster = (int)(blockIdx.x >> 1);
  volatile int* abort_flag = &ms.abort_flag;
  auto bar = [&](const uint64_t& b) { return smem_u32(&b); };
  const int tpc = kRows / a.G, tb = 2 * tpc;  // tokens of a CTA, of a block
  const int used = tpc * a.G;                 // rows of a CTA that hold tokens

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(ms.item_full[i]), 1);
      mbar_init(bar(ms.item_empty[i]), kSoftWarps + kEpiWarps + 3);  // + K, V, and warp 3
      mbar_init(bar(ms.stat_full[i]), kSoftWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(ms.k_full[i]), 1);  // (the leader's Q, K and V are full once the other CTA's are, too: twice the bytes)
      mbar_init(bar(ms.k_empty[i]), 1);
      mbar_init(bar(ms.v_full[i]), 1);
      mbar_init(bar(ms.v_empty[i]), 1);
      mbar_init(bar(ms.tail_v[i]), 1);
      mbar_init(bar(ms.tail_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ms.p_full[i][0]), 2 * kSoftWarps);
      mbar_init(bar(ms.p_full[i][1]), 2 * kSoftWarps);
      mbar_init(bar(ms.pv_done[i]), 1);
    }
    mbar_init(bar(ms.q_full), 1);
    mbar_init(bar(ms.q_empty), 1);
    mbar_init(bar(ms.s_full), 1);
    mbar_init(bar(ms.s_free), 2 * kSoftWarps);
    mbar_init(bar(ms.o_ready), 1);
    mbar_init(bar(ms.o_free), 2 * kEpiWarps);
    mbar_init(bar(ms.drain), 1);
    mbar_init(bar(ms.never), 1);
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) alloc2(smem_u32(&ms.tmem_base), kTmemCols);
  // rows of Q that no token has: zeros, once
  for (int i = tid; i < (kRows - used) * 32; i += kThreads) {
    const int qd = i & 3, c = (i >> 2) & 7, r = used + (i >> 5);
    *reinterpret_cast<uint4*>(smem + kOffQ + qd * kQQuarter + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  // the units of all prompts, and the prompt this cluster's range starts in: each thread a run of prompts
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, a.num_seqs), s1 = min(s0 + per, a.num_seqs);
  long long sum = 0, blocks = 0;
  for (int s = s0; s < s1; ++s) {
    int q0;
    const int nb = blocks_of(prompt_len(a, s, &q0), tb);
    blocks += nb;
    sum += a.Hkv * units(nb, tb);
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
    blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
  }
  if (lane == 31) {
    ms.scan[0][warp] = incl;
    ms.scan[1][warp] = blocks;
  }
  if (tid == 0) ms.start_seq = -1;
  tc_fence_before();
  __syncthreads();
  long long before = incl - sum, U = 0;
  blocks = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += ms.scan[0][w];
    U += ms.scan[0][w];
    blocks += ms.scan[1][w];
  }
  const int C = (int)max(1LL, min((long long)(gridDim.x >> 1), max(a.Hkv * blocks, U / kMinRange)));
  const Cut cut = {U, U / C, C, (int)(U % C)};
  const bool work = cluster < C && U > 0;
  const long long u0 = work ? cut.begin(cluster) : 0, u1 = work ? cut.begin(cluster + 1) : 0;
  if (work && before <= u0 && u0 < before + sum) {
    for (int s = s0; s < s1; ++s) {
      int q0;
      const long long c = a.Hkv * units(blocks_of(prompt_len(a, s, &q0), tb), tb);
      if (u0 < before + c) {
        ms.start_seq = s;
        ms.start_off = before;
        break;
      }
      before += c;
    }
  }
  tc_fence_before();
  cluster_sync();  // barriers, TMEM and the start are there in both CTAs
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;

  if (work) {
    // The ring: consumers read item i from entry i % kRing.
    auto take = [&](int i, Item& I) -> bool {
      const bool ok = mbar_wait(bar(ms.item_full[i % kRing]), (i / kRing) & 1, abort_flag, a.err);
      I = ms.item[i % kRing];
      return ok;
    };
    auto give = [&](int i) { mbar_arrive(bar(ms.item_empty[i % kRing])); };

    // (a warpgroup's four warps execute its setmaxnreg together, first thing in their branch)
    if (warp < kSoftWarp0) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == 2) {
        // ------------------------------------------------------------ the items, and their Q
        if (lane == 0) {
          tma_prefetch_desc(&tmap_q);
          const uint64_t policy = policy_evict_first();
          const uint32_t q_full = in_leader(bar(ms.q_full));
          int s = ms.start_seq, q0, n = prompt_len(a, s, &q0), nb = blocks_of(n, tb);
          long long off = u0 - ms.start_off;
          const long long head_units = units(nb, tb);
          int kvh = 0;
          for (; off >= head_units; ++kvh) off -= head_units;
          int b = block_at(off, nb, tb);
          long long u = u0 - off + units(b, tb);  // the block's first unit
          int i = 0;
          bool ok = true;
          while (ok && u < u1) {
            const int kv_end = min(n, (b + 1) * tb), tiles = (kv_end + kKeys - 1) / kKeys;
            const long long next = u + kFixed + (long long)(b + 1) * tb;
            auto first_tile = [&](int c) { return cut_tile(cut.begin(c) - u, tiles); };
            Item I;
            I.t0 = u < u0 ? first_tile(cluster) : 0;
            I.t1 = next > u1 ? first_tile(cluster + 1) : tiles;
            if (I.t0 < I.t1) {
              int c0 = u >= u0 ? cluster : cut.of(u), c1 = next <= u1 ? cluster : cut.of(next - 1);
              while (c0 < c1 && first_tile(c0 + 1) == 0) ++c0;
              while (c1 > c0 && first_tile(c1) == tiles) --c1;
              I.q0 = q0;
              I.n = n;
              I.tok0 = b * tb;
              I.kvh = kvh;
              I.kv_end = kv_end;
              I.split = cluster - c0;
              I.nsplit = c1 - c0 + 1;
              // a cluster has at most one piece that continues a block (slot 2c) and one that begins one (2c + 1)
              I.slot0 = 2 * c0 + (cut.begin(c0) <= u ? 1 : 0);
              I.slot1 = 2 * (c0 + 1);
              I.slot = I.split == 0 ? I.slot0 : I.slot1 + 2 * (I.split - 1);
              if (i >= kRing) ok = mbar_wait(bar(ms.item_empty[i % kRing]), ((i / kRing) - 1) & 1, abort_flag, a.err);
              if (!ok) break;
              ms.item[i % kRing] = I;
              mbar_arrive(bar(ms.item_full[i % kRing]));
              // Q can only be loaded once the item before has done with its own: bring it to L2 meanwhile
              for (int qd = 0; qd < 4; ++qd) tma_prefetch_3d(&tmap_q, qd * 64, kvh * a.G, q0 + I.tok0 + rank * tpc);
              if (i >= 1) ok = mbar_wait(bar(ms.q_empty), (i - 1) & 1, abort_flag, a.err);
              if (!ok) break;
              if (rank == 0) mbar_expect_tx(bar(ms.q_full), 2u * (uint32_t)used * 512u);
              for (int qd = 0; qd < 4; ++qd)
                tma_load_3d(sbase + kOffQ + qd * kQQuarter, &tmap_q, qd * 64, kvh * a.G, q0 + I.tok0 + rank * tpc, q_full, policy);
              ++i;
            }
            u = next;
            if (++b == nb) {
              b = 0;
              if (++kvh == a.Hkv) {
                kvh = 0;
                do {
                  if (++s >= a.num_seqs) break;
                  n = prompt_len(a, s, &q0);
                  nb = blocks_of(n, tb);
                } while (n == 0);
                if (s >= a.num_seqs) break;
              }
            }
          }
          // the end of the items
          if (ok && i >= kRing) ok = mbar_wait(bar(ms.item_empty[i % kRing]), ((i / kRing) - 1) & 1, abort_flag, a.err);
          if (ok) {
            ms.item[i % kRing].nsplit = 0;
            mbar_arrive(bar(ms.item_full[i % kRing]));
          }
          // the copies, the other CTA's too, have landed before the leader lets either CTA exit
          if (rank == 0 && i >= 1) mbar_drain(bar(ms.q_full), (i - 1) & 1, abort_flag, a.err);
          if (rank != 0 && !ok) outlast_copies();
        }
      } else if (warp == 0 || warp == 1) {
        // ------------------------------------------------------------ K (warp 0) and V (warp 1)
        if (lane == 0) {
          const bool is_k = warp == 0;
          const CUtensorMap* tmap = is_k ? &tmap_k : &tmap_v;
          uint64_t* full = is_k ? ms.k_full : ms.v_full;
          uint64_t* empty = is_k ? ms.k_empty : ms.v_empty;
          const uint32_t region = sbase + (is_k ? kOffK : kOffV);
          const uint32_t leader_full = in_leader(bar(full[0]));
          tma_prefetch_desc(tmap);
          const uint64_t policy = policy_evict_last();  // every block of a prompt reads them again
          uint32_t g = 0;
          bool ok = true;
          Item I;
          for (int i = 0; ok; ++i) {
            if (!(ok = take(i, I)) || I.nsplit == 0) break;
            for (int t = I.t0; t < I.t1; ++t, ++g) {
              const uint32_t st = g % kStages;
              if (g >= kStages && !(ok = mbar_wait(bar(empty[st]), ((g / kStages) - 1) & 1, abort_flag, a.err))) break;
              // V of a tail: the odd CTA's threads write into it first, so it completes there
              const bool tail = !is_k && t + 1 == I.t1 && (t + 1) * kKeys > I.kv_end;
              if (rank == 0) mbar_expect_tx(bar(full[st]), tail ? kTile : 2 * kTile);
              else if (tail) mbar_expect_tx(bar(ms.tail_v[st]), kTile);
              const uint32_t done = rank != 0 && tail ? bar(ms.tail_v[st]) : leader_full + st * 8;
              const uint32_t dst = region + st * kTile;
              const int key = I.q0 + t * kKeys;
              if (is_k) {
                for (int qd = 0; qd < 4; ++qd)
                  tma_load_3d(dst + qd * kKQuarter, tmap, qd * 64, I.kvh, key + rank * 64, done, policy);
              } else {
                for (int qd = 0; qd < 2; ++qd)
                  tma_load_3d(dst + qd * kVQuarter, tmap, rank * 128 + qd * 64, I.kvh, key, done, policy);
              }
            }
            if (ok) give(i);
          }
          if (rank != 0 && !ok) outlast_copies();
          for (uint32_t st = 0; rank == 0 && st < kStages; ++st) {  // every copy has landed before either CTA may exit
            if (g <= st) continue;
            const uint32_t last = (g - 1 - st) / kStages;  // the last use of the stage
            mbar_drain(bar(full[st]), last & 1, abort_flag, a.err);
          }
        }
      } else if (warp == 3 && rank != 0) {
        // ------------------------------------------------------------ the odd CTA's tails
        // Keys behind a block's last token: their V becomes zeros as soon as it has landed (in the leader the softmax
        // does that), mostly while the softmax is at the tile before, so that the release costs no one.
        const uint32_t tail_full = in_leader(bar(ms.tail_full[0]));
        uint32_t g = 0, tails = 0;  // tiles of the items so far; parity of each stage's tails
        Item I;
        for (int i = 0; __all_sync(0xffffffffu, take(i, I)) && I.nsplit > 0; ++i) {
          g += I.t1 - I.t0;
          const int end = I.kv_end - (I.t1 - 1) * kKeys;  // keys of the last tile that count
          if (end < kKeys) {
            const uint32_t st = (g - 1) % kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(bar(ms.tail_v[st]), tails >> st & 1, abort_flag, a.err))) break;
            tails ^= 1u << st;
            uint8_t* v = smem + kOffV + st * kTile;
            for (int x = end * 16 + lane; x < kKeys * 16; x += 32)  // 16 bytes: 8 of each d-quarter's row
              *reinterpret_cast<uint4*>(v + (x >> 3 & 1) * kVQuarter + (x >> 4) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) release_to_leader(tail_full + st * 8);
          }
          __syncwarp();
          if (lane == 0) give(i);
        }
      } else if (warp == 3) {
        // ------------------------------------------------------------ the leader's products
        // The lanes of the warp agree on every wait: the ones that see an abort and those that do not must not part.
        uint32_t g = 0;
        bool ok = true;
        Item I;
        auto waited = [&](const uint64_t& b, uint32_t parity) -> bool {
          return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, a.err));
        };
        uint32_t tails = 0;  // parity of each stage's tails
        auto pv = [&](uint32_t gg, bool first, bool last, bool tail, int i) -> bool {
          const uint32_t st = gg % kStages, b = gg & 1;
          // the first P.V of an item overwrites O: both CTAs' epilogues of the one before must be done
          if (first && i >= 1 && !waited(ms.o_free, (i - 1) & 1)) return false;
          if (!waited(ms.v_full[st], (gg / kStages) & 1)) return false;
          if (tail) {  // the odd CTA's V: landed, and zeroed behind the block's keys
            if (!__all_sync(0xffffffffu, wait_cluster(bar(ms.tail_full[st]), tails >> st & 1, abort_flag, a.err))) return false;
            tails ^= 1u << st;
          }
          // P comes in two parts, keys 0-31 and 64-95 of the tile and then the others
  #pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!waited(ms.p_full[b][h], (gg >> 1) & 1)) return false;
            tc_fence_after();
            if (elect_one()) {
              // V as one N = 256 MN-major operand, 128 of d in each CTA: 64-element atoms 16 KB apart, 8-key
              // groups 1 KB apart, 16 keys (2 KB) per instruction
              const uint64_t v0 = smem_desc(sbase + kOffV + st * kTile, kVQuarter, 1024, kSw128);
  #pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int kk = 2 * h + (x & 1) + (x >> 1) * 4;
                mma2_ts(tmem + kColO, tmem + kColP + b * kPBufCols + kk * 8, v0 + ((kk * 2048) >> 4), kIdescO, first && kk == 0 ? 0u : 1u);
              }
              if (h == 1) {
                commit2(bar(ms.v_empty[st]));
                commit2(bar(ms.pv_done[b]));
                if (last) commit2(bar(ms.o_ready));
              }
            }
            __syncwarp();
          }
          return true;
        };
        // The order: S of the next tile, also of the next item, goes before P.V of this one.
        int nt_before = 0;  // tiles of the item before
        bool tail_before = false;
        for (int i = 0; ok; ++i) {
          if (!(ok = __all_sync(0xffffffffu, take(i, I)))) break;
          const int nt = I.nsplit == 0 ? 0 : I.t1 - I.t0;
          for (int j = 0; j < nt; ++j, ++g) {
            const uint32_t st = g % kStages;
            if (j == 0 && !(ok = waited(ms.q_full, i & 1))) break;
            if (!(ok = waited(ms.k_full[st], (g / kStages) & 1))) break;
            if (g >= 1 && !(ok = waited(ms.s_free, (g - 1) & 1))) break;
            tc_fence_after();
            if (elect_one()) {
  #pragma unroll
              for (int qd = 0; qd < 4; ++qd) {
                const uint64_t q0 = smem_desc(sbase + kOffQ + qd * kQQuarter, 16, 1024, kSw128);
                const uint64_t k0 = smem_desc(sbase + kOffK + st * kTile + qd * kKQuarter, 16, 1024, kSw128);
  #pragma unroll
                for (int k = 0; k < 4; ++k)  // 16 values (32 bytes) of d per instruction
                  mma2(tmem + kColS, q0 + ((k * 32) >> 4), k0 + ((k * 32) >> 4), kIdescS, (qd | k) ? 1u : 0u);
              }
              commit2(bar(ms.s_full));
              commit2(bar(ms.k_empty[st]));
              if (j == nt - 1) commit2(bar(ms.q_empty));
            }
            __syncwarp();
            if (j >= 1) ok = pv(g - 1, j == 1, false, false, i);
            else if (i >= 1) ok = pv(g - 1, nt_before == 1, true, tail_before, i - 1);
            if (!ok) break;
          }
          if (nt == 0) {  // the end: the last item's last P.V
            if (i >= 1) ok = pv(g - 1, nt_before == 1, true, tail_before, i - 1);
            break;
          }
          nt_before = nt;
          tail_before = I.t1 * kKeys > I.kv_end;
          if (ok && lane == 0) give(i);
        }
        // every product has completed before either CTA may give its TMEM back
        if (elect_one()) commit2(bar(ms.drain));
        __syncwarp();
      }
    } else if (warp < kEpiWarp0) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
      // ------------------------------------------------------------ softmax
      const int sw = warp - kSoftWarp0;
      const int q4 = warp & 3, kh = sw >> 2;  // TMEM lane quarter; key half of the tile
      const int row = q4 * 32 + lane;
      const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
      const int pair_bar = 1 + q4;            // named barrier of the two warps that share these rows
      const uint32_t s_free = in_leader(bar(ms.s_free));
      const uint32_t p_full = in_leader(bar(ms.p_full[0][0]));  // (the four barriers lie in a row)
      const float c = a.score_scale_log2;
      const bool c_pos = c >= 0.f;
      const int my_t = row / a.G;
      uint32_t g = 0;
      // failure-path test: a bounded wait on a barrier nothing arrives on
      const bool stalled = a.stall_test_ns && !mbar_wait(bar(ms.never), 0, abort_flag, a.err, a.stall_test_ns);
      for (int i = 0; !stalled; ++i) {
        // All softmax threads leave together (they meet at barriers). A failed wait inside an item does not
        // leave it: the later ones then fail at once.
        Item I;
        if (barrier_or(10, kSoftThreads, !take(i, I)) || I.nsplit == 0) break;
        const int first_tok = I.tok0 + rank * tpc, tok = first_tok + my_t;  // this CTA's first, this row's token
        float m_ref = kMInit, l = 0.f;
        const int nt = I.t1 - I.t0;
        for (int j = 0; j < nt; ++j, ++g) {
          const uint32_t b = g & 1, st = g % kStages;
          const int key0 = (I.t0 + j) * kKeys, kbase = key0 + kh * 64;
          float t[64];
          mbar_wait(bar(ms.s_full), g & 1, abort_flag, a.err);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 64; k += 16) {
            float v[16];
            tmem_ld16(tmem + lane_addr + kColS + kh * 64 + k, v);
#pragma unroll
            for (int x = 0; x < 16; ++x) t[k + x] = v[x];
          }
          // P.V(g - 2) has read P buffer b (its barrier's next phase needs P(g)); long since, so the wait costs
          // nothing but its own latency, which the load above hides
          if (g >= 2) mbar_wait(bar(ms.pv_done[b]), ((g >> 1) - 1) & 1, abort_flag, a.err);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) signal_leader(s_free);  // S may be overwritten
          const bool need_mask = key0 + kKeys - 1 > first_tok;
          float mx;
          if (need_mask) {
#pragma unroll
            for (int x = 0; x < 64; ++x) t[x] = kbase + x <= tok ? t[x] * c : -INFINITY;
            mx = extreme_of<true>(t);
          } else {
            mx = (c_pos ? extreme_of<true>(t) : extreme_of<false>(t)) * c;
          }
          ms.red[b][kh][row] = mx;
          named_barrier(pair_bar, 64);
          const float mt = fmaxf(mx, ms.red[b][kh ^ 1][row]);
          float alpha = 1.f;
          const bool rescale = mt > m_ref + kTau;
          if (rescale) {
            alpha = ex2(m_ref - mt);
            m_ref = mt;
            l *= alpha;
          }
          // tcgen05.ld/st are warp-wide: a warp rescales if any of its rows must
          if (__any_sync(0xffffffffu, rescale && j > 0)) {
            mbar_wait(bar(ms.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort_flag, a.err);
            tc_fence_after();
            if (!rescale) alpha = 1.f;
#pragma unroll 1
            for (int k = 0; k < 128; k += 16) {  // this thread's half of its row of O
              float v[16];
              const uint32_t at = tmem + lane_addr + kColO + kh * 128 + k;
              tmem_ld16(at, v);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) v[x] *= alpha;
              tmem_st16(at, v);
            }
            tmem_wait_st();
          }
          const bool tail = rank == 0 && key0 + kKeys > I.kv_end;
          if (tail) {
            // keys behind the block's last token (other prompts', later ones'): their V becomes zeros;
            // thread (kh, row) zeroes d-quarter kh of key `row`, each lane of eight beginning with another
            // 16 bytes (another bank). This wait skips the phases of other tiles: V(g - 2) has landed
            // (P.V(g - 2) is done), V(g + 2) comes after P.V(g). (The odd CTA's warp 3 does its own.)
            mbar_wait(bar(ms.v_full[st]), (g / kStages) & 1, abort_flag, a.err);
            if (key0 + row >= I.kv_end) {
              uint4* dst = reinterpret_cast<uint4*>(smem + kOffV + st * kTile + kh * kVQuarter + row * 128);
#pragma unroll
              for (int x = 0; x < 8; ++x) dst[(x + lane) & 7] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          // P = 2^(s c - m + sigma), 32 keys at a time: P.V of the first begins while the second are computed. m is a
          // rounded s c, so P's largest value is off by 2^(m 2^-24), which cancels in the sums, but ends f16's range from
          // |m| = 2^26 on (rounding s c first too, where m is large, cost 1.5 % in every form tried).
          tc_fence_after();
          const float off = m_ref - kSigma, sc = need_mask ? 1.f : c;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
            float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float p0 = ex2(fmaf(t[32 * h + x], sc, -off)), p1 = ex2(fmaf(t[32 * h + x + 1], sc, -off));
              ls[(x >> 1) & 3] += p0 + p1;  // (the sums take P before its rounding: lse needs more than P.V does)
              pk[x / 2] = kF16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            }
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            tmem_st16u(tmem + lane_addr + kColP + b * kPBufCols + kh * 32 + 16 * h, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (tail) mbar_arrive(bar(ms.p_full[b][h]));
              else signal_leader(p_full + (2 * b + h) * 8);
            }
          }
        }
        ms.stat_l[i % kRing][kh][row] = l;
        if (kh == 0) ms.stat_m[i % kRing][row] = m_ref;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(ms.stat_full[i % kRing]));
          give(i);
        }
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
      // ------------------------------------------------------------ epilogue
      const int q4 = warp & 3, row = q4 * 32 + lane, gi = row;
      const uint32_t o_addr = tmem + ((uint32_t)(q4 * 32) << 16) + kColO;
      const uint32_t o_free = in_leader(bar(ms.o_free));
      const int my_t = row / a.G, my_g = row - my_t * a.G;
      // This call's counter tag (thread 0 uses it).
      const unsigned long long tag = (__ldcg(ws.epoch) ^ ((unsigned long long)ws.call_tag * 0x9E3779B97F4A7C15ull)) & kSplitTagMask;
      for (int i = 0;; ++i) {
        Item I;
        if (barrier_or(11, kEpiThreads, !take(i, I)) || I.nsplit == 0) break;
        const int tok = I.tok0 + rank * tpc + my_t;
        const bool valid = row < used && tok < I.n;
        mbar_wait(bar(ms.stat_full[i % kRing]), (i / kRing) & 1, abort_flag, a.err);
        const float lr = ms.stat_l[i % kRing][0][row] + ms.stat_l[i % kRing][1][row];
        // (a piece of which a row sees nothing has the sum 0; a NaN is not that)
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
        const float lse = lr == 0.f ? -INFINITY : ms.stat_m[i % kRing][row] - kSigma + log2f(lr);
        const int head = I.kvh * a.G + my_g;
        const long long out_at = valid ? (long long)(I.q0 + tok) * a.o_st + (long long)head * a.o_sh : -1;  // this row (-1: none)
        const long long lse_at = (long long)(I.q0 + tok) * a.lse_st + (long long)head * a.lse_sh;
        uint8_t* stage = smem + kOffStage + q4 * 32 * kStagePitch;
        // Chunks of 8 columns of each of the warp's rows, packed, go through shared memory, so that lanes side by
        // side store the bytes of a row (16 bytes of 32 rows a store were bound by the LSU): put() and flush().
        auto put = [&](const uint32_t* w, int chunk, int n) {
#pragma unroll
          for (int x = 0; x < n; ++x)
            *reinterpret_cast<uint4*>(stage + lane * kStagePitch + (chunk + x) * 16) = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        };
        auto flush = [&](auto chunks, int col) {
          constexpr int kN = decltype(chunks)::value;
          __syncwarp();
#pragma unroll
          for (int x = 0; x < kN; ++x) {
            const int idx = x * 32 + lane, r = idx / kN, ch = idx - r * kN;
            const long long at = __shfl_sync(0xffffffffu, out_at, r);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kStagePitch + ch * 16);
            if (at >= 0) *reinterpret_cast<uint4*>(a.out + at + col + ch * 8) = v;
          }
          __syncwarp();
        };
        auto load32 = [&](int col, float (&v)[32]) {
          float x0[16], x1[16];
          tmem_ld16(o_addr + col, x0);
          tmem_ld16(o_addr + col + 16, x1);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            v[x] = x0[x] * inv;
            v[16 + x] = x1[x] * inv;
          }
        };
        auto pack = [&](float x, float y) { return kF16 ? pack_f16x2(x, y) : pack_bf16x2(x, y); };
        // Have the other pieces of a cut block all arrived?
        unsigned long long* counter = ws.counters + 2 * I.slot0 + rank;
        if (I.nsplit > 1) {
          if (gi == 0) {
            ms.merge_flag = split_peek(counter) == (tag << 16 | (unsigned)(I.nsplit - 1));
            if (ms.merge_flag) split_clear(counter);
            __threadfence();
          }
          named_barrier(9, kEpiThreads);
        }
        mbar_wait(bar(ms.o_ready), i & 1, abort_flag, a.err);
        tc_fence_after();
        if (I.nsplit == 1) {
          // O leaves TMEM at once, part of it to the stage and the rest to registers, so that the next P.V may
          // overwrite it while the stores are still to come
          uint32_t w[80];
#pragma unroll
          for (int k = 0; k < kHeadDim; k += 32) {
            float v[32];
            load32(k, v);
            uint32_t p[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = pack(v[2 * x], v[2 * x + 1]);
            if (k < kStageCols) {
              put(p, k / 8, 4);
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) w[(k - kStageCols) / 2 + x] = p[x];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) signal_leader(o_free);
          flush(std::integral_constant<int, 12>(), 0);
          put(w, 0, 12);
          flush(std::integral_constant<int, 12>(), kStageCols);
          put(w + 48, 0, 8);
          flush(std::integral_constant<int, 8>(), 2 * kStageCols);
          if (a.lse && valid) a.lse[lse_at] = lse * 0.6931471805599453f;
        } else {
          // A piece whose block's other pieces have all arrived merges them with its own O at once. Any other
          // piece leaves its partial behind; should the others have arrived meanwhile, it merges too.
          auto slot_of = [&](int x) { return x == 0 ? I.slot0 : I.slot1 + 2 * (x - 1); };
          auto lse_of = [&](int x) { return ws.part_lse + (size_t)(2 * slot_of(x) + rank) * kRows + row; };
          auto part_of = [&](int x) {  // this row of a partial: four values every kRows * 4
            return reinterpret_cast<float4*>(ws.part_o) + (size_t)(2 * slot_of(x) + rank) * (kHeadDim / 4) * kRows + row;
          };
          bool last = ms.merge_flag;
          if (!last) {
            float4* part = part_of(I.split);
#pragma unroll 1
            for (int k = 0; k < kHeadDim; k += 32) {
              float v[32];
              load32(k, v);
#pragma unroll
              for (int x = 0; x < 32; x += 4) part[(k + x) / 4 * kRows] = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
            }
            *lse_of(I.split) = lse;
            __threadfence();
            named_barrier(9, kEpiThreads);
            if (gi == 0) {
              __threadfence();
              ms.merge_flag = split_arrive(counter, I.nsplit, tag);
              __threadfence();
            }
            named_barrier(9, kEpiThreads);
            last = ms.merge_flag;
          }
          if (last) {
            // out = sum_x 2^(lse_x - M) o_x / sum_x 2^(lse_x - M), in the order of the pieces: the same bits
            // whichever came last
            __threadfence();
            float M = -INFINITY, total = 0.f;
            for (int x = 0; x < I.nsplit; ++x) M = fmaxf(M, x == I.split ? lse : __ldcg(lse_of(x)));
            for (int x = 0; x < I.nsplit; ++x) total += exp2f((x == I.split ? lse : __ldcg(lse_of(x))) - M);
            const float scale = 1.f / total;  // (a token sees itself: some piece has weight 1)
            if (a.lse && valid) a.lse[lse_at] = (M + log2f(total)) * 0.6931471805599453f;
            // the next 32 columns of another piece are on their way while these are added up
            const int fx0 = I.split == 0 ? 1 : 0;
            int fx = fx0, fk = 0;
            float4 next[8];
            auto fetch = [&]() {
              const float4* o = part_of(fx) + fk / 4 * kRows;
#pragma unroll
              for (int y = 0; y < 8; ++y) next[y] = __ldcg(o + y * kRows);
              ++fx;
              fx += fx == I.split;
              if (fx >= I.nsplit) {
                fx = fx0;
                fk += 32;
              }
            };
            fetch();
#pragma unroll 1
            for (int k = 0; k < kHeadDim; k += 32) {
              float acc[32] = {};
#pragma unroll 1
              for (int x = 0; x < I.nsplit; ++x) {
                float v[32];
                if (x == I.split) {
                  load32(k, v);
                } else {
#pragma unroll
                  for (int y = 0; y < 8; ++y) {
                    v[4 * y] = next[y].x;
                    v[4 * y + 1] = next[y].y;
                    v[4 * y + 2] = next[y].z;
                    v[4 * y + 3] = next[y].w;
                  }
                  if (fk < kHeadDim) fetch();
                }
                const float wx = exp2f((x == I.split ? lse : __ldcg(lse_of(x))) - M) * scale;
#pragma unroll
                for (int y = 0; y < 32; ++y) acc[y] = fmaf(wx, v[y], acc[y]);
              }
              uint32_t w[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) w[y] = pack(acc[2 * y], acc[2 * y + 1]);
              put(w, 0, 4);
              flush(std::integral_constant<int, 4>(), k);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) signal_leader(o_free);
        }
        __syncwarp();
        if (lane == 0) give(i);
      }
    }
    // both CTAs wait for the leader's products (also after an abort)
    __syncwarp();
    if (warp == kSoftWarp0 && lane == 0) mbar_drain(bar(ms.drain), 0, abort_flag, a.err);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still arrive on its barriers
  if (warp == 0) {
    tc_fence_after();
    dealloc2(tmem, kTmemCols);
  }
}

namespace {

__global__ void prompt_epoch_kernel(unsigned long long* epoch) { *epoch += 1ull; }

bool encode(CUtensorMap* m, const void* data, bool f16, int heads, int T, long long sh, long long st, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)T};
  // (a dim of one entry has no stride that matters)
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? sh * 2 : 512), (cuuint64_t)(T > 1 ? st * 2 : 512)};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  return encode_tmap(m, f16, 3, data, dims, strides, box);
}

}  // namespace

int launch_prompt_tc(const PromptArgs& a, const PromptScratch& ws, int clusters, bool captured, cudaStream_t stream) {
  const long long strides[6] = {a.Hq > 1 ? a.q_sh : 1, a.T > 1 ? a.q_st : 1, a.Hkv > 1 ? a.k_sh : 1,
                                a.T > 1 ? a.k_st : 1, a.Hkv > 1 ? a.v_sh : 1, a.T > 1 ? a.v_st : 1};
  for (long long s : strides)
    if (s <= 0 || s >= 1LL << 38) return 0;  // what a tensor map cannot say (2^40 bytes): the warp-level kernel
  CUtensorMap q, k, v;
  const int tpc = kRows / a.G;
  if (!encode(&q, a.q, a.f16, a.Hq, a.T, a.q_sh, a.q_st, a.G, tpc) || !encode(&k, a.k, a.f16, a.Hkv, a.T, a.k_sh, a.k_st, 1, 64) ||
      !encode(&v, a.v, a.f16, a.Hkv, a.T, a.v_sh, a.v_st, 1, kKeys))
    return -1;
  auto kern = a.f16 ? prompt_tc_kernel<true> : prompt_tc_kernel<false>;
  static int attr_done[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  const int which = a.f16 ? 2 : 1;
  if (dev < 0 || dev >= 64 || !(attr_done[dev] & which)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    // setmaxnreg.inc waits for registers that are free: never launch a build whose split does not add up
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess && fa.numRegs != kLaunchRegs) {
      char buf[160];
      snprintf(buf, sizeof buf, "prompt kernel built with %d registers per thread; its warpgroup split needs %d", fa.numRegs, kLaunchRegs);
      set_tc_error(buf);
      return -1;
    }
    if (e == cudaSuccess && dev >= 0 && dev < 64) attr_done[dev] |= which;
  }
  // A graph replays its captured tag: the workspace's epoch word tells the replays apart.
  if (e == cudaSuccess && captured) {
    prompt_epoch_kernel<<<1, 1, 0, stream>>>(ws.epoch);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = launch_pdl(false, kern, 2 * clusters, kThreads, kSmemBytes, stream, q, k, v, a, ws);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    char buf[160];
    snprintf(buf, sizeof buf, "prompt kernel: %s", cudaGetErrorString(e));
    set_tc_error(buf);
    return -1;
  }
  return 1;
}

// Clusters that a call of these sizes can use: its blocks, or its units over the least range were all tokens one prompt's.
int prompt_clusters(long long T, int num_seqs, int Hkv, int G, int sms) {
  const int tb = 2 * (kRows / G);
  const double b = (double)((T + tb - 1) / tb) + num_seqs;
  const double ranges = Hkv * (b * kFixed + tb * b * (b + 1) / 2) / kMinRange;
  const double most = ranges > Hkv * b ? ranges : Hkv * b;
  const int all = sms / 2;
  return most < 1 ? 1 : most < all ? (int)most : all;
}

}  // namespace pgqa
