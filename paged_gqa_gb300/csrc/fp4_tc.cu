// fp4_tc.cu -- tcgen05 (TMEM) attention kernel over a 4-bit paged KV cache (fp4.cuh), bf16 Q,
// for verify blocks (kN = 64 rows: single tokens and MTP / speculative verify) and prefill
// blocks (kN = 128 rows), bottom-right causal.
//
// Both products take the cache as their A operand, with up to kN query rows as N:
//   S^T[key, row] = K Q^T          A = K   [128 keys, 256 d]
//   O^T[d, row] += V^T P^T         A = V^T [256 d, 128 keys], as two 128-lane tiles
// so the MMA's 128 lanes are full however few rows a block has, its cost follows the rows
// (N = rows rounded up to 16), and A can come from TMEM: the packed pages (144 bytes per key)
// go from HBM to shared memory by bulk copies, eight to twelve warps widen them to f16 (code * scale,
// exact) and store them with tcgen05.st, and no widened value ever passes through shared memory.
// (Through it, 1 KB per key written and read again would cost 16 of the ~12 cycles per key
// that a CTA has at full HBM bandwidth.) Widening thread t owns TMEM lane t: key t of the
// tile for K (its row's bytes are d pairs, K's order), code byte t of every key for V, i.e. d =
// 2t for tile 0 and 2t + 1 for tile 1; a V page's blocks hold 16 keys of a byte contiguously.
//
// Widening goes by halves of a tile (128 d of the 128 keys of K, 64 keys of both tiles of V: 64
// TMEM columns), each published to the MMA issuers and freed by them on its own, so a half is
// multiplied while the other is widened. With 64 rows K and V have two such halves each; with 128
// rows (S and O^T take 384 columns) they share two, K a tile ahead: K(0) K(1) V(0) K(2) V(1) ..
//
// Q is staged in f16 with a power of two per row (its largest value to [2^14, 2^15)): a bf16
// value has 8 significant bits, so everything within 2^-28 of the row's largest is exact, and
// the power goes into the row's score scale. P = 2^(s - m + 4) is rounded to f16 (2^-11), the
// row sums take it before that rounding: half the bytes and the rate of the f16 product, below the
// output's own rounding of 2^-8 (so is a split piece's f16 partial). The softmax, its lazy rescale, the split-KV pieces and
// their merge follow the FP8 verify kernel (verify_tc.cu): keys on lanes, rows on columns.
//
// Warp roles: warp 0 S issuer (+ TMEM owner), warp 1 P.V issuer, warp 2 K copies, warp 3 V
// copies, warps 4-19 softmax and epilogue (row group (w - 4) / 4 owns kN / 4 rows, lane quarter w % 4);
// with 64 rows (1024 threads) warps 20-23 widen K and 24-31 V, side by side; with 128 rows (896 threads) warps
// 20-27 widen both in turn, since the shared columns hold one at a time (2228 us for a 8192-token
// chunk on 32768 keys with the two groups of warps there, 2175 so).
//
// What bounds it. A 128-key tile takes about 10.4k warp instructions at 48-64 rows: ~3.2k widen, ~2.0k
// softmax, the rest hands tiles from role to role; issue slots are 65 % busy, the ALU pipe (conversions at
// half rate) 46 %, tensor cores 25 %, HBM 31 %. With either half of the work taken out (timing only): neither
// widening nor softmax 248 us, no widening 275, no softmax 337, all of it 431 then, 428 now (256 sequences of
// 8192 keys, 2-4 tokens, 32/2 heads: 1233 MB, 182 us at the HBM rate). 64 sequences of 1k-32k keys,
// 4 tokens, 16/1 heads: 128 us (46). With 128 rows widening and the products alternate in the shared
// columns, and a tile takes ~4700 cycles where the products alone take 2230: 2125 us, 905 TFLOP/s.
// A small call is a chain of cold steps. One CTA of a 128-row block, in cycles: set-up 1.7k, the item and its
// rows of Q 9k, the first S 2.4k, its softmax 10k (first references: 2.7k for each 16 rows; code
// fetched for the first time), each further tile 5k, epilogue 5.5k, the partial's store and count 6k, a merge of two
// pieces 11k: ~30 us, where the products take 2.
// Tried and slower: operands in quarters instead of halves (2910 us, a hand-over costs ~400
// cycles), both row halves of the softmax in registers (2370, spills), byte permutes for half of
// V's pairs (2337), one barrier arrival per softmax warp instead of per thread (2204, verify 439).
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

constexpr int kSoftWarp0 = 4, kSoftWarps = 16, kSoftThreads = kSoftWarps * 32;
constexpr int kWideWarp0 = kSoftWarp0 + kSoftWarps;
constexpr float kTau = 4.f;         // rescale when a score exceeds the reference by 2^kTau
constexpr float kSigma = 4.f;       // P is scaled by 2^kSigma (at most 2^8; f16 holds 2^-24)
constexpr float kMInit = -3.0e38f;  // reference of a row before its first key

constexpr uint32_t kTile = kTileKeys * kFp4Row;  // packed bytes of a tile of K or V (18 KB)
// V's scales of a tile, as widen_v multiplies by them: per 16-token block and group 16 words, f16
// {scale, 0} of even tokens and {0, scale} of odd ones.
constexpr uint32_t kScaleBuf = kTileKeys * 16 * 4;  // 8 KB
constexpr uint32_t kChunkCols = 64;              // TMEM columns of half a tile of K or V

template <int kN>
struct Cfg {
  static constexpr int kCols = kN / 4;  // rows per softmax thread
  // The widened operands in TMEM go by halves of 64 columns: 128 d of the 128 keys of K, 64 keys
  // of both tiles of V. With 64 rows K and V have two each; with 128 rows they share two.
  static constexpr bool kShared = kN == 128;
  // Warps that widen: 4 K and 8 V side by side, or, where the columns allow only one at a time,
  // the same 8 both in turn.
  static constexpr int kKWarps = kShared ? 8 : 4, kVWarps = 8;
  static constexpr int kVWarp0 = kWideWarp0 + (kShared ? 0 : kKWarps);
  static constexpr int kWarps = kVWarp0 + kVWarps, kThreads = kWarps * 32;
  // Registers of the warpgroups (their sum is what the launch gives: kLaunchRegs a thread).
  static constexpr int kLaunchRegs = kShared ? 72 : 64;
  static constexpr int kSoftRegs = kShared ? 96 : 72, kWideRegs = kShared ? 40 : 56, kOtherRegs = kShared ? 40 : 56;
  static_assert(kSoftWarps * kSoftRegs + (kWarps - kWideWarp0) * kWideRegs + kSoftWarp0 * kOtherRegs == kWarps * kLaunchRegs &&
                    kThreads * kLaunchRegs <= 65536, "register split");
  static constexpr int kKStages = kN == 64 ? 3 : 2, kVStages = kN == 64 ? 3 : 2;
  static constexpr int kSBufs = kN == 64 ? 2 : 1;
  static constexpr uint32_t kColS = 0, kColO = 128, kColK = 128 + 2 * kN, kColV = kColK + (kN == 64 ? 128 : 0);
  static_assert(kSBufs * kN <= 128 && kColV + 128 <= 512, "TMEM columns");
  static constexpr uint32_t kQQuarter = kN * 128;   // [kN rows][64 d] f16, 128-byte swizzle
  static constexpr uint32_t kPBlock = kTileKeys * 128;       // [128 keys][64 rows] f16
  static constexpr uint32_t kPBuf = kPBlock * (kN / 64);
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffP = kOffQ + 4 * kQQuarter;
  static constexpr uint32_t kOffK = kOffP + 2 * kPBuf;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTile;
  static constexpr uint32_t kOffScale = kOffV + kVStages * kTile;  // two tiles' V scales, kScaleBuf each
  static constexpr uint32_t kOffMisc = kOffScale + 2 * kScaleBuf;
  static_assert(2 * kPBuf >= kN * kHeadDim * 2, "a split piece's f16 partial fits the P buffers");
};

template <int kN, bool kFused>
struct Misc {
  using C = Cfg<kN>;
  alignas(16) float m[2][kN];
  alignas(16) float mo[2][kN];   // kSigma - m
  alignas(16) float cs[2][kN];   // score scale of the row (log2 units, Q's power of two removed)
  alignas(16) float red[4][kN];
  alignas(16) float alpha[kN];
  alignas(16) int lim[2][kN];
  alignas(16) long long out_off[2][kN];
  alignas(16) float lse_stage[kN];
  alignas(8) uint64_t k_full[C::kKStages], k_empty[C::kKStages], v_full[C::kVStages], v_empty[C::kVStages];
  uint64_t ak_full[2], av_full[2], ak_free[2], av_free[2], av_go[2];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t q_full, q_free, o_ready, o_free, drain[2];
  uint64_t never;  // no thread ever arrives (the failure-path test waits on it)
  uint32_t tmem_base;
  int abort_flag;
  int merge_flag;
  int fcount;
  int4 fitem[kFused ? kFusedMaxBlocks : 1];
  int4 fseq[kFused ? kFusedMaxBlocks : 1];
};

template <int kN, bool kFused>
constexpr size_t smem_bytes() {
  return Cfg<kN>::kOffMisc + sizeof(Misc<kN, kFused>) + 1024;
}
static_assert(smem_bytes<64, true>() <= 232448 && smem_bytes<128, false>() <= 232448, "shared memory of one CTA");
static_assert(sizeof(self_plan::Scratch) <= Cfg<64>::kKStages * kTile, "the self-plan scratch fits the K stages");

struct Item {
  int block, seq, kvh, row0, nrows, nsplit, split, slot_base;
  int tile_begin, ntiles, kv_hi;
  int q0, qn, L;
};

template <int kN, bool kFused>
__device__ __forceinline__ Item load_item(const Problem& p, const ClassPlan& cp, const Pointers& ptr,
                                          const Misc<kN, kFused>& ms, int it) {
  Item r;
  if (kFused) {
    const self_plan::Piece f = self_plan::unpack(p, ms.fitem[it]);
    const int4 sq = ms.fseq[it];
    r.block = f.block;
    r.seq = f.seq;
    r.kvh = f.kvh;
    r.tile_begin = f.tile_begin;
    r.ntiles = f.ntiles;
    r.split = f.split;
    r.nsplit = f.nsplit;
    r.slot_base = f.slot_base;
    r.q0 = sq.x;
    r.qn = sq.y;
    r.L = sq.z;
    r.row0 = 0;
    r.nrows = r.qn * p.G;
    r.kv_hi = min((r.tile_begin + r.ntiles) * kTileKeys, r.L);
  } else {
    const WorkItem w = cp.items[it];
    const RowBlock b = cp.blocks[w.block];
    r.block = w.block;
    r.seq = b.seq;
    r.kvh = b.kvh;
    r.row0 = b.row0;
    r.nrows = b.nrows;
    r.nsplit = b.nsplit;
    r.split = w.split;
    r.slot_base = b.slot_base;
    r.tile_begin = w.tile_begin;
    r.ntiles = w.tile_end - w.tile_begin;
    r.kv_hi = min(w.tile_end * kTileKeys, b.kv_end);
    r.q0 = ptr.qsl[b.seq];
    r.qn = ptr.qsl[b.seq + 1] - r.q0;
    r.L = ptr.seq_lens[b.seq];
  }
  return r;
}

// Byte mask of tokens 4w .. 4w + 3 of a 16-token block whose first n tokens are there.
__device__ __forceinline__ uint32_t token_mask(int n, int w) {
  const int k = n - 4 * w;
  return k >= 4 ? 0xffffffffu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
}

}  // namespace

template <int kN, bool kFused>
__global__ void __launch_bounds__(Cfg<kN>::kThreads, 1)
fp4_tc_kernel(Problem p, Pointers ptr, ClassPlan cp) {
  using C = Cfg<kN>;
  constexpr int kCols = C::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Misc<kN, kFused>& ms = *reinterpret_cast<Misc<kN, kFused>*>(smem + C::kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &ms.abort_flag;
  auto bar = [&](const uint64_t& b) { return smem_u32(&b); };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int item_begin = 0, item_end = 0;
  self_plan::Scratch& fs = *reinterpret_cast<self_plan::Scratch*>(smem + C::kOffK);
  if (kFused) {
    self_plan::load(p, ptr, fs);  // the set-up below overlaps these reads
    if (p.unplanned && blockIdx.x == 0) self_plan::flag_invalid(p, ptr, fs);
  } else {
    item_begin = cp.cta_item_begin[blockIdx.x];
    item_end = cp.cta_item_begin[blockIdx.x + 1];
    if (item_begin >= item_end) return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(bar(ms.k_full[s]), 1);
      mbar_init(bar(ms.k_empty[s]), C::kKWarps);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(bar(ms.v_full[s]), 1);
      mbar_init(bar(ms.v_empty[s]), C::kVWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(ms.ak_full[b]), C::kKWarps);
      mbar_init(bar(ms.av_full[b]), C::kVWarps);
      mbar_init(bar(ms.ak_free[b]), 1);
      mbar_init(bar(ms.av_free[b]), 1);
      mbar_init(bar(ms.av_go[b]), 1);
      mbar_init(bar(ms.s_full[b]), 1);
      mbar_init(bar(ms.s_free[b]), kSoftThreads);
      mbar_init(bar(ms.p_full[b]), kSoftThreads);
      mbar_init(bar(ms.pv_done[b]), 1);
    }
    mbar_init(bar(ms.q_full), kSoftThreads);
    mbar_init(bar(ms.q_free), 1);
    mbar_init(bar(ms.o_ready), 1);
    mbar_init(bar(ms.o_free), kSoftThreads);
    mbar_init(bar(ms.drain[0]), 1);
    mbar_init(bar(ms.drain[1]), 1);
    mbar_init(bar(ms.never), 1);
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_u32(&ms.tmem_base), 512);
    tmem_relinquish();
  }
  if (kFused) {
    __syncthreads();  // the sequences are staged
    if (warp == 1) self_plan::plan_warp(p, fs, cp.num_ctas, lane, ms.fitem, ms.fseq, &ms.fcount);
    fence_proxy_async_smem();  // the scratch lies where the copies go
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  if (kFused) {
    item_end = ms.fcount;
    if (item_end == 0) {  // no range or no tile in it: give the columns back and leave
      if (warp == 0) tmem_dealloc(tmem, 512);
      return;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int wg = warp >> 2;
  if (wg >= 1 && wg < kWideWarp0 / 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    // ------------------------------------------------------------ softmax + epilogue
    const int sw = warp - kSoftWarp0;
    const int gi = sw * 32 + lane;
    const int q4 = warp & 3;               // TMEM lane quarter
    const int rg = sw >> 2;                // row group
    const int c0 = rg * kCols;             // first row (column) this thread owns
    const int group_bar = 3 + rg;          // named barrier of the row group's four warps
    const int ti = q4 * 32 + lane;         // TMEM lane: key of the tile; for O^T, d = 2 ti and 2 ti + 1
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    uint64_t l[kCols / 2];  // row sums over this thread's keys, fp32, two rows each
#pragma unroll
    for (int n = 0; n < kCols / 2; ++n) l[n] = 0;
    // Failure-path test: every softmax thread's bounded wait on a barrier nothing arrives on
    // runs out; they skip the items, no Q is published, and every other role gives up and
    // drains what it has in flight.
    const bool stalled = p.stall_test_ns && !mbar_wait(bar(ms.never), 0, abort_flag, ptr.err, p.stall_test_ns);
    if (!stalled) {
      const unsigned long long ctag = gi == 0 ? split_tag(p, cp) : 0ull;

      auto q_prep = [&](const Item& I, int ii) {
        const int pi = ii & 1;
        // 128 rows: (token of the block << 16 | head) of each, worked out once (the division per load
        // makes a small call 1-2 us longer, and code to fetch); the epilogue's first barrier comes
        // before lse_stage is written
        uint32_t* where = reinterpret_cast<uint32_t*>(ms.lse_stage);
        const int t0 = I.row0 / p.G;
        if (ii >= 1) mbar_wait_polls(bar(ms.q_free), (ii - 1) & 1, abort_flag, ptr.err);
        if (gi < kN) {
          const int n = gi;
          const bool real = n < I.nrows;
          const RowMap m = map_row(I.row0 + n, p.G, I.kvh);
          ms.lim[pi][n] = real ? I.L - I.qn + m.t : -1;
          ms.out_off[pi][n] = real ? (long long)(I.q0 + m.t) * p.o_st + (long long)m.h * p.o_sh : 0;
          if (kN == 128) where[n] = (uint32_t)(m.t - t0) << 16 | (uint32_t)m.h;
          // padding rows: a finite reference, so their (discarded) scores never vote
          ms.m[pi][n] = real ? kMInit : 0.f;
          ms.mo[pi][n] = kSigma - ms.m[pi][n];
        }
        if (kN == 128) named_barrier(1, kSoftThreads);
        // A warp takes whole rows (32 lanes of 16 bytes), four at a time.
#pragma unroll 1
        for (int k0 = 0; k0 < kN / kSoftWarps; k0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (k0 + k) * kSoftWarps + sw;
            v[k] = make_uint4(0, 0, 0, 0);
            if (r < I.nrows) {
              RowMap m;
              if (kN == 128) {
                m.t = t0 + (int)(where[r] >> 16);
                m.h = (int)(where[r] & 0xffffu);
              } else {
                m = map_row(I.row0 + r, p.G, I.kvh);
              }
              v[k] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(ptr.q) +
                                                     (long long)(I.q0 + m.t) * p.q_st + (long long)m.h * p.q_sh + lane * 8);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (k0 + k) * kSoftWarps + sw;
            uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
            top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
            // 2^(141 - e) takes a row whose largest value has exponent field e to [2^14, 2^15)
            // (at most 2^127: a row below 2^-113 stays smaller, and exact all the same)
            const int e = max((int)(top >> 7), 14);
            const float up = __uint_as_float((uint32_t)(268 - e) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
            const int qd = lane >> 3, cc = lane & 7;
            *reinterpret_cast<uint4*>(smem + C::kOffQ + qd * C::kQQuarter + r * 128 + ((cc ^ (r & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
            if (lane == 0)  // times 2^(e - 141)
              ms.cs[pi][r] = p.score_scale_log2 * __uint_as_float(e > 14 ? (uint32_t)(e - 14) << 23 : 0x00400000u);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(ms.q_full));
      };

      // Rows cc .. cc + 15 of S buffer sb hold a score above the reference by more than 2^kTau: the
      // exact tile maximum of s c per row becomes the new reference, and O^T follows it (from the
      // item's second tile on). Called by the row group's four warps together; rare, so that it
      // trades speed for registers: a column at a time.
      auto new_reference = [&](int cc, int pi, uint32_t sb, bool have_o, uint32_t g, bool need_mask, int key, int kv_hi) {
        float r = -INFINITY;  // lane n: the warp's maximum of row cc + n
#pragma unroll 1
        for (int n = 0; n < 16; n += 4) {
          float v[4];
          tmem_ld4f(tmem + lane_addr + C::kColS + sb * kN + cc + n, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool vis = !need_mask || (key < kv_hi && key <= ms.lim[pi][cc + n + i]);
            const float x = warp_max(vis ? __fmul_rn(v[i], ms.cs[pi][cc + n + i]) : -INFINITY);
            if (lane == n + i) r = x;
          }
        }
        if (lane < 16) ms.red[q4][cc + lane] = r;
        named_barrier(group_bar, 128);
        if (q4 == 0 && lane < 16) {
          const int n = cc + lane;
          const float mt = fmaxf(fmaxf(ms.red[0][n], ms.red[1][n]), fmaxf(ms.red[2][n], ms.red[3][n]));
          const float m_old = ms.m[pi][n];
          const float mn = fmaxf(m_old, mt);
          ms.alpha[n] = ex2(m_old - mn);
          ms.m[pi][n] = mn;
          ms.mo[pi][n] = kSigma - mn;
        }
        named_barrier(group_bar, 128);
        if (have_o) {
          mbar_wait_polls(bar(ms.pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort_flag, ptr.err);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int n = 0; n < 32; n += 4) {
            const uint32_t a = tmem + lane_addr + C::kColO + (n >> 4) * kN + cc + (n & 15);
            float v[4];
            tmem_ld4f(a, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= ms.alpha[cc + (n & 15) + i];
            tmem_st4f(a, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
      };

      // The block's last piece joins all of them: w_i = 2^(lse_i - M) / sum_j 2^(lse_j - M), M the
      // largest, out = v_descale sum_i w_i o_i. A warp takes whole rows, 16 bytes a lane.
      auto merge = [&](const Item& I, int pi) {
        const float* lse = slot_lse(cp, I.slot_base);
        const uint16_t* part = slot_o(cp, I.slot_base);
        auto store_row = [&](int r, const float (&acc)[8], float k) {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(ptr.out) + ms.out_off[pi][r] + lane * 8) =
              make_uint4(pack_bf16x2(acc[0] * k, acc[1] * k), pack_bf16x2(acc[2] * k, acc[3] * k),
                         pack_bf16x2(acc[4] * k, acc[5] * k), pack_bf16x2(acc[6] * k, acc[7] * k));
        };
        if (I.nsplit <= 4) {
          // few pieces: the loads of all of them, for two rows at a time
#pragma unroll 1
          for (int r = sw; r < I.nrows; r += 2 * kSoftWarps) {
            float w[2][4];
            uint4 h[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rb = min(r + b * kSoftWarps, I.nrows - 1);
                w[b][i] = i < I.nsplit ? __ldcg(lse + i * kN + rb) : -INFINITY;
                h[b][i] = i < I.nsplit ? __ldcg(reinterpret_cast<const uint4*>(part + (i * kN + rb) * kHeadDim) + lane) : make_uint4(0, 0, 0, 0);
              }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (r + b * kSoftWarps >= I.nrows) break;
              const float M = fmaxf(fmaxf(w[b][0], w[b][1]), fmaxf(w[b][2], w[b][3]));
              float sum = 0.f, acc[8] = {};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float wi = ex2(w[b][i] - M);
                sum += wi;
                merge_add(acc, h[b][i], wi);
              }
              store_row(r + b * kSoftWarps, acc, p.out_scale / sum);
            }
          }
        } else {
#pragma unroll 1
          for (int r = sw; r < I.nrows; r += kSoftWarps) {
            float acc[8];
            const float sum = merge_row<4>(lse + r, kN, part + r * kHeadDim, kN * kHeadDim, I.nsplit, lane, acc);
            store_row(r, acc, p.out_scale / sum);
          }
        }
      };

      auto epilogue = [&](int it) {
        const int ii = it - item_begin, pi = ii & 1;
        const Item I = load_item<kN, kFused>(p, cp, ptr, ms, it);
        mbar_wait_polls(bar(ms.o_ready), ii & 1, abort_flag, ptr.err);
        __syncwarp();
        tc_fence_after();
        // row sums over the 128 key lanes: warp reduce-scatter, then across the quarters
#pragma unroll
        for (int cb = 0; cb < kCols; cb += 16) {
          float v[16];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float2 x = unpack2(l[cb / 2 + n]);
            v[2 * n] = x.x;
            v[2 * n + 1] = x.y;
            l[cb / 2 + n] = 0;
          }
#pragma unroll
          for (int w = 8, o = 16; o >= 2; w >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < w; ++i) {
              const float send = up ? v[i] : v[i + w];
              const float keep = up ? v[i + w] : v[i];
              v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          }
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
          // lanes 2r and 2r + 1 now hold row c0 + cb + r
          if ((lane & 1) == 0) ms.red[q4][c0 + cb + (lane >> 1)] = v[0];
        }
        named_barrier(1, kSoftThreads);
        const bool split = I.nsplit > 1;
        const int slot = I.slot_base + I.split;
        // 1 / (row sum), times v_descale unless this is a split piece (the merge applies it then);
        // and a split piece's log2-sum-exp
        if (gi < kN) {
          const float lr = ms.red[0][gi] + ms.red[1][gi] + ms.red[2][gi] + ms.red[3][gi];
          ms.alpha[gi] = lr > 0.f ? __fdividef(split ? 1.f : p.out_scale, lr) : lr == 0.f ? 0.f : lr;  // NaN stays
          if (split) ms.lse_stage[gi] = lr > 0.f ? ms.m[pi][gi] - kSigma + log2f(lr) : lr == 0.f ? -INFINITY : lr;
        }
        named_barrier(1, kSoftThreads);  // (the next item's barrier keeps its rescales off red and alpha)
#pragma unroll 1
        for (int cb = 0; cb < kCols; cb += 16) {
          const int cc = c0 + cb;
          if (cc >= I.nrows) break;  // warp-uniform
          float v[16], w[16];
          tmem_ld16(tmem + lane_addr + C::kColO + cc, v);
          tmem_ld16(tmem + lane_addr + C::kColO + kN + cc, w);
          tmem_wait_ld();
          if (split) {
            uint32_t* stage = reinterpret_cast<uint32_t*>(smem + C::kOffP);  // rows of 128 f16 pairs
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float inv = ms.alpha[cc + i];
              stage[(cc + i) * (kHeadDim / 2) + ti] = pack_f16x2(v[i] * inv, w[i] * inv);
            }
          } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(ptr.out) + 2 * ti;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (cc + i < I.nrows) {
                const float inv = ms.alpha[cc + i];
                *reinterpret_cast<uint32_t*>(out + ms.out_off[pi][cc + i]) = pack_bf16x2(v[i] * inv, w[i] * inv);
              }
          }
        }
        tc_fence_before();
        mbar_arrive(bar(ms.o_free));
        if (split) {
          // The f16 partial and its log2-sum-exp leave through the P buffers (every P.V of the
          // item has completed) by two bulk stores from one thread, before the counter moves.
          fence_proxy_async_smem();
          named_barrier(1, kSoftThreads);
          if (gi == 0) {
            const unsigned long long seen = split_peek(cp.counters + I.block);
            bulk_store(slot_o(cp, slot), sbase + C::kOffP, (uint32_t)I.nrows * kHeadDim * 2u);
            bulk_store(slot_lse(cp, slot), smem_u32(ms.lse_stage), kN * 4u);
            bulk_commit();
            bulk_wait_all();  // the partial is in global memory before the split counter moves
            fence_proxy_async_global();
            fence_acq_rel_gpu();
            ms.merge_flag = split_arrive_from(cp.counters + I.block, seen, I.nsplit, ctag);
            fence_acq_rel_gpu();
          }
          named_barrier(1, kSoftThreads);  // the stage is reused by the next item's P; merge_flag
          if (ms.merge_flag) merge(I, pi);
        }
      };

      uint32_t g = 0;
      // Per step: Q of item `it` (while the last P.V of the item before it runs), the epilogue of
      // the item before it, the tiles of item `it`.
      for (int it = item_begin;; ++it) {
        const int ii = it - item_begin;
        if (it < item_end) q_prep(load_item<kN, kFused>(p, cp, ptr, ms, it), ii);
        if (it > item_begin) {
          epilogue(it - 1);
          if (it == item_end) break;
        }
        const int pi = ii & 1;
        named_barrier(1, kSoftThreads);  // q_prep's shared writes are visible
        int ntiles, key0, kv_hi, min_lim;
        int nc;  // of this thread's rows (the same in the row group's four warps), a multiple of 16
        {
          const Item I = load_item<kN, kFused>(p, cp, ptr, ms, it);
          ntiles = I.ntiles;
          key0 = I.tile_begin * kTileKeys;
          kv_hi = I.kv_hi;
          nc = min(((I.nrows + 15) & ~15) - c0, kCols);
          min_lim = I.L - I.qn + map_row(I.row0, p.G, I.kvh).t;
        }
        // A failed wait (timeout or abort) does not leave the loops: every later wait then
        // fails fast, so all softmax warps still pass the same barriers and finish.
        for (int j = 0; j < ntiles; ++j, ++g, key0 += kTileKeys) {
          const uint32_t sb = g % C::kSBufs, pb = g & 1;
          const int key = key0 + ti;
          const bool need_mask = (key0 + kTileKeys > kv_hi) || (key0 + kTileKeys - 1 > min_lim);
          mbar_wait_polls(bar(ms.s_full[sb]), (g / C::kSBufs) & 1, abort_flag, ptr.err);
          __syncwarp();  // the TMEM loads are warp-wide
          tc_fence_after();
#pragma unroll
          for (int cb = 0; cb < kCols; cb += 16) {
            const bool active = cb < nc;
            uint64_t x[8];
            if (active) {
              // At most two passes: the one after a new reference asks for no other. With 64 rows it
              // leaves before the vote, with 128 the limit of the vote is out of reach then (the other way
              // round 436 for 428 us and 2205 for 2125 us: registers).
              float limit = kTau + kSigma;
              bool moved = false;
#pragma unroll 1
              for (;;) {
                tmem_ld16(tmem + lane_addr + C::kColS + sb * kN + c0 + cb, x);
                tmem_wait_ld();
                // x = s c - m + sigma, the exponent of P, from the rounded product that new_reference
                // takes its maxima of: with m >= s c, x is at most rn(m + rn(sigma - m)) <= kTau + kSigma
                // whatever the size of m (sigma - m is off by up to 4 where m is about 2^26 and is -m
                // beyond), so P fits f16, and equal scores weigh the same in every tile. A product fused
                // with the sum would be off from m by up to half a step of it, 64 for scores of 2^30
                // (256 sequences: 424 us so, 428 with rounded ones). The compiler fuses mul.rn.f32x2
                // with add.rn.f32x2 (measured), but cannot fuse an fma whose zero it does not know.
#pragma unroll
                for (int n = 0; n < 16; n += 4) {
                  const ulonglong2 o4 = *reinterpret_cast<const ulonglong2*>(&ms.mo[pi][c0 + cb + n]);
                  const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(&ms.cs[pi][c0 + cb + n]);
                  x[n / 2] = add2(fma2(x[n / 2], s4.x, p.zero2), o4.x);
                  x[n / 2 + 1] = add2(fma2(x[n / 2 + 1], s4.y, p.zero2), o4.y);
                }
                if (need_mask) {
                  const int seen = key < kv_hi ? key : 0x7fffffff;
#pragma unroll
                  for (int n = 0; n < 16; n += 2) {
                    const int2 l2 = *reinterpret_cast<const int2*>(&ms.lim[pi][c0 + cb + n]);
                    const float2 v = unpack2(x[n / 2]);
                    x[n / 2] = pack2(seen <= l2.x ? v.x : -INFINITY, seen <= l2.y ? v.y : -INFINITY);
                  }
                }
                if (kN == 64 && moved) break;
                float xmax = -INFINITY;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                  const float2 v = unpack2(x[n]);
                  xmax = max3f(xmax, v.x, v.y);
                }
                // does any score of these 16 rows exceed its row's reference by more than 2^kTau?
                if (!barrier_or(group_bar, 128, xmax > (kN == 128 ? limit : kTau + kSigma))) break;
                new_reference(c0 + cb, pi, sb, j > 0, g, need_mask, key, kv_hi);
#pragma unroll
                for (int n = 0; n < 16; n += 2)
                  l[(cb + n) / 2] = mul2(l[(cb + n) / 2], *reinterpret_cast<const uint64_t*>(&ms.alpha[c0 + cb + n]));
                if (kN == 128) limit = INFINITY;
                else moved = true;
              }
            }
            if (cb + 16 == kCols) {  // S has been read for the last time
              tc_fence_before();
              mbar_arrive(bar(ms.s_free[sb]));
            }
            // P buffer g & 1 is free once P.V(g-2) has completed (the barrier's next phase needs a
            // P these threads have not written yet, so a late parity wait cannot miss it)
            if (cb == 0 && g >= 2) mbar_wait_polls(bar(ms.pv_done[pb]), ((g >> 1) - 1) & 1, abort_flag, ptr.err);
            if (active) {
              // P^T row of key ti (128-byte swizzle): 16 of this thread's rows
              const uint32_t row = sbase + C::kOffP + pb * C::kPBuf + (c0 >> 6) * C::kPBlock + ti * 128;
#pragma unroll
              for (int n = 0; n < 16; n += 8) {
                uint32_t pk[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 v = unpack2(x[n / 2 + k]);
                  const float e0 = ex2(v.x), e1 = ex2(v.y);
                  l[(cb + n) / 2 + k] = add2(l[(cb + n) / 2 + k], pack2(e0, e1));
                  pk[k] = pack_f16x2(e0, e1);
                }
                st_shared_v4(row + (((((c0 & 63) + cb + n) >> 3) ^ (ti & 7)) << 4), pk);
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(bar(ms.p_full[pb]));
        }
      }
    }  // !stalled
  } else if (wg >= kWideWarp0 / 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kWideRegs));
    // ------------------------------------------------------------ widening: packed tiles to TMEM
    const int q4 = warp & 3;
    const int ti = q4 * 32 + lane;  // TMEM lane
    const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
    // A failed wait (timeout or abort) does not leave the loops: the V warps share a barrier, and
    // every later wait then fails fast.
    // The warp is converged after a wait and after an arrival: the tcgen05.st that follow are
    // warp-wide instructions, and neither a poll's exit nor a one-lane arrival brings the lanes
    // together by itself.
    auto wait = [&](uint32_t b, uint32_t parity) {
      mbar_wait_polls(b, parity & 1, abort_flag, ptr.err);
      __syncwarp();
    };
    auto arrive = [&](uint32_t b) {
      mbar_arrive_warp(b, lane);
      __syncwarp();
    };
    // Before half h of tile g's K or V is written: its columns are free. Shared columns are used
    // in the order K(0) K(1) V(0) K(2) V(1) .. V(last): what was there last is K(0) before K(1), then
    // V(g - 2) before K(g), and K(g + 1), or V(g - 1) if g is the last tile, before V(g). Every
    // barrier here has one set of waiters that waits for its phases in turn, none of them more
    // than one ahead of the waiters (a parity wait cannot tell a phase from the one two before
    // it): so QK(0) arrives at ak_free for K(1), every later QK(g + 1) at av_go for V(g).
    auto k_cols_free = [&](uint32_t g, int h) {
      if (g < 1) return;
      if (!C::kShared || g == 1) wait(bar(ms.ak_free[0]) + 8 * h, g - 1);
      else wait(bar(ms.av_free[0]) + 8 * h, g);
    };
    auto v_cols_free = [&](uint32_t g, bool last, int h) {
      if (!C::kShared) {
        if (g >= 1) wait(bar(ms.av_free[0]) + 8 * h, g - 1);
      } else if (last && g >= 1) {
        wait(bar(ms.av_free[0]) + 8 * h, g - 1);
      } else {
        wait(bar(ms.av_go[0]) + 8 * h, g);
      }
    };
    auto publish = [&](uint32_t full) {
      tmem_wait_st();
      tc_fence_before();
      arrive(full);
    };
    // K of tile g: this thread's key, 64 d at a time (of both segments of a half, or of one)
    uint32_t kst = 0, kph = 0;  // stage and its phase
    const int kseg0 = C::kShared ? (warp - kWideWarp0) >> 2 : 0;  // of a half's two 64-d segments
    auto widen_k = [&](uint32_t g) {
      wait(bar(ms.k_full[0]) + 8 * kst, kph);
      const uint8_t* row = smem + C::kOffK + kst * kTile + ti * kFp4Row;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        k_cols_free(g, h);
        tc_fence_after();
#pragma unroll 1
        for (int seg = 2 * h + kseg0; seg < 2 * h + (C::kShared ? kseg0 + 1 : 2); ++seg) {
          const uint4* src = reinterpret_cast<const uint4*>(row + 32 * seg);
          const uint4 x[2] = {src[0], src[1]};
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(row + kFp4Codes + 4 * seg);
          const uint32_t dst = tmem + lane_addr + C::kColK + 32 * seg;
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // 32 values: two groups
            const uint32_t s2 = fp4::scales2(i ? sc >> 16 : sc);
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hh[4];
              fp4::codes4(w[k], hh);
#pragma unroll
              for (int b = 0; b < 4; ++b) o[4 * k + b] = k < 2 ? fp4::mul_f16x2_lo(hh[b], s2) : fp4::mul_f16x2_hi(hh[b], s2);
            }
            tmem_st16u(dst + 16 * i, o);
          }
        }
        publish(bar(ms.ak_full[0]) + 8 * h);
      }
      arrive(bar(ms.k_empty[0]) + 8 * kst);
      if (++kst == C::kKStages) {
        kst = 0;
        kph ^= 1;
      }
    };
    // V of tile g: code byte ti (d = 2 ti, 2 ti + 1) of keys 64 j + 32 half + [0, 32) of half j.
    // First these warps' threads widen the tile's scales once for all (8 bytes each), keys from
    // n_keys on (stale slots, or never copied) to zeros.
    uint32_t vst = 0, vph = 0;
    const int vt = (warp - C::kVWarp0) * 32 + lane;  // 0..255
    const int half = (vt >> 7) & 1;               // which 32 keys of a half tile
    auto widen_v = [&](uint32_t g, bool last, int n_keys) {
      wait(bar(ms.v_full[0]) + 8 * vst, vph);
      const uint8_t* tile = smem + C::kOffV + vst * kTile;
      uint8_t* scales = smem + C::kOffScale + (g & 1) * kScaleBuf;
      {
        const int blk = vt >> 5, grp = (vt & 31) >> 1, t8 = (vt & 1) * 8;
        uint2 w = *reinterpret_cast<const uint2*>(tile + blk * kFp4BlockBytes + kFp4BlockScales + grp * 16 + t8);
        if (n_keys < kTileKeys) {
          const int n = n_keys - blk * kFp4Block - t8;
          w.x &= token_mask(n, 0);
          w.y &= token_mask(n, 1);
        }
        uint4* dst = reinterpret_cast<uint4*>(scales + (blk * 16 + grp) * 64 + t8 * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = k ? w.y : w.x, e = x & 0x00ff00ffu, o = x & 0xff00ff00u;
          dst[k] = make_uint4(fp4::scales2(e), fp4::scales2(o), fp4::scales2(e >> 16), fp4::scales2(o >> 16));
        }
      }
      named_barrier(8, C::kVWarps * 32);
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        v_cols_free(g, last, j);
        tc_fence_after();
        const uint32_t dst = tmem + lane_addr + C::kColV + j * kChunkCols + 16 * half;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int blk = 4 * j + 2 * half + i;
          const uint4 x = *reinterpret_cast<const uint4*>(tile + blk * kFp4BlockBytes + ti * 16);
          const uint4* sc = reinterpret_cast<const uint4*>(scales + (blk * 16 + (ti >> 3)) * 64);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t lo[8], hi[8];  // tiles 0 and 1: key pairs
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hh[4];
            fp4::codes4(w[k], hh);
            const uint4 s = sc[k];
            fp4::pair_keys(hh[0], hh[1], s.x, s.y, lo[2 * k], hi[2 * k]);
            fp4::pair_keys(hh[2], hh[3], s.z, s.w, lo[2 * k + 1], hi[2 * k + 1]);
          }
          tmem_st8u(dst + 8 * i, lo);
          tmem_st8u(dst + 32 + 8 * i, hi);
        }
        publish(bar(ms.av_full[0]) + 8 * j);
      }
      arrive(bar(ms.v_empty[0]) + 8 * vst);
      if (++vst == C::kVStages) {
        vst = 0;
        vph ^= 1;
      }
    };
    // the CTA's tiles
    const bool is_k = warp < C::kVWarp0, is_v = warp >= C::kVWarp0;
    uint32_t g = 0;
    for (int it = item_begin; it < item_end; ++it) {
      const Item I = load_item<kN, kFused>(p, cp, ptr, ms, it);
      int left = I.kv_hi - I.tile_begin * kTileKeys;  // keys from tile j on that are there
#pragma unroll 1
      for (int j = 0; j < I.ntiles; ++j, ++g, left -= kTileKeys) {
        const bool last = it + 1 == item_end && j + 1 == I.ntiles;
        // one after the other: K a tile ahead
        const uint32_t k_end = C::kShared ? g + (last ? 1 : 2) : is_k ? g + 1 : g;
#pragma unroll 1
        for (uint32_t kg = C::kShared && g > 0 ? g + 1 : g; kg < k_end; ++kg) widen_k(kg);
        if (is_v) widen_v(g, last, left);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == 0 || warp == 1) {
      // ------------------------------------------------------------ MMA issuers
      // The whole warp walks the tiles and waits; one elected lane issues. With uniform control
      // flow the descriptors live in uniform registers, which tcgen05.mma takes: issued from a
      // one-lane loop, each instruction first moved its operands there. The lanes have to leave
      // every wait together for that (the vote): a suspended poll ends lane by lane, and uniform
      // registers belong to the warp, not to a part of it that runs ahead.
      auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_polls(b, parity & 1, abort_flag, ptr.err));
      };
      const bool is_s = warp == 0;
      const bool lead = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sm0 = __shfl_sync(0xffffffffu, sbase, 0);
      // B: Q (K-major, 64-d quarters) or P (MN-major: 64-row blocks kPBlock apart, 8-key groups
      // 1 KB apart, 16 keys or 2 KB per instruction)
      const uint64_t bdesc = is_s ? smem_desc(sm0 + C::kOffQ, 16, 1024, kSw128)
                                  : smem_desc(sm0 + C::kOffP, C::kPBlock, 1024, kSw128);
      uint32_t g = 0;
      int ii = 0;
      bool ok = true;
      for (int it = item_begin; it < item_end && ok; ++it, ++ii) {
        const Item I = load_item<kN, kFused>(p, cp, ptr, ms, it);
        const uint32_t n16 = (uint32_t)(__shfl_sync(0xffffffffu, I.nrows, 0) + 15) & ~15u;
        const int ntiles = __shfl_sync(0xffffffffu, I.ntiles, 0);
        const uint32_t idesc = idesc_f16(128, 0, false, !is_s) | (n16 >> 3 << 17);
        for (int j = 0; j < ntiles; ++j, ++g) {
          if (is_s) {
            const uint32_t sb = g % C::kSBufs, su = g / C::kSBufs;
            const bool last = it + 1 == item_end && j + 1 == ntiles;
            if (j == 0 && !(ok = wait(bar(ms.q_full), ii))) break;
            if (su >= 1 && !(ok = wait(bar(ms.s_free[sb]), su - 1))) break;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!(ok = wait(bar(ms.ak_full[0]) + 8 * h, g))) break;
              tc_fence_after();
              if (lead) {
                const uint32_t a = tm + C::kColK + h * kChunkCols, d = tm + C::kColS + sb * kN;
                const uint64_t q = bdesc + ((2 * h * C::kQQuarter) >> 4);
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 d (8 columns of A) per instruction
                  mma_f16_ts(d, a + i * 8, q + (((i >> 2) * C::kQQuarter + (i & 3) * 32) >> 4), idesc, (h | i) ? 1u : 0u);
                mma_commit((!C::kShared || (g == 0 && !last) ? bar(ms.ak_free[0]) : bar(ms.av_go[0])) + 8 * h);
                if (h == 1) {
                  mma_commit(bar(ms.s_full[sb]));
                  if (j == ntiles - 1) mma_commit(bar(ms.q_free));
                }
              }
              __syncwarp();
            }
          } else {
            // the first P.V of an item overwrites O^T: the previous epilogue must be done
            if (j == 0 && ii >= 1 && !(ok = wait(bar(ms.o_free), ii - 1))) break;
            if (!(ok = wait(bar(ms.p_full[g & 1]), g >> 1))) break;
#pragma unroll 1
            for (int c64 = 0; c64 < 2; ++c64) {
              if (!(ok = wait(bar(ms.av_full[0]) + 8 * c64, g))) break;
              tc_fence_after();
              if (lead) {
                const uint32_t a = tm + C::kColV + c64 * kChunkCols, d = tm + C::kColO;
                const uint64_t pd = bdesc + (((g & 1) * C::kPBuf + c64 * 8192) >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    mma_f16_ts(d + h * kN, a + h * 32 + kk * 8, pd + ((kk * 2048) >> 4), idesc,
                               (j == 0 && c64 == 0 && kk == 0) ? 0u : 1u);
                mma_commit(bar(ms.av_free[0]) + 8 * c64);
                if (c64 == 1) {
                  mma_commit(bar(ms.pv_done[g & 1]));
                  if (j == ntiles - 1) mma_commit(bar(ms.o_ready));
                }
              }
              __syncwarp();
            }
          }
          if (!ok) break;
        }
      }
      // Every MMA this warp's leader issued has completed before the CTA may release TMEM.
      if (lead) {
        uint64_t& drain = is_s ? ms.drain[0] : ms.drain[1];
        mma_commit(bar(drain));
        mbar_drain(bar(drain), 0, abort_flag, ptr.err);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ bulk copies of pages
      // One warp for K, one for V; lane i copies page i of a tile (up to 8 pages).
      const bool is_k = warp == 2;
      const uint32_t nst = is_k ? C::kKStages : C::kVStages;
      const uint32_t region = sbase + (is_k ? C::kOffK : C::kOffV);
      uint64_t* full = is_k ? ms.k_full : ms.v_full;
      uint64_t* empty = is_k ? ms.k_empty : ms.v_empty;
      const uint8_t* cache = static_cast<const uint8_t*>(is_k ? ptr.k : ptr.v);
      const long long sb = is_k ? p.k_sb : p.v_sb, sh = is_k ? p.k_sh : p.v_sh;
      // verify: every page is read once; prefill: the row blocks of a sequence read it again
      const uint64_t policy = kN == 64 ? policy_evict_first() : policy_evict_last();
      const int ppt = kTileKeys / p.P;  // pages per tile (1, 2, 4 or 8)
      uint32_t g = 0;
      bool ok = true;
      for (int it = item_begin; it < item_end && ok; ++it) {
        const Item I = load_item<kN, kFused>(p, cp, ptr, ms, it);
        const int32_t* bt_row = ptr.block_table + (size_t)I.seq * p.bt_stride;
        const uint8_t* head = cache + (long long)I.kvh * sh;
        int left = I.kv_hi - I.tile_begin * kTileKeys - lane * p.P;  // keys from this lane's page on
        if (lane >= ppt) left = 0;
        // a window of 32 block-table entries, one per lane, and the next one in flight; an index
        // past the row is clamped, and such an entry is not used
        int at = I.tile_begin * ppt + lane;
        int cur = bt_row[min(at, p.W - 1)], next = bt_row[min(at + 32, p.W - 1)];
        int first = 0;  // of the tile's pages in the window
        if (is_k) {
          // the softmax warps read this item's Q soon: bring its rows into L2
          for (int r = lane; r < I.nrows; r += 32) {
            const RowMap m = map_row(I.row0 + r, p.G, I.kvh);
            const uint8_t* row = static_cast<const uint8_t*>(ptr.q) + ((long long)(I.q0 + m.t) * p.q_st + (long long)m.h * p.q_sh) * 2;
#pragma unroll
            for (int c = 0; c < 512; c += 128) prefetch_l2(row + c);
          }
        }
#pragma unroll 1
        for (int j = 0; j < I.ntiles; ++j, ++g) {
          int blk = __shfl_sync(0xffffffffu, cur, (first + lane) & 31);
          first += ppt;
          if (first == 32) {
            first = 0;
            at += 32;
            cur = next;
            next = bt_row[min(at + 32, p.W - 1)];
          }
          // tokens to copy: all of a page, but of the piece's last one the 16-token blocks with keys
          const int tokens = min(p.P, (left + kFp4Block - 1) & ~(kFp4Block - 1));
          const uint32_t st = g % nst;
          if (lane == 0) {
            // what all lanes copy: the tile's keys, rounded up to whole blocks
            const uint32_t bytes = (uint32_t)min(kTileKeys, (left + kFp4Block - 1) & ~(kFp4Block - 1)) * kFp4Row;
            ok = mbar_wait_polls(bar(empty[st]), ((g / nst) & 1) ^ 1, abort_flag, ptr.err);
            if (ok) mbar_expect_tx(bar(full[st]), bytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          __syncwarp();  // the other lanes' copies come after lane 0's wait
          if (tokens > 0) {
            if (blk < 0 || blk >= p.NB) {
              atomicOr(ptr.err, kErrPage);
              blk = 0;
            }
            bulk_load_hint(region + st * kTile + (uint32_t)(lane * p.P) * kFp4Row, head + (long long)blk * sb,
                           (uint32_t)tokens * kFp4Row, bar(full[st]), policy);
          }
          left -= lane < ppt ? kTileKeys : 0;
        }
      }
      // Every issued copy has landed before the CTA may exit.
      if (lane == 0) {
        for (uint32_t t = g > nst ? g - nst : 0; t < g; ++t)  // the last tile of each stage
          mbar_drain(bar(full[t % nst]), (t / nst) & 1, abort_flag, ptr.err);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

template <int kN, bool kFused>
int launch(const Problem& p, const Pointers& ptr, const ClassPlan& cp, cudaStream_t stream, bool dependent) {
  auto kern = fp4_tc_kernel<kN, kFused>;
  constexpr size_t smem = smem_bytes<kN, kFused>();
  static bool done[64] = {};  // one per instance of this template
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
      char buf[160];
      snprintf(buf, sizeof buf, "cudaFuncSetAttribute(4-bit attention): %s", cudaGetErrorString(e));
      set_tc_error(buf);
      return -1;
    }
    // setmaxnreg.inc waits until the registers it asks for are free; the split adds up only
    // if the kernel starts with exactly kLaunchRegs registers per thread, so never launch otherwise.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess || fa.numRegs != Cfg<kN>::kLaunchRegs) {
      char buf[160];
      snprintf(buf, sizeof buf, "4-bit attention kernel built with %d registers per thread; its warpgroup split needs %d",
               e == cudaSuccess ? fa.numRegs : -1, Cfg<kN>::kLaunchRegs);
      set_tc_error(buf);
      return -1;
    }
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  e = launch_pdl(dependent, kern, cp.num_ctas, Cfg<kN>::kThreads, smem, stream, p, ptr, cp);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    char buf[160];
    snprintf(buf, sizeof buf, "4-bit attention kernel launch: %s", cudaGetErrorString(e));
    set_tc_error(buf);
    return -1;
  }
  return 1;
}

}  // namespace

int launch_fp4_tc(const Problem& p, const Pointers& ptr, const ClassPlan& cp, int cls, cudaStream_t stream,
                  bool dependent) {
  if (cls == 1) return launch<128, false>(p, ptr, cp, stream, dependent);
  return p.fused_verify ? launch<64, true>(p, ptr, cp, stream, dependent) : launch<64, false>(p, ptr, cp, stream, dependent);
}

}  // namespace pgqa
