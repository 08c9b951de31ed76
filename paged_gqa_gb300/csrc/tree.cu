// tree.cu -- what surrounds the attention of a token tree: the tokens' masks and positions from
// their parents, and the accepted tokens' K and V into their final places in the cache.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "step.cuh"

namespace pgqa {

// A CTA per sequence, a thread per token: token t's mask holds the tokens of its path, t itself
// among them, and its position is the context's length plus its depth. The parents lie in shared
// memory; a token climbs to the context by itself (one shared load a step, no synchronisation),
// and since parents come before their children it meets the words of its mask from the last to
// the first, so a word is written once and the mask needs no storage. Bound by latency: 7 trees of 13 tokens take
// 2.1 us from a graph, 256 of 64 tokens 3.4 (0.3 MB); a call from Python 8 us.
__global__ void __launch_bounds__(32 * kMaxMaskWords) tree_mask_kernel(TreeMaskArgs a) {
  __shared__ int par[32 * kMaxMaskWords];
  const int s = blockIdx.x, t = threadIdx.x;
  const int q0 = a.qsl[s], q1 = a.qsl[s + 1], qn = q1 - q0, L = a.seq_lens[s];
  if (q0 < 0 || q1 < q0 || q1 > a.T || qn > L || qn > 32 * a.words) {
    if (t == 0) atomicOr(a.err, kErrBounds);
    for (int i = max(q0, 0) + t; i < min(q1, a.T); i += blockDim.x) {
      for (int w = 0; w < a.words; ++w) a.masks[(long long)i * a.masks_st + w] = 0;
      for (int x = 0; x < a.axes; ++x) a.positions[x * a.positions_sa + i] = 0;
    }
    return;
  }
  if (t < qn) {
    int p = a.parents[q0 + t];
    if (p < -1 || p >= t) {
      atomicOr(a.err, kErrBounds);
      p = -1;
    }
    par[t] = p;
  }
  __syncthreads();
  if (t >= qn) return;
  int32_t* row = a.masks + (long long)(q0 + t) * a.masks_st;
  int word = a.words - 1, depth = -1;
  uint32_t bits = 0;
  for (int at = t; at >= 0; at = par[at]) {
    while (word > (at >> 5)) {
      row[word--] = (int32_t)bits;
      bits = 0;
    }
    bits |= 1u << (at & 31);
    ++depth;
  }
  while (word >= 0) {
    row[word--] = (int32_t)bits;
    bits = 0;
  }
  for (int x = 0; x < a.axes; ++x) a.positions[x * a.positions_sa + q0 + t] = L - qn + depth;
}

cudaError_t launch_tree_masks(const TreeMaskArgs& a, cudaStream_t stream) {
  tree_mask_kernel<<<a.S, 32 * a.words, 0, stream>>>(a);
  return cudaGetLastError();
}

namespace {
constexpr int kKeepWarps = 4;
constexpr int kKeepRows = 8;  // rows in flight
}  // namespace

// A warp per (sequence, kv head, K or V). Kept token k moves from position ctx + kept[k] to ctx + k;
// kept is increasing, so a place is never written before it has been read (k' < k <= kept[k] for
// every earlier destination k'), and since a lane moves the same bytes of every row, its own
// program order is all the order that takes. Piece: a lane's 16 bytes of a bf16 row, 8 of an e4m3 one. Bound by latency
// (lengths, the kept list, two page ids, the rows): 5 sequences take 3.7 us from a graph, 256 with up to 7 kept tokens
// and 2 heads 3.0.
template <typename Piece>
__global__ void __launch_bounds__(kKeepWarps * 32) cache_keep_kernel(KeepArgs a) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kKeepWarps + (threadIdx.x >> 5);
  const long long per_seq = 2LL * a.Hkv;
  if (unit >= a.S * per_seq) return;
  const int s = (int)(unit / per_seq), part = (int)(unit - s * per_seq);
  const int which = part & 1, head = part >> 1;
  const int q0 = a.qsl[s], q1 = a.qsl[s + 1], qn = q1 - q0, L = a.seq_lens[s], n = a.num_kept[s];
  const bool first = part == 0 && lane == 0;
  if (q0 < 0 || q1 < q0 || qn > L || (long long)L > (long long)a.W * a.P) {
    if (first) {
      atomicOr(a.err, kErrBounds);
      a.lens_out[s] = L;
    }
    return;
  }
  const int ctx = L - qn;
  const int32_t* kept = a.kept + (long long)s * a.kept_st;
  bool bad = n < 0 || n > a.D || n > qn;
  if (!bad)
    for (int k = lane; k < n; k += 32) bad |= kept[k] >= qn || kept[k] <= (k ? kept[k - 1] : -1);
  bad = __any_sync(0xffffffffu, bad);
  if (first) {
    if (bad) atomicOr(a.err, kErrBounds);
    a.lens_out[s] = ctx + (bad ? 0 : n);
  }
  if (bad) return;
  uint8_t* cache = a.cache[which] + (long long)head * a.sh[which] + lane * sizeof(Piece);
  const int32_t* bt = a.bt + (long long)s * a.bt_stride;
  for (int k0 = 0; k0 < n; k0 += 32) {
    // lane i: the places of kept token k0 + i (-1: nothing to move)
    long long src = -1, dst = -1;
    const int k = k0 + lane;
    if (k < n && kept[k] != k) {
      const int from = ctx + kept[k], to = ctx + k;
      const int pf = bt[from >> a.p_shift], pt = bt[to >> a.p_shift];
      if (pf < 0 || pf >= a.NB || pt < 0 || pt >= a.NB) {
        atomicOr(a.err, kErrPage);
      } else {
        src = pf * a.sb[which] + (from & (a.P - 1)) * a.sp[which];
        dst = pt * a.sb[which] + (to & (a.P - 1)) * a.sp[which];
      }
    }
    for (int i0 = 0; i0 < 32 && k0 + i0 < n; i0 += kKeepRows) {
      Piece x[kKeepRows];
#pragma unroll
      for (int i = 0; i < kKeepRows; ++i) {
        const long long o = __shfl_sync(0xffffffffu, src, i0 + i);
        if (o >= 0) x[i] = *reinterpret_cast<const Piece*>(cache + o);
      }
#pragma unroll
      for (int i = 0; i < kKeepRows; ++i) {
        const long long o = __shfl_sync(0xffffffffu, dst, i0 + i);
        if (o >= 0) *reinterpret_cast<Piece*>(cache + o) = x[i];
      }
    }
  }
}

cudaError_t launch_cache_keep(const KeepArgs& a, cudaStream_t stream) {
  const long long units = 2LL * a.S * a.Hkv;
  const int grid = (int)((units + kKeepWarps - 1) / kKeepWarps);
  if (a.row_bytes == 512) cache_keep_kernel<uint4><<<grid, kKeepWarps * 32, 0, stream>>>(a);
  else cache_keep_kernel<uint2><<<grid, kKeepWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pgqa
