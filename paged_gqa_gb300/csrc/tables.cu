// tables.cu -- block tables, slot maps and the page pool behind them, from request lengths.
//
// A request s with q new tokens on ctx cached ones holds L = ctx + q tokens and needs
// ceil(L / P) pages. The pages it already holds are the first page_counts[row] entries of its
// row of the pool; what is missing comes from the top of a stack of free pages, what ended
// requests held goes onto it first. With t_s = max(0, need_s - held_s) and r_s = sum of t over
// the requests before s, page i of the t_s new ones is free[avail - 1 - (r_s + i)]: every
// request finds its pages by a prefix sum, and the answer does not depend on any order of
// execution. query_start_loc is the prefix sum of the new tokens, the slot of a token at
// position p is page * P + p % P.
//
// Two launches. The first, one CTA, does what needs every request: the prefix sums, the pages
// given back and taken, the counts. The second copies the pool's rows into the batch's block
// table and writes the slots, over as many CTAs as there are table rows; it is the one that
// moves bytes (4 W per request), and starts as a programmatic dependent.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "step.cuh"
#include "tc_kernels.cuh"

namespace pgqa {

namespace {

constexpr int kPoolThreads = 1024;
constexpr int kFillThreads = 128;
constexpr int kSegment = 512;  // table columns per CTA of the second launch: four per thread

// Exclusive block-wide prefix sums of two values; *ta and *tb get the sums.
__device__ void scan2(long long& a, long long& b, long long* ta, long long* tb) {
  __shared__ long long sa[32], sb[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sa[warp] = a;
    sb[warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    long long x = sa[lane], y = sb[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    sa[lane] = x;
    sb[lane] = y;
  }
  __syncthreads();
  a += (warp ? sa[warp - 1] : 0) - a0;
  b += (warp ? sb[warp - 1] : 0) - b0;
  *ta = sa[31];
  *tb = sb[31];
  __syncthreads();  // sa and sb may be written again
}

// Calls f(lane's value of x, i) for i < n of every lane in turn, the lanes of the warp sharing the i.
template <typename F>
__device__ __forceinline__ void warp_each(int n, F f) {
  unsigned todo = __ballot_sync(0xffffffffu, n > 0);
  while (todo) {
    const int j = __ffs(todo) - 1;
    todo &= todo - 1;
    f(j, __shfl_sync(0xffffffffu, n, j));
  }
}

}  // namespace

// Every thread serves the same requests in each phase. A request's held pages are kept in its
// entry of seq_lens in between (-1: flagged), since page_counts may be page_counts_out.
__global__ void __launch_bounds__(kPoolThreads, 1) pool_kernel(TableArgs a) {
  const int tid = threadIdx.x, lane = tid & 31;
  __shared__ int s_flag, s_free, s_given, s_taken;
  if (tid == 0) {
    s_flag = s_given = s_taken = 0;
    int nf = *a.num_free;
    if (nf < 0 || nf > a.F) {  // no such stack: nothing can be given back or taken
      s_flag = 1;
      nf = nf < 0 ? 0 : a.F;
    }
    s_free = nf;
  }
  // 1. the rows' counts; a request whose row or lengths cannot be is flagged
  for (int s = tid; s < a.S; s += kPoolThreads) {
    const int row = a.rows[s];
    int held = 0;
    if (row >= 0 && row < a.R) {
      held = a.counts[row];
      if (held < 0 || held > a.Wp) held = -1;
    } else if (row != -1) {
      held = -1;
    }
    a.seq_lens[s] = held;
  }
  if (a.counts_out != a.counts)
    for (int r = tid; r < a.R; r += kPoolThreads) a.counts_out[r] = a.counts[r];
  __syncthreads();
  // 2. a row that two requests name belongs to the first of them: each puts its number there, the
  // largest of INT_MAX - s stays
  for (int s = tid; s < a.S; s += kPoolThreads)
    if (a.rows[s] >= 0 && a.seq_lens[s] >= 0) atomicMax(a.counts_out + a.rows[s], INT_MAX - s);
  __syncthreads();
  for (int s = tid; s < a.S; s += kPoolThreads)
    if (a.rows[s] >= 0 && a.seq_lens[s] >= 0 &&
        *const_cast<volatile int*>(a.counts_out + a.rows[s]) != INT_MAX - s)
      a.seq_lens[s] = -1;
  __syncthreads();
  // 3. ended requests give their pages back, on top of the stack, in the batch's order
  long long base = 0;
  const int nf = s_free;
  for (int s0 = 0; s0 < a.S; s0 += kPoolThreads) {
    const int s = s0 + tid;
    int n = 0, row = -1;
    bool mine = false;
    if (s < a.S && a.rows[s] >= 0 && a.seq_lens[s] >= 0) {
      row = a.rows[s];
      mine = a.q_lens[s] == -1;
      n = mine ? a.seq_lens[s] : 0;
    }
    long long off = n, none = 0, total, total2;
    scan2(off, none, &total, &total2);
    off += base + nf;
    const bool fits = off + n <= a.F;
    if (mine) {
      a.counts_out[row] = fits ? 0 : n;
      if (!fits) s_flag = 1;
    }
    if (!fits) n = 0;
    if (n) atomicMax(&s_given, (int)(off + n) - nf);
    warp_each(n, [&](int j, int nj) {
      const int rj = __shfl_sync(0xffffffffu, row, j);
      const int to = (int)__shfl_sync(0xffffffffu, off, j);
      for (int i = lane; i < nj; i += 32) a.free_pages[to + i] = a.pages[(long long)rj * a.pages_st + i];
    });
    base += total;
  }
  __syncthreads();
  // 4. the others take theirs; the first token of each
  const int avail = nf + s_given;
  long long tokens = 0;
  base = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPoolThreads) {
    const int s = s0 + tid;
    int q = 0, row = -1, held = 0, take = 0;
    long long L = 0;
    bool ok = false;
    if (s < a.S) {
      const int given = a.q_lens[s];
      row = a.rows[s];
      held = a.seq_lens[s];
      if (row == -1) {
        if (given > 0) s_flag = 1;  // tokens of no request
      } else {
        q = max(given, 0);
        if (given < -1 || held < 0) {
          s_flag = 1;
        } else if (given >= 0) {
          const int ctx = a.ctx_lens[s];
          L = (long long)ctx + q;
          const long long need = (L + a.P - 1) >> a.p_shift;
          ok = ctx >= 0 && L <= INT_MAX && need <= min(a.W, a.Wp);
          if (ok) take = max(0, (int)need - held);
        }
      }
    }
    long long first = take, tok = q, total, total_q;
    scan2(first, tok, &total, &total_q);
    first += base;
    tok += tokens;
    const bool mine = s < a.S && row >= 0 && held >= 0 && a.q_lens[s] != -1;  // its entry holds the mark of step 2
    if (take && first + take > avail) {  // out of pages: this request, and those behind it that need some
      take = 0;
      ok = false;
    }
    if (mine) {
      if (!ok) s_flag = 1;
      a.counts_out[row] = held + take;
    }
    if (take) atomicMax(&s_taken, (int)(first + take));
    if (s < a.S) {
      a.seq_lens[s] = ok ? (int)L : 0;
      a.qsl[s + 1] = (int)min(tok + q, (long long)INT_MAX);
    }
    warp_each(take, [&](int j, int nj) {
      const int rj = __shfl_sync(0xffffffffu, row, j), hj = __shfl_sync(0xffffffffu, held, j);
      const int from = avail - 1 - (int)__shfl_sync(0xffffffffu, first, j);
      for (int i = lane; i < nj; i += 32) a.pages[(long long)rj * a.pages_st + hj + i] = a.free_pages[from - i];
    });
    base += total;
    tokens += total_q;
  }
  __syncthreads();
  if (tid == 0) {
    a.qsl[0] = 0;
    *a.num_free_out = avail - s_taken;
    if (s_flag || tokens > a.T) atomicOr(a.err, kErrBounds);
  }
}

// CTA (s, segment): kSegment columns of the request's table row and, of its tokens, every
// (number of segments)-th run of kFillThreads; the tokens behind the last request's get -1.
__global__ void __launch_bounds__(kFillThreads) table_fill_kernel(TableArgs a, int segments) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int s = blockIdx.x / segments, seg = blockIdx.x - s * segments;
  const int L = a.seq_lens[s], row = a.rows[s];
  const int need = (int)(((long long)L + a.P - 1) >> a.p_shift);
  const int32_t* src = a.pages + (long long)(row < 0 ? 0 : row) * a.pages_st;
  int32_t* dst = a.table + (long long)s * a.table_st;
#pragma unroll
  for (int i = 0; i < kSegment / kFillThreads; ++i) {
    const int c = seg * kSegment + i * kFillThreads + tid;
    if (c < a.W) dst[c] = c < need ? src[c] : -1;
  }
  const int t0 = a.qsl[s], t1 = min(a.qsl[s + 1], a.T);
  const int n = a.qsl[s + 1] - t0, ctx = L - n;
  for (int t = t0 + seg * kFillThreads + tid; t < t1; t += segments * kFillThreads) {
    int slot = -1;
    if (L > 0) {
      const int pos = ctx + t - t0;
      const int page = src[pos >> a.p_shift];
      const long long x = (long long)page * a.P + (pos & (a.P - 1));
      if (page >= 0 && x <= INT_MAX) slot = (int)x;
      else atomicOr(a.err, kErrPage);
    }
    a.slots[t] = slot;
  }
  if (s == a.S - 1)
    for (int t = max(0, a.qsl[a.S]) + seg * kFillThreads + tid; t < a.T; t += segments * kFillThreads) a.slots[t] = -1;
}

cudaError_t launch_build_tables(const TableArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_pdl(false, pool_kernel, 1, kPoolThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
  if (a.S == 0) return a.T > 0 ? cudaMemsetAsync(a.slots, 0xff, sizeof(int32_t) * (size_t)a.T, stream) : cudaGetLastError();
  const int segments = a.W > 0 ? (a.W + kSegment - 1) / kSegment : 1;
  e = launch_pdl(true, table_fill_kernel, a.S * segments, kFillThreads, 0, stream, a, segments);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pgqa
