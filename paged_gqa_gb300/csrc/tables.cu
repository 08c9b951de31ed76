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
// Two launches. The first, one CTA, does what needs every request: who has which row, the prefix sums,
// the pages given back and taken, the counts. It is a chain of dependent reads, so a thread keeps what it has
// read of its requests in registers, rows are told apart by a hash table in shared memory, one scan carries
// all three sums, and what is copied in bulk is shared out over the warps. The second copies the pool's
// rows into the batch's block table and writes the slots, over as many CTAs as there are table rows; it is the
// one that moves bytes (4 W per request), and is resident before the first one ends.
//
// Bound by latency and by the host: 250 requests of up to 2080 columns take 7.5 us from a graph (2.1 MB; 0.5 us at the
// copy rate) and 17 as a call from Python (13 tensors described, two launches); 1500 requests of 160 columns, 41 of them
// new with up to 64 pages each, 15.4 and 17. With the first launch written plainly (three scans, rows told apart in global
// memory, each thread copying its own pages) the 250 requests took 17 us from a graph.
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
static_assert(kMaxRequests % kPoolThreads == 0, "requests per thread of the first launch");

struct Sums {
  long long given, taken, tokens;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return Sums{a.given + b.given, a.taken + b.taken, a.tokens + b.tokens};
}
__device__ __forceinline__ Sums shfl_up(Sums a, int o) {
  return Sums{__shfl_up_sync(0xffffffffu, a.given, o), __shfl_up_sync(0xffffffffu, a.taken, o),
              __shfl_up_sync(0xffffffffu, a.tokens, o)};
}
// Block-wide exclusive prefix sums; *all gets the sums.
__device__ __forceinline__ Sums scan(Sums v, Sums* warps, Sums* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = shfl_up(x, o);
    if (lane >= o) x = x + y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sums w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = shfl_up(w, o);
      if (lane >= o) w = w + y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  *all = warps[31];
  const Sums before = warp ? warps[warp - 1] : Sums{0, 0, 0};
  return Sums{before.given + x.given - v.given, before.taken + x.taken - v.taken, before.tokens + x.tokens - v.tokens};
}

// Copies of page ids between a row of the pool and the stack. A few are made by the request's own thread;
// longer ones become jobs of kJob ids, which the warps share.
constexpr int kFew = 4, kJob = 256, kMaxJobs = 1024;
struct Job {
  int row, at, n, stack;  // ids pages[row][at ..), stack[stack ..) upwards (back) or downwards (taken)
};
struct Jobs {
  int count;
  Job job[kMaxJobs];
};
__device__ __forceinline__ void copy_ids(const TableArgs& a, const Job& j, bool back, int from, int step) {
  int32_t* row = a.pages + (long long)j.row * a.pages_st + j.at;
  for (int i0 = from; i0 < j.n; i0 += step * 8) {
    int32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * step;
      if (i < j.n) v[k] = back ? row[i] : a.free_pages[j.stack - i];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * step;
      if (i < j.n) {
        if (back) a.free_pages[j.stack + i] = v[k];
        else row[i] = v[k];
      }
    }
  }
}
__device__ __forceinline__ void copy_or_queue(const TableArgs& a, Jobs& jobs, const Job& j, bool back) {
  if (j.n <= kFew) {
    copy_ids(a, j, back, 0, 1);
    return;
  }
  for (int i = 0; i < j.n; i += kJob) {
    const Job part = {j.row, j.at + i, min(kJob, j.n - i), back ? j.stack + i : j.stack - i};
    const int at = atomicAdd(&jobs.count, 1);
    if (at < kMaxJobs) jobs.job[at] = part;
    else copy_ids(a, part, back, 0, 1);
  }
}
__device__ __forceinline__ void do_jobs(const TableArgs& a, const Jobs& jobs, bool back) {
  const int n = min(jobs.count, kMaxJobs);
  for (int i = threadIdx.x >> 5; i < n; i += kPoolThreads / 32) copy_ids(a, jobs.job[i], back, threadIdx.x & 31, 32);
}

struct PoolSmem {
  Sums warps[32];
  int flag, given, taken;
  Jobs back, take;
};

}  // namespace

// Thread t serves `per` requests from t * per on, at most kPer. `slots`: entries of the hash table, a power of two,
// twice the requests at least.
template <int kPer>
__global__ void __launch_bounds__(kPoolThreads, 1) pool_kernel(TableArgs a, int per, int slots) {
  extern __shared__ __align__(16) unsigned char pool_smem[];
  PoolSmem& sm = *reinterpret_cast<PoolSmem*>(pool_smem);
  int* key = reinterpret_cast<int*>(&sm + 1);  // row of the pool (-1: none yet)
  int* owner = key + slots;                    // the first request that names it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (tid == 0) sm.flag = sm.given = sm.taken = sm.back.count = sm.take.count = 0;
  int nf = *a.num_free;
  int row[kPer], q[kPer], ctx[kPer], held[kPer];  // held: -1 where the request cannot be served
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid * per + i;
    const bool there = i < per && s < a.S;
    row[i] = there ? a.rows[s] : -1;
    q[i] = there ? a.q_lens[s] : 0;
    ctx[i] = there ? a.ctx_lens[s] : 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) held[i] = row[i] >= 0 && row[i] < a.R ? a.counts[row[i]] : row[i] == -1 ? 0 : -1;
  if (a.counts_out != a.counts)
    for (int r = tid; r < a.R; r += kPoolThreads) a.counts_out[r] = a.counts[r];
  for (int i = tid; i < slots; i += kPoolThreads) {
    key[i] = -1;
    owner[i] = INT_MAX;
  }
  __syncthreads();
  // a row that two requests name belongs to the first of them
  bool flag = false;
  int slot[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (held[i] > a.Wp || held[i] < 0) held[i] = -1;
    slot[i] = -1;
    if (row[i] < 0 || held[i] < 0) continue;
    int h = (int)(((unsigned)row[i] * 2654435761u) >> 8) & (slots - 1);
    for (;;) {  // (at most half of the table is taken)
      const int k = atomicCAS(key + h, -1, row[i]);
      if (k == -1 || k == row[i]) break;
      h = (h + 1) & (slots - 1);
    }
    atomicMin(owner + h, tid * per + i);
    slot[i] = h;
  }
  __syncthreads();
  if (nf < 0 || nf > a.F) {  // no such stack: taken as the nearer end
    flag = true;
    nf = nf < 0 ? 0 : a.F;
  }
  // what each request gives, needs and brings
  Sums mine = {0, 0, 0};
  int take[kPer], give[kPer], ok[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (slot[i] >= 0 && owner[slot[i]] != tid * per + i) held[i] = -1;
    take[i] = give[i] = ok[i] = 0;
    if (row[i] == -1) {
      flag |= q[i] > 0;  // tokens of no request
      q[i] = 0;
      continue;
    }
    flag |= held[i] < 0 || q[i] < -1;
    if (held[i] >= 0 && q[i] == -1) {
      give[i] = held[i];
    } else if (held[i] >= 0 && q[i] >= 0) {
      const long long L = (long long)ctx[i] + q[i], need = (L + a.P - 1) >> a.p_shift;
      ok[i] = ctx[i] >= 0 && L <= INT_MAX && need <= min(a.W, a.Wp);
      if (ok[i]) take[i] = max(0, (int)need - held[i]);
    }
    mine = mine + Sums{give[i], take[i], max(q[i], 0)};
  }
  Sums all;
  const Sums start = scan(mine, sm.warps, &all);
  // ended requests give their pages back, on top of the stack
  Sums at = start;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long to = nf + at.given;
    at.given += give[i];
    if (row[i] >= 0 && held[i] >= 0 && q[i] == -1) {
      const bool fits = to + give[i] <= a.F;
      if (fits && give[i]) {
        atomicMax(&sm.given, (int)(to + give[i]) - nf);
        copy_or_queue(a, sm.back, Job{row[i], 0, give[i], (int)to}, true);
      }
      flag |= !fits;
      a.counts_out[row[i]] = fits ? 0 : held[i];
    }
  }
  __syncthreads();
  do_jobs(a, sm.back, true);
  __syncthreads();
  // the others take theirs from the top
  const int avail = nf + sm.given;
  at = start;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid * per + i;
    if (i >= per || s >= a.S) break;
    const long long first = at.taken;
    at.taken += take[i];
    at.tokens += max(q[i], 0);
    if (take[i] && first + take[i] > avail) {  // out of pages: this request, and those behind it that need some
      take[i] = 0;
      ok[i] = 0;
    }
    if (row[i] >= 0 && held[i] >= 0 && q[i] >= 0) {
      flag |= !ok[i];
      a.counts_out[row[i]] = held[i] + take[i];
    }
    if (take[i]) {
      atomicMax(&sm.taken, (int)(first + take[i]));
      copy_or_queue(a, sm.take, Job{row[i], held[i], take[i], avail - 1 - (int)first}, false);
    }
    a.seq_lens[s] = ok[i] ? ctx[i] + q[i] : 0;
    a.qsl[s + 1] = (int)min(at.tokens, (long long)INT_MAX);
  }
  if (flag) sm.flag = 1;
  __syncthreads();
  do_jobs(a, sm.take, false);
  if (tid == 0) {
    a.qsl[0] = 0;
    *a.num_free_out = avail - sm.taken;
    if (sm.flag || all.tokens > a.T) atomicOr(a.err, kErrBounds);
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
  // (query_start_loc may pass T, up to 2^31 - 1: no token is counted from there)
  const int t0 = min(a.qsl[s], a.T), t1 = min(a.qsl[s + 1], a.T), ctx = a.ctx_lens[s];
  for (int t = t0 + seg * kFillThreads + tid; t < t1; t += segments * kFillThreads) {
    int slot = -1;
    if (L > 0) {
      const int pos = ctx + (t - t0);
      const int page = src[pos >> a.p_shift];
      const long long x = (long long)page * a.P + (pos & (a.P - 1));
      if (page >= 0 && x <= INT_MAX) slot = (int)x;
      else atomicOr(a.err, kErrPage);
    }
    a.slots[t] = slot;
  }
  if (s == a.S - 1)
    for (int t = min(a.qsl[a.S], a.T) + seg * kFillThreads + tid; t < a.T; t += segments * kFillThreads) a.slots[t] = -1;
}

cudaError_t launch_build_tables(const TableArgs& a, cudaStream_t stream) {
  int slots = 64;
  while (slots < 2 * a.S) slots *= 2;
  const size_t smem = sizeof(PoolSmem) + 2 * sizeof(int) * (size_t)slots;
  static_assert(sizeof(PoolSmem) + 2 * sizeof(int) * 2 * kMaxRequests <= 232448, "hash table of the most requests");
  const bool one = a.S <= kPoolThreads;  // a request per thread
  auto kern = one ? pool_kernel<1> : pool_kernel<kMaxRequests / kPoolThreads>;
  static int attr_done[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  if (dev < 0 || dev >= 64 || !(attr_done[dev] & (one ? 1 : 2))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(PoolSmem) + 2 * sizeof(int) * 2 * kMaxRequests));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] |= one ? 1 : 2;
  }
  e = launch_pdl(false, kern, 1, kPoolThreads, smem, stream, a, (a.S + kPoolThreads - 1) / kPoolThreads, slots);
  if (e != cudaSuccess) return e;
  if (a.S == 0) return a.T > 0 ? cudaMemsetAsync(a.slots, 0xff, sizeof(int32_t) * (size_t)a.T, stream) : cudaGetLastError();
  const int segments = a.W > 0 ? (a.W + kSegment - 1) / kSegment : 1;
  e = launch_pdl(true, table_fill_kernel, a.S * segments, kFillThreads, 0, stream, a, segments);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pgqa
