// fp4_cache.cu -- the 4-bit paged cache's write (new tokens' K and V quantised into their
// pages) and read (pages dequantised back to bf16 rows).
//
// Write, for each group g of 16 consecutive values x of a (token, kv head) row:
//   y = x * inv (fp32; inv = 1 / descale rounded to fp32 once per call)
//   scale = e4m3(max |y| * fp32(1/6)), round to nearest even, at most 448
//   code  = e2m1(y * r), r = fp32(1 / scale) (0 for a zero scale), nearest even, at most 6
// so a group's largest value takes the code 6 up to the scale's rounding. The products and r
// are rounded to 24 bits, far finer than either format's steps; they are the definition (a
// true division can differ at a tie). A NaN in a group makes its scale NaN.
// Read: bf16(code * scale * descale), code * scale exact.
//
// Both are HBM-bound: 1024 bytes of bf16 and 288 of cache per (token, kv head). The unit of
// work is the tokens of one sequence inside one 16-token block of a page, for one kv head:
// one warp, lane l holding values 8l .. 8l + 7, i.e. code bytes 4l .. 4l + 3. A whole block
// of V leaves as 64 contiguous bytes per lane; a part of one as single bytes (16 apart).
// Measured: writing 8 chunks of 8001-8192 tokens, 2 heads, and reading them back 67 us (339 MB, 5.0 TB/s; 50 us
// at the copy rate); alone, from a graph, the write takes 40 us (25 at the copy rate) and the read 31 (25).
// Reading 6 prefixes of up to 16384 tokens, 2 heads: 31 us (158 MB, 5.1 TB/s; 23 us). A step's 256 tokens take
// 3.7 us to write and 3.3 to read, from a graph: launch and two dependent reads (table, row).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "device_util.cuh"
#include "fp4.cuh"
#include "plan.cuh"
#include "tc_util.cuh"

namespace pgqa {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;       // tokens whose rows are in flight at once in a warp
constexpr int kWarpsPerSm = 16; // A call with fewer (token, head) rows than this many warps per SM launches a
                                // warp for each; only those whose token starts a block of 16 or a sequence
                                // have a unit to move, the others look their sequence up and leave. A
                                // larger call gives a warp a window of up to 16 tokens.

// The units of the warps' windows: every unit belongs to the window that holds its first
// token. fn(t, n, slot, page): tokens [t, t + n) lie in slots [slot, slot + n) of `page`
// (-1: not there, or flagged).
template <typename F>
__device__ __forceinline__ void for_each_unit(const Fp4CacheArgs& a, int t, int t_end, int lane, F&& fn) {
  int s = seq_of_token(a.qsl, a.num_seqs, t, lane);
  int q0 = __ldg(a.qsl + s), q1 = __ldg(a.qsl + s + 1), L = __ldg(a.seq_lens + s);
  while (t < t_end) {
    while (t >= q1 && s < a.num_seqs - 1) {
      ++s;
      q0 = q1;
      q1 = __ldg(a.qsl + s + 1);
      L = __ldg(a.seq_lens + s);
    }
    // As in the attention, a sequence whose tokens do not lie in [0, T) has no valid token: its
    // units are cut at q1, and so end by T.
    const long long qn = (long long)q1 - q0, pos = L - qn + (t - q0);
    if (q0 < 0 || q1 > a.T || t < q0 || t >= q1 || qn > L || pos < 0 || (pos >> a.p_shift) >= a.W) {
      if (lane == 0) atomicOr(a.err, kErrBounds);
      fn(t, 1, 0, -1);  // a token without a place
      ++t;
      continue;
    }
    const int off = (int)(pos & (kFp4Block - 1));
    const int n = min(kFp4Block - off, q1 - t);
    if (t == q0 || off == 0) {
      int page = __ldg(a.bt + (long long)s * a.bt_stride + (pos >> a.p_shift));
      if (page < 0 || page >= a.NB) {
        if (lane == 0) atomicOr(a.err, kErrPage);
        page = -1;
      }
      fn(t, n, (int)(pos & (a.P - 1)), page);
    }  // else the window starts inside a unit of the one before
    t += n;
  }
}

// 8 values of one row -> their codes; *scale8 the group's scale byte (lanes 2g and 2g + 1
// hold group g).
__device__ __forceinline__ uint32_t quantise8(uint4 v, float inv, uint32_t* scale8) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // The largest |x| of the group as bf16 bits: integer order is the order of magnitudes, with
  // NaN above infinity, so a NaN survives the maximum. |x| * inv rounds monotonically, so the
  // largest product is the product of the largest.
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  m = max(m >> 16, m & 0xffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const float amax = __fmul_rn(__uint_as_float(m << 16), inv);
  const uint32_t s8 = tc::e4m3x2(__fmul_rn(amax, 1.f / 6.f), 0.f) & 0xffu;
  *scale8 = s8;
  const float s = fp4::scale_value(s8);
  const float r = s == 0.f ? 0.f : __frcp_rn(s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __fmul_rn(__fmul_rn(__uint_as_float(w[i] << 16), inv), r);
    y[2 * i + 1] = __fmul_rn(__fmul_rn(__uint_as_float(w[i] & 0xffff0000u), inv), r);
  }
  return fp4::encode8(y);
}

// 8 codes and their scale byte -> 8 bf16 values.
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t scale8, float descale) {
  uint32_t h[4], out[4];
  fp4::codes4(codes, h);
  const float s = fp4::scale_value(scale8);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_f16x2(h[i]);
    out[i] = pack_bf16x2(__fmul_rn(x.x * s, descale), __fmul_rn(x.y * s, descale));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <bool kFull>
__device__ __forceinline__ void write_unit(const Fp4CacheArgs& a, int t, int n, int slot, int page, int h, int lane) {
  const uint16_t* kx = a.kx + (long long)t * a.kx_st + (long long)h * a.kx_sh + lane * 8;
  const uint16_t* vx = a.vx + (long long)t * a.vx_st + (long long)h * a.vx_sh + lane * 8;
  uint8_t* krow = a.kc + page * a.kc_sb + h * a.kc_sh + slot * kFp4Row;
  uint8_t* vblk = a.vc + page * a.vc_sb + h * a.vc_sh + (slot / kFp4Block) * kFp4BlockBytes;
  const int tok = slot % kFp4Block;
  uint32_t vw[kFp4Block], vs[kFp4Block / 4] = {};
  const int cnt = kFull ? kFp4Block : n;
#pragma unroll
  for (int j0 = 0; j0 < kFp4Block; j0 += kBatch) {
    if (!kFull && j0 >= cnt) break;
    uint4 k[kBatch], v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (kFull || j0 + j < cnt) {
        k[j] = __ldcs(reinterpret_cast<const uint4*>(kx + (j0 + j) * a.kx_st));
        v[j] = __ldcs(reinterpret_cast<const uint4*>(vx + (j0 + j) * a.vx_st));
      }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (!kFull && j0 + j >= cnt) break;
      uint32_t s8;
      const uint32_t kw = quantise8(k[j], a.k_mul, &s8);
      uint8_t* row = krow + (j0 + j) * kFp4Row;
      *reinterpret_cast<uint32_t*>(row + lane * 4) = kw;
      if (!(lane & 1)) row[kFp4Codes + lane / 2] = (uint8_t)s8;
      const uint32_t c = quantise8(v[j], a.v_mul, &s8);
      if (kFull) {
        vw[j0 + j] = c;
        vs[(j0 + j) / 4] |= s8 << (8 * ((j0 + j) & 3));
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) vblk[(lane * 4 + b) * kFp4Block + tok + j0 + j] = (uint8_t)(c >> (8 * b));
        if (!(lane & 1)) vblk[kFp4BlockScales + (lane / 2) * kFp4Block + tok + j0 + j] = (uint8_t)s8;
      }
    }
  }
  if (kFull) {
    // byte b of each token's word -> the 16 tokens of code byte 4 lane + b
    uint32_t q[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {vw[4 * j], vw[4 * j + 1], vw[4 * j + 2], vw[4 * j + 3]};
      uint32_t r[4];
      fp4::transpose4(w, r);
#pragma unroll
      for (int b = 0; b < 4; ++b) q[b][j] = r[b];
    }
    uint4* dst = reinterpret_cast<uint4*>(vblk + lane * 64);
#pragma unroll
    for (int b = 0; b < 4; ++b) dst[b] = make_uint4(q[b][0], q[b][1], q[b][2], q[b][3]);
    if (!(lane & 1))
      *reinterpret_cast<uint4*>(vblk + kFp4BlockScales + (lane / 2) * kFp4Block) = make_uint4(vs[0], vs[1], vs[2], vs[3]);
  }
}

__device__ __forceinline__ void read_unit(const Fp4CacheArgs& a, int t, int n, int slot, int page, int h, int lane) {
  uint16_t* kx = a.kx + (long long)t * a.kx_st + (long long)h * a.kx_sh + lane * 8;
  uint16_t* vx = a.vx + (long long)t * a.vx_st + (long long)h * a.vx_sh + lane * 8;
  if (page < 0) {
    for (int j = 0; j < n; ++j) {
      *reinterpret_cast<uint4*>(kx + j * a.kx_st) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(vx + j * a.vx_st) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const uint8_t* krow = a.kc + page * a.kc_sb + h * a.kc_sh + slot * kFp4Row;
  const uint8_t* vblk = a.vc + page * a.vc_sb + h * a.vc_sh + (slot / kFp4Block) * kFp4BlockBytes;
  const int tok = slot % kFp4Block;
  uint4 vv[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) vv[b] = __ldcs(reinterpret_cast<const uint4*>(vblk + lane * 64) + b);
  const uint4 vs = __ldcs(reinterpret_cast<const uint4*>(vblk + kFp4BlockScales + (lane / 2) * kFp4Block));
  const uint32_t* vq = reinterpret_cast<const uint32_t*>(vv);
  const uint32_t sq[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
  for (int j0 = 0; j0 < kFp4Block; j0 += kBatch) {
    // tokens tok .. tok + n - 1 of the block, in block order (so that registers are indexed
    // by constants)
    uint32_t kw[kBatch], ks[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = j0 + j - tok;  // token of the unit
      if (r >= 0 && r < n) {
        kw[j] = __ldcs(reinterpret_cast<const uint32_t*>(krow + r * kFp4Row + lane * 4));
        ks[j] = __ldcs(krow + r * kFp4Row + kFp4Codes + lane / 2);
      }
    }
    const uint32_t w[4] = {vq[j0 / 4], vq[4 + j0 / 4], vq[8 + j0 / 4], vq[12 + j0 / 4]};
    uint32_t c[4];
    fp4::transpose4(w, c);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = j0 + j - tok;
      if (r >= 0 && r < n) {
        __stcs(reinterpret_cast<uint4*>(kx + r * a.kx_st), dequantise8(kw[j], ks[j], a.k_mul));
        __stcs(reinterpret_cast<uint4*>(vx + r * a.vx_st), dequantise8(c[j], (sq[j0 / 4] >> (8 * j)) & 0xffu, a.v_mul));
      }
    }
  }
}

}  // namespace

template <bool kWrite>
__global__ void __launch_bounds__(kWarps * 32) fp4_cache_kernel(Fp4CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int h = (int)(w % a.Hkv);
  const long long t0 = w / a.Hkv * a.window;
  if (t0 >= a.T) return;
  const int t_end = (int)min(t0 + a.window, (long long)a.T);
  for_each_unit(a, (int)t0, t_end, lane, [&](int t, int n, int slot, int page) {
    if (kWrite) {
      if (page < 0) return;
      if (n == kFp4Block) write_unit<true>(a, t, n, slot, page, h, lane);
      else write_unit<false>(a, t, n, slot, page, h, lane);
    } else {
      read_unit(a, t, n, slot, page, h, lane);
    }
  });
}

namespace {

template <bool kWrite>
cudaError_t launch(Fp4CacheArgs a, int sms, cudaStream_t stream) {
  if (a.T == 0 || a.Hkv == 0) return cudaSuccess;
  const long long per = (long long)a.T * a.Hkv / ((long long)sms * kWarpsPerSm);
  a.window = (int)std::min<long long>(kFp4Block, std::max<long long>(1, per));
  const long long warps = ((long long)a.T + a.window - 1) / a.window * a.Hkv;
  fp4_cache_kernel<kWrite><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_cache_write(const Fp4CacheArgs& a, int sms, cudaStream_t stream) {
  return launch<true>(a, sms, stream);
}
cudaError_t launch_fp4_cache_read(const Fp4CacheArgs& a, int sms, cudaStream_t stream) {
  return launch<false>(a, sms, stream);
}

}  // namespace pgqa
