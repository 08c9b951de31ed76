// rope.cu -- rotary positions with up to four axes (time, height, width, ...) for q and k.
//
// Pair i of the first `rot` values of a head turns by the angle pos[axis(i)][t] * inv_freq[i]:
//   (u, w) -> (u cos - w sin, w cos + u sin)
// in fp32, rounded to bf16 once; the other values pass through. Pairs are (i, i + rot / 2),
// or (2i, 2i + 1) if `adjacent`.
//
// The angle: an fp32 product would be off by whole turns' worth of phase for far positions
// (2^20 * 2^-24 = 1/16 rad at an inv_freq of 1). inv_freq / (2 pi) is taken as a 64-bit
// fraction of a turn (fixed point, from an integer product of the frequency's 24 bits with the 96 bits of
// 1 / (2 pi) that matter at its exponent, as Payne and Hanek reduce angles), off by less than one
// unit of 2^-64 for every finite frequency; the position times it, modulo 2^64, wraps whole turns away
// exactly (2^31 units at most: 2^-33 turns), and its top 32 bits are the phase (2^-32 turns more), off
// by less than 2^-31 turns for every 32-bit position, before the cosine and sine of a number in
// [-1, 1) half turns. With 64 bits of 1 / (2 pi) for all exponents the phase was off by 4e-8
// turns at a frequency of 1e5 and by 0.004 at 1e10.
//
// HBM-bound: each rotated row is read and written once (in place, only its rotated part).
// 16 lanes take a row, 16 values a lane (two 16-byte loads and stores): values
// 8c .. 8c + 7 and rot / 2 + 8c .. of the halves order, 16c .. 16c + 15 of the adjacent one, so
// a lane holds both values of its 8 pairs and its 8 angles serve every head of a token.
// A half-warp loads four rows before it works out the angles and stores any (an in-place store keeps the
// compiler from moving later loads up): 16384 tokens of 26 heads, 256 values, 76 us (5.75 TB/s of
// reads and writes; 64 us at the measured copy rate); when that was 78, row by row 98, two rows 81, six 77
// but more registers. 16 warps an SM, 4 KB in flight each: with 24 warps the registers spill (92 us). A decoding
// step's 256 tokens of 17 heads take 7.1 us from a graph, one token 5.7 (an empty kernel 1.1): a chain of
// frequencies, positions, rows and eight sines and cosines per lane, in code fetched for the first time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "device_util.cuh"
#include "plan.cuh"

namespace pgqa {

namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 4;
constexpr int kBatch = 4;  // rows a half-warp has in flight

// 1 / (2 pi), 224 bits after the point: enough for the 96 from the highest exponent on.
__constant__ uint32_t kInv2Pi[7] = {0x28be60dbu, 0x9391054au, 0x7f09d5f4u, 0x7d4d3770u, 0x36d8a566u, 0x4f10e410u, 0x7f9458eau};

// x / (2 pi) modulo 1 as a 64-bit fraction; x finite.
__device__ __forceinline__ uint64_t turns_of(float x) {
  const uint32_t b = __float_as_uint(x), be = (b >> 23) & 0xffu;
  const uint64_t m = be ? (b & 0x7fffffu) | 0x800000u : (b & 0x7fffffu);
  const int e = (int)(be ? be : 1u) - 150;  // |x| = m 2^e
  // For e > 0 the first e bits of 1 / (2 pi) only make whole turns: start after them.
  const int skip = max(e, 0), k = skip >> 5, r = skip & 31;
  const uint64_t p2 = m * __funnelshift_l(kInv2Pi[k + 3], kInv2Pi[k + 2], r);
  const uint64_t p1 = m * __funnelshift_l(kInv2Pi[k + 2], kInv2Pi[k + 1], r) + (p2 >> 32);
  const uint64_t hi = m * __funnelshift_l(kInv2Pi[k + 1], kInv2Pi[k], r) + (p1 >> 32);
  const uint64_t lo = (p1 << 32) | (p2 & 0xffffffffu);
  // |x| / (2 pi) = (hi 2^64 + lo) 2^(-96 + min(e, 0)) and whole turns; hi < 2^56
  const int s = 32 + max(-e, 0);
  const uint64_t f = s < 64 ? (lo >> s) | (hi << (64 - s)) : s < 128 ? hi >> (s - 64) : 0;
  return (b >> 31) ? 0ull - f : f;
}

__device__ __forceinline__ int axis_of(const RopeArgs& a, int i) {
  if (a.interleaved) {
    const int x = i % a.axes;
    return i < a.axes * a.sections[x] ? x : 0;
  }
  int x = 0, end = a.sections[0];
  while (i >= end && x + 1 < a.axes) end += a.sections[++x];
  return x;
}

__device__ __forceinline__ void turn2(uint32_t& u, uint32_t& w, float c0, float s0, float c1, float s1) {
  const float u0 = __uint_as_float(u << 16), u1 = __uint_as_float(u & 0xffff0000u);
  const float w0 = __uint_as_float(w << 16), w1 = __uint_as_float(w & 0xffff0000u);
  u = pack_bf16x2(u0 * c0 - w0 * s0, u1 * c1 - w1 * s1);
  w = pack_bf16x2(w0 * c0 + u0 * s0, w1 * c1 + u1 * s1);
}
// An adjacent pair in one word.
__device__ __forceinline__ uint32_t turn1(uint32_t v, float c, float s) {
  const float u = __uint_as_float(v << 16), w = __uint_as_float(v & 0xffff0000u);
  return pack_bf16x2(u * c - w * s, w * c + u * s);
}

}  // namespace

// Work unit: (token, `chunk` consecutive heads of q then k). Half-warps take alternate heads.
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) rope_kernel(RopeArgs a, int chunk, int nchunks) {
  const int lane = threadIdx.x & 31, c = lane & 15, half = lane >> 4;
  const bool rotated = c < a.rot / 16;
  const int off0 = rotated && !a.adjacent ? 8 * c : 16 * c;
  const int off1 = rotated && !a.adjacent ? a.rot / 2 + 8 * c : 16 * c + 8;
  uint64_t f[8];
  uint32_t axes = 0;  // 4 bits per pair
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = 0;
    if (rotated) {
      const float x = __ldg(a.inv_freq + 8 * c + j);
      if (isfinite(x)) f[j] = turns_of(x);
      else bad = true;
      axes |= (uint32_t)axis_of(a, 8 * c + j) << (4 * j);
    }
  }
  const int rows = a.heads[0] + a.heads[1];
  const long long units = (long long)a.T * nchunks, step = (long long)gridDim.x * kWarps;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += step) {
    const long long t = u / nchunks;
    const int r0 = (int)(u - t * nchunks) * chunk, r1 = min(rows, r0 + chunk);
    float co[8], si[8];
    bool first = true;
    for (int r = r0 + half; r < r1; r += 2 * kBatch) {
      uint4 p[kBatch], q[kBatch];
      uint16_t* dst[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int rb = r + 2 * b;
        const int i = rb < a.heads[0] ? 0 : 1, h = i ? rb - a.heads[0] : rb;
        dst[b] = nullptr;
        if (rb >= r1 || (!rotated && a.in_place[i])) continue;
        const uint16_t* src = a.x[i] + t * a.x_st[i] + h * a.x_sh[i];
        dst[b] = a.y[i] + t * a.y_st[i] + h * a.y_sh[i];
        p[b] = *reinterpret_cast<const uint4*>(src + off0);
        q[b] = *reinterpret_cast<const uint4*>(src + off1);
      }
      if (rotated && first) {
        first = false;
        int pos[kRopeMaxAxes];
#pragma unroll
        for (int x = 0; x < kRopeMaxAxes; ++x) pos[x] = x < a.axes ? __ldg(a.pos + x * a.pos_sa + t) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int x = (axes >> (4 * j)) & 15;
          const int ps = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
          const int phase = (int)(((uint64_t)(int64_t)ps * f[j]) >> 32);  // of a turn, 2^32 to the turn
          sincospif((float)phase * 4.656612873077393e-10f, &si[j], &co[j]);  // * 2^-31: half turns
        }
        if (bad)
#pragma unroll
          for (int j = 0; j < 8; ++j) co[j] = si[j] = __int_as_float(0x7fc00000);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!dst[b]) continue;
        if (rotated) {
          uint4 &u = p[b], &w = q[b];
          if (a.adjacent) {
            u = make_uint4(turn1(u.x, co[0], si[0]), turn1(u.y, co[1], si[1]), turn1(u.z, co[2], si[2]), turn1(u.w, co[3], si[3]));
            w = make_uint4(turn1(w.x, co[4], si[4]), turn1(w.y, co[5], si[5]), turn1(w.z, co[6], si[6]), turn1(w.w, co[7], si[7]));
          } else {
            turn2(u.x, w.x, co[0], si[0], co[1], si[1]);
            turn2(u.y, w.y, co[2], si[2], co[3], si[3]);
            turn2(u.z, w.z, co[4], si[4], co[5], si[5]);
            turn2(u.w, w.w, co[6], si[6], co[7], si[7]);
          }
        }
        *reinterpret_cast<uint4*>(dst[b] + off0) = p[b];
        *reinterpret_cast<uint4*>(dst[b] + off1) = q[b];
      }
    }
  }
}

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  const int rows = a.heads[0] + a.heads[1];
  if (a.T == 0 || rows == 0) return cudaSuccess;
  // Heads per warp: all of a token's where there are tokens enough for every warp, else as few
  // as two, so that a decoding step's rows spread over the SMs.
  const long long warps = (long long)sms * kCtasPerSm * kWarps;
  const long long split = std::max<long long>(1, warps / a.T);
  const int chunk = (int)std::max<long long>(2, (rows + split - 1) / split + 1) / 2 * 2;
  const int nchunks = (rows + chunk - 1) / chunk;
  const long long want = ((long long)a.T * nchunks + kWarps - 1) / kWarps;
  const int grid = (int)std::min<long long>(want, (long long)sms * kCtasPerSm);
  rope_kernel<<<grid, kWarps * 32, 0, stream>>>(a, chunk, nchunks);
  return cudaGetLastError();
}

}  // namespace pgqa
