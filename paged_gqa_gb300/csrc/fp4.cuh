// fp4.cuh -- the 4-bit cache format: e2m1 codes with one e4m3 scale per 16 values.
//
// A value is code * scale * descale: the code is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), the scale an e4m3 byte of the value's group of 16 consecutive d, descale the
// tensor's factor, which the caller passes. code * scale has at most 6 significant bits and
// lies in [2^-10, 2688] or is 0, so it is exact in f16, bf16 and tf32.
//
// A (token, kv head) row has 128 code bytes (byte i: d = 2i in the low nibble, 2i + 1 in the
// high one) and 16 scale bytes. A page of one kv head is P * 144 contiguous bytes:
//   K  token by token: [128 codes][16 scales]. A 144-byte pitch puts 8 consecutive rows'
//      16-byte chunks in different banks, so threads that own one key each read their row
//      from a copied page without conflicts;
//   V  in blocks of 16 tokens: [128 bytes][16 tokens] codes, then [16 groups][16 tokens]
//      scales. A thread that owns byte i (two d) reads 16 tokens of it at once: the
//      attention's P.V product wants V^T, whose rows are d and whose columns are tokens.
// Every byte belongs to one token, so a token is written without reading its neighbours.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace pgqa {
namespace fp4 {

// Four code bytes -> f16 pairs (byte k: h[k] = {low nibble, high nibble}), exact.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// One code byte -> its two values.
__device__ __forceinline__ float2 code_pair(uint32_t byte) {
  uint32_t h[4];
  codes4(byte, h);
  return __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
}
// Two scale bytes (low byte first) -> an f16 pair, exact.
__device__ __forceinline__ uint32_t scales2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return h;
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t h = scales2(byte);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}
// Eight values -> eight codes, value 0 in the lowest nibble; rounded to nearest even,
// saturating at +-6.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// An f16 pair times the low (high) half of another.
__device__ __forceinline__ uint32_t mul_f16x2_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// {lo(a) * lo(s), lo(b) * hi(t)} and {hi(a) * lo(s), hi(b) * hi(t)} for s = {x, 0}, t = {0, y}: two
// f16 pairs of codes (one key each) to two pairs of keys, times their scales, exact. Selecting by
// zeros keeps the work on the FMA pipes; byte permutes would share the ALU pipe with the codes'
// conversions, which is the fuller one.
__device__ __forceinline__ void pair_keys(uint32_t a, uint32_t b, uint32_t s, uint32_t t, uint32_t& lo, uint32_t& hi) {
  const __half2 ha = *reinterpret_cast<const __half2*>(&a), hb = *reinterpret_cast<const __half2*>(&b);
  const __half2 hs = *reinterpret_cast<const __half2*>(&s), ht = *reinterpret_cast<const __half2*>(&t);
  const __half2 l = __hfma2(__low2half2(hb), ht, __hmul2(__low2half2(ha), hs));
  const __half2 h = __hfma2(__high2half2(hb), ht, __hmul2(__high2half2(ha), hs));
  lo = *reinterpret_cast<const uint32_t*>(&l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
}

// 4 x 4 bytes transposed: byte k of r[j] = byte j of w[k].
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&r)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  r[0] = __byte_perm(a, b, 0x5410);
  r[1] = __byte_perm(a, b, 0x7632);
  r[2] = __byte_perm(c, d, 0x5410);
  r[3] = __byte_perm(c, d, 0x7632);
}

}  // namespace fp4
}  // namespace pgqa
