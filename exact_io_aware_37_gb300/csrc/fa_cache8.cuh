// The 8-bit key/value cache's number format, shared by the kernels that write,
// read and attend to it.  A row of D values is held as D e4m3 codes and one
// exponent byte b: value = code * 2^(b - 127), b in 0 .. 254.  The exponent is
// the smallest for which the row's largest magnitude is at most 448 (the
// largest e4m3 value), so the codes use the format's whole range; a power of
// two makes scaling exact, and e4m3 keeps its relative step at any scale, so
// nothing is lost against a scale with a mantissa except the last bit of
// range.  One byte instead of a float32 scale keeps the cache at D + 1 bytes a
// row.  Values that are not finite become the NaN code and do not count
// towards the largest magnitude.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

namespace fa {
namespace c8 {

// Exponent byte of a row whose largest finite magnitude is `amax`: amax =
// m * 2^x with m in [0.5, 1); 448 = 0.875 * 2^9, so the exponent is x - 9,
// one more when m > 0.875; at least -127.
__device__ __forceinline__ int exp_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -127) + 127;
}
// 2^(127 - b), for b of exp_byte (0 .. 247): always a normal float.
__device__ __forceinline__ float inv_scale(int b) { return __uint_as_float((uint32_t)(254 - b) << 23); }
// 2^(b - 127); b = 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale(int b) { return __uint_as_float(b > 0 ? (uint32_t)b << 23 : 0x00400000u); }

// |x| as counted towards the row's largest magnitude
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // false for NaN too
}

// Two values of magnitude at most 448, or NaN, to two codes (round to nearest
// even), `lo` in the low byte.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes (low 16 bits of u) to an fp16 pair, exactly.
__device__ __forceinline__ uint32_t decode2_f16(uint32_t u) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)u));
  return r;
}
__device__ __forceinline__ float2 decode2(uint32_t u) {
  const uint32_t h = decode2_f16(u);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two fp16 values of magnitude at most 256 (or NaN) as sums of three codes each, x =
// c0 + c1 / 32 + c2 / 1024: 4 bits a term, 12 in all (fp16 has 11), down to 2^-20 absolute (half
// of c2's smallest step, 2^-9 / 1024).  A term's error is at most 8, so the next one is at most
// 256 again; every difference is exact in fp16.
constexpr float kTerm = 1.f / 32;
__device__ __forceinline__ uint32_t encode2_f16(__half2 h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
  return r;
}
__device__ __forceinline__ void encode2_terms(__half2 h, uint32_t (&t)[3]) {
  const __half2 up = __float2half2_rn(32.f), down = __float2half2_rn(-32.f);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    t[k] = encode2_f16(h);
    if (k < 2) {
      const uint32_t c = decode2_f16(t[k]);
      h = __hfma2(*reinterpret_cast<const __half2*>(&c), down, __hmul2(h, up));
    }
  }
}

}  // namespace c8
}  // namespace fa
