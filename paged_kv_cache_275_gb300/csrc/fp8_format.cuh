// The 8-bit cache's format on the device: a row's exponent, its codes, and the way back (fp8_cache.h).
//
// The scale of a row is a power of two: e4m3 is a floating type, so a finer scale would keep no more significant bits, and
// with a power of two the codes and the values they stand for are exact, in whatever arithmetic they are formed: bf16 holds
// every value, a code times its scale (but that of 2^128, and those below 2^-133).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {
namespace {

// 2^(e - 127); e = 255 gives infinity (the append writes none above 247).
__device__ __forceinline__ float fp8_scale(uint32_t e) { return __uint_as_float(max(e << 23, 0x00400000u)); }
// e - 127 as a number, by way of 2^23 + e, whose last bit is one.
__device__ __forceinline__ float fp8_power(uint32_t e) { return __uint_as_float(0x4b000000u | e) - 8388735.f; }

// The exponent byte of a row whose largest finite magnitude has the bf16 bits `top`: the least e >= 0 with
// top <= 448 * 2^(e - 127).  448 = 1.75 * 2^8, so the mantissa is compared with 0.75 * 128.
__device__ __forceinline__ uint32_t fp8_exponent(uint32_t top) {
  const int e = static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 96u);
  return e < 0 ? 0u : static_cast<uint32_t>(e);
}
// What takes the row's values to its codes: 2^(127 - e), e <= 247.
__device__ __forceinline__ float fp8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Two codes, lo in the low byte; round to nearest even.  (Values are within 448 in magnitude, or not a number.)
__device__ __forceinline__ uint32_t fp8_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of two codes as fp16, exactly.
__device__ __forceinline__ uint32_t fp8_halves(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ float2 fp8_floats(uint16_t codes) {
  const uint32_t h = fp8_halves(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace
}  // namespace pkv
