// Conversions of quantized coefficient codes to fp16, shared by the decode kernels and the
// prefill's page-widening pass.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace rcp {

// Two 4-bit codes (byte B of w: the even coefficient in the low nibble, two's complement) times
// their group's scale, as an fp16 pair.  The byte goes to both halves; the low nibble n becomes
// the fp16 1024 + (n ^ 8) (exponent bits 0x6400 with n ^ 8 as the low mantissa bits), the high
// one, four bits up, 64 + (n ^ 8) (0x5400); minus 1032 and 72 the signed codes, exactly; the
// product with the scale rounds once.  (Four instructions a pair, seven when the nibbles were
// put together by shifts: 554 -> 533 us for a 4-bit decode at 64 x 8192.)
template <int B>
__device__ __forceinline__ uint32_t int4x2_to_half2_bits(uint32_t w, __half2 scale) {
  uint32_t b;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(b) : "r"(w), "n"(0x4040 + 0x0101 * B));
  b = (b & 0x00F0000Fu) ^ 0x54806408u;
  const __half2 code = __hsub2(*reinterpret_cast<const __half2*>(&b),
                               __floats2half2_rn(1032.f, 72.f));
  const __half2 v = __hmul2(code, scale);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace rcp
