// kv4_common.cuh — the 4-bit row format shared by the kernels of the paged cache.
//
// A row of 512 values is 256 bytes of codes and 16 bytes of scales.  A code is e2m1 (sign, two
// exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), element 2i in the
// low nibble of byte i.  Each group of 32 values shares one scale byte b, the power of two 2^(b - 127);
// b = 255 marks a group that held a NaN.  The library writes exponents in [-23, 13] only, where every
// code * scale is exact in fp16 and in bf16 (0.5 * 2^-23 is fp16's least value, 6 * 2^13 = 49152).
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace ds4x {

constexpr int kKv4Dim = 512;
constexpr int kKv4CodeBytes = kKv4Dim / 2;    // of one row
constexpr int kKv4ScaleBytes = kKv4Dim / 32;  // of one row
constexpr int kKv4ExpMin = -23, kKv4ExpMax = 13;

// The eight codes of `w` (nibble i = element i) as four fp16 pairs; exact.
__device__ __forceinline__ void kv4_decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(b - 127) as fp32 (b = 0, which the library never writes, reads as 0), NaN for b = 255.
__device__ __forceinline__ float kv4_scale(uint32_t b) {
  return __uint_as_float((b << 23) | (b == 255u ? 0x400000u : 0u));
}

}  // namespace ds4x
