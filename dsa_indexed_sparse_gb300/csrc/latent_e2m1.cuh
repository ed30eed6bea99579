// The 4-bit latent row (DSA_E2M1), 432 bytes:
//   [0, 256)    512 E2M1 codes, latent dim 2 i in the low nibble of byte i, dim 2 i + 1 in the high one
//   [256, 288)  32 E4M3 scales, scale b for dims [16 b, 16 b + 16)
//   [288, 292)  fp32 row scale
//   [292, 304)  reserved (written as zero)
//   [304, 432)  64 bf16 rope values
// Dim d stands for e2m1(code_d) * e4m3(scale_{d / 16}) * row scale.  A code has two
// significant bits and a scale four, so with a power-of-two row scale (what the
// writer stores) the value has at most six: exact in bf16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_device.cuh"

namespace dsa {

constexpr int kE2m1Row = 432;
constexpr int kE2m1Scales = 256;     // byte offset of the block scales
constexpr int kE2m1RowScale = 288;   // byte offset of the row scale
constexpr int kE2m1Rope = 304;       // byte offset of the rope values

// Two codes (a byte) -> two floats, exact.
__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight codes (a 32-bit word, low nibble first) -> four pairs of halves, exact.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Exponent of the row scale of a row whose largest latent magnitude is amax:
// floor(log2 amax) - 10, so that amax / 2^e lies in [1024, 2048) and the largest
// block scale amax / 2^e / 6 in [170, 342): below E4M3's 448 after rounding.  0
// for an all-zero row; infinite magnitudes take the largest finite exponent.
__device__ __forceinline__ int e2m1_row_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  return max(-126, min(117, ilogbf(amax) - 10));
}

}  // namespace dsa
