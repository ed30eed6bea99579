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

// Value of latent dim d (< 512) of a row.
__device__ __forceinline__ float e2m1_latent(const uint8_t* row, int d) {
  const float2 v = e2m1x2_to_float2(row[d >> 1]);
  return ((d & 1) ? v.y : v.x) * (e4m3_to_float(row[kE2m1Scales + (d >> 4)]) *
                                  *reinterpret_cast<const float*>(row + kE2m1RowScale));
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
