// Rotary positions: the cosine and sine of one (position, pair).
//
// A pair's angle at position p is p * inv_freq.  Formed in fp32 the product is
// off by up to 2^-24 of itself -- 0.06 radians at a position of a million -- and
// the argument reduction of a large angle is slow.  So a pair's frequency is kept
// as turns per position (inv_freq / 2 pi) in 64-bit fixed point: the product with
// the integer position, taken modulo 2^64, is the exact fraction of a turn (off by
// at most p * 2^-53 of the frequency, its rounding on the host).  Its upper 32 bits are
// split into the nearest quarter turn and a rest of at most 1/4 half turn, which
// goes to the half-turn sine and cosine: in fp32 the rest is off by 2^-27 half turns, the
// whole (up to one half turn) by 2^-25, more than the functions themselves (fp32 heads
// against 64 bits 3.9e-8, 5.6e-8 without the split; 262,144 tokens of one head 27.0 us,
// 25.1 without, the other cases the same).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsa {

struct RopeArgs {
  const uint64_t* turns;   // [d_rot / 2] turns per position, in units of 2^-64
  int32_t d_rot;
  bool half;               // pair i is (i, i + d_rot / 2), else (2 i, 2 i + 1)
  float magnitude;         // factor on cosine and sine
};

// (magnitude cos, magnitude sin) of the pair's angle at position pos.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turns, int32_t pos, float magnitude) {
  const uint64_t phase = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t hi = static_cast<uint32_t>(phase >> 32), quarter = (hi + 0x20000000u) >> 30;
  const float rest = static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * 4.656612873077393e-10f;  // 2^-31
  float s0, c0;
  sincospif(rest, &s0, &c0);
  const float c1 = quarter & 1u ? s0 : c0, s1 = quarter & 1u ? c0 : s0;
  const float c = __uint_as_float(__float_as_uint(c1) ^ (((quarter + 1u) & 2u) << 30));
  const float s = __uint_as_float(__float_as_uint(s1) ^ ((quarter & 2u) << 30));
  return make_float2(magnitude * c, magnitude * s);
}

// The rotated pair, in one order of operations everywhere: the same values come out
// whatever alignment or layout a caller's tensors have.
__device__ __forceinline__ float2 rope_pair(float a, float b, float2 cs) {
  return make_float2(fmaf(a, cs.x, -__fmul_rn(b, cs.y)), fmaf(a, cs.y, __fmul_rn(b, cs.x)));
}

}  // namespace dsa
