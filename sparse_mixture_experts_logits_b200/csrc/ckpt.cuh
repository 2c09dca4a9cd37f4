// The 8-bit form of a block of MOE_CKPT_BLOCK values: its exponent byte E and
// q = clamp(round(x 2^(133 - E)), -127, 127) (see ckpt.cu).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kBlk = MOE_CKPT_BLOCK;

// 2^(127 - E): takes the block's largest magnitude into [1, 2).  E = 255: 0.
__device__ __forceinline__ float ckpt_inv_scale(uint32_t e) {
  return __uint_as_float(e < 254u ? (254u - e) << 23 : (e == 254u ? 0x00400000u : 0u));
}
// 2^(E - 133), subnormal for E <= 6; E = 255: NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t e) {
  return __uint_as_float(e >= 255u ? 0x7fc00000u : (e >= 7u ? (e - 6u) << 23 : 1u << (16u + e)));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace moe
