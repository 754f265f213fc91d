// cache_common.hpp -- internal helpers of the quantised cache: groups of 32
// values as E4M3 (8 bits) or E2M1 (4 bits) codes with a power of two each.
#pragma once

#include "kernels.hpp"
#include "token_common.hpp"

namespace dlrm {

constexpr int kGroup = 32;      // values that share a scale
constexpr int kMinScale = 10;   // 2^-117

// The power of two that a scale's byte stands for; 255 makes the conversions
// below give NaN.
__device__ __forceinline__ float unit_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes, the first in the lowest bits.
template <int BITS>
struct Codes {
  uint32_t w[BITS / 4];
};

// Values 2I and 2I + 1 of eight, in float32 and in bfloat16 (exact in both).
template <int I>
__device__ __forceinline__ auto pair_f32(const Codes<4> &c, float unit) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.w[0], unit, I);
}
template <int I>
__device__ __forceinline__ auto pair_f32(const Codes<8> &c, float unit) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.w[I / 2], unit, I % 2 != 0);
}
template <int I>
__device__ __forceinline__ uint32_t pair_bf16(const Codes<4> &c, float unit) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.w[0], unit, I));
}
template <int I>
__device__ __forceinline__ uint32_t pair_bf16(const Codes<8> &c, float unit) {
  return __builtin_bit_cast(
      uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.w[I / 2], unit, I % 2 != 0));
}

template <int BITS>
__device__ __forceinline__ void values_of(const Codes<BITS> &c, float unit, float (&v)[8]) {
  const auto a = pair_f32<0>(c, unit), b = pair_f32<1>(c, unit), d = pair_f32<2>(c, unit),
             e = pair_f32<3>(c, unit);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
  v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
}

}  // namespace dlrm
