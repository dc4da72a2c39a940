// Device and host pieces shared by the kernels on 4-bit operands (MX4: blocks
// of 32 E2M1 values that share a power of two), gfx950.
#pragma once

#include "../../include/mc2_serve.h"
#include "mc2_common.hpp"
#include "mc2_host.hpp"

namespace mc2 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

inline int64_t mx4_blocks(int64_t k) { return (k + 31) / 32; }
inline int64_t mx4_pitch(int64_t k) { return (mx4_blocks(k) + 15) / 16 * 16; }

// The power of two that a scale byte stands for, as the conversions take it:
// they use the fp32 number's exponent field alone, so that field 0 is 2^-127
// here, and 255 gives NaN (checked on the device for all 256).
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two values of byte B of `c` times a power of two, as 16-bit pairs or fp32.
template <int B>
__device__ __forceinline__ uint32_t mx4_pair_bf16(uint32_t c, float s) {
  return bit_cast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, B));
}
template <int B>
__device__ __forceinline__ uint32_t mx4_pair_f16(uint32_t c, float s) {
  return bit_cast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, B));
}
template <int B>
__device__ __forceinline__ f32x2_t mx4_pair_f32(uint32_t c, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, B);
}

// Eight values (one dword of codes) as bf16: four dwords.
__device__ __forceinline__ u32x4_t mx4_bf16x8(uint32_t c, float s) {
  return u32x4_t{mx4_pair_bf16<0>(c, s), mx4_pair_bf16<1>(c, s), mx4_pair_bf16<2>(c, s),
                 mx4_pair_bf16<3>(c, s)};
}

}  // namespace mc2
