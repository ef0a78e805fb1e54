// Element types of the history-cache and sampling kernels.
#pragma once

#include "hlr_common.hpp"

namespace hlr {

// bfloat16: conversions round to nearest even.
struct bf16 {
  uint16_t bits;
  bf16() = default;
  __device__ __forceinline__ explicit bf16(float f) {
    uint32_t u = __builtin_bit_cast(uint32_t, f);
    if (f != f)
      u |= 0x400000u;  // stays a NaN when the low half is cut off
    else
      u += 0x7fffu + ((u >> 16) & 1u);
    bits = static_cast<uint16_t>(u >> 16);
  }
  __device__ __forceinline__ explicit operator float() const {
    return __builtin_bit_cast(float, static_cast<uint32_t>(bits) << 16);
  }
};

}  // namespace hlr
