// Element types and launch sizes of the history-cache and sampling kernels.
#pragma once

#include "hlr_common.hpp"

namespace hlr {

// bfloat16: conversions round to nearest even.
struct bf16 {
  uint16_t bits;
  bf16() = default;
  __device__ __forceinline__ explicit bf16(float f) : bits(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f))) {}
  __device__ __forceinline__ explicit operator float() const {
    return __builtin_bit_cast(float, static_cast<uint32_t>(bits) << 16);
  }
};

// Blocks of one launch: it holds fewer than 2^32 threads (more wrap around without an error: 2^22 + 5 blocks of 1,024 ran
// as 5), so larger calls are several launches.
constexpr int64_t most_blocks(int threads) { return 0xffffffffll / threads; }

}  // namespace hlr
