// The scales of the FP8 cache with a scale per block and kv head.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace kvfp8 {

// Scales are powers of two from 2^-60 to 2^120.  120 is what the largest float needs (448 * 2^120 >= 2^128).
// -60 keeps 1 / s, which the attention kernels sum weights by, and such a sum over 2^31 tokens within float's
// range.
constexpr int kMinScaleExp = -60, kMaxScaleExp = 120;

// (0 is a block that nothing was written to)
__device__ __forceinline__ bool block_scale_ok(float s) {
    const uint32_t bits = __float_as_uint(s);
    constexpr uint32_t kLow = static_cast<uint32_t>(kMinScaleExp + 127) << 23, kHigh = static_cast<uint32_t>(kMaxScaleExp + 127) << 23;
    return (bits & 0x7FFFFFu) == 0u && bits - kLow <= kHigh - kLow;
}
// 1 / s, exactly
__device__ __forceinline__ float block_scale_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }

}  // namespace kvfp8
