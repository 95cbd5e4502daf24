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

// V scales ride in the exponent of the attention's weights, 2^(s + log2 vs - m) with m 2^7 below a row's highest, and the row's sum adds
// them times 1 / vs.  A weight below 2^-126 is 0 in that sum, where 2^(s - m) should be added: under 2^(-126 - log2 vs), while the
// highest one adds 2^(7 - log2 of its vs) at least.  And when m rises by more than 126, what was summed before (under 2^(15 - log2 vs) a token)
// is multiplied by 0.  While the V scales met so far are within 2^kSumSpan of each other, that loses under 2^-54 of the sum for each
// token; from there on the sum takes 2^(s - m) itself, and its factors in two halves.
constexpr int kSumSpan = 64;

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }

}  // namespace kvfp8
