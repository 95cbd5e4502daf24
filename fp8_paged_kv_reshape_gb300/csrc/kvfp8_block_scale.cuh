// The scales of the FP8 cache with a scale per block and kv head.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace kvfp8 {

// Scales lie between 2^-60 and 2^120.  120 is what the largest float needs (448 * 2^120 >= 2^128).  -60
// keeps 1 / s, which the attention kernels sum weights by, and such a sum over 2^31 tokens within float's
// range.
constexpr int kMinScaleExp = -60, kMaxScaleExp = 120;

// (false for a NaN; 0 is a block that nothing was written to)
__device__ __forceinline__ bool block_scale_ok(float s) { return s >= 0x1p-60f && s <= 0x1p120f; }

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }

}  // namespace kvfp8
