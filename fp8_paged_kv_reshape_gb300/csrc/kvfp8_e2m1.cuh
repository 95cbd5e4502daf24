// Device helpers of the 4-bit cache (sm_103a): E2M1 by the hardware's packed converters.  Apart from
// kvfp8_device.cuh, so that the 8-bit kernels' sources are their own.
#pragma once

#include <cstdint>

namespace kvfp8 {

// Eight floats -> eight E2M1 codes (x[0] in the lowest nibble): nearest even, saturating at 6;
// the sign bit is the operand's.
__device__ __forceinline__ uint32_t e2m1x8_from_f32(const float *x) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight E2M1 codes -> four fp16 pairs (nibbles 2i, 2i+1 in the halves of r[i]).
__device__ __forceinline__ void f16x2_from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

}  // namespace kvfp8
