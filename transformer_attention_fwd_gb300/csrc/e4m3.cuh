// e4m3.cuh -- the 8-bit element of the quantised cache: 4 exponent and 3
// mantissa bits, largest value 448, NaN but no infinity.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "sm100.cuh"

namespace attn {

constexpr float kE4m3Max = 448.0f;
// A scale is never below this: 448 * 2^-100 is far under any cache's content.
constexpr float kE4m3MinScale = 0x1p-100f;

// Two fp32 values to two codes (a in the low byte): round to nearest even,
// beyond 448 to 448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pack2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
    return e4m3_pack2(a, b) | (e4m3_pack2(c, d) << 16);
}
// Four codes to two pairs of fp16 values (lower two codes, upper two): exact.
__device__ __forceinline__ void e4m3_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}

// Four codes times a ratio, rounded to codes again (exact for a power of two,
// but for results under 2^-6).
__device__ __forceinline__ uint32_t e4m3_rescale(uint32_t codes, float ratio) {
    uint32_t lo, hi;
    e4m3_to_f16x4(codes, lo, hi);
    return e4m3_pack4(f16_lo_to_f32(lo) * ratio, f16_hi_to_f32(lo) * ratio,
                      f16_lo_to_f32(hi) * ratio, f16_hi_to_f32(hi) * ratio);
}

}  // namespace attn
