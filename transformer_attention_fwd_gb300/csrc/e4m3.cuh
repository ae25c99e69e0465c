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
// Two codes (the low 16 bits) to two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r) : "r"(codes));
    return r;
}

// Four codes times a ratio, rounded to codes again (exact for a power of two,
// but for results under 2^-6).
__device__ __forceinline__ uint32_t e4m3_rescale(uint32_t codes, float ratio) {
    const uint32_t lo = e4m3_to_f16x2(codes & 0xffffu), hi = e4m3_to_f16x2(codes >> 16);
    return e4m3_pack4(f16_lo_to_f32(lo) * ratio, f16_hi_to_f32(lo) * ratio,
                      f16_lo_to_f32(hi) * ratio, f16_hi_to_f32(hi) * ratio);
}

}  // namespace attn
