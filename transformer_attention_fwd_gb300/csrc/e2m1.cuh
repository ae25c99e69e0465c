// e2m1.cuh -- the 4-bit element of the quantised cache (sign, 2 exponent bits and 1
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and its scales, one e4m3 value for each 16
// elements of a row.  Two codes share a byte, the even element in the low half.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "e4m3.cuh"

namespace attn {

constexpr float kE2m1Max = 6.0f;
constexpr float kRowScaleMin = 0x1p-9f;  // the smallest e4m3 value above 0
constexpr int kRowScaleSpan = 16;        // elements of a scale

// The four bytes' codes as pairs of fp16 values: exact.
__device__ __forceinline__ void e2m1_to_f16x8(uint32_t codes, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(codes));
}
// Eight fp32 values to codes: to the nearest, halfway to the even code, beyond 6 to 6.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// Two e4m3 values (the low 16 bits) as fp16: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t codes) {
    uint32_t v;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(v) : "r"(codes));
    return v;
}
// Each half of a word in both halves of one.
__device__ __forceinline__ void both_halves(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 %0, {l, l};\n\tmov.b32 %1, {h, h};\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(x));
}
// Products of fp16 pairs.  A code times its scale is exact: 2 and 4 significant bits,
// between 2^-10 and 2688.
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes times scales in fp16 or bf16, exact in either.  Two groups' scales as factors:
template <bool kF16>
__device__ __forceinline__ void e2m1_scales(uint32_t codes, uint32_t (&by)[2]) {
    const uint32_t f = e4m3_to_f16x2(codes);
    if (kF16) {
        both_halves(f, by[0], by[1]);
    } else {
        const float lo = f16_lo_to_f32(f) * 0x1p112f, hi = f16_hi_to_f32(f) * 0x1p112f;
        by[0] = pack_bf16x2(lo, lo);
        by[1] = pack_bf16x2(hi, hi);
    }
}
// fp16 values of two codes times such a factor.  In bf16 their bits, three places down, are the
// values times 2^-112 (the low bits are 0): no conversion, and the factor has 2^112.
template <bool kF16>
__device__ __forceinline__ uint32_t e2m1_times(uint32_t v, uint32_t by) {
    if (kF16) return f16x2_mul(v, by);
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(((v >> 3) & 0x0fff0fffu) | (v & 0x80008000u)), "r"(by));
    return d;
}

}  // namespace attn
