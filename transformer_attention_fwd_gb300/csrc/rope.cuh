// rope.cuh -- rotary positions on rows of D elements held by groups of lanes,
// shared by the rotation kernels (rope.cu) and the paged appends (append.cu,
// append_e4m3.cu).
//
// A pair (a, b) of one head at position t turns by the angle t * f of its
// frequency f:  (a cos - b sin, b cos + a sin), times the rotation's
// magnitude.  f arrives as a fraction of a turn per position in units of
// 2^-64 turn, so t * f modulo one turn is the low 64 bits of one integer
// product: exact, whatever the position.  The angle's error is |t| times the
// table's (2^-65 turns where it was rounded to nearest once; attn_rope_turns
// computes in double, 2^-53 turns) and the 2^-33 turns of its top 32 bits.
//
// A lane holds two 16-byte chunks of a row, chosen so that both elements of
// each of its pairs are its own: chunks j and j + half for the halves layout,
// any two for adjacent pairs.  Then nothing is exchanged between lanes, and
// pairs are worked on two at a time as packed fp32 (first elements A, second
// elements B).  Only halves that are no whole number of chunks go through
// shared memory.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "sm100.cuh"

namespace attn {

enum RopeLayout {
    kRopeAdjacent = 0,  // pairs (2i, 2i+1)
    kRopeHalves = 1,    // pairs (i, i + half), half a whole number of 16-byte chunks
    kRopeHalvesOdd = 2  // pairs (i, i + half), any half
};

// Element types: words of a chunk to and from fp32.
struct RopeBf16 {
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo_to_f32(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi_to_f32(w); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
};
struct RopeF16 {
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ float lo(uint32_t w) { return f16_lo_to_f32(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return f16_hi_to_f32(w); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_f16x2(a, b); }
};
struct RopeF32 {
    static constexpr int kBytes = 4;
};

// The rotation of one call.
struct RopeTable {
    const unsigned long long* turns;  // [half], 2^-64 turns per position
    int half;                         // rotated pairs; the head's first 2 * half elements turn
    float magnitude;
};

// magnitude * (cos, sin) of a pair's angle.  Of the phase's top 32 bits (half turns of
// 2^-31), the multiple of 128 next to them is exact as a float; its sine and cosine are
// turned by the rest, at most 2^-25 half turns, to first order (the second is under 2^-47).
// The float nearest to all 32 bits instead would leave an error of that size, more than
// sincospif's own.
__device__ __forceinline__ float2 rope_cos_sin(const RopeTable& t, int pair, int position) {
    const unsigned long long phase =
        static_cast<unsigned long long>(static_cast<long long>(position)) * t.turns[pair];
    const unsigned near = static_cast<unsigned>((phase + 0x80000000u) >> 32) + 64u;  // wraps by whole turns
    const float rest = static_cast<float>(static_cast<int>(near & 127u) - 64) * (0x1p-31f * 3.14159265f);
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(near & ~127u)) * 0x1p-31f, &s, &c);
    return make_float2(fmaf(-s, rest, c) * t.magnitude, fmaf(c, rest, s) * t.magnitude);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// kWeights: elements are multiplied by weights (the norm's) on the way.
template <typename E, int D, int kLayout, bool kWeights = false>
struct Rope {
    static constexpr int kChunk = 16 / E::kBytes;       // elements of a 16-byte chunk; pairs of a lane
    static constexpr int kLanes = D / (2 * kChunk);     // lanes of a row
    static constexpr int kRows = 32 / kLanes;           // rows of a warp step
    static constexpr int kP2 = kChunk / 2;              // pairs of pairs of a lane
    static constexpr int kScratch = kLayout == kRopeHalvesOdd ? kRows * D : 0;  // floats a warp needs

    struct Raw {
        uint4 c0, c1;
    };
    struct Pairs {  // pairs 2k, 2k + 1: first elements, second elements
        uint64_t a[kP2], b[kP2];
    };
    // A row's result from its pairs: a' = a * aa + b * ab, b' = b * bb + a * ba.
    // Without weights aa = bb = cos and ab = -ba = -sin, of which one each is
    // kept.
    struct Coef {
        uint64_t aa[kP2], ab[kP2], bb[kWeights ? kP2 : 1], ba[kWeights ? kP2 : 1];
    };

    // First elements of lane j's chunks.
    static __device__ __forceinline__ int first(int j, int half) {
        if (kLayout != kRopeHalves) return j * kChunk;
        const int hc = half / kChunk;
        return (j < hc ? j : 2 * hc + 2 * (j - hc)) * kChunk;
    }
    static __device__ __forceinline__ int second(int j, int half) {
        if (kLayout != kRopeHalves) return (j + kLanes) * kChunk;
        const int hc = half / kChunk;
        return (j < hc ? j + hc : 2 * hc + 2 * (j - hc) + 1) * kChunk;
    }
    // Pair i of lane j.
    static __device__ __forceinline__ int pair(int j, int i) {
        if (kLayout == kRopeAdjacent)
            return i < kP2 ? j * kP2 + i : (j + kLanes) * kP2 + i - kP2;
        return j * kChunk + i;
    }

    static __device__ __forceinline__ Raw load(const void* first_chunk, const void* second_chunk) {
        return Raw{*static_cast<const uint4*>(first_chunk), *static_cast<const uint4*>(second_chunk)};
    }
    static __device__ __forceinline__ Raw zero() { return Raw{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }

    static __device__ __forceinline__ Pairs ones() {
        Pairs p;
#pragma unroll
        for (int i = 0; i < kP2; ++i) p.a[i] = p.b[i] = f2_pack(1.0f, 1.0f);
        return p;
    }
    static __device__ __forceinline__ Pairs unpack(const Raw& r) {
        Pairs p;
        if constexpr (E::kBytes == 4) {
            const float x[4] = {__uint_as_float(r.c0.x), __uint_as_float(r.c0.y), __uint_as_float(r.c0.z), __uint_as_float(r.c0.w)};
            const float y[4] = {__uint_as_float(r.c1.x), __uint_as_float(r.c1.y), __uint_as_float(r.c1.z), __uint_as_float(r.c1.w)};
            if (kLayout == kRopeAdjacent) {
                p.a[0] = f2_pack(x[0], x[2]); p.b[0] = f2_pack(x[1], x[3]);
                p.a[1] = f2_pack(y[0], y[2]); p.b[1] = f2_pack(y[1], y[3]);
            } else {
                p.a[0] = f2_pack(x[0], x[1]); p.a[1] = f2_pack(x[2], x[3]);
                p.b[0] = f2_pack(y[0], y[1]); p.b[1] = f2_pack(y[2], y[3]);
            }
        } else {
            const uint32_t x[4] = {r.c0.x, r.c0.y, r.c0.z, r.c0.w}, y[4] = {r.c1.x, r.c1.y, r.c1.z, r.c1.w};
            if (kLayout == kRopeAdjacent) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    p.a[k] = f2_pack(E::lo(x[2 * k]), E::lo(x[2 * k + 1]));
                    p.b[k] = f2_pack(E::hi(x[2 * k]), E::hi(x[2 * k + 1]));
                    p.a[kP2 - 2 + k] = f2_pack(E::lo(y[2 * k]), E::lo(y[2 * k + 1]));
                    p.b[kP2 - 2 + k] = f2_pack(E::hi(y[2 * k]), E::hi(y[2 * k + 1]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < kP2; ++k) {
                    p.a[k] = f2_pack(E::lo(x[k]), E::hi(x[k]));
                    p.b[k] = f2_pack(E::lo(y[k]), E::hi(y[k]));
                }
            }
        }
        return p;
    }

    // The elements in the chunks' order.
    static __device__ __forceinline__ void elements(const Pairs& p, float (&x)[kChunk], float (&y)[kChunk]) {
        if (kLayout == kRopeAdjacent) {
#pragma unroll
            for (int k = 0; k < kP2 / 2; ++k) {
                f2_unpack(p.a[k], x[4 * k], x[4 * k + 2]);
                f2_unpack(p.b[k], x[4 * k + 1], x[4 * k + 3]);
                f2_unpack(p.a[kP2 / 2 + k], y[4 * k], y[4 * k + 2]);
                f2_unpack(p.b[kP2 / 2 + k], y[4 * k + 1], y[4 * k + 3]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kP2; ++k) {
                f2_unpack(p.a[k], x[2 * k], x[2 * k + 1]);
                f2_unpack(p.b[k], y[2 * k], y[2 * k + 1]);
            }
        }
    }

    static __device__ __forceinline__ uint4 pack(const float (&x)[kChunk]) {
        if constexpr (E::kBytes == 4)
            return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else
            return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7]));
    }
    static __device__ __forceinline__ void store(void* first_chunk, void* second_chunk, const Pairs& p) {
        float x[kChunk], y[kChunk];
        elements(p, x, y);
        *static_cast<uint4*>(first_chunk) = pack(x);
        *static_cast<uint4*>(second_chunk) = pack(y);
    }

    static __device__ __forceinline__ void store(void* first_chunk, void* second_chunk, const Raw& r) {
        *static_cast<uint4*>(first_chunk) = r.c0;
        *static_cast<uint4*>(second_chunk) = r.c1;
    }

    // Which of lane j's pairs turn.
    static __device__ __forceinline__ unsigned turning(int half, int j) {
        unsigned on = 0;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) on |= pair(j, i) < half ? 1u << i : 0u;
        return on;
    }
    // Lane j's coefficients from a token's table, and from its weights.
    static __device__ __forceinline__ void coefficients(const float* table, int j, Coef& k,
                                                        const Pairs* w = nullptr) {
        if constexpr (kLayout != kRopeHalvesOdd) {  // the odd layout reads them where they are used
#pragma unroll
            for (int i = 0; i < kP2; i += 2) {  // four pairs next to one another (fp32 adjacent: two)
                k.aa[i] = *reinterpret_cast<const uint64_t*>(table + pair(j, 2 * i));
                k.ab[i] = *reinterpret_cast<const uint64_t*>(table + D / 2 + pair(j, 2 * i));
                k.aa[i + 1] = *reinterpret_cast<const uint64_t*>(table + pair(j, 2 * i + 2));
                k.ab[i + 1] = *reinterpret_cast<const uint64_t*>(table + D / 2 + pair(j, 2 * i + 2));
            }
            if constexpr (kWeights) {
#pragma unroll
                for (int i = 0; i < kP2; ++i) {
                    k.bb[i] = f2_mul(k.aa[i], w->b[i]);
                    k.ba[i] = f2_mul(f2_mul(k.ab[i], f2_pack(-1.0f, -1.0f)), w->a[i]);
                    k.aa[i] = f2_mul(k.aa[i], w->a[i]);
                    k.ab[i] = f2_mul(k.ab[i], w->b[i]);
                }
            }
        }
    }

    // Turns a row; on: turning().  All 32 lanes call it; table and scratch (the
    // lane group's D floats) are used in the HalvesOdd layout only.
    static __device__ __forceinline__ void turn(Pairs& p, const Coef& k, unsigned on, int half, int j,
                                                const float* table, float* scratch) {
        if constexpr (kLayout == kRopeHalvesOdd) {
            float x[kChunk], y[kChunk];
            elements(p, x, y);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                scratch[j * kChunk + i] = x[i];
                scratch[(j + kLanes) * kChunk + i] = y[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                x[i] = turned(scratch, table, half, j * kChunk + i);
                y[i] = turned(scratch, table, half, (j + kLanes) * kChunk + i);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kP2; ++i) {
                p.a[i] = f2_pack(x[2 * i], x[2 * i + 1]);
                p.b[i] = f2_pack(y[2 * i], y[2 * i + 1]);
            }
        } else {
            const bool whole = 2 * half == D;
#pragma unroll
            for (int i = 0; i < kP2; ++i) {
                // What does not turn takes nothing of its partner (0 * infinity would): its
                // coefficients are 1 and -0, and the zeros below are signed so that a is
                // added -0 and b is subtracted +0, which change no value, not -0 either.
                const uint64_t pa = whole ? p.a[i] : masked(p.a[i], on >> (2 * i), -0.0f);
                const uint64_t pb = whole ? p.b[i] : masked(p.b[i], on >> (2 * i), 0.0f);
                if constexpr (kWeights) {
                    p.a[i] = f2_fma(pb, k.ab[i], f2_mul(p.a[i], k.aa[i]));
                    p.b[i] = f2_fma(pa, k.ba[i], f2_mul(p.b[i], k.bb[i]));
                } else {
                    p.a[i] = f2_fma(pb, k.ab[i], f2_mul(p.a[i], k.aa[i]));
                    p.b[i] = f2_sub(f2_mul(p.b[i], k.aa[i]), f2_mul(pa, k.ab[i]));
                }
            }
        }
    }

    static __device__ __forceinline__ void scale(Pairs& p, float f) {
        const uint64_t ff = f2_pack(f, f);
#pragma unroll
        for (int i = 0; i < kP2; ++i) {
            p.a[i] = f2_mul(p.a[i], ff);
            p.b[i] = f2_mul(p.b[i], ff);
        }
    }
    static __device__ __forceinline__ void multiply(Pairs& p, const Pairs& w) {
#pragma unroll
        for (int i = 0; i < kP2; ++i) {
            p.a[i] = f2_mul(p.a[i], w.a[i]);
            p.b[i] = f2_mul(p.b[i], w.b[i]);
        }
    }
    // 1 / sqrt(mean(x^2) + eps) of a row.
    static __device__ __forceinline__ float rms_scale(const Pairs& p, float eps) {
        uint64_t ss = f2_mul(p.a[0], p.a[0]);
        ss = f2_fma(p.b[0], p.b[0], ss);
#pragma unroll
        for (int i = 1; i < kP2; ++i) {
            ss = f2_fma(p.a[i], p.a[i], ss);
            ss = f2_fma(p.b[i], p.b[i], ss);
        }
        float u, v;
        f2_unpack(ss, u, v);
        u += v;
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) u += __shfl_xor_sync(0xffffffffu, u, m);
        return rsqrtf(u * (1.0f / D) + eps);
    }

  private:
    // The two floats, each `none` unless its bit of `on` is set.
    static __device__ __forceinline__ uint64_t masked(uint64_t v, unsigned on, float none) {
        float lo, hi;
        f2_unpack(v, lo, hi);
        return f2_pack((on & 1u) ? lo : none, (on & 2u) ? hi : none);
    }
    static __device__ __forceinline__ float turned(const float* row, const float* table, int half, int i) {
        if (i >= 2 * half) return row[i];
        const int q = i < half ? i : i - half;
        const float c = table[q], n = table[D / 2 + q];
        return i < half ? fmaf(row[i + half], n, row[i] * c) : fmaf(row[i - half], -n, row[i] * c);
    }
};

// A token's table: cos of every pair (1 for those that do not turn), then the
// negated sines; entry i of D/2.
template <int D>
__device__ __forceinline__ void rope_entry(const RopeTable& t, int i, int position, float* table) {
    const float2 cs = i < t.half ? rope_cos_sin(t, i, position) : make_float2(1.0f, 0.0f);
    table[i] = cs.x;
    table[D / 2 + i] = -cs.y;
}
template <int D>
__device__ __forceinline__ void rope_fill(const RopeTable& t, int position, int lane, float* table) {
    for (int i = lane; i < D / 2; i += 32) rope_entry<D>(t, i, position, table);
    __syncwarp();
}

}  // namespace attn
