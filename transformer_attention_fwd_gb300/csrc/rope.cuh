// rope.cuh -- rotary positions on rows of D elements held by lane groups of a
// warp, shared by the rotation kernels (rope.cu) and the paged append
// (append.cu, append_e4m3.cu).
//
// A pair (a, b) of one head at position t turns by the angle t * f of its
// frequency f:  (a cos - b sin, b cos + a sin), times the rotation's
// magnitude.  f arrives as a fraction of a turn per position in units of
// 2^-64 turn, so t * f modulo one turn is the low 64 bits of one integer
// product: exact, whatever the position.  The angle's error is the table's
// rounding, |t| * 2^-65 turns, and the 2^-25 half turns of the float the top
// 32 bits are rounded to.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "sm100.cuh"

namespace attn {

constexpr int kRopeChunk = 8;  // elements of a row one lane holds

// How the pairs of a head are laid out, as far as the exchange between lanes
// goes.
enum RopeLayout {
    kRopeAdjacent = 0,  // (2i, 2i+1): inside one lane
    kRopeHalves = 1,    // (i, i + rot/2), rot/2 a multiple of 8: whole chunks trade lanes
    kRopeHalvesOdd = 2  // (i, i + rot/2), any even rot: elements traded through shared memory
};

// Element types: eight elements of a row as loaded (Raw), and as fp32.
struct RopeBf16 {
    using Raw = uint4;
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ Raw load(const void* p) { return *static_cast<const uint4*>(p); }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void unpack(const Raw& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo_to_f32(w[i]);
            f[2 * i + 1] = bf16_hi_to_f32(w[i]);
        }
    }
    static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
        *static_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ void store_raw(void* p, const Raw& u) { *static_cast<uint4*>(p) = u; }
    static __device__ __forceinline__ Raw shuffle(const Raw& u, int lane) {
        return make_uint4(__shfl_sync(0xffffffffu, u.x, lane), __shfl_sync(0xffffffffu, u.y, lane),
                          __shfl_sync(0xffffffffu, u.z, lane), __shfl_sync(0xffffffffu, u.w, lane));
    }
};

struct RopeF16 {
    using Raw = uint4;
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ Raw load(const void* p) { return *static_cast<const uint4*>(p); }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void unpack(const Raw& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = f16_lo_to_f32(w[i]);
            f[2 * i + 1] = f16_hi_to_f32(w[i]);
        }
    }
    static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
        *static_cast<uint4*>(p) = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]),
                                             pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ void store_raw(void* p, const Raw& u) { *static_cast<uint4*>(p) = u; }
    static __device__ __forceinline__ Raw shuffle(const Raw& u, int lane) { return RopeBf16::shuffle(u, lane); }
};

struct RopeF32 {
    struct Raw {
        float4 a, b;
    };
    static constexpr int kBytes = 4;
    static __device__ __forceinline__ Raw load(const void* p) {
        const float4* q = static_cast<const float4*>(p);
        return Raw{q[0], q[1]};
    }
    static __device__ __forceinline__ Raw zero() {
        return Raw{make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    }
    static __device__ __forceinline__ void unpack(const Raw& u, float (&f)[8]) {
        f[0] = u.a.x; f[1] = u.a.y; f[2] = u.a.z; f[3] = u.a.w;
        f[4] = u.b.x; f[5] = u.b.y; f[6] = u.b.z; f[7] = u.b.w;
    }
    static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
        float4* q = static_cast<float4*>(p);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
    static __device__ __forceinline__ void store_raw(void* p, const Raw& u) {
        float4* q = static_cast<float4*>(p);
        q[0] = u.a;
        q[1] = u.b;
    }
    static __device__ __forceinline__ Raw shuffle(const Raw& u, int lane) {
        Raw r;
        r.a.x = __shfl_sync(0xffffffffu, u.a.x, lane); r.a.y = __shfl_sync(0xffffffffu, u.a.y, lane);
        r.a.z = __shfl_sync(0xffffffffu, u.a.z, lane); r.a.w = __shfl_sync(0xffffffffu, u.a.w, lane);
        r.b.x = __shfl_sync(0xffffffffu, u.b.x, lane); r.b.y = __shfl_sync(0xffffffffu, u.b.y, lane);
        r.b.z = __shfl_sync(0xffffffffu, u.b.z, lane); r.b.w = __shfl_sync(0xffffffffu, u.b.w, lane);
        return r;
    }
};

// The rotation of one call.
struct RopeTable {
    const unsigned long long* turns;  // [half], 2^-64 turns per position
    int half;                         // rotated pairs; the head's first 2 * half elements turn
    float magnitude;
};

__device__ __forceinline__ void rope_sincos(const RopeTable& t, int pair, int position, float* s,
                                            float* c) {
    const unsigned long long phase =
        static_cast<unsigned long long>(static_cast<long long>(position)) * t.turns[pair];
    const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f;
    sincospif(half_turns, s, c);
}

// What a lane multiplies its eight elements and their partners by:
// y[e] = x[e] * own[e] + partner[e] * other[e].
struct RopeCoef {
    float own[8], other[8];
};

// Pair and sign of element i of a head: the pair it belongs to (-1 outside the
// rotated part) and whether it is the pair's first element.
template <int kLayout>
__device__ __forceinline__ int rope_pair(int i, int half, bool* first) {
    if (i >= 2 * half) return -1;
    if (kLayout == kRopeAdjacent) {
        *first = (i & 1) == 0;
        return i >> 1;
    }
    *first = i < half;
    return *first ? i : i - half;
}

// Element a lane's element i trades with (itself outside the rotated part).
template <int kLayout>
__device__ __forceinline__ int rope_partner(int i, int half) {
    if (i >= 2 * half) return i;
    if (kLayout == kRopeAdjacent) return i ^ 1;
    return i < half ? i + half : i - half;
}

// weight: nullptr, or the norm's weight row (fp32 values come from Row::unpack
// of its chunks); the partner's element carries the partner's weight.
template <typename Row, int kLayout>
__device__ __forceinline__ void rope_coefficients(const RopeTable& t, int chunk0, int position,
                                                  const void* weight, RopeCoef& k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bool first = true;
        const int pair = rope_pair<kLayout>(chunk0 + e, t.half, &first);
        float s = 0.0f, c = 1.0f;
        if (pair >= 0) {
            if (kLayout == kRopeAdjacent && (e & 1)) {  // the pair's even element has them already
                k.own[e] = k.own[e - 1];
                k.other[e] = -k.other[e - 1];
                continue;
            }
            rope_sincos(t, pair, position, &s, &c);
            s *= t.magnitude;
            c *= t.magnitude;
        }
        k.own[e] = c;
        k.other[e] = first ? -s : s;
    }
    if (weight != nullptr) {
        float w[8];
        const uint8_t* base = static_cast<const uint8_t*>(weight);
        Row::unpack(Row::load(base + static_cast<int64_t>(chunk0) * Row::kBytes), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) k.own[e] *= w[e];
        if (kLayout == kRopeAdjacent) {
#pragma unroll
            for (int e = 0; e < 8; ++e) k.other[e] *= w[e ^ 1];
        } else if (kLayout == kRopeHalves) {
            const int p0 = rope_partner<kLayout>(chunk0, t.half);
            Row::unpack(Row::load(base + static_cast<int64_t>(p0) * Row::kBytes), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) k.other[e] *= w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int p = rope_partner<kLayout>(chunk0 + e, t.half);
                float wp[8];
                Row::unpack(Row::load(base + static_cast<int64_t>(p & ~7) * Row::kBytes), wp);
                float v = wp[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) v = (p & 7) == j ? wp[j] : v;
                k.other[e] *= v;
            }
        }
    }
}

// The partners of a lane's eight elements.  All 32 lanes call it; `row` is the
// lane group's D floats of shared memory (kRopeHalvesOdd only).  Elements
// outside the rotated part get 0, so that 0 * infinity does not reach them.
template <typename Row, int kLayout, int D>
__device__ __forceinline__ void rope_exchange(const typename Row::Raw& raw, const float (&x)[8],
                                              int half, int lane, float* row, float (&xp)[8]) {
    const int sub = lane % (D / 8);
    if (kLayout == kRopeAdjacent) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
    } else if (kLayout == kRopeHalves) {
        const int hc = half / 8;
        const int to = sub >= 2 * hc ? lane : (sub < hc ? lane + hc : lane - hc);
        Row::unpack(Row::shuffle(raw, to), xp);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) row[sub * 8 + e] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = row[rope_partner<kLayout>(sub * 8 + e, half)];
        __syncwarp();
    }
    if (2 * half < D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = sub * 8 + e < 2 * half ? xp[e] : 0.0f;
    }
}

// 1 / sqrt(mean(x^2) + eps) over a row held by D/8 neighbouring lanes.
template <int D>
__device__ __forceinline__ float rope_rms_scale(const float (&x)[8], float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int m = D / 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    return rsqrtf(ss * (1.0f / D) + eps);
}

}  // namespace attn
