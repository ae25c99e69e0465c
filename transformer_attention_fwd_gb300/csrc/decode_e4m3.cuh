// decode_e4m3.cuh -- shared by the two decodes over the 8-bit cache: the arithmetic
// of one 16-key tile, the copies that feed it, and the merge of partial results.
// decode_e4m3.cu says what is computed and how.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "e4m3.cuh"
#include "sm100.cuh"

namespace attn {

constexpr int kTile = 16;          // keys of a tile
constexpr int kMaxPrefixB = 1024;  // requests whose tile counts a CTA sums itself
constexpr float kSlack = 6.0f;
// A weight is held as two fp16 terms, what the first leaves out in the second, relative
// to 2^mv, mv lying kLift under the maximum it follows: the largest weights are 2^kLift to
// 2^(kLift + kSlack), inside fp16.  The two terms are within 2^-24 of a weight from 1/2 on
// and within 2^-25 of the smaller ones: from 2^-kLow on (kLift + kLow binades under the
// reference) within 2^-14 of itself.  Still smaller ones get products of their own,
// relative to the largest of them (unit_tile).
constexpr float kLift = 9.0f;
constexpr float kLow = 11.0f;
// A weight this many binades under 2^mv, 2^-125 of the reference, is 0.
constexpr float kGone = 116.0f;
// References start here: below any score, and finite, so that no difference of
// two of them is NaN.
constexpr float kLowest = -3.0e38f;
constexpr float kLn2 = 0.69314718055994531f;

// A tile in shared memory: K rows, V rows, their scales.
template <int D>
constexpr int kStageBytes = 2 * kTile * D + 2 * kTile * 4;

struct E4m3Params {
    const uint16_t* q;
    const uint8_t* kv;
    const float* scales;
    const int* block_table;
    const int* seq_lens;
    uint16_t* o;
    float* lse;
    long long* cum;  // [B + 1] tiles before each request (global: more than kMaxPrefixB requests)
    longlong2* geom;  // {all tiles, tiles of a CTA's slice}
    int4* first;     // [grid] {request, unit, tile, tiles} a CTA's slice starts in
    float* ws_o;     // [2 * grid, HC, D] pieces of cut units, not normalised
    float4* ws_ml;   // [2 * grid, HC] their {m, sum, mv}
    unsigned* status;
    PageDivider page;
    int B, Hq, Hkv, group, chunks, max_pages, num_blocks;
    float scale_log2;
};

// n / d for n, d >= 0: most fit in 32 bits, whose division is several times shorter.
__device__ __forceinline__ long long divide(long long n, int d) {
    return (n >> 32) == 0 ? static_cast<long long>(static_cast<unsigned>(n) / static_cast<unsigned>(d)) : n / d;
}

// One place in the sequence of tiles.
struct Cursor {
    int b, unit, tile, tiles, len;
};

// A length inside the block table (bad ones are reported by tile_prefix).
__device__ __forceinline__ int clamped(const E4m3Params& p, int L) {
    const int most = p.max_pages * p.page.size;
    return L < 0 ? 0 : (L > most ? most : L);
}
__device__ __forceinline__ int clamped_len(const E4m3Params& p, int b) { return clamped(p, p.seq_lens[b]); }

// The next tile; there has to be one.
__device__ __forceinline__ void cursor_next(const E4m3Params& p, const long long* cum, Cursor& c) {
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    if (++c.unit < p.Hkv * p.chunks) return;
    c.unit = 0;
    do {
        ++c.b;
        c.tiles = static_cast<int>(cum[c.b + 1] - cum[c.b]);
    } while (c.tiles == 0);
    c.len = clamped_len(p, c.b);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 (4) bytes into shared memory; 0 bytes of them: zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Place of a row's 16-byte chunk: rows of eight chunks rotate theirs by the row,
// rows of four by the row pair, so that both products' reads spread over the banks.
template <int D>
__device__ __forceinline__ int chunk_at(int row, int chunk) {
    return D == 128 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3));
}

// The 2 or 4 words of a lane's D/8 columns of a V row.
template <int D>
__device__ __forceinline__ void load_v(const uint8_t* rows, int row, int g, uint32_t (&w)[D / 32]) {
    if (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(rows + row * D + chunk_at<D>(row, g) * 16);
        w[0] = u.x; w[1] = u.y; w[D / 32 - 2] = u.z; w[D / 32 - 1] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(rows + row * D + chunk_at<D>(row, g >> 1) * 16 + (g & 1) * 8);
        w[0] = u.x; w[1] = u.y;
    }
}

template <bool kF16>
__device__ __forceinline__ float elem_f32(uint16_t x) {
    return kF16 ? f16_lo_to_f32(x) : bf16_lo_to_f32(x);
}

// The state of the unit a warp is in.  Lane (g, t) = (lane / 4, lane % 4) works
// on heads 2t and 2t + 1 (of each half of eight).
template <int D, int HC>
struct UnitState {
    static constexpr int kR = HC / 8;       // halves of eight heads
    uint32_t qb[D / 16][kR][2];             // Q^T operand: head g, two runs of inner indices
    float qs[kR][2];                        // what a product with it is multiplied by
    float m[kR][2], l[kR][2], mv[kR][2];    // reference and this lane's sum of the p; O's reference
    float o[kR][D / 16][4];                 // O^T: two columns of V, two heads
};

// Q fragments of heads hq0 .. hq0 + heads - 1, each times a power of two that
// takes its largest element to [512, 1024).  Elements down to 2^-24 of the largest are
// then exact in fp16 (bf16's 8 bits, fp16's 11), smaller ones off by at most 2^-34 of the
// largest: a thousandth of the rounding of the largest's product in an fp32 sum.
template <int D, int HC, bool kF16>
__device__ __forceinline__ void unit_begin(const E4m3Params& p, const Cursor& c, int lane,
                                           UnitState<D, HC>& s) {
    const int g = lane >> 2, t = lane & 3;
    const int hkv = p.chunks == 1 ? c.unit : c.unit / p.chunks, chunk = c.unit - hkv * p.chunks;
    const int heads = min(HC, p.group - chunk * HC);
    const int hq0 = hkv * p.group + chunk * HC;
#pragma unroll
    for (int r = 0; r < HC / 8; ++r) {
        const int h = r * 8 + g;
        uint32_t w[D / 8];  // the lane's D/4 columns, t * D/4 on
        float most = 0.0f;
        if (h < heads) {
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + (static_cast<int64_t>(c.b) * p.Hq + hq0 + h) * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 u = src[i];
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            most = fmaxf(most, fmaxf(fabsf(elem_f32<kF16>(w[i] & 0xffffu)), fabsf(elem_f32<kF16>(w[i] >> 16))));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // up = 2^(9 - floor(log2 most)), 1 for zero, subnormal or non-finite rows.
        const int e = static_cast<int>(__float_as_uint(most) >> 23);
        const int k = (e == 0 || e == 255) ? 0 : max(-126, min(126, 9 - (e - 127)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
        const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        s.qs[r][0] = __shfl_sync(0xffffffffu, back, 8 * t);
        s.qs[r][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
        // Product step j takes columns 4 j .. 4 j + 3 of the lane's: the first two as
        // inner indices 2t, 2t + 1, the others as 2t + 8, 2t + 9.
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            s.qb[i / 2][r][i & 1] =
                pack_f16x2(elem_f32<kF16>(w[i] & 0xffffu) * up, elem_f32<kF16>(w[i] >> 16) * up);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s.m[r][i] = s.mv[r][i] = kLowest;
            s.l[r][i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s.o[r][j][i] = 0.0f;
    }
}

// Maximum over the lanes that hold the same heads.
__device__ __forceinline__ float heads_max(float m) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
    return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
}
__device__ __forceinline__ float heads_sum(float l) {
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    return l + __shfl_xor_sync(0xffffffffu, l, 16);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Factor from sum w v to O, 2^(mv - m) / l, but for the 2^-kLift that the sum is multiplied
// by first (out_of): V's scales reach down to where the whole factor would be no normal number.
__device__ __forceinline__ float out_factor(float m, float l, float mv) { return ex2_approx(mv - m + kLift) / l; }
__device__ __forceinline__ float out_of(float sum, float factor) { return sum * 0x1p-9f * factor; }
static_assert(kLift == 9.0f, "out_of");

// Folds {m, sum, mv} of a piece into e.
__device__ __forceinline__ void fold(float4& e, const float4& x) {
    const float m = fmaxf(e.x, x.x);
    e.y = e.y * ex2_approx(e.x - m) + x.y * ex2_approx(x.x - m);
    e.x = m;
    e.z = fmaxf(e.z, x.z);
}
// The same over lanes kFrom, 2 kFrom, .. 16 apart; every lane gets the result.
template <int kFrom>
__device__ __forceinline__ void fold_lanes(float4& e) {
    float m = e.x;
#pragma unroll
    for (int o = kFrom; o < 32; o <<= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        e.z = fmaxf(e.z, __shfl_xor_sync(0xffffffffu, e.z, o));
    }
    e.y *= ex2_approx(e.x - m);
    e.x = m;
#pragma unroll
    for (int o = kFrom; o < 32; o <<= 1) e.y += __shfl_xor_sync(0xffffffffu, e.y, o);
}

// A lane's D/32 neighbouring columns.
template <int D>
struct Columns {
    float c[D / 32];
    __device__ __forceinline__ void load(const float* row, int lane) {
        if constexpr (D == 128) {
            const float4 v = reinterpret_cast<const float4*>(row)[lane];
            c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
        } else {
            const float2 v = reinterpret_cast<const float2*>(row)[lane];
            c[0] = v.x; c[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(float* row, int lane) const {
        if constexpr (D == 128) reinterpret_cast<float4*>(row)[lane] = make_float4(c[0], c[1], c[2], c[3]);
        else reinterpret_cast<float2*>(row)[lane] = make_float2(c[0], c[1]);
    }
    __device__ __forceinline__ void add(const Columns& x, float w) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) c[i] = fmaf(x.c[i], w, c[i]);
    }
    template <bool kF16>
    __device__ __forceinline__ void store16(uint16_t* row, int lane, float f) const {
        using E = Elem16<kF16>;
        if constexpr (D == 128)
            reinterpret_cast<uint2*>(row)[lane] =
                make_uint2(E::pack(out_of(c[0], f), out_of(c[1], f)), E::pack(out_of(c[2], f), out_of(c[3], f)));
        else reinterpret_cast<uint32_t*>(row)[lane] = E::pack(out_of(c[0], f), out_of(c[1], f));
    }
};

// The merge of up to kParts parts of a unit by one warp: all heads' weights at
// once, lane h + HC * k holding those of head h's parts k, k + 32 / HC, ..
template <int D, int HC, int kParts>
struct MergedHeads {
    static constexpr int kApart = 32 / HC, kHeld = (kParts + kApart - 1) / kApart;
    float4 all;  // head lane % HC: the common references and sum
    float weight[kHeld];

    // part(k, h): {m, l, mv} of head h in part k < n.
    template <typename Part>
    __device__ __forceinline__ MergedHeads(int n, int lane, Part part) {
        float4 e[kHeld];
        all = make_float4(kLowest, 0.0f, kLowest, 0.0f);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int k = lane / HC + i * kApart;
            e[i] = k < n ? part(k, lane % HC) : make_float4(kLowest, 0.0f, kLowest, 0.0f);
            fold(all, e[i]);
        }
        fold_lanes<HC>(all);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) weight[i] = ex2_approx(e[i].z - all.z);
    }
    // Head h's sum of w v, and its {m, l, mv}; load(k, x): the lane's columns in part k.
    template <typename Load>
    __device__ __forceinline__ Columns<D> head(int h, int n, int lane, Load load, float4* ml) const {
        Columns<D> acc{};
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const float wt = __shfl_sync(0xffffffffu, weight[k / kApart], h + HC * (k % kApart));
            if (k >= n) continue;
            Columns<D> x;
            load(k, x);
            acc.add(x, wt);
        }
        *ml = make_float4(__shfl_sync(0xffffffffu, all.x, h), __shfl_sync(0xffffffffu, all.y, h),
                          __shfl_sync(0xffffffffu, all.z, h), 0.0f);
        return acc;
    }
};

// Two weights as two terms each, P^T's operand.
struct Weights {
    uint32_t hi, lo;
    __device__ __forceinline__ void set(float a, float b) {
        const uint32_t h = pack_f16x2(a, b);
        hi = transpose8x8(h);
        lo = transpose8x8(pack_f16x2(a - f16_lo_to_f32(h), b - f16_hi_to_f32(h)));
    }
};

// A head's heaviest weights out of the exponents left, and what the products with them are
// multiplied by; a lane's two keys.  Those taken are -inf from then on.
__device__ __forceinline__ float heaviest(float& e0, float& e1, float& w0, float& w1) {
    const float top = heads_max(fmaxf(e0, e1));
    const float down = top < 0.0f && top > -kGone ? floorf(top - kLift) : 0.0f;
    const bool later0 = e0 - down < -kLow, later1 = e1 - down < -kLow;  // false for NaN
    w0 = later0 ? 0.0f : ex2_approx(e0 - down);
    w1 = later1 ? 0.0f : ex2_approx(e1 - down);
    e0 = later0 ? e0 : -INFINITY;
    e1 = later1 ? e1 : -INFINITY;
    return ex2_approx(down);
}

// One tile of a warp's ring: scores, weights, and the weighted V rows.
template <int D, int HC, bool kWholePages>
__device__ __forceinline__ void unit_tile(const uint8_t* stage, int valid, int lane, UnitState<D, HC>& s) {
    constexpr int kR = HC / 8, kS = D / 16;
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* vrows = stage + kTile * D;
    const float* ks = reinterpret_cast<const float*>(stage + 2 * kTile * D);
    const float* vs = ks + kTile;
    // Key g's and key g + 8's columns of this lane, four to a product step.
    uint32_t kw[2][kS];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int row = n * 8 + g;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int chunk = D == 128 ? 2 * t + i : t;
            const uint4 u = *reinterpret_cast<const uint4*>(stage + row * D + chunk_at<D>(row, chunk) * 16);
            kw[n][4 * i] = u.x; kw[n][4 * i + 1] = u.y; kw[n][4 * i + 2] = u.z; kw[n][4 * i + 3] = u.w;
        }
    }
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int j = 0; j < 4; ++j) load_v<D>(vrows, 2 * t + (j & 1) + 8 * (j >> 1), g, vw[j]);
    float sc[kR][4], sd[kR][4];  // two chains of products
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[r][i] = sd[r][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kS; ++j) {
        uint32_t a0, a1, a2, a3;
        e4m3_to_f16x4(kw[0][j], a0, a2);
        e4m3_to_f16x4(kw[1][j], a1, a3);
#pragma unroll
        for (int r = 0; r < kR; ++r) mma_f16((j & 1) ? sd[r] : sc[r], a0, a1, a2, a3, s.qb[j][r][0], s.qb[j][r][1]);
    }
    // V^T's operand (with eight heads all of it now, while the products run): bytes 2i, 2i + 1 of two keys' words are
    // (k0, k1) of one column, then of the next.
    uint32_t va[kS][4];
    auto convert = [&](int i) {
        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
        e4m3_to_f16x4(__byte_perm(vw[0][i / 2], vw[1][i / 2], sel), va[i][0], va[i][1]);
        e4m3_to_f16x4(__byte_perm(vw[2][i / 2], vw[3][i / 2], sel), va[i][2], va[i][3]);
    };
    if (HC == 8)
#pragma unroll
        for (int i = 0; i < kS; ++i) convert(i);
    // Factors and lifts (log2 of V's scales) of keys g and g + 8: one pair for a tile
    // inside one page.
    constexpr int kF = kWholePages ? 1 : 2;
    float kk[kF], lift[kF];
#pragma unroll
    for (int n = 0; n < kF; ++n) {
        kk[n] = ks[kWholePages ? 0 : n * 8 + g];
        lift[n] = __log2f(vs[kWholePages ? 0 : n * 8 + g]);
    }
    float x[kR][4];  // exponents of p; those of w are x + lift
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[r][i] = (sc[r][i] + sd[r][i]) * (kk[(i >> 1) % kF] * s.qs[r][i & 1]);
    if (valid < kTile) {  // the unit's last tile
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((i >> 1) * 8 + g >= valid) x[r][i] = -INFINITY;
    }
    bool need = false;
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            need |= x[r][i] > fminf(s.m[r][i & 1], (s.mv[r][i & 1] + kLift) - lift[(i >> 1) % kF]) + kSlack;
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float m = fmaxf(s.m[r][i], heads_max(fmaxf(x[r][i], x[r][i + 2])));
                const float mv =
                    fmaxf(s.mv[r][i], heads_max(fmaxf(x[r][i] + lift[0], x[r][i + 2] + lift[kF - 1])) - kLift);
                const float alpha = ex2_approx(s.mv[r][i] - mv);
                s.l[r][i] *= ex2_approx(s.m[r][i] - m);
                s.m[r][i] = m;
                s.mv[r][i] = mv;
#pragma unroll
                for (int j = 0; j < kS; ++j) {
                    s.o[r][j][i] *= alpha;
                    s.o[r][j][i + 2] *= alpha;
                }
            }
        }
    }
    float e[kR][4], w[kR][4], least = INFINITY;  // the weights' exponents, the weights
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s.l[r][i & 1] += ex2_approx(x[r][i] - s.m[r][i & 1]);
            e[r][i] = x[r][i] + (lift[(i >> 1) % kF] - s.mv[r][i & 1]);
            w[r][i] = ex2_approx(e[r][i]);
            least = fminf(least, e[r][i]);
        }
    if (__all_sync(0xffffffffu, least >= -kLow)) {
        Weights pb[kR][2];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            pb[r][0].set(w[r][0], w[r][1]);
            pb[r][1].set(w[r][2], w[r][3]);
        }
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            if (HC != 8) convert(i);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                mma_f16(s.o[r][i], va[i][0], va[i][1], va[i][2], va[i][3], pb[r][0].hi, pb[r][1].hi);
                mma_f16(s.o[r][i], va[i][0], va[i][1], va[i][2], va[i][3], pb[r][0].lo, pb[r][1].lo);
            }
        }
        return;
    }
    // Some keys are far below their head's reference (or past the unit's end).  The
    // weights go in groups of kLift + kLow binades, from the largest down, each with
    // products of its own relative to 2^(mv + down): so a head whose reference is one
    // heavy key with an empty value still has the others'.
    bool more = true;
    while (more) {
        Weights pb[kR][2];
        float back[kR][2];
        float most = -INFINITY;
        auto half = [&](int r) {
            back[r][0] = heaviest(e[r][0], e[r][2], w[r][0], w[r][2]);
            back[r][1] = heaviest(e[r][1], e[r][3], w[r][1], w[r][3]);
            most = fmaxf(most, fmaxf(fmaxf(e[r][0], e[r][1]), fmaxf(e[r][2], e[r][3])));
            pb[r][0].set(w[r][0], w[r][1]);
            pb[r][1].set(w[r][2], w[r][3]);
        };
        half(0);  // (a loop here is not unrolled, and puts the arrays in memory)
        if (kR == 2) half(kR - 1);
        more = __any_sync(0xffffffffu, most > -kGone);
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            if (HC != 8) convert(i);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(part, va[i][0], va[i][1], va[i][2], va[i][3], pb[r][0].hi, pb[r][1].hi);
                mma_f16(part, va[i][0], va[i][1], va[i][2], va[i][3], pb[r][0].lo, pb[r][1].lo);
#pragma unroll
                for (int n = 0; n < 4; ++n) s.o[r][i][n] = fmaf(part[n], back[r][n & 1], s.o[r][i][n]);
            }
        }
    }
}

template <bool kF16, int N>
__device__ __forceinline__ void store_row(uint16_t* dst, const float (&v)[N]) {
    using E = Elem16<kF16>;
#pragma unroll
    for (int i = 0; i < N; i += 8)
        *reinterpret_cast<uint4*>(dst + i) = make_uint4(E::pack(v[i], v[i + 1]), E::pack(v[i + 2], v[i + 3]),
                                                        E::pack(v[i + 4], v[i + 5]), E::pack(v[i + 6], v[i + 7]));
}

// A warp's tiles into its ring: copies in order, a stage a tile, each tile's block
// ids loaded one step ahead.
template <int D, int kStages, bool kWholePages>
struct Feed {
    static constexpr int kPerRow = D / 16, kRowsPer = 32 / kPerRow, kCopies = kTile / kRowsPer;
    const E4m3Params& p;
    const long long* cum;
    Cursor lc;        // the next tile to copy
    int loaded = 0;   // tiles whose copies have been issued
    const int count, lane;
    int id = 0, row = 0;
    // Where a lane's copies go in a stage: row r0 + i * kRowsPer, chunk col.  The
    // chunks' order repeats every eight rows.
    const int r0, col, put0, put1;
    const int64_t page_bytes, to_v;
    const uint32_t ring;
    uint32_t fill;    // the stage copied into next

    __device__ __forceinline__ Feed(const E4m3Params& params, const long long* prefix, const Cursor& at, int tiles,
                                    const uint8_t* stages, int lane_id)
        : p(params), cum(prefix), lc(at), count(tiles), lane(lane_id), r0(lane_id / kPerRow), col(lane_id % kPerRow),
          put0(r0 * D + chunk_at<D>(r0, col) * 16),
          put1((r0 + kRowsPer) * D + chunk_at<D>(r0 + kRowsPer, col) * 16),
          page_bytes(static_cast<int64_t>(params.page.size) * D), to_v(params.Hkv * page_bytes),
          ring(smem_u32(stages)), fill(ring) {
        look_up();
    }
    __device__ __forceinline__ int put(int i) const { return ((i & 1) ? put1 : put0) + (i / 2) * 2 * kRowsPer * D; }
    __device__ __forceinline__ void look_up() {
        const int key = lc.tile * kTile + (kWholePages ? 0 : lane & 15);
        const int page = p.page.split(kWholePages || key < lc.len ? key : lc.len - 1, &row);
        id = p.block_table[static_cast<int64_t>(lc.b) * p.max_pages + page];
    }
    __device__ __forceinline__ void issue() {
        if (loaded < count) {
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) {
                atomicOr(p.status, ATTN_DEV_BAD_INPUT);
                id = 0;
            }
            const int hkv = p.chunks == 1 ? lc.unit : lc.unit / p.chunks;
            const int valid = lc.len - lc.tile * kTile;  // 16 and more: the whole tile
            const int64_t block = static_cast<int64_t>(id) * 2 * p.Hkv + hkv;  // of K; V's is Hkv further
            // Lanes 0 .. 15: K's scales, 16 .. 31: V's (a tile in one page: lanes 0 and 16).
            if (kWholePages ? (lane & 15) == 0 : true)
                copy4(fill + 2 * kTile * D + lane * 4, p.scales + block + (lane >> 4) * p.Hkv,
                      (lane & 15) < valid ? 4 : 0);
            if (kWholePages) {  // one run of rows
                const uint8_t* src = p.kv + block * page_bytes + static_cast<int64_t>(row) * D + lane * 16;
                if (valid >= kTile) {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        copy16(fill + put(i), src + i * 512);
                        copy16(fill + kTile * D + put(i), src + to_v + i * 512);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const bool in = r0 + i * kRowsPer < valid;
                        const uint8_t* at = in ? src + i * 512 : p.kv;
                        copy16_or_zero(fill + put(i), at, in);
                        copy16_or_zero(fill + kTile * D + put(i), in ? at + to_v : p.kv, in);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int r = r0 + i * kRowsPer;
                    const int rid = __shfl_sync(0xffffffffu, id, r), rrow = __shfl_sync(0xffffffffu, row, r);
                    const uint8_t* src = p.kv + (static_cast<int64_t>(rid) * 2 * p.Hkv + hkv) * page_bytes +
                                         static_cast<int64_t>(rrow) * D + col * 16;
                    copy16_or_zero(fill + put(i), src, r < valid);
                    copy16_or_zero(fill + kTile * D + put(i), src + to_v, r < valid);
                }
            }
            fill += kStageBytes<D>;
            if (fill == ring + kStages * kStageBytes<D>) fill = ring;
            if (++loaded < count) {
                const int tile = lc.tile;
                cursor_next(p, cum, lc);
                if (kWholePages && lc.tile == tile + 1 && row + kTile < p.page.size) row += kTile;  // the same page
                else look_up();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// The unit's result: a warp had all its keys.
template <int D, int HC, bool kF16>
__device__ __forceinline__ void unit_out(const UnitState<D, HC>& s, const E4m3Params& p, int64_t row0, int heads,
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < HC / 8; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = r * 8 + 2 * t + i;
            const float l = heads_sum(s.l[r][i]), f = out_factor(s.m[r][i], l, s.mv[r][i]);
            float c[D / 8];
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                c[2 * j] = out_of(s.o[r][j][i], f);
                c[2 * j + 1] = out_of(s.o[r][j][i + 2], f);
            }
            if (h < heads) store_row<kF16>(p.o + (row0 + h) * D + g * (D / 8), c);
            if (p.lse && g == 0 && h < heads) p.lse[row0 + h] = (s.m[r][i] + __log2f(l)) * kLn2;
        }
    }
}

// A warp's part of a unit: its sums [HC][D] and {m, l, mv} [HC] in shared memory.
template <int D, int HC>
__device__ __forceinline__ void unit_piece(const UnitState<D, HC>& s, float* piece, float4* ml, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < HC / 8; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = r * 8 + 2 * t + i;
            const float l = heads_sum(s.l[r][i]);
#pragma unroll
            for (int j = 0; j < D / 16; j += 2)
                *reinterpret_cast<float4*>(piece + h * D + g * (D / 8) + 2 * j) =
                    make_float4(s.o[r][j][i], s.o[r][j][i + 2], s.o[r][j + 1][i], s.o[r][j + 1][i + 2]);
            if (g == 0) ml[h] = make_float4(s.m[r][i], l, s.mv[r][i], 0.0f);
        }
    }
}

// Query heads a CTA serves at a time: one or two 8-row halves of the product.
inline int heads_at_once(int group) { return group <= 8 ? 8 : 16; }


}  // namespace attn
