// decode_e2m1.cuh -- the 4-bit format of the decodes in decode_cache.cuh: a tile's
// copies, its scores, weights and weighted V rows.  decode_e2m1.cu says how.
#pragma once

#include "decode_cache.cuh"
#include "e2m1.cuh"

namespace attn {

// Place of a row's 16-byte chunk (two or four of them): a line of 128 bytes holds two
// (four) rows, their order and that of the chunks changed from line to line so that the
// reads of both products, rows 0 .. 7 and rows 0, 2, 4, 6 at a time, meet no bank twice.
template <int D>
__device__ __forceinline__ int chunk4_at(int row, int chunk) {
    if (D == 128)
        return (row >> 1) * 128 + ((row ^ (row >> 1)) & 1) * 64 + (chunk ^ ((row >> 1) & 2)) * 16;
    return (row >> 2) * 128 + ((row & 3) ^ ((row >> 2) & 1)) * 32 + chunk * 16;
}

struct E2m1Cache {
    // K rows, V rows, their scales.
    template <int D>
    static constexpr int kStageBytes = 2 * kTile * (D / 2 + D / 16);
    static constexpr bool kTwoReferences = false, kFactors = true;
    // The long kernel: CTAs to an SM, as registers allow, and the stages of a warp's ring.
    template <int D, int HC>
    static constexpr int kLongPerSm = D == 128 ? (HC == 8 ? 3 : 2) : (HC == 8 ? 4 : 3);
    template <int D, int HC>
    static constexpr int kLongStages = D == 128 && HC == 8 ? 5 : 6;

    // Where things are in a stage.
    template <int D>
    struct Stage {
        static constexpr int kV = kTile * D / 2, kScales = 2 * kV, kVScales = kScales + kTile * (D / 16);
    };

    template <int D, bool kWholePages>
    struct Copies {
        static constexpr int kPerRow = D / 32, kCopies = kTile * kPerRow / 32;
        static constexpr int kScaleRow = D / kRowScaleSpan, kScaleChunks = kTile * kScaleRow / 16;
        const int lane;
        int put[kCopies];
        const int64_t row_bytes, to_v;  // of codes; scales have an eighth

        __device__ __forceinline__ Copies(const CacheParams& p, int lane_id)
            : lane(lane_id), row_bytes(D / 2), to_v(static_cast<int64_t>(p.Hkv) * p.page.size * (D / 2)) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                put[i] = chunk4_at<D>((lane + 32 * i) / kPerRow, (lane + 32 * i) % kPerRow);
        }

        // valid: keys of the tile (kTile and more: all); id, row: of key 0, or (pages that end
        // inside a tile) of key lane % 16.
        __device__ __forceinline__ void issue(const CacheParams& p, uint32_t fill, int id, int row, int hkv,
                                              int valid) const {
            using S = Stage<D>;
            if (kWholePages) {  // one run of rows
                const int64_t first = (static_cast<int64_t>(id) * 2 * p.Hkv + hkv) * p.page.size + row;
                const uint8_t* src = p.kv + first * row_bytes + lane * 16;
                if (valid >= kTile) {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        copy16(fill + put[i], src + i * 512);
                        copy16(fill + S::kV + put[i], src + to_v + i * 512);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const bool in = (lane + 32 * i) / kPerRow < valid;
                        const uint8_t* at = in ? src + i * 512 : p.kv;
                        copy16_or_zero(fill + put[i], at, in);
                        copy16_or_zero(fill + S::kV + put[i], in ? at + to_v : p.kv, in);
                    }
                }
                if (lane < 2 * kScaleChunks) {  // K's scales, then V's
                    const int c = lane % kScaleChunks;
                    const int bytes = min(16, max(0, valid * kScaleRow - c * 16));
                    const uint8_t* at = p.row_scales + first * kScaleRow + (lane < kScaleChunks ? 0 : to_v / 8) + c * 16;
                    copy16_part(fill + S::kScales + lane * 16, bytes > 0 ? at : p.row_scales, bytes);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int r = (lane + 32 * i) / kPerRow;
                    const int rid = __shfl_sync(0xffffffffu, id, r), rrow = __shfl_sync(0xffffffffu, row, r);
                    const uint8_t* src = p.kv + ((static_cast<int64_t>(rid) * 2 * p.Hkv + hkv) * p.page.size + rrow) * row_bytes +
                                         (lane + 32 * i) % kPerRow * 16;
                    copy16_or_zero(fill + put[i], src, r < valid);
                    copy16_or_zero(fill + S::kV + put[i], src + to_v, r < valid);
                }
                // Lanes 0 .. 15: K's scales, 16 .. 31: V's.
                const uint8_t* at = p.row_scales + ((static_cast<int64_t>(id) * 2 * p.Hkv + hkv) * p.page.size + row) * kScaleRow +
                                    (lane < kTile ? 0 : to_v / 8);
                copy_scales<kScaleRow>(fill + S::kScales + lane * kScaleRow, at, lane % kTile < valid);
            }
        }

      private:
        // `bytes` of 16, zeros behind them.
        static __device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, int bytes) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
        }
        template <int kBytes>
        static __device__ __forceinline__ void copy_scales(uint32_t dst, const void* src, bool read) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                         :: "r"(dst), "l"(src), "n"(kBytes), "r"(read ? kBytes : 0) : "memory");
        }
    };

    // One tile of a warp's ring: scores, weights, and the weighted V rows.
    template <int D, int HC, bool kWholePages>
    static __device__ __forceinline__ void tile(const uint8_t* stage, int valid, int lane, UnitState<D, HC>& s,
                                                const TileScores& scores) {
        using S = Stage<D>;
        constexpr int kR = HC / 8, kS = D / 16, kScaleRow = D / kRowScaleSpan;
        const int g = lane >> 2, t = lane & 3;
        // Key g's and key g + 8's columns of this lane, D/4 from t * D/4 on, and their scales,
        // each in both halves of a word.
        uint32_t kw[2][D / 32], kscale[2][D / 64];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int row = n * 8 + g;
            const uint8_t* at = stage + S::kScales + row * kScaleRow;
            if constexpr (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(stage + chunk4_at<D>(row, t));
                kw[n][0] = u.x; kw[n][1] = u.y; kw[n][2] = u.z; kw[n][3] = u.w;
                const uint32_t f = e4m3_to_f16x2(*reinterpret_cast<const uint16_t*>(at + 2 * t));
                kscale[n][0] = __byte_perm(f, f, 0x1010);
                kscale[n][1] = __byte_perm(f, f, 0x3232);
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(stage + chunk4_at<D>(row, t >> 1) + (t & 1) * 8);
                kw[n][0] = u.x; kw[n][1] = u.y;
                const uint32_t f = e4m3_to_f16x2(at[t]);
                kscale[n][0] = __byte_perm(f, f, 0x1010);
            }
        }
        // Keys 2t, 2t + 1, 2t + 8 and 2t + 9: this lane's D/8 columns of V from g * D/8 on, and
        // the scales, two keys' in a word.
        uint32_t vw[4][D / 64], vscale[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 2 * t + (j & 1) + 8 * (j >> 1);
            if constexpr (D == 128) {
                const uint2 u = *reinterpret_cast<const uint2*>(stage + S::kV + chunk4_at<D>(row, g >> 1) + (g & 1) * 8);
                vw[j][0] = u.x; vw[j][1] = u.y;
            } else {
                vw[j][0] = *reinterpret_cast<const uint32_t*>(stage + S::kV + chunk4_at<D>(row, g >> 2) + (g & 3) * 4);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t* at = stage + S::kVScales + (2 * t + 8 * j) * kScaleRow + (D == 128 ? g : g >> 1);
            vscale[j] = e4m3_to_f16x2(at[0] | (static_cast<uint32_t>(at[kScaleRow]) << 8));
        }
        float sc[kR][4], sd[kR][4];  // two chains of products
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[r][i] = sd[r][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < kS; j += 2) {  // two product steps out of a word of eight columns
            uint32_t a[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                e2m1_to_f16x8(kw[n][j / 2], a[n]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[n][i] = f16x2_mul(a[n][i], kscale[n][j / 4]);
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                mma_f16(sc[r], a[0][0], a[1][0], a[0][1], a[1][1], s.qb[j][r][0], s.qb[j][r][1]);
                mma_f16(sd[r], a[0][2], a[1][2], a[0][3], a[1][3], s.qb[j + 1][r][0], s.qb[j + 1][r][1]);
            }
        }
        // V^T's operand (with eight heads all of it now, while the products run): the low halves of two
        // keys' bytes are one column's codes, the high halves the next column's.
        uint32_t va[kS][4];
        auto columns = [&](int word, int key, int i0) {  // steps i0 .. i0 + 3, keys `key` of 0 or 2
            const uint32_t x = vw[key][word], y = vw[key + 1][word];
            uint32_t even[4], odd[4];
            e2m1_to_f16x8((x & 0x0f0f0f0fu) | ((y & 0x0f0f0f0fu) << 4), even);
            e2m1_to_f16x8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), odd);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                va[i0 + i][key] = f16x2_mul(even[i], vscale[key / 2]);
                va[i0 + i][key + 1] = f16x2_mul(odd[i], vscale[key / 2]);
            }
        };
        auto convert = [&](int i) {
            if (i % 4 != 0) return;
            columns(i / 4, 0, i);
            columns(i / 4, 2, i);
        };
        if (HC == 8)
#pragma unroll
            for (int i = 0; i < kS; ++i) convert(i);
        float x[kR][4], e[kR][4], w[kR][4];  // exponents, the same under the reference, weights
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[r][i] = (sc[r][i] + sd[r][i]) * s.qs[r][i & 1];
        if (scores.at != nullptr) {
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i >> 1) * 8 + g, h = r * 8 + 2 * t + (i & 1);
                    if (key < valid && h < scores.heads) scores.at[key * scores.group + h] = x[r][i];
                }
        }
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
            for (int i = 0; i < 4; ++i) {
                e[r][i] = x[r][i] - s.mv[r][i & 1];
                need |= e[r][i] > kLift + kSlack;
            }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mv = fmaxf(s.mv[r][i], heads_max(fmaxf(x[r][i], x[r][i + 2])) - kLift);
                    const float alpha = ex2_approx(s.mv[r][i] - mv);
                    s.l[r][i] *= alpha;
                    s.mv[r][i] = mv;
                    e[r][i] = x[r][i] - mv;
                    e[r][i + 2] = x[r][i + 2] - mv;
#pragma unroll
                    for (int j = 0; j < kS; ++j) {
                        s.o[r][j][i] *= alpha;
                        s.o[r][j][i + 2] *= alpha;
                    }
                }
            }
        }
        float least = INFINITY;
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[r][i] = ex2_approx(e[r][i]);
                s.l[r][i & 1] += w[r][i];
                least = fminf(least, e[r][i]);
            }
        weighted_rows<D, HC>(e, w, least, va, convert, s);
    }
};

}  // namespace attn
