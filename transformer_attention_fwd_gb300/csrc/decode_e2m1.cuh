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
    // Two products' keys to a tile: their chains of dependent instructions run side by side,
    // and one check of the reference serves both.
    static constexpr int kKeys = 32, kParts = kKeys / kTile;
    static_assert(kParts == 2, "sixteen lanes to a part");
    // Of each part: K rows, V rows, their scales.
    template <int D>
    static constexpr int kPartBytes = 2 * kTile * (D / 2 + D / 16);
    template <int D>
    static constexpr int kStageBytes = kParts * kPartBytes<D>;
    static constexpr bool kFourHeads = true, kTwoReferences = false, kFactors = true;
    // The long kernel: CTAs to an SM, as registers allow, and the stages of a warp's ring.
    template <int D, int HC>
    static constexpr int kLongPerSm = D == 128 ? (HC <= 8 ? 3 : 2) : (HC <= 8 ? 4 : 3);
    template <int D, int HC>
    static constexpr int kLongStages = D == 128 && HC <= 8 ? 2 : 3;
    static constexpr int kShortStages = 3;

    // Where things are in a part.
    template <int D>
    struct Stage {
        static constexpr int kV = kTile * D / 2, kScales = 2 * kV, kVScales = kScales + kTile * (D / 16);
    };

    // A lane's copies.  Pages that hold a part's keys: sixteen lanes to a part, each copying
    // chunks l, l + 16, .. of its run of rows, whose places repeat every 256 bytes but for
    // a swap of chunk pairs.  Else a row at a time.
    template <int D, bool kWholePages>
    struct Copies {
        static constexpr int kPerRow = D / 32, kCopies = kTile * kPerRow / 16;
        static constexpr int kScaleRow = D / kRowScaleSpan, kScaleChunks = kTile * kScaleRow / 16;
        static constexpr uint32_t kSwap = D == 128 ? 32 : 0;
        const int lane;
        const uint32_t put0;     // of the lane's first chunk, in the tile
        const int64_t to_v;      // of codes; scales have an eighth

        __device__ __forceinline__ Copies(const CacheParams& p, int lane_id)
            : lane(lane_id), put0((lane_id >> 4) * kPartBytes<D> + chunk4_at<D>((lane_id & 15) / kPerRow, lane_id % kPerRow)),
              to_v(static_cast<int64_t>(p.Hkv) * p.page.size * (D / 2)) {}
        __device__ __forceinline__ uint32_t put(int i) const { return ((i & 1) ? put0 ^ kSwap : put0) + i * 256; }

        // valid: keys of the tile (kKeys and more: all); id, row: of key lane, or (pages that hold a
        // part's keys) of key 0 of the lane's part.
        __device__ __forceinline__ void issue(const CacheParams& p, uint32_t fill, int id, int row, int hkv,
                                              int valid) const {
            using S = Stage<D>;
            const int64_t first = (static_cast<int64_t>(id) * 2 * p.Hkv + hkv) * p.page.size + row;
            if (kWholePages) {
                const int l = lane & 15, c = l % kScaleChunks;
                const uint8_t* src = p.kv + first * (D / 2) + l * 16;
                const uint8_t* scales = p.row_scales + first * kScaleRow + (l < kScaleChunks ? 0 : to_v / 8) + c * 16;
                const uint32_t scales_to = fill + (lane >> 4) * kPartBytes<D> + S::kScales + l * 16;  // K's, then V's
                if (valid >= kKeys) {
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        copy16(fill + put(i), src + i * 256);
                        copy16(fill + S::kV + put(i), src + to_v + i * 256);
                    }
                    if (l < 2 * kScaleChunks) copy16(scales_to, scales);
                } else {
                    valid -= lane & 16;  // of the part
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const bool in = (l + 16 * i) / kPerRow < valid;
                        const uint8_t* at = in ? src + i * 256 : p.kv;
                        copy16_or_zero(fill + put(i), at, in);
                        copy16_or_zero(fill + S::kV + put(i), in ? at + to_v : p.kv, in);
                    }
                    const int bytes = min(16, max(0, valid * kScaleRow - c * 16));
                    if (l < 2 * kScaleChunks) copy16_part(scales_to, bytes > 0 ? scales : p.row_scales, bytes);
                }
            } else {
#pragma unroll
                for (int n = 0; n < kKeys * kPerRow / 32; ++n) {
                    const int r = (lane + 32 * n) / kPerRow, chunk = lane % kPerRow;
                    const int64_t at = __shfl_sync(0xffffffffu, first, r);
                    const uint8_t* src = p.kv + at * (D / 2) + chunk * 16;
                    const uint32_t to = fill + (r / kTile) * kPartBytes<D> + chunk4_at<D>(r % kTile, chunk);
                    copy16_or_zero(to, src, r < valid);
                    copy16_or_zero(to + S::kV, src + to_v, r < valid);
                }
                const uint32_t to = fill + (lane >> 4) * kPartBytes<D> + S::kScales + (lane & 15) * kScaleRow;
                copy_scales<kScaleRow>(to, p.row_scales + first * kScaleRow, lane < valid);
                copy_scales<kScaleRow>(to + kTile * kScaleRow, p.row_scales + first * kScaleRow + to_v / 8, lane < valid);
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
        constexpr int kR = kHalves<HC>, kS = D / 16, kScaleRow = D / kRowScaleSpan;
        const int g = lane >> 2, t = lane & 3;
        float sc[kParts][kR][4], sd[kParts][kR][4];  // two chains of products each
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int n = 0; n < 4; ++n) sc[i][r][n] = sd[i][r][n] = 0.0f;
        {
            // Key g's and key g + 8's columns of this lane, D/4 from t * D/4 on, and their scales,
            // each in both halves of a word.
            uint32_t kw[kParts][2][D / 32], kscale[kParts][2][D / 64];
            const uint8_t* codes = stage + (D == 128 ? chunk4_at<D>(g, t) : chunk4_at<D>(g, t >> 1) + (t & 1) * 8);
            const uint8_t* scale = stage + S::kScales + g * kScaleRow + t * (D / 64);
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint8_t* c = codes + i * kPartBytes<D> + n * (8 * D / 2);  // eight rows on: the same place
                    const uint8_t* at = scale + i * kPartBytes<D> + n * 8 * kScaleRow;
                    if constexpr (D == 128) {
                        const uint4 u = *reinterpret_cast<const uint4*>(c);
                        kw[i][n][0] = u.x; kw[i][n][1] = u.y; kw[i][n][2] = u.z; kw[i][n][3] = u.w;
                        both_halves(e4m3_to_f16x2(*reinterpret_cast<const uint16_t*>(at)), kscale[i][n][0], kscale[i][n][1]);
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(c);
                        kw[i][n][0] = u.x; kw[i][n][1] = u.y;
                        uint32_t none;
                        both_halves(e4m3_to_f16x2(*at), kscale[i][n][0], none);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kS; j += 2) {  // two product steps out of a word of eight columns
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        e2m1_to_f16x8(kw[i][n][j / 2], a[n]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[n][k] = f16x2_mul(a[n][k], kscale[i][n][j / 4]);
                    }
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        mma_f16(sc[i][r], a[0][0], a[1][0], a[0][1], a[1][1], s.qb[j][r][0], s.qb[j][r][1]);
                        mma_f16(sd[i][r], a[0][2], a[1][2], a[0][3], a[1][3], s.qb[j + 1][r][0], s.qb[j + 1][r][1]);
                    }
                }
            }
        }
        float x[kParts][kR][4], e[kParts][kR][4], w[kParts][kR][4];  // exponents, under the reference, weights
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int n = 0; n < 4; ++n) x[i][r][n] = (sc[i][r][n] + sd[i][r][n]) * s.qs[r][n & 1];
        if (scores.at != nullptr) {
            const bool pairs = scores.group % 2 == 0;  // a lane's two heads are 8-byte aligned
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int n = 0; n < 4; n += 2) {
                        const int key = i * kTile + (n >> 1) * 8 + g, h = r * 8 + 2 * t;
                        float* to = scores.at + key * scores.group + h;
                        if (key >= valid || h >= scores.heads) continue;
                        if (pairs) {
                            *reinterpret_cast<float2*>(to) = make_float2(x[i][r][n], x[i][r][n + 1]);
                        } else {
                            to[0] = x[i][r][n];
                            if (h + 1 < scores.heads) to[1] = x[i][r][n + 1];
                        }
                    }
        }
        if (valid < kKeys) {  // the unit's last tile
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (i * kTile + (n >> 1) * 8 + g >= valid) x[i][r][n] = -INFINITY;
        }
        bool need = false;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    e[i][r][n] = x[i][r][n] - s.mv[r][n & 1];
                    need |= e[i][r][n] > kLift + kSlack;
                }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float most = fmaxf(x[0][r][n], x[0][r][n + 2]);
#pragma unroll
                    for (int i = 1; i < kParts; ++i) most = fmaxf(most, fmaxf(x[i][r][n], x[i][r][n + 2]));
                    const float mv = fmaxf(s.mv[r][n], heads_max(most) - kLift);
                    const float alpha = ex2_approx(s.mv[r][n] - mv);
                    s.l[r][n] *= alpha;
                    s.mv[r][n] = mv;
#pragma unroll
                    for (int i = 0; i < kParts; ++i) {
                        e[i][r][n] = x[i][r][n] - mv;
                        e[i][r][n + 2] = x[i][r][n + 2] - mv;
                    }
#pragma unroll
                    for (int j = 0; j < kS; ++j) {
                        s.o[r][j][n] *= alpha;
                        s.o[r][j][n + 2] *= alpha;
                    }
                }
            }
        }
        float least[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            least[i] = INFINITY;
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    w[i][r][n] = ex2_approx(e[i][r][n]);
                    s.l[r][n & 1] += w[i][r][n];
                    least[i] = fminf(least[i], e[i][r][n]);
                }
        }
        if (__all_sync(0xffffffffu, fminf(least[0], least[kParts - 1]) >= -kLow)) {
            // In one stretch, so that a part's operand is made under the other's products.
            Weights<HC> pb[kParts][kR][2];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    pb[i][r][0].set(w[i][r][0], w[i][r][1], t);
                    pb[i][r][1].set(w[i][r][2], w[i][r][3], t);
                }
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const Values<D> v(stage + i * kPartBytes<D>, g, t);
#pragma unroll
                for (int j = 0; j < kS; j += 4) {
                    uint32_t va[4][4];
                    v.columns(j / 4, va);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            mma_f16(s.o[r][j + k], va[k][0], va[k][1], va[k][2], va[k][3], pb[i][r][0].hi, pb[i][r][1].hi);
                            if (HC >= 8)
                                mma_f16(s.o[r][j + k], va[k][0], va[k][1], va[k][2], va[k][3], pb[i][r][0].lo,
                                        pb[i][r][1].lo);
                        }
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const Values<D> v(stage + i * kPartBytes<D>, g, t);
            uint32_t va[kS][4];
            auto convert = [&](int k) {
                if (k % 4 != 0) return;
                uint32_t c[4][4];
                v.columns(k / 4, c);
#pragma unroll
                for (int n = 0; n < 16; ++n) va[k + n / 4][n % 4] = c[n / 4][n % 4];
            };
            if (HC <= 8)
#pragma unroll
                for (int k = 0; k < kS; ++k) convert(k);
            weighted_rows<D, HC>(e[i], w[i], least[i], va, convert, lane, s);
        }
    }

  private:
    // A part's V as this lane needs it: keys 2t, 2t + 1, 2t + 8 and 2t + 9, D/8 columns from
    // g * D/8 on, and the scales, two keys' in a word.
    template <int D>
    struct Values {
        uint32_t w[4][D / 64], scale[2];
        __device__ __forceinline__ Values(const uint8_t* part, int g, int t) {
            using S = Stage<D>;
            constexpr int kScaleRow = D / kRowScaleSpan;
            // Row 2t + 1 is in the next half (quarter) of row 2t's line, or the one before.
            const uint32_t even = D == 128 ? chunk4_at<D>(2 * t, g >> 1) + (g & 1) * 8 : chunk4_at<D>(2 * t, g >> 2) + (g & 3) * 4;
            const uint32_t odd = even ^ (D / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t* c = part + S::kV + ((j & 1) ? odd : even) + (j >> 1) * (8 * D / 2);
                if constexpr (D == 128) {
                    const uint2 u = *reinterpret_cast<const uint2*>(c);
                    w[j][0] = u.x; w[j][1] = u.y;
                } else {
                    w[j][0] = *reinterpret_cast<const uint32_t*>(c);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* at = part + S::kVScales + (2 * t + 8 * j) * kScaleRow + (D == 128 ? g : g >> 1);
                scale[j] = e4m3_to_f16x2(at[0] | (static_cast<uint32_t>(at[kScaleRow]) << 8));
            }
        }
        // V^T's operand of eight columns, two to a product step: the low halves of two keys' bytes are
        // one column's codes, the high halves the next column's.
        __device__ __forceinline__ void columns(int word, uint32_t (&va)[4][4]) const {
#pragma unroll
            for (int key = 0; key < 4; key += 2) {
                const uint32_t u = w[key][word], v = w[key + 1][word];
                uint32_t even[4], odd[4];
                e2m1_to_f16x8((u & 0x0f0f0f0fu) | ((v & 0x0f0f0f0fu) << 4), even);
                e2m1_to_f16x8(((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u), odd);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    va[k][key] = f16x2_mul(even[k], scale[key / 2]);
                    va[k][key + 1] = f16x2_mul(odd[k], scale[key / 2]);
                }
            }
        }
    };
};

}  // namespace attn
