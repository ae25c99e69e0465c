// decode_e4m3.cuh -- the 8-bit format of the decodes in decode_cache.cuh: a tile's
// copies, its scores, weights and weighted V rows.  decode_e4m3.cu says how.
#pragma once

#include "decode_cache.cuh"
#include "e4m3.cuh"

namespace attn {

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

struct E4m3Cache {
    static constexpr int kKeys = kTile;
    // K rows, V rows, their scales.
    template <int D>
    static constexpr int kStageBytes = 2 * kTile * D + 2 * kTile * 4;
    static constexpr bool kFourHeads = false, kTwoReferences = true, kFactors = false;
    // The long kernel: CTAs to an SM, as registers allow, and the stages of a warp's ring.
    template <int D, int HC>
    static constexpr int kLongPerSm = D == 128 ? (HC == 8 ? 3 : 2) : (HC == 8 ? 4 : 3);
    template <int D, int HC>
    static constexpr int kLongStages = HC == 8 ? 3 : 4;
    static constexpr int kShortStages = 4;

    // Where a lane's copies go in a stage: row r0 + i * kRowsPer, chunk col.  The
    // chunks' order repeats every eight rows.
    template <int D, bool kWholePages>
    struct Copies {
        static constexpr int kPerRow = D / 16, kRowsPer = 32 / kPerRow, kCopies = kTile / kRowsPer;
        const int lane, r0, col, put0, put1;
        const int64_t page_bytes, to_v;

        __device__ __forceinline__ Copies(const CacheParams& p, int lane_id)
            : lane(lane_id), r0(lane_id / kPerRow), col(lane_id % kPerRow),
              put0(r0 * D + chunk_at<D>(r0, col) * 16),
              put1((r0 + kRowsPer) * D + chunk_at<D>(r0 + kRowsPer, col) * 16),
              page_bytes(static_cast<int64_t>(p.page.size) * D), to_v(p.Hkv * page_bytes) {}
        __device__ __forceinline__ int put(int i) const { return ((i & 1) ? put1 : put0) + (i / 2) * 2 * kRowsPer * D; }

        // valid: keys of the tile (kTile and more: all); id, row: of key 0, or (pages that end
        // inside a tile) of key lane % 16.
        __device__ __forceinline__ void issue(const CacheParams& p, uint32_t fill, int id, int row, int hkv,
                                              int valid) const {
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
        }
    };

    // One tile of a warp's ring: scores, weights, and the weighted V rows.
    template <int D, int HC, bool kWholePages>
    static __device__ __forceinline__ void tile(const uint8_t* stage, int valid, int lane, UnitState<D, HC>& s,
                                                const TileScores&) {
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
        weighted_rows<D, HC>(e, w, least, va, convert, lane, s);
    }
};

}  // namespace attn
