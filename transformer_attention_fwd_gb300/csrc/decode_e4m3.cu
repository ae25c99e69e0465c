// decode_e4m3.cu -- decode (one query row per (request, head)) over the paged
// 8-bit cache with one scale for each block, K or V, and head
// (attn_fwd_decode_paged_e4m3).
//
//   O = sum_j p_j vs_j v_j / sum_j p_j,  p_j = 2^x_j,
//   x_j = log2(e) * scale * ks_j * (q . k_j)
//
// with k_j, v_j the codes and ks_j, vs_j the scales of key j's block.  HBM bound:
// 2 * D bytes per key and KV head are read once.  Half the bytes of the 16-bit
// cache leave half the time per key, so the products go to the tensor cores
// (mma.sync m16n8k16 in fp16, fp32 sums; the codes convert exactly): S^T = K Q^T
// with 16 keys as rows and eight query heads of their KV head as columns, and
// O^T = V^T P^T with 16 columns of V as rows.  P^T's operand is S^T's result with
// each 8 x 8 block transposed (movmatrix).  The order of a product's inner index
// is free, so K's columns and V's rows are dealt to lanes so that each reads 16
// contiguous bytes.
//
// Two running references.  The sum of the p_j is taken relative to 2^m, m a
// maximum over x_j, in fp32.  What multiplies a code is w_j = p_j vs_j, taken
// relative to 2^mv, mv a maximum over x_j + log2 vs_j, in fp16: the weights that
// matter keep 11 bits and none overflows, however far apart the scales are.  The
// result is (sum w_j v_j) / (sum p_j) * 2^(mv - m).  A reference moves only when
// a key exceeds it by 2^kSlack.
//
// Work: all 16-key tiles of all (request, KV head, head chunk) units are laid
// end to end, cut into one equal slice per CTA and that into one per warp.  A
// warp streams its tiles through a ring of its own with 16-byte asynchronous
// copies; nothing in the loop waits for another warp.  Units inside one warp's
// range are written at once; the pieces of the others are merged in the CTA at
// its end, and those that a CTA boundary cuts by the combine kernel.  Two
// small CTAs share an SM, so that one's start and end pass under the other's
// streaming.  (More of them than fit at once, to even out the SMs, lost 5 us for
// each further wave: a start costs that much.)
//
// 64 requests of 4096 keys, Hq 32, Hkv 8, D 128, 16-token blocks (539 MB): 91 us,
// 5.9 TB/s.  Every CTA sums the lengths and finds its place in 2.8 us, the first
// tiles are there after 5.9, the SMs run dry between 78 and 88 us (together they
// stream at 7 TB/s), merging takes 1 to 2 us and the combine kernel 3.  With 8
// query heads per KV head and ragged lengths (231 MB) 44 us, by the same fixed
// costs; at D = 64 94 us for 540 MB.  With 16 heads per KV head instruction issue
// bounds it: 105 us (D = 128), 123 us (D = 64).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "e4m3.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace attn {
namespace {

constexpr int kTile = 16;          // keys of a tile
constexpr int kMaxPrefixB = 1024;  // requests whose tile counts a CTA sums itself
constexpr float kSlack = 6.0f;
// References start here: below any score, and finite, so that no difference of
// two of them is NaN.
constexpr float kLowest = -3.0e38f;
constexpr float kLn2 = 0.69314718055994531f;

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

template <int D, int HC>
struct E4m3Layout {
    static constexpr int kWarps = 4;
    static constexpr int kPerSm = D == 128 ? 2 : (HC == 8 ? 4 : 3);  // CTAs, as registers allow
    static constexpr int kStage = 2 * kTile * D + 2 * kTile * 4;  // K rows, V rows, scales
    static constexpr int kPiece = HC * D * 4;
    static constexpr int kStages = D == 128 ? 4 : (HC == 8 ? 4 : 5);
    static constexpr int kPieceOff = kWarps * kStages * kStage;
    static constexpr int kMlOff = kPieceOff + kWarps * kPiece;  // [warp][2][HC] float4
    static constexpr int kMetaOff = kMlOff + kWarps * 2 * HC * 16;
    static constexpr int kCumOff = kMetaOff + kWarps * 2 * 16;
    static constexpr int kBytes = kCumOff + (kMaxPrefixB + 1) * 8 + 40 * 8;
    static_assert(kStages * kStage >= kPiece, "a warp's ring holds its second piece");
    static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "CTAs to an SM");
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

__device__ __forceinline__ Cursor cursor_at(const E4m3Params& p, const long long* cum, long long v) {
    const long long U = static_cast<long long>(p.Hkv) * p.chunks;
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] * U <= v) lo = mid; else hi = mid - 1;
    }
    Cursor c;
    c.b = lo;
    c.tiles = static_cast<int>(cum[lo + 1] - cum[lo]);
    const long long r = v - cum[lo] * U;
    c.unit = static_cast<int>(divide(r, c.tiles));
    c.tile = static_cast<int>(r - static_cast<long long>(c.unit) * c.tiles);
    c.len = clamped_len(p, lo);
    return c;
}

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

// cum[b] = tiles of requests 0 .. b - 1, by the whole block.
__device__ void tile_prefix(const E4m3Params& p, long long* cum, long long* scan, bool report) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + nt - 1) / nt;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = p.seq_lens[b], L = clamped(p, n);
        if (report && L != n) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        mine += (L + kTile - 1) / kTile;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long run = incl - mine;
    for (int i = 0; i < warp; ++i) run += scan[i];
    const long long end = run + mine;
    for (int b = b0; b < b1; ++b) {  // one request: nothing to read again
        run = b + 1 == b1 ? end : run + (clamped_len(p, b) + kTile - 1) / kTile;
        cum[b + 1] = run;
    }
    if (tid == 0) cum[0] = 0;
    __syncthreads();
}

__global__ void __launch_bounds__(1024) e4m3_prefix_kernel(const E4m3Params p) {
    __shared__ long long scan[32];
    tile_prefix(p, p.cum, scan, true);
}

// Tiles of a CTA's slice: at least one a warp.
__device__ __forceinline__ long long slice_tiles(long long total, int grid, int warps) {
    const long long per = divide(total + grid - 1, grid);
    return per < warps ? warps : per;
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
// takes its largest element to [512, 1024).
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

// Factor from sum w v to O: 2^(mv - m) / l.
__device__ __forceinline__ float out_factor(float m, float l, float mv) { return ex2_approx(mv - m) / l; }

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
            reinterpret_cast<uint2*>(row)[lane] = make_uint2(E::pack(c[0] * f, c[1] * f), E::pack(c[2] * f, c[3] * f));
        else reinterpret_cast<uint32_t*>(row)[lane] = E::pack(c[0] * f, c[1] * f);
    }
};

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
            need |= x[r][i] > fminf(s.m[r][i & 1], s.mv[r][i & 1] - lift[(i >> 1) % kF]) + kSlack;
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float m = fmaxf(s.m[r][i], heads_max(fmaxf(x[r][i], x[r][i + 2])));
                const float mv = fmaxf(s.mv[r][i], heads_max(fmaxf(x[r][i] + lift[0], x[r][i + 2] + lift[kF - 1])));
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
    uint32_t pb[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s.l[r][i & 1] += ex2_approx(x[r][i] - s.m[r][i & 1]);
            w[i] = ex2_approx(x[r][i] + (lift[(i >> 1) % kF] - s.mv[r][i & 1]));
        }
        pb[r][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        pb[r][1] = transpose8x8(pack_f16x2(w[2], w[3]));
    }
#pragma unroll
    for (int i = 0; i < kS; ++i) {
        if (HC != 8) convert(i);
#pragma unroll
        for (int r = 0; r < kR; ++r) mma_f16(s.o[r][i], va[i][0], va[i][1], va[i][2], va[i][3], pb[r][0], pb[r][1]);
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

// What a warp leaves of a unit it has not covered alone.
struct PieceMeta {
    long long unit;  // request << 32 | unit, -1: none
    int begins, ends;  // the piece holds the unit's first (last) tile; begins = 2: not at the slice's start
};

template <int D, int HC, bool kF16, bool kWholePages>
__global__ void __launch_bounds__(E4m3Layout<D, HC>::kWarps * 32, E4m3Layout<D, HC>::kPerSm)
decode_e4m3_kernel(const E4m3Params p, int prefix_in_kernel) {
    using L = E4m3Layout<D, HC>;
    constexpr int kWarps = L::kWarps;
    constexpr int kR = HC / 8, kCols = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;  // as in UnitState
    uint8_t* ring = smem + warp * L::kStages * L::kStage;
    float4* ml = reinterpret_cast<float4*>(smem + L::kMlOff);
    PieceMeta* meta = reinterpret_cast<PieceMeta*>(smem + L::kMetaOff);
    long long* s_cum = reinterpret_cast<long long*>(smem + L::kCumOff);
    const long long* cum = p.cum;
    grid_wait();
    grid_launch_next();
    if (prefix_in_kernel) {
        tile_prefix(p, s_cum, s_cum + kMaxPrefixB + 1, blockIdx.x == 0);
        cum = s_cum;
    }
    const int grid = static_cast<int>(gridDim.x);
    const int U = p.Hkv * p.chunks;

    // Requests without keys.
    for (int b = blockIdx.x; b < p.B; b += grid) {
        if (cum[b + 1] != cum[b]) continue;
        const int64_t row0 = static_cast<int64_t>(b) * p.Hq;
        for (int i = threadIdx.x; i < p.Hq * (D / 8); i += kWarps * 32)
            reinterpret_cast<uint4*>(p.o + row0 * D)[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = threadIdx.x; i < p.Hq; i += kWarps * 32) p.lse[row0 + i] = -INFINITY;
    }

    const long long total = cum[p.B] * U;
    const long long per = slice_tiles(total, grid, kWarps);
    const long long v0 = per * blockIdx.x, v1 = v0 + per < total ? v0 + per : total;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.geom = make_longlong2(total, per);
    if (v0 >= total) return;
    const int wper = static_cast<int>((v1 - v0 + kWarps - 1) / kWarps);
    const long long va = v0 + static_cast<long long>(warp) * wper;
    const int count = va >= v1 ? 0 : static_cast<int>(va + wper < v1 ? wper : v1 - va);
    if (lane < 2) meta[2 * warp + lane].unit = -1;
    __syncwarp();

    if (count > 0) {
        Cursor lc = cursor_at(p, cum, va), cc = lc;
        if (threadIdx.x == 0) p.first[blockIdx.x] = make_int4(lc.b, lc.unit, lc.tile, lc.tiles);  // va = v0
        int loaded = 0;  // tiles whose copies have been issued
        // The next tile to copy: its block ids are loaded one step ahead.
        int id = 0, row = 0, page = 0;
        auto look_up = [&]() {
            const int key = lc.tile * kTile + (kWholePages ? 0 : lane & 15);
            page = p.page.split(kWholePages || key < lc.len ? key : lc.len - 1, &row);
            id = p.block_table[static_cast<int64_t>(lc.b) * p.max_pages + page];
        };
        look_up();
        // Where a lane's copies go in a stage: row r0 + i * kRowsPer, chunk col.  The
        // chunks' order repeats every eight rows.
        constexpr int kPerRow = D / 16, kRowsPer = 32 / kPerRow, kCopies = kTile / kRowsPer;
        const int r0 = lane / kPerRow, col = lane % kPerRow;
        const int put0 = r0 * D + chunk_at<D>(r0, col) * 16;
        const int put1 = (r0 + kRowsPer) * D + chunk_at<D>(r0 + kRowsPer, col) * 16;
        auto put = [&](int i) { return ((i & 1) ? put1 : put0) + (i / 2) * 2 * kRowsPer * D; };
        const int64_t page_bytes = static_cast<int64_t>(p.page.size) * D, to_v = p.Hkv * page_bytes;
        const uint32_t ring32 = smem_u32(ring);
        uint32_t fill = ring32;  // the stage copied into next
        auto issue = [&]() {
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
                        const uint8_t* src = p.kv +
                            (static_cast<int64_t>(rid) * 2 * p.Hkv + hkv) * page_bytes + static_cast<int64_t>(rrow) * D + col * 16;
                        copy16_or_zero(fill + put(i), src, r < valid);
                        copy16_or_zero(fill + kTile * D + put(i), src + to_v, r < valid);
                    }
                }
                fill += L::kStage;
                if (fill == ring32 + L::kStages * L::kStage) fill = ring32;
                if (++loaded < count) {
                    const int tile = lc.tile;
                    cursor_next(p, cum, lc);
                    if (kWholePages && lc.tile == tile + 1 && row + kTile < p.page.size) row += kTile;  // the same page
                    else look_up();
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) issue();

        UnitState<D, HC> s;
        const uint8_t* stage = ring;
        int pieces = 0;
        int from = cc.tile;  // the unit's first tile of this warp
        unit_begin<D, HC, kF16>(p, cc, lane, s);
        for (int n = 0; n < count; ++n) {
            asm volatile("cp.async.wait_group %0;" :: "n"(L::kStages - 2) : "memory");
            __syncwarp();  // the tile is there, and the stage filled next has been read
            issue();
            unit_tile<D, HC, kWholePages>(stage, min(kTile, cc.len - cc.tile * kTile), lane, s);
            stage += L::kStage;
            if (stage == ring + L::kStages * L::kStage) stage = ring;
            const bool unit_done = cc.tile + 1 == cc.tiles;
            if (!unit_done && n + 1 < count) {
                ++cc.tile;
                continue;
            }
            // The unit, or this warp's part of it, is done.
            const int hkv = p.chunks == 1 ? cc.unit : cc.unit / p.chunks, chunk = cc.unit - hkv * p.chunks;
            const int heads = min(HC, p.group - chunk * HC);
            const int64_t row0 = static_cast<int64_t>(cc.b) * p.Hq + hkv * p.group + chunk * HC;
            const bool whole = unit_done && from == 0;
            float* piece = reinterpret_cast<float*>(pieces == 0 ? smem + L::kPieceOff + warp * L::kPiece : ring);
            if (!whole && pieces == 1) {  // the warp's last: no copy is in flight into its ring
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const int h0 = r * 8 + 2 * t;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = h0 + i;
                    const float l = heads_sum(s.l[r][i]);
                    float c[kCols];
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        c[2 * j] = s.o[r][j][i];
                        c[2 * j + 1] = s.o[r][j][i + 2];
                    }
                    if (whole) {
                        const float f = out_factor(s.m[r][i], l, s.mv[r][i]);
#pragma unroll
                        for (int k = 0; k < kCols; ++k) c[k] *= f;
                        if (h < heads) store_row<kF16>(p.o + (row0 + h) * D + g * kCols, c);
                        if (p.lse && g == 0 && h < heads) p.lse[row0 + h] = (s.m[r][i] + __log2f(l)) * kLn2;
                    } else {
#pragma unroll
                        for (int k = 0; k < kCols; k += 4)
                            *reinterpret_cast<float4*>(piece + h * D + g * kCols + k) =
                                make_float4(c[k], c[k + 1], c[k + 2], c[k + 3]);
                        if (g == 0) ml[(2 * warp + pieces) * HC + h] = make_float4(s.m[r][i], l, s.mv[r][i], 0.0f);
                    }
                }
            }
            if (!whole) {
                if (lane == 0) {
                    const long long at = va + n - (cc.tile - from);  // the piece's first tile in the sequence
                    meta[2 * warp + pieces] = PieceMeta{(static_cast<long long>(cc.b) << 32) | cc.unit,
                                                        from == 0 ? (at > v0 ? 2 : 1) : 0, unit_done ? 1 : 0};
                }
                ++pieces;
            }
            if (n + 1 < count) {
                cursor_next(p, cum, cc);
                from = 0;
                unit_begin<D, HC, kF16>(p, cc, lane, s);
            }
        }
    }
    __syncthreads();

    // Merge the pieces of each unit that is not one warp's, its heads dealt to the
    // warps.  Lane i holds place i of the pieces' list (two places a warp, in the
    // order of the sequence); a unit's pieces after its first are in first places.
    static_assert(2 * kWarps <= 32, "a lane for each place");
    const long long place = lane < 2 * kWarps ? meta[lane].unit : -1;
    const long long back1 = __shfl_up_sync(0xffffffffu, place, 1), back2 = __shfl_up_sync(0xffffffffu, place, 2);
    const bool is_first = place >= 0 && ((lane & 1) || lane == 0 || (back1 >= 0 ? back1 : back2) != place);
    for (unsigned left = __ballot_sync(0xffffffffu, is_first); left != 0; left &= left - 1) {
        const int from = __ffs(left) - 1, w0 = from >> 1;
        const PieceMeta head_piece = meta[from];
        const unsigned others =
            __ballot_sync(0xffffffffu, place == head_piece.unit && lane > from && (lane & 1) == 0);
        const int n = 1 + __popc(others);
        const bool ends = n == 1 ? head_piece.ends : meta[2 * (w0 + n - 1)].ends;
        const int b = static_cast<int>(head_piece.unit >> 32), unit = static_cast<int>(head_piece.unit & 0x7fffffff);
        const int hkv = p.chunks == 1 ? unit : unit / p.chunks, chunk = unit - hkv * p.chunks;
        const int heads = min(HC, p.group - chunk * HC);
        const int64_t row0 = static_cast<int64_t>(b) * p.Hq + hkv * p.group + chunk * HC;
        const bool whole = head_piece.begins && ends;
        const int64_t ws = 2ll * blockIdx.x + (head_piece.begins == 2 ? 1 : 0);
        // Lane h + HC * k: the references, sums and weights of head h's pieces k, k + 32 / HC, ..
        constexpr int kApart = 32 / HC, kHeld = (kWarps + kApart - 1) / kApart;
        float4 e[kHeld], all = make_float4(kLowest, 0.0f, kLowest, 0.0f);
        float weight[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int k = lane / HC + i * kApart;
            e[i] = k < n ? ml[(k == 0 ? from : 2 * (w0 + k)) * HC + lane % HC] : make_float4(kLowest, 0.0f, kLowest, 0.0f);
            fold(all, e[i]);
        }
        fold_lanes<HC>(all);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) weight[i] = ex2_approx(e[i].z - all.z);
#pragma unroll
        for (int i = 0; i < HC / kWarps; ++i) {
            const int h = warp + i * kWarps;
            Columns<D> acc{};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float wt = __shfl_sync(0xffffffffu, weight[k / kApart], h + HC * (k % kApart));
                if (k >= n) continue;
                Columns<D> x;
                x.load(reinterpret_cast<const float*>(k == 0 && (from & 1) ? smem + w0 * L::kStages * L::kStage
                                                                           : smem + L::kPieceOff + (w0 + k) * L::kPiece) + h * D,
                       lane);
                acc.add(x, wt);
            }
            const float m = __shfl_sync(0xffffffffu, all.x, h), l = __shfl_sync(0xffffffffu, all.y, h);
            const float mv = __shfl_sync(0xffffffffu, all.z, h);
            if (h >= heads) continue;
            if (whole) {
                acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor(m, l, mv));
                if (p.lse && lane == 0) p.lse[row0 + h] = (m + __log2f(l)) * kLn2;
            } else {
                acc.store(p.ws_o + (ws * HC + h) * D, lane);
                if (lane == 0) p.ws_ml[ws * HC + h] = make_float4(m, l, mv, 0.0f);
            }
        }
    }
}

// Merge the pieces of the units that CTA boundaries cut: block j takes the unit
// that the boundary between the slices of CTAs j and j + 1 cuts, if it is the
// unit's first one.  Its warps share out the heads, and a head's pieces where there
// are more warps than heads; of few units, with many pieces each, the heads go to
// grid.y blocks.
// Launched with programmatic stream serialisation: it waits for the kernel before
// it reads.
constexpr int kCombineWarps = 8;

template <int D, int HC, bool kF16>
__global__ void __launch_bounds__(kCombineWarps * 32) decode_e4m3_combine_kernel(const E4m3Params p) {
    __shared__ __align__(16) float s_acc[kCombineWarps][D];
    grid_wait();
    const longlong2 geom = *p.geom;  // {tiles, tiles of a slice}
    const int4 f = p.first[blockIdx.x + 1];  // not written past the last slice
    const long long at = geom.y * (blockIdx.x + 1ll);
    if (at >= geom.x) return;
    if (f.z == 0 || f.z > geom.y) return;  // not cut here, or cut at an earlier boundary
    const int hkv = p.chunks == 1 ? f.y : f.y / p.chunks, chunk = f.y - hkv * p.chunks;
    const int heads = min(HC, p.group - chunk * HC);
    // The unit starts in the slice before the boundary; its pieces: of CTA blockIdx.x,
    // in its second place unless its slice starts with the unit, and on.
    const int n = 2 + static_cast<int>(divide(f.w - f.z - 1, static_cast<int>(min(geom.y, 0x7fffffffll))));
    const long long slot0 = 2ll * blockIdx.x + (f.z != geom.y ? 1 : 0);
    const int64_t row0 = static_cast<int64_t>(f.x) * p.Hq + hkv * p.group + chunk * HC;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto slot = [&](int i, int h) {
        return (i == 0 ? slot0 : 2 * (blockIdx.x + static_cast<long long>(i))) * HC + h;
    };
    // Heads at a time, and the warps that share a head's pieces.
    int abreast = 1;
    while (gridDim.y == 1 && abreast < heads && abreast < kCombineWarps) abreast *= 2;
    const int sharers = kCombineWarps / abreast, sharer = warp % sharers;
    for (int h0 = blockIdx.y * abreast; h0 < heads; h0 += gridDim.y * abreast) {
        const int h = min(heads - 1, h0 + warp / sharers);
        float4 all = make_float4(kLowest, 0.0f, kLowest, 0.0f);
        for (int i = lane; i < n; i += 32) fold(all, p.ws_ml[slot(i, h)]);
        fold_lanes<1>(all);
        Columns<D> acc{};
#pragma unroll 4
        for (int i = sharer; i < n; i += sharers) {
            Columns<D> x;
            x.load(p.ws_o + slot(i, h) * D, lane);
            acc.add(x, ex2_approx(p.ws_ml[slot(i, h)].z - all.z));
        }
        if (sharers > 1) {
            acc.store(s_acc[warp], lane);
            __syncthreads();
            if (sharer == 0)
                for (int i = 1; i < sharers; ++i) {
                    Columns<D> x;
                    x.load(s_acc[warp + i], lane);
                    acc.add(x, 1.0f);
                }
            __syncthreads();
        }
        if (sharer == 0 && h0 + warp / sharers < heads) {
            acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor(all.x, all.y, all.z));
            if (lane == 0 && p.lse) p.lse[row0 + h] = (all.x + __log2f(all.y)) * kLn2;
        }
    }
}

// Query heads a CTA serves at a time: one or two 8-row halves of the product.
int heads_at_once(int group) { return group <= 8 ? 8 : 16; }

int ctas_per_sm(const PagedShape& s) {
    if (heads_at_once(s.Hq / s.Hkv) == 8) return s.D == 64 ? E4m3Layout<64, 8>::kPerSm : E4m3Layout<128, 8>::kPerSm;
    return s.D == 64 ? E4m3Layout<64, 16>::kPerSm : E4m3Layout<128, 16>::kPerSm;
}

// Workspace: cum (long long [B + 1]), geom (longlong2), first (int4 [grid]), the
// pieces of the cut units and their references and sums.
struct WsLayout {
    size_t geom, first, ws_o, ws_ml, bytes;
    WsLayout(const PagedShape& s, int grid) {
        const size_t rows = 2ull * grid * heads_at_once(s.Hq / s.Hkv);
        auto up16 = [](size_t x) { return (x + 15) / 16 * 16; };
        geom = up16(8ull * (s.B + 1));
        first = geom + sizeof(longlong2);
        ws_o = first + 16ull * grid;
        ws_ml = ws_o + rows * s.D * sizeof(float);
        bytes = ws_ml + rows * sizeof(float4);
    }
};

template <int D, int HC, bool kF16, bool kWholePages>
cudaError_t launch_main(const E4m3Params& p, int grid, int prefix, int device, cudaStream_t st) {
    using L = E4m3Layout<D, HC>;
    auto* kern = decode_e4m3_kernel<D, HC, kF16, kWholePages>;
    static bool attr_set[64] = {};  // device < 64 (device_env)
    cudaError_t e = cudaSuccess;
    if (!attr_set[device]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[device] = true;
    }
    e = launch_serial(kern, dim3(grid), L::kWarps * 32, L::kBytes, st, p, prefix);
    if (e != cudaSuccess || grid < 2) return e;
    // Few units: each has many pieces, and its heads are shared out to more blocks.
    const bool few = static_cast<long long>(p.B) * p.Hkv * p.chunks * 4 < grid;
    return launch_serial(decode_e4m3_combine_kernel<D, HC, kF16>, dim3(grid - 1, few ? std::min(HC, p.group) : 1),
                         kCombineWarps * 32, 0, st, p);
}

template <int D, int HC>
cudaError_t launch_types(const E4m3Params& p, bool f16, bool whole, int grid, int prefix,
                         const LaunchEnv& env) {
    const int dev = env.device;
    cudaStream_t st = env.stream;
    if (f16)
        return whole ? launch_main<D, HC, true, true>(p, grid, prefix, dev, st)
                     : launch_main<D, HC, true, false>(p, grid, prefix, dev, st);
    return whole ? launch_main<D, HC, false, true>(p, grid, prefix, dev, st)
                 : launch_main<D, HC, false, false>(p, grid, prefix, dev, st);
}

}  // namespace

size_t decode_e4m3_workspace_bytes(const PagedShape& s, int num_sms) {
    return WsLayout(s, ctas_per_sm(s) * num_sms).bytes;
}

cudaError_t launch_decode_paged_e4m3(const uint16_t* q, const uint8_t* kv, const float* scales,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     uint16_t* o, float* lse, void* ws, const PagedShape& s,
                                     const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    const int grid = ctas_per_sm(s) * env.num_sms;
    const WsLayout lay(s, grid);
    uint8_t* base = static_cast<uint8_t*>(ws);
    const bool prefix = s.B <= kMaxPrefixB;
    E4m3Params p{};
    p.q = q;
    p.kv = kv;
    p.scales = scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.cum = prefix ? nullptr : reinterpret_cast<long long*>(base);
    p.geom = reinterpret_cast<longlong2*>(base + lay.geom);
    p.first = reinterpret_cast<int4*>(base + lay.first);
    p.ws_o = reinterpret_cast<float*>(base + lay.ws_o);
    p.ws_ml = reinterpret_cast<float4*>(base + lay.ws_ml);
    p.status = env.status;
    p.page = PageDivider(s.page);
    p.B = s.B;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.group = s.Hq / s.Hkv;
    const int hc = heads_at_once(p.group);
    p.chunks = (p.group + hc - 1) / hc;
    p.max_pages = s.max_pages;
    p.num_blocks = s.num_blocks;
    p.scale_log2 = s.scale * 1.4426950408889634f;

    cudaError_t e = cudaSuccess;
    if (!prefix) {
        e4m3_prefix_kernel<<<1, 1024, 0, env.stream>>>(p);
        e = cudaGetLastError();
    }
    const bool f16 = s.f16 != 0, whole = s.page % kTile == 0;
    if (e == cudaSuccess) {
        if (s.D == 64)
            e = hc == 8 ? launch_types<64, 8>(p, f16, whole, grid, prefix, env)
                        : launch_types<64, 16>(p, f16, whole, grid, prefix, env);
        else
            e = hc == 8 ? launch_types<128, 8>(p, f16, whole, grid, prefix, env)
                        : launch_types<128, 16>(p, f16, whole, grid, prefix, env);
    }
    if (grid_out) *grid_out = grid;
    if (kernels_launched) *kernels_launched = (prefix ? 1 : 2) + (grid > 1 ? 1 : 0);
    return e;
}

}  // namespace attn
