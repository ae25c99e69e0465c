// decode_cache_long.cuh -- the decode over a quantised cache for long contexts and many
// requests: all tiles laid end to end, cut into equal slices.  decode_e4m3.cu says how;
// what depends on the format is in the class C (decode_cache.cuh).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "decode_cache.cuh"
#include "pdl.cuh"

namespace attn {

// What one CTA of the long kernel holds; C::kLongPerSm<D, HC> CTAs share an SM and a warp's
// ring has C::kLongStages<D, HC> stages.
template <class C, int D, int HC>
struct LongLayout {
    static constexpr int kWarps = 4;
    static constexpr int kPerSm = C::template kLongPerSm<D, HC>;
    static constexpr int kStage = C::template kStageBytes<D>;
    static constexpr int kPiece = HC * D * 4;
    static constexpr int kStages = C::template kLongStages<D, HC>;
    static constexpr int kPieceOff = kWarps * kStages * kStage;
    static constexpr int kMlOff = kPieceOff + kWarps * kPiece;  // [warp][2][HC] float4
    static constexpr int kMetaOff = kMlOff + kWarps * 2 * HC * 16;
    static constexpr int kCumOff = kMetaOff + kWarps * 2 * 16;
    static constexpr int kBytes = kCumOff + (kMaxPrefixB + 1) * 8 + 40 * 8;
    static_assert(kStages * kStage >= kPiece, "a warp's ring holds its second piece");
    static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "CTAs to an SM");
};

__device__ __forceinline__ Cursor cursor_at(const CacheParams& p, const long long* cum, long long v) {
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

// cum[b] = tiles of requests 0 .. b - 1, by the whole block.
template <class C>
__device__ void tile_prefix(const CacheParams& p, long long* cum, long long* scan, bool report) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + nt - 1) / nt;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = p.seq_lens[b], L = clamped(p, n);
        if (report && L != n) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        mine += (L + C::kKeys - 1) / C::kKeys;
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
        run = b + 1 == b1 ? end : run + (clamped_len(p, b) + C::kKeys - 1) / C::kKeys;
        cum[b + 1] = run;
    }
    if (tid == 0) cum[0] = 0;
    __syncthreads();
}

template <class C>
__global__ void __launch_bounds__(1024) decode_prefix_kernel(const CacheParams p) {
    __shared__ long long scan[32];
    tile_prefix<C>(p, p.cum, scan, true);
}

// Tiles of a CTA's slice: at least one a warp.
__device__ __forceinline__ long long slice_tiles(long long total, int grid, int warps) {
    const long long per = divide(total + grid - 1, grid);
    return per < warps ? warps : per;
}

// What a warp leaves of a unit it has not covered alone.
struct PieceMeta {
    long long unit;  // request << 32 | unit, -1: none
    int begins, ends;  // the piece holds the unit's first (last) tile; begins = 2: not at the slice's start
};

template <class C, int D, int HC, bool kF16, bool kWholePages>
__global__ void __launch_bounds__(LongLayout<C, D, HC>::kWarps * 32, LongLayout<C, D, HC>::kPerSm)
decode_long_kernel(const CacheParams p, int prefix_in_kernel) {
    using L = LongLayout<C, D, HC>;
    constexpr int kWarps = L::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* ring = smem + warp * L::kStages * L::kStage;
    float4* ml = reinterpret_cast<float4*>(smem + L::kMlOff);
    PieceMeta* meta = reinterpret_cast<PieceMeta*>(smem + L::kMetaOff);
    long long* s_cum = reinterpret_cast<long long*>(smem + L::kCumOff);
    const long long* cum = p.cum;
    grid_wait();
    grid_launch_next();
    if (prefix_in_kernel) {
        tile_prefix<C>(p, s_cum, s_cum + kMaxPrefixB + 1, blockIdx.x == 0);
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
        const Cursor lc = cursor_at(p, cum, va);
        Cursor cc = lc;
        if (threadIdx.x == 0) p.first[blockIdx.x] = make_int4(lc.b, lc.unit, lc.tile, lc.tiles);  // va = v0
        Feed<C, D, L::kStages, kWholePages> feed(p, cum, lc, count, ring, lane);
#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) feed.issue();

        UnitState<D, HC> s;
        const uint8_t* stage = ring;
        int pieces = 0;
        int from = cc.tile;  // the unit's first tile of this warp
        unit_begin<C, D, HC, kF16>(p, cc, lane, s);
        for (int n = 0; n < count; ++n) {
            asm volatile("cp.async.wait_group %0;" :: "n"(L::kStages - 2) : "memory");
            __syncwarp();  // the tile is there, and the stage filled next has been read
            feed.issue();
            C::template tile<D, HC, kWholePages>(stage, min(C::kKeys, cc.len - cc.tile * C::kKeys), lane, s,
                                                 tile_scores<C, HC>(p, cc));
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
            if (whole) unit_out<C, D, HC, kF16>(s, p, hkv, row0, heads, lane);
            else unit_piece<C, D, HC>(s, piece, ml + (2 * warp + pieces) * HC, lane);
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
                unit_begin<C, D, HC, kF16>(p, cc, lane, s);
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
        auto slot = [&](int k) { return k == 0 ? from : 2 * (w0 + k); };
        MergedHeads<D, HC, kWarps> merged(n, lane, [&](int k, int h) { return ml[slot(k) * HC + h]; });
#pragma unroll
        for (int i = 0; i < HC / kWarps; ++i) {
            const int h = warp + i * kWarps;
            float4 all;
            const Columns<D> acc = merged.head(h, n, lane, [&](int k, Columns<D>& x) {
                x.load(reinterpret_cast<const float*>(k == 0 && (from & 1) ? smem + w0 * L::kStages * L::kStage
                                                                           : smem + L::kPieceOff + (w0 + k) * L::kPiece) + h * D,
                       lane);
            }, &all);
            if (h >= heads) continue;
            if (whole) {
                acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor<C>(p, hkv, all.x, all.y, all.z));
                if (p.lse && lane == 0) p.lse[row0 + h] = (all.x + __log2f(all.y)) * kLn2;
            } else {
                acc.store(p.ws_o + (ws * HC + h) * D, lane);
                if (lane == 0) p.ws_ml[ws * HC + h] = all;
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

template <class C, int D, int HC, bool kF16>
__global__ void __launch_bounds__(kCombineWarps * 32) decode_combine_pieces_kernel(const CacheParams p) {
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
            acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor<C>(p, hkv, all.x, all.y, all.z));
            if (lane == 0 && p.lse) p.lse[row0 + h] = (all.x + __log2f(all.y)) * kLn2;
        }
    }
}

template <class C>
int long_per_sm(const PagedShape& s) {
    return by_shape<C>(s.D, s.Hq / s.Hkv, [](auto d, auto h) {
        return LongLayout<C, decltype(d)::value, decltype(h)::value>::kPerSm;
    });
}

// Workspace: cum (long long [B + 1]), geom (longlong2), first (int4 [grid]), the
// pieces of the cut units and their references and sums.
struct WsLayout {
    size_t geom, first, ws_o, ws_ml, bytes;
    WsLayout(const PagedShape& s, int grid, int heads) {
        const size_t rows = 2ull * grid * heads;
        auto up16 = [](size_t x) { return (x + 15) / 16 * 16; };
        geom = up16(8ull * (s.B + 1));
        first = geom + sizeof(longlong2);
        ws_o = first + 16ull * grid;
        ws_ml = ws_o + rows * s.D * sizeof(float);
        bytes = ws_ml + rows * sizeof(float4);
    }
};

template <class C, int D, int HC, bool kF16, bool kWholePages>
cudaError_t launch_main(const CacheParams& p, int grid, int prefix, int device, cudaStream_t st) {
    using L = LongLayout<C, D, HC>;
    auto* kern = decode_long_kernel<C, D, HC, kF16, kWholePages>;
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
    return launch_serial(decode_combine_pieces_kernel<C, D, HC, kF16>, dim3(grid - 1, few ? std::min(HC, p.group) : 1),
                         kCombineWarps * 32, 0, st, p);
}

template <class C, int D, int HC>
cudaError_t launch_types(const CacheParams& p, bool f16, bool whole, int grid, int prefix,
                         const LaunchEnv& env) {
    const int dev = env.device;
    cudaStream_t st = env.stream;
    if (f16)
        return whole ? launch_main<C, D, HC, true, true>(p, grid, prefix, dev, st)
                     : launch_main<C, D, HC, true, false>(p, grid, prefix, dev, st);
    return whole ? launch_main<C, D, HC, false, true>(p, grid, prefix, dev, st)
                 : launch_main<C, D, HC, false, false>(p, grid, prefix, dev, st);
}

// The launches of one call; ws: WsLayout's bytes.
template <class C>
cudaError_t launch_decode_long(CacheParams p, const PagedShape& s, void* ws, const LaunchEnv& env, int* grid_out,
                               int* kernels_launched) {
    const int grid = long_per_sm<C>(s) * env.num_sms;
    const WsLayout lay(s, grid, heads_at_once<C>(p.group));
    uint8_t* base = static_cast<uint8_t*>(ws);
    const bool prefix = s.B <= kMaxPrefixB;
    p.cum = prefix ? nullptr : reinterpret_cast<long long*>(base);
    p.geom = reinterpret_cast<longlong2*>(base + lay.geom);
    p.first = reinterpret_cast<int4*>(base + lay.first);
    p.ws_o = reinterpret_cast<float*>(base + lay.ws_o);
    p.ws_ml = reinterpret_cast<float4*>(base + lay.ws_ml);

    cudaError_t e = cudaSuccess;
    if (!prefix) {
        decode_prefix_kernel<C><<<1, 1024, 0, env.stream>>>(p);
        e = cudaGetLastError();
    }
    const bool f16 = s.f16 != 0, whole = s.page % kTile == 0;
    if (e == cudaSuccess)
        e = by_shape<C>(s.D, p.group, [&](auto d, auto h) {
            return launch_types<C, decltype(d)::value, decltype(h)::value>(p, f16, whole, grid, prefix, env);
        });
    *grid_out = grid;
    *kernels_launched = (prefix ? 1 : 2) + (grid > 1 ? 1 : 0);
    return e;
}

template <class C>
size_t decode_long_workspace(const PagedShape& s, int num_sms) {
    return WsLayout(s, long_per_sm<C>(s) * num_sms, heads_at_once<C>(s.Hq / s.Hkv)).bytes;
}

}  // namespace attn
