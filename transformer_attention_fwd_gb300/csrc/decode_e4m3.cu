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
// relative to 2^mv, mv following a maximum over x_j + log2 vs_j, as two fp16 terms
// with a product each: one alone, 11 bits, made results that are small differences of
// large sums wrong by their own size.  A tile with keys 2^20 or more under the reference
// takes its weights in groups, each relative to its largest, so what light keys add up
// to behind a heavy one with no value is there too.  (The second term costs 1 % at
// 64 x 4096 keys with up to 8 heads per KV head of 128, 8 % of 64, and 15 % with 16
// heads; products in another order, both checks in one vote and the second term made
// behind the first one's products change nothing.)  The result is (sum w_j v_j) / (sum p_j) * 2^(mv - m).  A reference moves
// only when a key exceeds it by 2^kSlack.
//
// Work: all 16-key tiles of all (request, KV head, head chunk) units are laid
// end to end, cut into one equal slice per CTA and that into one per warp.  A
// warp streams its tiles through a ring of its own with 16-byte asynchronous
// copies; nothing in the loop waits for another warp.  Units inside one warp's
// range are written at once; the pieces of the others are merged in the CTA at
// its end, and those that a CTA boundary cuts by the combine kernel.  Two to four
// small CTAs share an SM, as registers allow, so that one's start and end pass
// under the others' streaming (three instead of two, with rings of three tiles
// instead of four, took 3.4 us off below, and 1.1 off the ragged one).  More of them
// than fit at once, to even out the SMs, lost 5 us for each further wave: a start
// costs that much.
//
// 64 requests of 4096 keys, Hq 32, Hkv 8, D 128, 16-token blocks (539 MB): 89.6 us,
// 6.0 TB/s.  Every CTA sums the lengths and finds its place in 2.8 us, the first
// tiles are there after 5.6, the SMs run dry between 75 and 81 us (together they
// stream at 7.2 TB/s; these before the weights' second terms, at 88.6 us), merging
// takes 1 to 2 us and the combine kernel 3.  With 8 query heads per KV head and ragged
// lengths (231 MB) 44.6 us, by the same fixed costs (short contexts, for which they
// are all of the time, are in decode_e4m3_short.cu); at D = 64 101 us for 540 MB.
// With 16 heads per KV head 118 us (D = 128) and 139 us (D = 64): two and three warps
// to a scheduler, each waiting out the latencies of its own instructions (issue active
// 43 and 58 %, tensor pipe 38 and 32 %).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_internal.h"
#include "decode_e4m3.cuh"
#include "pdl.cuh"

namespace attn {
namespace {

template <int D, int HC>
struct E4m3Layout {
    static constexpr int kWarps = 4;
    static constexpr int kPerSm = D == 128 ? (HC == 8 ? 3 : 2) : (HC == 8 ? 4 : 3);  // CTAs, as registers allow
    static constexpr int kStage = kStageBytes<D>;
    static constexpr int kPiece = HC * D * 4;
    static constexpr int kStages = HC == 8 ? 3 : 4;
    static constexpr int kPieceOff = kWarps * kStages * kStage;
    static constexpr int kMlOff = kPieceOff + kWarps * kPiece;  // [warp][2][HC] float4
    static constexpr int kMetaOff = kMlOff + kWarps * 2 * HC * 16;
    static constexpr int kCumOff = kMetaOff + kWarps * 2 * 16;
    static constexpr int kBytes = kCumOff + (kMaxPrefixB + 1) * 8 + 40 * 8;
    static_assert(kStages * kStage >= kPiece, "a warp's ring holds its second piece");
    static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "CTAs to an SM");
};

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
        const Cursor lc = cursor_at(p, cum, va);
        Cursor cc = lc;
        if (threadIdx.x == 0) p.first[blockIdx.x] = make_int4(lc.b, lc.unit, lc.tile, lc.tiles);  // va = v0
        Feed<D, L::kStages, kWholePages> feed(p, cum, lc, count, ring, lane);
#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) feed.issue();

        UnitState<D, HC> s;
        const uint8_t* stage = ring;
        int pieces = 0;
        int from = cc.tile;  // the unit's first tile of this warp
        unit_begin<D, HC, kF16>(p, cc, lane, s);
        for (int n = 0; n < count; ++n) {
            asm volatile("cp.async.wait_group %0;" :: "n"(L::kStages - 2) : "memory");
            __syncwarp();  // the tile is there, and the stage filled next has been read
            feed.issue();
            unit_tile<D, HC, kWholePages>(stage, min(kTile, cc.len - cc.tile * kTile), lane, s);
            stage += kStageBytes<D>;
            if (stage == ring + L::kStages * kStageBytes<D>) stage = ring;
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
            if (whole) unit_out<D, HC, kF16>(s, p, row0, heads, lane);
            else unit_piece<D, HC>(s, piece, ml + (2 * warp + pieces) * HC, lane);
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
                acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor(all.x, all.y, all.z));
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
    return decode_e4m3_short_ranks(s, num_sms) > 0 ? 0 : WsLayout(s, ctas_per_sm(s) * num_sms).bytes;
}

cudaError_t launch_decode_paged_e4m3(const uint16_t* q, const uint8_t* kv, const float* scales,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     uint16_t* o, float* lse, void* ws, const PagedShape& s,
                                     const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    E4m3Params p{};
    p.q = q;
    p.kv = kv;
    p.scales = scales;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
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
    int grid = 0;
    if (const int ranks = decode_e4m3_short_ranks(s, env.num_sms); ranks > 0) {
        const cudaError_t e = launch_decode_e4m3_short(p, s, ranks, env, &grid);
        if (grid_out) *grid_out = grid;
        if (kernels_launched) *kernels_launched = 1;
        return e;
    }
    grid = ctas_per_sm(s) * env.num_sms;
    const WsLayout lay(s, grid);
    uint8_t* base = static_cast<uint8_t*>(ws);
    const bool prefix = s.B <= kMaxPrefixB;
    p.cum = prefix ? nullptr : reinterpret_cast<long long*>(base);
    p.geom = reinterpret_cast<longlong2*>(base + lay.geom);
    p.first = reinterpret_cast<int4*>(base + lay.first);
    p.ws_o = reinterpret_cast<float*>(base + lay.ws_o);
    p.ws_ml = reinterpret_cast<float4*>(base + lay.ws_ml);

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
