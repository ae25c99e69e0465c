// decode_cache_short.cuh -- the decode over a quantised cache for short contexts and few
// requests: a cluster takes each unit.  decode_e4m3_short.cu says how; what depends on
// the format is in the class C (decode_cache.cuh).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "decode_cache.cuh"
#include "pdl.cuh"

namespace attn {

constexpr int kShortWarps = 4;
constexpr int kMaxRanks = 8;  // CTAs of a cluster
// When a cluster takes each unit, with both kernels' times at head dim 128, Hkv 8,
// Hq 32, page 16:
//  - a warp has at most 16 tiles of 16 by the table's width (one request of 1024, 4096
//    and 8192 keys: 6.4, 8.9 and 13.5 us against 9.1, 11.9 and 13.8; of 32768, 64
//    tiles a warp: 41.1 against 19.8);
//  - the units fill the GPU at most twice (64 and 96 requests of 200 keys: 10.1 and
//    12.6 us against 14.6 and 16.6; 256 requests of one key, 4.5 times: 15.3
//    against 9.8, and 1024 of 200 keys, 18 times: 109 against 77).
constexpr int kMaxKeys = 256, kMaxFills = 2;  // of a warp
// A rank more only for over 16 such tiles of the unit (8 requests of 200 keys: 4.8, 5.2
// and 6.0 us with 1, 2 and 8 CTAs; of 1024: 12.0, 8.9 and 8.5 with 1, 2 and 4).
constexpr int kRankKeys = 256;

template <class C, int D, int HC>
struct ShortLayout {
    static constexpr int kPerSm = D == 128 ? (HC <= 8 ? 3 : 2) : (HC <= 8 ? 4 : 3);  // CTAs, as registers allow
    static constexpr int kPartOff = kShortWarps * C::kShortStages * C::template kStageBytes<D>;  // the CTA's part [HC][D]
    static constexpr int kMlOff = kPartOff + HC * D * 4;                // the warps' {m, l, mv} [kShortWarps][HC]
    static constexpr int kPartMlOff = kMlOff + kShortWarps * HC * 16;        // the CTA's [HC]
    static constexpr int kBytes = kPartMlOff + HC * 16;
    static_assert(C::kShortStages * C::template kStageBytes<D> >= HC * D * 4, "a warp's ring holds its part");
    static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "CTAs to an SM");
};

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The end of a CTA that has nothing to add up: it takes part in both barriers all
// the same.  So no CTA reads the shared memory of one that is gone, even if the
// lengths change under the kernel and its CTAs do not see the same.
__device__ __forceinline__ void leave(int ranks) {
    if (ranks == 1) return;
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
}

// Shared memory of another CTA of the cluster, at this CTA's address.
__device__ __forceinline__ uint32_t of_rank(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 remote4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 remote2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

template <class C, int D, int HC, bool kF16, bool kWholePages>
__global__ void __launch_bounds__(kShortWarps * 32, ShortLayout<C, D, HC>::kPerSm)
decode_short_kernel(const CacheParams p, int ranks) {
    using L = ShortLayout<C, D, HC>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* ring = smem + warp * C::kShortStages * C::template kStageBytes<D>;
    float* part = reinterpret_cast<float*>(smem + L::kPartOff);
    float4* ml = reinterpret_cast<float4*>(smem + L::kMlOff);
    float4* part_ml = reinterpret_cast<float4*>(smem + L::kPartMlOff);
    grid_wait();
    grid_launch_next();

    const int U = p.Hkv * p.chunks;
    const int cluster = static_cast<int>(blockIdx.x) / ranks, rank = static_cast<int>(blockIdx.x) - cluster * ranks;
    Cursor cc;
    cc.b = cluster / U;
    cc.unit = cluster - cc.b * U;
    const int asked = p.seq_lens[cc.b];
    cc.len = clamped(p, asked);
    cc.tiles = (cc.len + C::kKeys - 1) / C::kKeys;
    const int hkv = p.chunks == 1 ? cc.unit : cc.unit / p.chunks, chunk = cc.unit - hkv * p.chunks;
    const int heads = min(HC, p.group - chunk * HC);
    const int64_t row0 = static_cast<int64_t>(cc.b) * p.Hq + hkv * p.group + chunk * HC;
    if (asked != cc.len && cc.unit == 0 && rank == 0 && threadIdx.x == 0) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
    if (cc.tiles == 0) {  // no keys
        if (rank > 0) return leave(ranks);
        for (int i = threadIdx.x; i < heads * (D / 8); i += kShortWarps * 32)
            reinterpret_cast<uint4*>(p.o + row0 * D)[i] = make_uint4(0, 0, 0, 0);
        if (p.lse && threadIdx.x < heads) p.lse[row0 + threadIdx.x] = -INFINITY;
        return leave(ranks);
    }

    // Tiles of a warp, and the CTAs and this CTA's warps that have any.
    const int per = (cc.tiles + ranks * kShortWarps - 1) / (ranks * kShortWarps);
    const int parts = (cc.tiles + per * kShortWarps - 1) / (per * kShortWarps);
    const int first = (rank * kShortWarps + warp) * per;
    const int count = max(0, min(per, cc.tiles - first));
    const int active = min(kShortWarps, max(0, (cc.tiles - rank * kShortWarps * per + per - 1) / per));
    if (count > 0) {
        cc.tile = first;
        Feed<C, D, C::kShortStages, kWholePages> feed(p, nullptr, cc, count, ring, lane);
#pragma unroll
        for (int i = 0; i < C::kShortStages - 1; ++i) feed.issue();
        UnitState<D, HC> s;
        const uint8_t* stage = ring;
        unit_begin<C, D, HC, kF16>(p, cc, lane, s);
        for (int n = 0; n < count; ++n) {
            asm volatile("cp.async.wait_group %0;" :: "n"(C::kShortStages - 2) : "memory");
            __syncwarp();  // the tile is there, and the stage filled next has been read
            feed.issue();
            C::template tile<D, HC, kWholePages>(stage, min(C::kKeys, cc.len - cc.tile * C::kKeys), lane, s,
                                                 tile_scores<C, HC>(p, cc));
            stage += C::template kStageBytes<D>;
            if (stage == ring + C::kShortStages * C::template kStageBytes<D>) stage = ring;
            ++cc.tile;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        unit_piece<C, D, HC>(s, reinterpret_cast<float*>(ring), ml + warp * HC, lane);
    }
    __syncthreads();
    if (active > 0) {
        constexpr int kPer = HC / kShortWarps;
        MergedHeads<D, HC, kShortWarps> m(active, lane, [&](int k, int h) { return ml[k * HC + h]; });
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int h = warp + i * kShortWarps;
            float4 all;
            const Columns<D> acc = m.head(h, active, lane, [&](int k, Columns<D>& x) {
                x.load(reinterpret_cast<const float*>(smem + k * C::kShortStages * C::template kStageBytes<D>) + h * D, lane);
            }, &all);
            if (parts == 1) {  // this CTA had all of the unit
                if (h >= heads) continue;
                acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor<C>(p, hkv, all.x, all.y, all.z));
                if (p.lse && lane == 0) p.lse[row0 + h] = (all.x + __log2f(all.y)) * kLn2;
            } else {
                acc.store(part + h * D, lane);
                if (lane == 0) part_ml[h] = all;
            }
        }
    }
    if (parts == 1) return leave(ranks);
    cluster_arrive();
    cluster_wait();
    // Heads rank, rank + ranks, ..: a warp each.
    for (int h = rank + warp * ranks; h < heads; h += kShortWarps * ranks) {
        float4 all = make_float4(kLowest, 0.0f, kLowest, 0.0f);
        if (lane < parts) all = remote4(of_rank(part_ml + h, lane));
        const float z = all.z;
        fold_lanes<1>(all);
        const float weight = ex2_approx(z - all.z);
        Columns<D> acc{};
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
            const float wt = __shfl_sync(0xffffffffu, weight, k);
            if (k >= parts) continue;
            Columns<D> x;
            if constexpr (D == 128) {
                const float4 v = remote4(of_rank(part + h * D + lane * 4, k));
                x.c[0] = v.x; x.c[1] = v.y; x.c[2] = v.z; x.c[3] = v.w;
            } else {
                const float2 v = remote2(of_rank(part + h * D + lane * 2, k));
                x.c[0] = v.x; x.c[1] = v.y;
            }
            acc.add(x, wt);
        }
        acc.template store16<kF16>(p.o + (row0 + h) * D, lane, out_factor<C>(p, hkv, all.x, all.y, all.z));
        if (p.lse && lane == 0) p.lse[row0 + h] = (all.x + __log2f(all.y)) * kLn2;
    }
    cluster_arrive();  // the others have read this CTA's shared memory
    cluster_wait();
}

template <class C, int D, int HC, bool kF16, bool kWholePages>
cudaError_t launch_short_kernel(const CacheParams& p, int ranks, unsigned grid, const LaunchEnv& env) {
    using L = ShortLayout<C, D, HC>;
    auto* kern = decode_short_kernel<C, D, HC, kF16, kWholePages>;
    static bool attr_set[64] = {};  // device < 64 (device_env)
    if (!attr_set[env.device]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[env.device] = true;
    }
    return launch_serial_clusters(kern, dim3(grid), kShortWarps * 32, L::kBytes, ranks, env.stream, p, ranks);
}

template <class C, int D, int HC>
cudaError_t launch_short_types(const CacheParams& p, bool f16, bool whole, int ranks, unsigned grid, const LaunchEnv& env) {
    if (f16)
        return whole ? launch_short_kernel<C, D, HC, true, true>(p, ranks, grid, env)
                     : launch_short_kernel<C, D, HC, true, false>(p, ranks, grid, env);
    return whole ? launch_short_kernel<C, D, HC, false, true>(p, ranks, grid, env)
                 : launch_short_kernel<C, D, HC, false, false>(p, ranks, grid, env);
}

// CTAs of a cluster that takes each unit; 0: the long kernel takes the call.
template <class C>
int decode_short_ranks(const PagedShape& s, int num_sms) {
    const int group = s.Hq / s.Hkv, hc = heads_at_once<C>(group);
    const long long units = static_cast<long long>(s.B) * s.Hkv * ((group + hc - 1) / hc);
    const long long keys = static_cast<long long>(s.max_pages) * s.page;  // at most
    const int per_sm = by_shape<C>(s.D, group, [](auto d, auto h) {
        return ShortLayout<C, decltype(d)::value, decltype(h)::value>::kPerSm;
    });
    const long long room = static_cast<long long>(per_sm) * num_sms;
    int ranks = 1;
    while (ranks < kMaxRanks && 2 * ranks * units <= room && keys > kRankKeys * ranks) ranks *= 2;
    return units <= kMaxFills * room && keys <= kMaxKeys * kShortWarps * ranks ? ranks : 0;
}

template <class C>
cudaError_t launch_decode_short(const CacheParams& p, const PagedShape& s, int ranks, const LaunchEnv& env,
                                     int* grid_out) {
    const unsigned grid = static_cast<unsigned>(s.B) * static_cast<unsigned>(p.Hkv * p.chunks) * ranks;
    const bool f16 = s.f16 != 0, whole = s.page % kTile == 0;
    *grid_out = static_cast<int>(grid);
    return by_shape<C>(s.D, p.group, [&](auto d, auto h) {
        return launch_short_types<C, decltype(d)::value, decltype(h)::value>(p, f16, whole, ranks, grid, env);
    });
}

}  // namespace attn
