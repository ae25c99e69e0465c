// evict.cu -- eviction from a paged cache by accumulated attention weight
// (attn_evict_paged, attn_evict_paged_e2m1).
//
// Of a request with more than `keep` keys, each KV head keeps its last `recent` slots and
// the keep - recent heaviest of the others, and the kept rows move to slots 0 .. keep - 1 in
// their order.  Two kernels.  evict_select_kernel, a CTA for each (request, KV head): the
// weights as ordered integers, the smallest kept one found digit by digit from histograms
// (radix selection: 11, 11 and 10 bits), then the kept slots written in order and the
// weights moved.  evict_move_kernel: the rows.  A kept row never moves up, so in place is
// safe if a row is read before its slot is written: slots are taken in order, a chunk is
// read whole before any of it is written.  Columns of a row have nothing to do with one
// another: where (request, KV head) pairs are few their columns go to CTAs of their own,
// instead of CTAs that would have to wait for one another.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "e2m1.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace attn {
namespace {

struct EvictParams {
    uint8_t* cache;
    uint8_t* scales;
    float* weights;
    const int *block_table, *lens;
    int *new_lens, *kept;
    unsigned* status;
    PageDivider page;
    int B, Hkv, max_pages, num_blocks, keep, recent;
};

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeldKeys = 8192;  // in shared memory; those behind are read again

// Integers in the order of the weights: -0 as 0, NaN under everything.
__device__ __forceinline__ uint32_t ordered(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A request's slots; len: 0 if out of range (reported by the first kernel).
struct Slots {
    const EvictParams& p;
    const int* table;
    int len;
    __device__ __forceinline__ Slots(const EvictParams& params, int b, bool report)
        : p(params), table(params.block_table + static_cast<int64_t>(b) * params.max_pages) {
        const int n = p.lens[b], most = p.max_pages * p.page.size;
        len = n < 0 ? 0 : (n > most ? most : n);
        if (report && len != n) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
    }
    // Block and row of a slot; the block is -1 (reported) if its id is outside the pool.
    __device__ __forceinline__ int find(int slot, int* row) const {
        const int id = table[p.page.split(slot, row)];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) return id;
        atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        return -1;
    }
    __device__ __forceinline__ float* weight(int slot, int hkv) const {
        int row;
        const int id = find(slot, &row);
        return id < 0 ? nullptr : p.weights + (static_cast<int64_t>(id) * p.Hkv + hkv) * p.page.size + row;
    }
};

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
    __shared__ uint32_t s_key[kHeldKeys];
    __shared__ int s_bin[kBins];
    __shared__ int s_warp[kSelectWarps][2];
    __shared__ int s_digit, s_above;
    grid_wait();
    grid_launch_next();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    for (long long unit = blockIdx.x; unit < static_cast<long long>(p.B) * p.Hkv; unit += gridDim.x) {
        const int b = static_cast<int>(unit / p.Hkv), hkv = static_cast<int>(unit % p.Hkv);
        const Slots slots(p, b, hkv == 0 && tid == 0);
        int* kept = p.kept + unit * p.keep;
        if (hkv == 0 && tid == 0) p.new_lens[b] = min(slots.len, p.keep);
        if (slots.len <= p.keep) {
            for (int i = tid; i < p.keep; i += kSelectThreads) kept[i] = i < slots.len ? i : -1;
            continue;
        }
        const int n = slots.len - p.recent, want = p.keep - p.recent;  // candidates, those of them kept
        auto load = [&](int i) {
            const float* w = slots.weight(i, hkv);
            return w ? ordered(*w) : 0u;
        };
        __syncthreads();  // the unit before has been read
        for (int i = tid; i < min(n, kHeldKeys); i += kSelectThreads) s_key[i] = load(i);
        auto key = [&](int i) { return i < kHeldKeys ? s_key[i] : load(i); };

        // The key of the last kept one, from the highest digit on: `left` of those that share
        // the digits so far are kept.
        uint32_t prefix = 0;
        int left = want, shift = 32;
        for (int bits = 11; shift > 0 && want > 0; shift -= bits, bits = shift < 11 ? shift : 11) {
            const int low = shift - bits;
            for (int i = tid; i < kBins; i += kSelectThreads) s_bin[i] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kSelectThreads) {
                const uint32_t k = key(i);
                if (shift == 32 || (k >> shift) == prefix) atomicAdd(&s_bin[(k >> low) & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            // Thread i has bins 4 i .. 4 i + 3; counts from the top bin down.
            constexpr int kPer = kBins / kSelectThreads;
            int mine[kPer], own = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) own += mine[i] = s_bin[tid * kPer + i];
            int above = own;  // in this and all higher lanes, then warps
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_down_sync(0xffffffffu, above, o);
                if (lane + o < 32) above += x;
            }
            if (lane == 0) s_warp[warp][0] = above;
            __syncthreads();
            for (int i = warp + 1; i < kSelectWarps; ++i) above += s_warp[i][0];
            above -= own;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {
                if (above < left && left <= above + mine[i]) {
                    s_digit = tid * kPer + i;
                    s_above = above;
                }
                above += mine[i];
            }
            __syncthreads();
            prefix = prefix << bits | static_cast<uint32_t>(s_digit);
            left -= s_above;
        }

        // Kept slots in order: a warp has a run of them, and counts first.
        const int run = (n + kSelectWarps - 1) / kSelectWarps, from = min(n, warp * run), to = min(n, from + run);
        int over = 0, equal = 0;
        for (int i = from; i < to; i += 32) {
            const uint32_t k = i + lane < to ? key(i + lane) : 0u;
            over += __popc(__ballot_sync(0xffffffffu, i + lane < to && k > prefix));
            equal += __popc(__ballot_sync(0xffffffffu, i + lane < to && k == prefix));
        }
        __syncthreads();  // s_warp has been read
        if (lane == 0) {
            s_warp[warp][0] = over;
            s_warp[warp][1] = equal;
        }
        __syncthreads();
        over = equal = 0;
        for (int i = 0; i < warp; ++i) {
            over += s_warp[i][0];
            equal += s_warp[i][1];
        }
        if (want > 0)
            for (int i = from; i < to; i += 32) {
                const uint32_t k = i + lane < to ? key(i + lane) : 0u;
                const unsigned o = __ballot_sync(0xffffffffu, i + lane < to && k > prefix);
                const unsigned e = __ballot_sync(0xffffffffu, i + lane < to && k == prefix);
                const unsigned below = (1u << lane) - 1;
                const int before = equal + __popc(e & below);  // equal ones in front: the lowest stay
                if ((o >> lane & 1) || ((e >> lane & 1) && before < left))
                    kept[over + __popc(o & below) + min(before, left)] = i + lane;
                over += __popc(o);
                equal += __popc(e);
            }
        for (int i = tid; i < p.recent; i += kSelectThreads) kept[want + i] = n + i;
        __syncthreads();

        // The weights follow, then zeros.
        for (int i0 = 0; i0 < p.keep; i0 += kSelectThreads) {
            const int i = i0 + tid;
            float w = 0.0f;
            if (i < p.keep) {
                const float* at = slots.weight(kept[i], hkv);
                if (at) w = *at;
            }
            __syncthreads();
            if (i < p.keep) {
                float* at = slots.weight(i, hkv);
                if (at) *at = w;
            }
        }
        __syncthreads();
        for (int i = p.keep + tid; i < slots.len; i += kSelectThreads) {
            float* at = slots.weight(i, hkv);
            if (at) *at = 0.0f;
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveDepth = 4;  // pieces of a thread in flight

// Moves one column range of the kept rows of (request, KV head, K or V): pieces of T, `pieces`
// (a power of two) to a row, at byte `first` of rows of row_bytes.
template <typename T>
__device__ __forceinline__ void move_rows(const EvictParams& p, uint8_t* base, int row_bytes, int first, int pieces,
                                          const Slots& slots, const int* kept, int side, int hkv) {
    const int tid = threadIdx.x, piece = tid & (pieces - 1), r0 = tid / pieces, rows = kMoveThreads / pieces;
    auto at = [&](int slot) -> T* {
        int row;
        const int id = slots.find(slot, &row);
        if (id < 0) return nullptr;
        const int64_t n = (static_cast<int64_t>(id) * 2 + side) * p.Hkv + hkv;
        return reinterpret_cast<T*>(base + (n * p.page.size + row) * row_bytes + first) + piece;
    };
    for (int i0 = 0; i0 < p.keep; i0 += rows * kMoveDepth) {
        T v[kMoveDepth];
        bool moves[kMoveDepth];
#pragma unroll
        for (int u = 0; u < kMoveDepth; ++u) {
            const int i = i0 + u * rows + r0, from = i < p.keep ? kept[i] : i;
            const T* src = from != i ? at(from) : nullptr;
            moves[u] = src != nullptr;
            if (moves[u]) v[u] = *src;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveDepth; ++u) {
            T* dst = moves[u] ? at(i0 + u * rows + r0) : nullptr;
            if (dst) *dst = v[u];
        }
        // (The next chunk's rows lie above every slot written here.)
    }
}

// Block (x, y): unit y of (request, KV head), part x: sides times column ranges, then sides of
// the scales.
template <int kRowBytes, int kScaleBytes>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int ranges) {
    grid_wait();
    grid_launch_next();
    for (long long unit = blockIdx.y; unit < static_cast<long long>(p.B) * p.Hkv; unit += gridDim.y) {
        const int b = static_cast<int>(unit / p.Hkv), hkv = static_cast<int>(unit % p.Hkv);
        const Slots slots(p, b, false);
        if (slots.len <= p.keep) continue;
        const int* kept = p.kept + unit * p.keep;
        const int part = blockIdx.x;
        if (part < 2 * ranges) {
            const int bytes = kRowBytes / ranges;
            move_rows<uint4>(p, p.cache, kRowBytes, part / 2 * bytes, bytes / 16, slots, kept, part % 2, hkv);
        } else if constexpr (kScaleBytes == 8) {
            move_rows<uint2>(p, p.scales, 8, 0, 1, slots, kept, part % 2, hkv);
        } else if constexpr (kScaleBytes == 4) {
            move_rows<uint32_t>(p, p.scales, 4, 0, 1, slots, kept, part % 2, hkv);
        }
        __syncthreads();
    }
}

template <int kRowBytes, int kScaleBytes>
cudaError_t launch_move(const EvictParams& p, const LaunchEnv& env, int* grid_out) {
    const long long units = static_cast<long long>(p.B) * p.Hkv;
    int ranges = 1;
    while (ranges * 32 < kRowBytes && 2 * ranges * units < 4ll * env.num_sms) ranges *= 2;
    const dim3 grid(2 * ranges + (kScaleBytes ? 2 : 0), static_cast<unsigned>(std::min(units, 65535ll)));
    *grid_out = static_cast<int>(grid.x * grid.y);
    return launch_serial(evict_move_kernel<kRowBytes, kScaleBytes>, grid, kMoveThreads, 0, env.stream, p, ranges);
}

}  // namespace

cudaError_t launch_evict_paged(const EvictShape& s, const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    EvictParams p{};
    p.cache = static_cast<uint8_t*>(s.cache);
    p.scales = s.scales;
    p.weights = s.weights;
    p.block_table = s.block_table;
    p.lens = s.seq_lens;
    p.new_lens = s.new_lens;
    p.kept = s.kept;
    p.status = env.status;
    p.page = PageDivider(s.page);
    p.B = s.B;
    p.Hkv = s.Hkv;
    p.max_pages = s.max_pages;
    p.num_blocks = s.num_blocks;
    p.keep = s.keep;
    p.recent = s.recent;
    const long long units = static_cast<long long>(s.B) * s.Hkv;
    cudaError_t e = launch_serial(evict_select_kernel, dim3(static_cast<unsigned>(std::min(units, 0x7fffffffll))),
                                  kSelectThreads, 0, env.stream, p);
    if (e != cudaSuccess) return e;
    *kernels_launched = 2;
    if (s.scales) return s.D == 64 ? launch_move<32, 4>(p, env, grid_out) : launch_move<64, 8>(p, env, grid_out);
    return s.D == 64 ? launch_move<128, 0>(p, env, grid_out) : launch_move<256, 0>(p, env, grid_out);
}

}  // namespace attn
