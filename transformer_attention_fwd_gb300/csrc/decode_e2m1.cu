// decode_e2m1.cu -- decode (one query row per (request, head)) over the paged 4-bit
// cache with one scale for each 16 elements of a row (attn_fwd_decode_paged_e2m1), and
// the sums of its attention weights.
//
//   O = sum_j p_j v_j / sum_j p_j,  p_j = 2^x_j,  x_j = log2(e) * scale * (q . k_j)
//
// with k_j, v_j = code * scale * the head's factor.  HBM bound: 2 * (D/2 + D/16) bytes
// per key and KV head are read once.  The work, its split and its merge are the 8-bit
// decode's (decode_e4m3.cu).  A code times its scale is exact in fp16, so the operands
// of the tensor cores are made from both in registers: two codes of K to one word by a
// conversion, V's by the same conversion once the nibbles of two keys' rows share a
// byte, each then times its scale; the heads' factors multiply the query and the result.
// V's sizes are in the operand, so one reference serves the sum of the weights and the
// weighted sum (the 8-bit decode has a scale per block in its weights).
//
// Measured (64 requests of 4096 keys, 32 + 8 heads, D 128): 67.6 us, 302 MB; the copies alone
// take 58, 12 of them start, tail and combine.  Conversions and products fill 59% of the issue
// slots: no limit, but three warps to a scheduler wait out their own instructions in the rest.
// Tiles of 32 keys instead of 16: 91 -> 81 us; V's products of both halves in one stretch: 79; for up
// to four heads the weights' second terms in the free columns: 77; half a warp copying each half: 68.
//
// Weights added up: the tiles leave their scores (fp32, one for each key and head) in a
// workspace, and once the log-sum-exp is known a second kernel adds 2^(x - lse) over a KV
// head's query heads to each key's weight: 2 * 4 * group bytes per key and KV head
// instead of the row of K that a second look at the keys would read.  (88.4 us; a pass of
// attn_weights_paged_e2m1 behind the decode would add 48.)
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_cache_long.cuh"
#include "decode_e2m1.cuh"

namespace attn {
namespace {

constexpr int kAddThreads = 128;
constexpr int kAddKeys = 4;  // of a thread, their reads in flight together
constexpr float kLog2e = 1.4426950408889634f;

// weights[slot] += sum over a KV head's query heads of 2^(score - lse).  Block (x, y): runs of
// kAddKeys * kAddThreads keys, gridDim.x runs apart, of (request, KV head) y, y + gridDim.y, ..
// Four heads at a time (16 bytes) where the group allows: 55.6 us instead of 59.6 with eight heads
// to a KV head, no difference with four.  A thread's chain is the length, the block ids, the weights; with one key at a time the blocks
// took 20 us at 64 x 4096 keys, most of them waiting.
template <bool kFours>
__global__ void __launch_bounds__(kAddThreads) add_scores_kernel(const CacheParams p, float* weights) {
    grid_wait();
    grid_launch_next();
    const int units = p.B * p.Hkv;
    for (int u = blockIdx.y; u < units; u += gridDim.y) {
        const int b = u / p.Hkv, hkv = u - b * p.Hkv;
        const int len = clamped_len(p, b);
        const float* lse = p.lse + static_cast<int64_t>(b) * p.Hq + hkv * p.group;
        const int* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
        const float* scores = p.scores + static_cast<int64_t>(u) * p.max_pages * p.page.size * p.group;
        // (Unsigned: a step behind the last keys of the longest tables passes 2^31.)
        for (unsigned from = blockIdx.x * (kAddKeys * kAddThreads) + threadIdx.x; from < static_cast<unsigned>(len);
             from += gridDim.x * (kAddKeys * kAddThreads)) {
            const int key0 = static_cast<int>(from);
            int id[kAddKeys], row[kAddKeys];
#pragma unroll
            for (int i = 0; i < kAddKeys; ++i) {
                const int key = key0 + i * kAddThreads;
                id[i] = key < len ? table[p.page.split(key, &row[i])] : -1;
            }
            float sum[kAddKeys] = {};
            for (int h = 0; h < p.group; h += kFours ? 4 : 1) {
                if constexpr (kFours) {  // 16 bytes at a time: the workspace is aligned to them
                    float4 v[kAddKeys];
#pragma unroll
                    for (int i = 0; i < kAddKeys; ++i) {
                        const int key = min(key0 + i * kAddThreads, len - 1);
                        v[i] = *reinterpret_cast<const float4*>(scores + static_cast<int64_t>(key) * p.group + h);
                    }
                    const float z[4] = {lse[h] * kLog2e, lse[h + 1] * kLog2e, lse[h + 2] * kLog2e, lse[h + 3] * kLog2e};
#pragma unroll
                    for (int i = 0; i < kAddKeys; ++i)
                        sum[i] += (ex2_approx(v[i].x - z[0]) + ex2_approx(v[i].y - z[1])) +
                                  (ex2_approx(v[i].z - z[2]) + ex2_approx(v[i].w - z[3]));
                } else {
                    const float z = lse[h] * kLog2e;
#pragma unroll
                    for (int i = 0; i < kAddKeys; ++i) {
                        const int key = min(key0 + i * kAddThreads, len - 1);
                        sum[i] += ex2_approx(scores[static_cast<int64_t>(key) * p.group + h] - z);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kAddKeys; ++i)
                if (static_cast<unsigned>(id[i]) < static_cast<unsigned>(p.num_blocks))  // others: reported by the decode
                    atomicAdd(weights + (static_cast<int64_t>(id[i]) * p.Hkv + hkv) * p.page.size + row[i], sum[i]);
        }
    }
}

struct AddLayout {
    size_t scores, lse, bytes;  // behind the decode's own workspace
    AddLayout(const PagedShape& s, size_t at, bool weights, bool own_lse) {
        auto up16 = [](size_t x) { return (x + 15) / 16 * 16; };
        scores = up16(at);
        lse = up16(scores + (weights ? 4ull * s.B * s.Hq * s.max_pages * s.page : 0));
        bytes = weights ? lse + (own_lse ? 4ull * s.B * s.Hq : 0) : at;
    }
};

size_t decode_bytes(const PagedShape& s, int num_sms) {
    return decode_e2m1_short_ranks(s, num_sms) > 0 ? 0 : decode_long_workspace<E2m1Cache>(s, num_sms);
}

}  // namespace

size_t decode_e2m1_workspace_bytes(const PagedShape& s, int num_sms, bool weights, bool own_lse) {
    return AddLayout(s, decode_bytes(s, num_sms), weights, own_lse).bytes;
}

cudaError_t launch_decode_paged_e2m1(const uint16_t* q, const uint8_t* kv, const uint8_t* scales, const float* factors,
                                     const int32_t* block_table, const int32_t* seq_lens, uint16_t* o, float* lse,
                                     float* weights, void* ws, const PagedShape& s, const LaunchEnv& env,
                                     int* grid_out, int* kernels_launched) {
    CacheParams p = cache_params<E2m1Cache>(q, kv, block_table, seq_lens, o, lse, s, env);
    p.row_scales = scales;
    p.factors = factors;
    if (weights) {
        uint8_t* base = static_cast<uint8_t*>(ws);
        const AddLayout lay(s, decode_bytes(s, env.num_sms), true, lse == nullptr);
        p.scores = reinterpret_cast<float*>(base + lay.scores);
        if (!lse) p.lse = reinterpret_cast<float*>(base + lay.lse);
    }
    cudaError_t e;
    if (const int ranks = decode_e2m1_short_ranks(s, env.num_sms); ranks > 0) {
        *kernels_launched = 1;
        e = launch_decode_e2m1_short(p, s, ranks, env, grid_out);
    } else {
        e = launch_decode_long<E2m1Cache>(p, s, ws, env, grid_out, kernels_launched);
    }
    if (e != cudaSuccess || !weights) return e;
    ++*kernels_launched;
    const long long keys = static_cast<long long>(s.max_pages) * s.page, units = static_cast<long long>(s.B) * s.Hkv;
    // Not more blocks than there are keys for by the table's width.
    const unsigned y = static_cast<unsigned>(std::min(units, 65535ll));
    const long long want = std::max(1ll, 32ll * env.num_sms / y), run = kAddKeys * kAddThreads;
    const unsigned x = static_cast<unsigned>(std::min(want, (keys + run - 1) / run));
    return launch_serial(p.group % 4 == 0 ? add_scores_kernel<true> : add_scores_kernel<false>, dim3(x, y), kAddThreads, 0,
                         env.stream, p, weights);
}

}  // namespace attn
