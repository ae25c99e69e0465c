// weights.cu -- attention weights of packed queries, added up over the keys of a paged
// cache (attn_weights_paged, attn_weights_paged_e2m1):
//
//   weights[key j] += sum over the request's queries i that see j and over the query
//                     heads of the KV head of 2^(x_ij - log2(e) lse_i),
//   x_ij = log2(e) * scale * (q_i . k_j)
//
// the column sums of the probabilities, which are never written down.  S^T = K Q^T on the
// tensor cores (mma.sync m16n8k16, fp32 sums) with 16 keys as rows: a key's sum then stays in
// the four lanes that hold its row.  A warp keeps 32 rows of K in registers and passes all
// query rows that see them by; each key belongs to one warp, so nothing is added twice or in
// a changing order.  The order of a product's inner index is free, so each lane reads what suits
// the reads.  For decode steps: up to eight query rows are one column block, held in registers
// while the keys stream by.  HBM bound in 16 bits (64 requests of 4096 keys, 8 KV heads, D 128:
// 88 us, 554 MB at 6.3 TB/s); in 4 bits by the conversions' instructions (47 us, 168 MB).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "e2m1.cuh"
#include "pdl.cuh"
#include "sm100.cuh"
#include "weights.cuh"
#include "weights_counts.h"

namespace attn {
namespace {

// A block is a warp: with four, that leave together, a step over 64 x 4096 4-bit keys took 66 us
// instead of 47, over 16-bit ones 103 instead of 88.
constexpr int kPerSm = 16;  // blocks an SM has room for (128 registers)
constexpr int kMostRun = 8;  // chunks of a block
constexpr int kKeys = 32;  // of a chunk, which a warp reads at a time

template <bool kF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's D/4 elements of a K row as they are in the cache: a run of 4-bit ones, every fourth eight
// of 16-bit ones, so that four lanes' reads are whole sectors.  Zeros without a row.
template <int D, bool kFour>
struct RawKey {
    static constexpr int kWords = kFour ? D / 32 : D / 8;
    uint32_t w[kWords], scale;
    __device__ __forceinline__ void load(const WeightsParams& p, int64_t row, int t) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        scale = 0;
        if (row < 0) return;
        if constexpr (!kFour) {
            const uint4* src = reinterpret_cast<const uint4*>(p.cache + row * (D * 2)) + t;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 u = src[4 * i];
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        } else {
            const uint8_t* codes = p.cache + row * (D / 2) + t * (D / 8);
            const uint8_t* scales = p.scales + row * (D / kRowScaleSpan) + t * (D / 64);
            if constexpr (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(codes);
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                scale = *reinterpret_cast<const uint16_t*>(scales);
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(codes);
                w[0] = u.x; w[1] = u.y;
                scale = *scales;
            }
        }
    }
    // As words of the products' type: a code times its scale is exact in fp16.
    __device__ __forceinline__ void words(uint32_t (&out)[D / 8]) const {
        if constexpr (!kFour) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) out[i] = w[i];
        } else {
            uint32_t by[2];
            both_halves(e4m3_to_f16x2(scale), by[0], by[1]);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                uint32_t v[4];
                e2m1_to_f16x8(w[i], v);
#pragma unroll
                for (int k = 0; k < 4; ++k) out[4 * i + k] = f16x2_mul(v[k], by[i / 2]);
            }
        }
    }
};

// Eight query rows of a KV head, from r0 on: token by token, the head's query heads within.
// Token i sees keys up to len - n + i.  Over a 4-bit cache they are fp16, bf16 ones times a power
// of two that takes a row's largest element to [512, 1024): what is exact is the decode's.
template <int D, bool kF16, bool kFour>
struct QueryRows {
    uint32_t qb[D / 8];  // row g's elements, those that the lane has of a K row
    float by[2], lse[2];  // of rows 2t and 2t + 1: what a product is multiplied by, log2(e) times the lse
    int last[2];          // the last key they see; -1: no row
    __device__ __forceinline__ void load(const WeightsParams& p, const WeightsRequest& req, int hkv, float scale, int r0,
                                         int g, int t) {
        const int n = req.end - req.begin, rows = n * p.group;  // checked on the host: fits
        const int mine = r0 + g;
        {
            const int token = mine / p.group, head = mine - token * p.group;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (req.begin + token) * p.q_token +
                                                              (hkv * p.group + head) * p.q_head);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 u = mine < rows ? src[kFour ? t * (D / 32) + i : 4 * i + t] : make_uint4(0, 0, 0, 0);
                qb[4 * i] = u.x; qb[4 * i + 1] = u.y; qb[4 * i + 2] = u.z; qb[4 * i + 3] = u.w;
            }
        }
        by[0] = by[1] = scale;
        if constexpr (kFour && !kF16) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                most = fmaxf(most, fmaxf(fabsf(bf16_lo_to_f32(qb[i])), fabsf(bf16_hi_to_f32(qb[i]))));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // 2^k; 1 for zero, subnormal or non-finite rows.
            const int e = static_cast<int>(__float_as_uint(most) >> 23);
            const int k = (e == 0 || e == 255) ? 0 : max(-126, min(126, 9 - (e - 127)));
            const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            const float back = scale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            by[0] = __shfl_sync(0xffffffffu, back, 8 * t);
            by[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) qb[i] = pack_f16x2(bf16_lo_to_f32(qb[i]) * up, bf16_hi_to_f32(qb[i]) * up);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = r0 + 2 * t + i, token = rr / p.group, head = rr - token * p.group;
            lse[i] = 0.0f;
            last[i] = -1;
            if (rr < rows) {
                lse[i] = p.lse[(hkv * p.group + head) * p.lse_head + (req.begin + token) * p.lse_token] * kWeightsLog2e;
                last[i] = lse[i] == -INFINITY ? -1 : req.len - n + token;
            }
        }
    }
    // Adds the weights of keys key0 + g and key0 + g + 8 (kw) to sum.
    __device__ __forceinline__ void add(const uint32_t (&kw0)[D / 8], const uint32_t (&kw1)[D / 8], int key0, int g,
                                        float (&sum)[2]) const {
        float s[2][4] = {};  // two chains
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const uint32_t a[4] = {kw0[2 * j], kw1[2 * j], kw0[2 * j + 1], kw1[2 * j + 1]};
            mma16<kF16 || kFour>(s[j % 2], a, qb[2 * j], qb[2 * j + 1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float w = ex2_approx(fmaf(s[0][2 * i + k] + s[1][2 * i + k], by[k], -lse[k]));
                sum[i] += key0 + i * 8 + g <= last[k] ? w : 0.0f;
            }
    }
};

// The keys of [key0, end) of one (request, KV head), by a warp.  Of 4-bit rows the next chunk is
// read while one is worked on, and the blocks of the one after are looked up; of 16-bit rows a warp
// has one chunk.
template <int D, bool kF16, bool kFour>
__device__ __forceinline__ void weights_keys(const WeightsParams& p, const WeightsRequest& req, int b, int hkv, int key0,
                                             int end, int g, int t) {
    const int* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
    // This lane's own key of a chunk is 8 t + g: {block id, row in it}; id < 0: none.
    auto find = [&](int from) {
        const int key = from + t * 8 + g;
        int2 at = make_int2(-1, 0);
        if (key < end) {
            at.x = table[p.page.split(key, &at.y)];
            if (static_cast<unsigned>(at.x) >= static_cast<unsigned>(p.num_blocks)) {
                atomicOr(p.status, ATTN_DEV_BAD_INPUT);
                at.x = -1;
            }
        }
        return at;
    };
    auto read = [&](int2 at, RawKey<D, kFour> (&raw)[4]) {
        const int64_t own = at.x < 0 ? -1 : (static_cast<int64_t>(at.x) * 2 * p.Hkv + hkv) * p.page.size + at.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i].load(p, __shfl_sync(0xffffffffu, own, 4 * g + i), t);
    };
    const int n = req.end - req.begin, rows = n * p.group;
    const float scale = p.scale_log2 * (p.factors ? p.factors[hkv] : 1.0f);
    int2 at = find(key0), next = make_int2(-1, 0);
    RawKey<D, kFour> raw[4];
    read(at, raw);
    if (kFour && key0 + kKeys < end) next = find(key0 + kKeys);
    QueryRows<D, kF16, kFour> q;
    if (rows <= 8) q.load(p, req, hkv, scale, 0, g, t);
    while (true) {
        RawKey<D, kFour> now[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = raw[i];
        const int2 here = at;
        if constexpr (kFour) {
            at = next;
            if (key0 + kKeys < end) read(at, raw);
            next = key0 + 2 * kKeys < end ? find(key0 + 2 * kKeys) : make_int2(-1, 0);
        }
        float sum[2][2] = {};
        // The query rows pass by: 16-bit rows of K all at once; 4-bit ones as they are converted, sixteen
        // at a time (all of them spilled registers).
        constexpr int kAtOnce = kFour ? 1 : 2;
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += kAtOnce) {
            uint32_t kw[2 * kAtOnce][D / 8];
#pragma unroll
            for (int i = 0; i < 2 * kAtOnce; ++i) now[2 * h0 + i].words(kw[i]);
            for (int r0 = weights_first_row(key0 + 16 * h0, req.len, n, p.group) / 8 * 8; r0 < rows; r0 += 8) {
                if (rows > 8) q.load(p, req, hkv, scale, r0, g, t);
#pragma unroll
                for (int h = 0; h < kAtOnce; ++h) q.add(kw[2 * h], kw[2 * h + 1], key0 + (h0 + h) * 16, g, sum[h0 + h]);
            }
        }
        float own = 0.0f;  // this lane's key's sum
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = sum[i / 2][i % 2];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (t == i) own = x;
        }
        if (here.x >= 0)  // (another request may share the block)
            atomicAdd(p.weights + (static_cast<int64_t>(here.x) * p.Hkv + hkv) * p.page.size + here.y, own);
        key0 += kKeys;
        if (!kFour || key0 >= end) break;
    }
}

// Block (x, y, z): runs x, x + gridDim.x, .. of `run` chunks of KV heads y, y + gridDim.y, .. of requests z,
// z + gridDim.z, ..
template <int D, bool kF16, bool kFour>
__global__ void __launch_bounds__(32, kPerSm)
weights_kernel(const WeightsParams p, int run) {
    grid_wait();
    grid_launch_next();
    const int g = threadIdx.x / 4, t = threadIdx.x % 4;
    const int keys = run * kKeys;
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const WeightsRequest r = weights_request(p, b);
        if (!r.ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        if (!r.ok || r.end == r.begin) continue;
        for (long long key0 = static_cast<long long>(blockIdx.x) * keys; key0 < r.len;
             key0 += static_cast<long long>(gridDim.x) * keys) {
            const int first = static_cast<int>(key0), end = first + min(r.len - first, keys);
            for (int hkv = blockIdx.y; hkv < p.Hkv; hkv += gridDim.y)
                weights_keys<D, kF16, kFour>(p, r, b, hkv, first, end, g, t);
        }
    }
}

template <int D, bool kFour>
cudaError_t launch_type(const WeightsParams& p, const LaunchEnv& env, bool f16, int* grid_out) {
    const long long chunks = (static_cast<long long>(p.max_pages) * p.page.size + kKeys - 1) / kKeys;
    // Of 4-bit rows even runs, long enough to read ahead in where that leaves three blocks for every two
    // places.
    long long run = 1;
    if (kFour) {
        const double per = static_cast<double>(chunks) * p.B * p.Hkv / (1.5 * kPerSm * env.num_sms);
        run = per >= kMostRun ? kMostRun : per < 1 ? 1 : static_cast<long long>(per);
        const long long runs = (chunks + run - 1) / run;
        run = (chunks + runs - 1) / runs;
    }
    // Not many more blocks than it takes, however wide the table is: one that has nothing to do costs too.
    const unsigned y = std::min(p.Hkv, 65535), z = std::min(p.B, 65535);
    // (64 requests of 4096 4-bit keys in tables eight times as wide: 78 us with 32 blocks to a place, 47 with
    // tables as wide as the requests.)
    const long long most = std::max(1ll, (kFour ? 6ll : 32ll) * kPerSm * env.num_sms / (static_cast<long long>(y) * z));
    const dim3 grid(static_cast<unsigned>(std::min((chunks + run - 1) / run, most)), y, z);
    *grid_out = static_cast<int>(grid.x);
    return f16 ? launch_serial(weights_kernel<D, true, kFour>, grid, 32, 0, env.stream, p, static_cast<int>(run))
               : launch_serial(weights_kernel<D, false, kFour>, grid, 32, 0, env.stream, p, static_cast<int>(run));
}

}  // namespace

cudaError_t launch_weights_paged(const WeightsShape& s, const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    const WeightsParams p = weights_params(s, env);
    *kernels_launched = 1;
    if (s.scales)
        return s.D == 64 ? launch_type<64, true>(p, env, s.f16, grid_out) : launch_type<128, true>(p, env, s.f16, grid_out);
    return s.D == 64 ? launch_type<64, false>(p, env, s.f16, grid_out) : launch_type<128, false>(p, env, s.f16, grid_out);
}

}  // namespace attn
