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
// a changing order.  The order of a product's inner index is free, so each lane reads runs of
// D/4 contiguous elements of its rows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "e2m1.cuh"
#include "pdl.cuh"
#include "sm100.cuh"
#include "weights.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kWarpKeys = 32;
constexpr int kBlockKeys = kWarps * kWarpKeys;

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

// A lane's D/4 elements of a K row as words of the queries' type; zeros without a row.
template <int D, bool kF16, bool kFour>
__device__ __forceinline__ void load_key(const WeightsParams& p, int64_t row, int t, uint32_t (&w)[D / 8]) {
    if (kFour) {
        const uint8_t* codes = p.cache + row * (D / 2) + t * (D / 8);
        const uint8_t* scales = p.scales + row * (D / kRowScaleSpan) + t * (D / 64);
        uint32_t c[D / 32] = {}, s = 0;
        if (row >= 0) {
            if (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(codes);
                c[0] = u.x; c[1] = u.y; c[D / 32 - 2] = u.z; c[D / 32 - 1] = u.w;
                s = *reinterpret_cast<const uint16_t*>(scales);
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(codes);
                c[0] = u.x; c[1] = u.y;
                s = *scales;
            }
        }
        s = e4m3_to_f16x2(s);
        const uint32_t by[2] = {__byte_perm(s, s, 0x1010), __byte_perm(s, s, 0x3232)};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint32_t v[4];
            e2m1_to_f16x8(c[i], v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = f16x2_mul(v[k], by[i / 2]);  // exact, in bf16 too: six significant bits
                w[4 * i + k] = kF16 ? x : pack_bf16x2(f16_lo_to_f32(x), f16_hi_to_f32(x));
            }
        }
    } else {
        const uint4* src = reinterpret_cast<const uint4*>(p.cache + (row * D + t * (D / 4)) * 2);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 u = row >= 0 ? src[i] : make_uint4(0, 0, 0, 0);
            w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
        }
    }
}

// Adds up the 32 keys from key0 on of one (request, KV head), by a warp.
template <int D, bool kF16, bool kFour>
__device__ __forceinline__ void weights_keys(const WeightsParams& p, const WeightsRequest& req, int b, int hkv, int key0,
                                             int g, int t) {
    const int len = req.len, begin = req.begin, n = req.end - req.begin;
    // Rows g, g + 8, g + 16, g + 24 of the warp's keys.
    uint32_t kw[4][D / 8];
    int64_t slot[4];  // of the weights; negative: none
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = key0 + i * 8 + g;
        slot[i] = -1;
        int64_t row = -1;
        if (key < len) {
            int in_page;
            const int id = p.block_table[static_cast<int64_t>(b) * p.max_pages + p.page.split(key, &in_page)];
            if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) {
                row = (static_cast<int64_t>(id) * 2 * p.Hkv + hkv) * p.page.size + in_page;
                slot[i] = (static_cast<int64_t>(id) * p.Hkv + hkv) * p.page.size + in_page;
            } else {
                atomicOr(p.status, ATTN_DEV_BAD_INPUT);
            }
        }
        load_key<D, kF16, kFour>(p, row, t, kw[i]);
    }
    const float by = p.scale_log2 * (p.factors ? p.factors[hkv] : 1.0f);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};

    // Query rows: token by token, a KV head's query heads within.  Token i sees keys up to
    // len - n + i.
    const int rows = n * p.group;  // checked on the host: fits
    const int first_token = max(0, key0 - (len - n));
    for (int r0 = first_token * p.group / 8 * 8; r0 < rows; r0 += 8) {
        const int mine = r0 + g;
        uint32_t qb[D / 8];
        {
            const int token = mine / p.group, head = mine - token * p.group;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (begin + token) * p.q_token +
                                                              (hkv * p.group + head) * p.q_head + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 u = mine < rows ? src[i] : make_uint4(0, 0, 0, 0);
                qb[4 * i] = u.x; qb[4 * i + 1] = u.y; qb[4 * i + 2] = u.z; qb[4 * i + 3] = u.w;
            }
        }
        float lse[2];
        int last[2];  // the last key that rows r0 + 2t, r0 + 2t + 1 see; -1: no row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = r0 + 2 * t + i, token = rr / p.group, head = rr - token * p.group;
            lse[i] = 0.0f;
            last[i] = -1;
            if (rr < rows) {
                lse[i] = p.lse[(hkv * p.group + head) * p.lse_head + (begin + token) * p.lse_token] * kWeightsLog2e;
                last[i] = lse[i] == -INFINITY ? -1 : len - n + token;
            }
        }
        float s[2][4] = {};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {kw[2 * h][2 * j], kw[2 * h + 1][2 * j], kw[2 * h][2 * j + 1], kw[2 * h + 1][2 * j + 1]};
                mma16<kF16>(s[h], a, qb[2 * j], qb[2 * j + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float w = ex2_approx(fmaf(s[i / 2][(i % 2) * 2 + k], by, -lse[k]));
                sum[i] += key0 + i * 8 + g <= last[k] ? w : 0.0f;
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        if (t == 0 && slot[i] >= 0) atomicAdd(p.weights + slot[i], sum[i]);  // another request may share the block
    }
}

// Block (x, y, z): keys x * kBlockKeys .. of KV heads y, y + gridDim.y, .. of requests z, z + gridDim.z, ..
template <int D, bool kF16, bool kFour>
__global__ void __launch_bounds__(kWarps * 32)
weights_kernel(const WeightsParams p) {
    grid_wait();
    grid_launch_next();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const WeightsRequest r = weights_request(p, b);
        if (!r.ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        const int key0 = blockIdx.x * kBlockKeys + warp * kWarpKeys;
        if (!r.ok || r.end == r.begin || key0 >= r.len) continue;
        for (int hkv = blockIdx.y; hkv < p.Hkv; hkv += gridDim.y)
            weights_keys<D, kF16, kFour>(p, r, b, hkv, key0, g, t);
    }
}

template <int D, bool kFour>
cudaError_t launch_type(const WeightsParams& p, dim3 grid, bool f16, cudaStream_t st) {
    return f16 ? launch_serial(weights_kernel<D, true, kFour>, grid, kWarps * 32, 0, st, p)
               : launch_serial(weights_kernel<D, false, kFour>, grid, kWarps * 32, 0, st, p);
}

}  // namespace

cudaError_t launch_weights_paged(const WeightsShape& s, const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    const WeightsParams p = weights_params(s, env);
    const long long keys = static_cast<long long>(s.max_pages) * s.page;
    const dim3 grid(static_cast<unsigned>((keys + kBlockKeys - 1) / kBlockKeys), std::min(s.Hkv, 65535), std::min(s.B, 65535));
    *grid_out = static_cast<int>(grid.x);
    *kernels_launched = 1;
    if (s.scales)
        return s.D == 64 ? launch_type<64, true>(p, grid, s.f16, env.stream)
                         : launch_type<128, true>(p, grid, s.f16, env.stream);
    return s.D == 64 ? launch_type<64, false>(p, grid, s.f16, env.stream)
                     : launch_type<128, false>(p, grid, s.f16, env.stream);
}

}  // namespace attn
