// append_e4m3.cu -- new keys and values into the paged 8-bit cache, with one
// scale for each block, K or V, and head (attn_append_paged_e4m3).
//
// A block's scale is the smallest power of two s with b * max|x| <= 448 s over
// its finite elements (448: the largest e4m3 value), b = sqrt(2) * magnitude
// for rotated keys, else 1.  A rotation raises no component above sqrt(2) times
// the pair's larger one, so the scale needs the elements before the rotation
// only: it is an exact comparison of input values, the same whatever the
// rounding of the rotation.  A power of two costs e4m3 no precision (only the
// subnormal end moves), and the rows a partly filled block holds follow a
// scale that grows by an exact division.
//
// Work: an item is one page of one request, in which the call's new tokens fill
// some rows.  A CTA takes one item and eight of its 2 * Hkv (K or V, head)
// tasks, a warp each: it loads up to 16 rows, takes their largest magnitude
// from the raw bits, fixes the scale, rotates from registers with the sines and
// cosines the CTA shares, rounds and stores.  Longer pages run in groups of 16
// rows and read their rows a second time (out of L2).  Query rows are taken by
// further CTAs of the same launch, as in append.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "append.cuh"
#include "e4m3.cuh"

namespace attn {
namespace {

constexpr int kGroup = 16;  // rows in registers at a time

// The smallest power of two s >= 2^-100 with amax <= limit * s.
__device__ __forceinline__ float block_scale(float amax, float limit) {
    const float q = amax / limit;
    float s = fmaxf(__uint_as_float(__float_as_uint(q) & 0x7f800000u), kE4m3MinScale);
    while (amax > limit * s) s *= 2.0f;  // at most twice: the quotient was rounded down
    return s > kE4m3MinScale && amax <= limit * (0.5f * s) ? 0.5f * s : s;
}

// Largest finite magnitude of the two 16-bit elements of each word.
template <typename Row>
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w) {
    constexpr uint32_t kInf = Row::kInfinity;
    const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    return max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u);
}

struct BlockBf16 : RopeBf16 {
    static constexpr uint32_t kInfinity = 0x7f80u;
    static __device__ __forceinline__ float value(uint32_t bits) { return bf16_lo_to_f32(bits); }
};
struct BlockF16 : RopeF16 {
    static constexpr uint32_t kInfinity = 0x7c00u;
    static __device__ __forceinline__ float value(uint32_t bits) { return f16_lo_to_f32(bits); }
};

template <typename Row, int D, int kLayout>
__global__ void __launch_bounds__(kAppendWarps * 32)
append_e4m3_kernel(const AppendParams p) {
    constexpr int kLanes = D / kRopeChunk, kRowsPerStep = 32 / kLanes;
    constexpr int kSteps = kGroup / kRowsPerStep;
    __shared__ float s_row[kLayout == kRopeHalvesOdd ? kAppendWarps * kRowsPerStep * D : 1];
    __shared__ float2 s_cs[kGroup][D / 2];  // cos, sin of a row's pairs
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int sub = lane % kLanes, grp = lane / kLanes;
    float* row = s_row + (kLayout == kRopeHalvesOdd ? (warp * kRowsPerStep + grp) * D : 0);
    const unsigned kv_blocks = p.items * p.splits;
    if (blockIdx.x == gridDim.x - 1) append_report(p);

    if (blockIdx.x >= kv_blocks) {  // query rows
        const long long w = static_cast<long long>(blockIdx.x - kv_blocks) * kAppendWarps + warp;
        if (w >= p.warps) return;
        const int token = static_cast<int>(w / p.q_segs);
        const int seg = static_cast<int>(w - static_cast<long long>(token) * p.q_segs);
        int b, slot;
        if (!append_slot(p, token, lane, &b, &slot)) return;
        RopeCoef coef;
        rope_coefficients<Row, kLayout>(p.table, sub * kRopeChunk,
                                        p.positions ? p.positions[token] : slot, nullptr, coef);
        const uint8_t* x = static_cast<const uint8_t*>(p.q.x) +
                           (token * p.q.x_token + sub * kRopeChunk) * Row::kBytes;
        uint8_t* y = static_cast<uint8_t*>(p.q.y) +
                     (token * p.q.y_token + sub * kRopeChunk) * Row::kBytes;
        const int h0 = seg * p.steps * kRowsPerStep;
        const int h1 = min(p.q.heads, h0 + p.steps * kRowsPerStep);
        for (int h = h0; h < h1; h += kRowsPerStep) {
            const int head = h + grp;
            const typename Row::Raw raw =
                head < h1 ? Row::load(x + head * p.q.x_head * Row::kBytes) : Row::zero();
            float v[8], vp[8];
            Row::unpack(raw, v);
            rope_exchange<Row, kLayout, D>(raw, v, p.table.half, lane, row, vp);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], coef.own[e], vp[e] * coef.other[e]);
            if (head < h1) Row::store(y + head * p.q.y_head * Row::kBytes, v);
        }
        return;
    }

    // The item's request, page and rows: the same in every warp.
    const int item = static_cast<int>(blockIdx.x / p.splits);
    const int b = warp_last_at_most(p.B, item, lane, [&](int i) {
        return static_cast<long long>(p.page.quotient(max(0, p.cu[i]))) + 2ll * i;
    });
    const AppendRequest rq = append_request(p, b);
    if (!rq.ok || rq.begin == rq.end) return;
    const int start = rq.len - (rq.end - rq.begin);  // first new slot
    const int base = p.page.quotient(rq.begin) + 2 * b;
    if (item < base) return;
    const long long page0 = static_cast<long long>(p.page.quotient(start) + (item - base)) * p.page.size;
    if (page0 >= rq.len) return;
    const int r0 = static_cast<int>(max(0ll, start - page0));
    const int r1 = static_cast<int>(min(static_cast<long long>(p.page.size), rq.len - page0));
    const int rows = r1 - r0;
    const int token0 = rq.begin + static_cast<int>(page0 + r0 - start);
    const int groups = (rows + kGroup - 1) / kGroup;

    const int Hkv = p.k.heads;
    const int first_task = static_cast<int>(blockIdx.x % p.splits) * kAppendWarps;
    const int task = first_task + warp;
    const bool active = task < 2 * Hkv, is_v = task >= Hkv, cta_has_k = first_task < Hkv;
    const int head = is_v ? task - Hkv : task;
    const RopeRows& src = is_v ? p.v : p.k;
    const uint8_t* x = static_cast<const uint8_t*>(src.x) +
                       (token0 * src.x_token + head * src.x_head + sub * kRopeChunk) * Row::kBytes;
    const int id = append_block(p, b, p.page.quotient(static_cast<int>(page0)));

    typename Row::Raw raw[kSteps];
    auto load = [&](int g) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int rr = g * kGroup + i * kRowsPerStep + grp;
            raw[i] = active && rr < rows ? Row::load(x + rr * src.x_token * Row::kBytes) : Row::zero();
        }
    };
    load(0);
    uint32_t packed = 0;
    for (int g = 0;;) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            packed = __vmaxu2(packed, raw[i].x & 0x7fff7fffu);
            packed = __vmaxu2(packed, raw[i].y & 0x7fff7fffu);
            packed = __vmaxu2(packed, raw[i].z & 0x7fff7fffu);
            packed = __vmaxu2(packed, raw[i].w & 0x7fff7fffu);
        }
        if (++g == groups) break;
        load(g);
    }
    uint32_t most = __reduce_max_sync(0xffffffffu, max(packed & 0xffffu, packed >> 16));
    if (most >= Row::kInfinity) {  // infinities or NaN among them: the finite ones alone
        most = 0;
        for (int g = 0; g < groups; ++g) {
            if (groups > 1) load(g);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                most = max(most, max(finite_magnitude<Row>(raw[i].x), finite_magnitude<Row>(raw[i].y)));
                most = max(most, max(finite_magnitude<Row>(raw[i].z), finite_magnitude<Row>(raw[i].w)));
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
    }
    const bool write = active && id >= 0;
    float scale = block_scale(Row::value(most), is_v ? kE4m3Max : p.k_limit);
    uint8_t* block = p.cache + ((static_cast<int64_t>(id) * 2 + (is_v ? 1 : 0)) * Hkv + head) * p.page.size * D;
    if (write) {
        float* scale_at = p.scales + (static_cast<int64_t>(id) * 2 + (is_v ? 1 : 0)) * Hkv + head;
        if (r0 > 0) {
            const float old = *scale_at;
            if (scale > old) {  // the older rows follow
                const float ratio = old / scale;
                for (int c = lane; c < r0 * (D / 16); c += 32) {
                    uint4* at = reinterpret_cast<uint4*>(block) + c;
                    uint4 w = *at;
                    w.x = e4m3_rescale(w.x, ratio);
                    w.y = e4m3_rescale(w.y, ratio);
                    w.z = e4m3_rescale(w.z, ratio);
                    w.w = e4m3_rescale(w.w, ratio);
                    *at = w;
                }
            }
            scale = fmaxf(scale, old);
        }
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *scale_at = scale;
    }
    const float inv = 1.0f / scale;

    // From the last group, which is in registers, to the first.
    for (int g = groups - 1; g >= 0; --g) {
        if (cta_has_k && p.table.half > 0) {
            __syncthreads();
            const int here = min(kGroup, rows - g * kGroup);
            for (int i = threadIdx.x; i < here * p.table.half; i += kAppendWarps * 32) {
                const int rr = i / p.table.half, pair = i - rr * p.table.half;
                const int at = g * kGroup + rr;
                float s, c;
                rope_sincos(p.table, pair, p.positions ? p.positions[token0 + at] : start + (token0 - rq.begin) + at,
                            &s, &c);
                s_cs[rr][pair] = make_float2(c * p.table.magnitude, s * p.table.magnitude);
            }
            __syncthreads();
        }
        if (!active) continue;
        if (g != groups - 1) load(g);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int in_group = i * kRowsPerStep + grp, rr = g * kGroup + in_group;
            if (g * kGroup + i * kRowsPerStep >= rows) break;  // the same for the whole warp
            float v[8];
            Row::unpack(raw[i], v);
            if (!is_v) {
                float vp[8];
                rope_exchange<Row, kLayout, D>(raw[i], v, p.table.half, lane, row, vp);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    bool first = true;
                    const int pair = rope_pair<kLayout>(sub * kRopeChunk + e, p.table.half, &first);
                    if (pair < 0) continue;
                    const float2 cs = s_cs[in_group][pair];
                    v[e] = fmaf(v[e], cs.x, vp[e] * (first ? -cs.y : cs.y));
                }
                if (rr < rows && p.k.y != nullptr)
                    Row::store(static_cast<uint8_t*>(p.k.y) +
                                   ((token0 + rr) * p.k.y_token + head * p.k.y_head + sub * kRopeChunk) * Row::kBytes,
                               v);
            }
            if (rr < rows && write) {
                uint2 out;
                out.x = e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                out.y = e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
                *reinterpret_cast<uint2*>(block + static_cast<int64_t>(r0 + rr) * D + sub * kRopeChunk) = out;
            }
        }
    }
}

template <typename Row, int D>
cudaError_t launch_layout(const AppendParams& p, int layout, unsigned blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent:
            append_e4m3_kernel<Row, D, kRopeAdjacent><<<blocks, kAppendWarps * 32, 0, st>>>(p);
            break;
        case kRopeHalves:
            append_e4m3_kernel<Row, D, kRopeHalves><<<blocks, kAppendWarps * 32, 0, st>>>(p);
            break;
        default:
            append_e4m3_kernel<Row, D, kRopeHalvesOdd><<<blocks, kAppendWarps * 32, 0, st>>>(p);
            break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_paged_e4m3(const AppendShape& s, const RopeShape& r, const RopeRows* q,
                                     const RopeRows& k, const RopeRows& v, const LaunchEnv& env,
                                     int* grid_out, int* kernels_launched) {
    AppendParams p = append_params(s, r, q, k, v, env);
    p.k_limit = r.rot_dim > 0
                    ? static_cast<float>(448.0 / (1.4142135623730951 * static_cast<double>(r.magnitude)))
                    : kE4m3Max;
    // Request b's pages are items cu[b] / page + 2 b and on: it touches at most
    // n / page + 2 of them, so the ranges do not meet.
    p.splits = static_cast<unsigned>((2 * k.heads + kAppendWarps - 1) / kAppendWarps);
    const long long items = s.total / s.page + 2ll * s.B;
    const int rows = 32 / (r.D / kRopeChunk);
    const int q_steps = (p.q.heads + rows - 1) / rows;
    const long long per = static_cast<long long>(s.total) * q_steps / (static_cast<long long>(env.num_sms) * 32);
    p.steps = static_cast<int>(std::max<long long>(1, std::min<long long>(per, q_steps)));
    p.q_segs = (q_steps + p.steps - 1) / p.steps;
    p.warps = static_cast<long long>(s.total) * p.q_segs;
    const long long blocks = items * p.splits + (p.warps + kAppendWarps - 1) / kAppendWarps;
    if (items > 0x7fffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.items = static_cast<unsigned>(items);
    const unsigned g = static_cast<unsigned>(blocks);
    const int layout = rope_layout(r.rot_dim, r.interleaved);
    cudaError_t e;
    if (r.dtype == ATTN_F16)
        e = r.D == 64 ? launch_layout<BlockF16, 64>(p, layout, g, env.stream)
                      : launch_layout<BlockF16, 128>(p, layout, g, env.stream);
    else
        e = r.D == 64 ? launch_layout<BlockBf16, 64>(p, layout, g, env.stream)
                      : launch_layout<BlockBf16, 128>(p, layout, g, env.stream);
    if (grid_out) *grid_out = static_cast<int>(g);
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
