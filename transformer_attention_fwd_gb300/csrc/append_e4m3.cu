// append_e4m3.cu -- new keys and values into the paged 8-bit cache, with one
// scale for each block, K or V, and head (attn_append_paged_e4m3).
//
// A block's scale is the smallest power of two s with b * max|x| <= 448 s over
// its finite elements (448: the largest e4m3 value), b = sqrt(2) * magnitude
// for rotated keys (at least 1 if part of the head passes through), else 1.  A
// rotation raises no component above sqrt(2) times the pair's larger one, so the
// scale needs the elements before the rotation
// only: it is an exact comparison of input values, the same whatever the
// rounding of the rotation.  A power of two costs e4m3 no precision (only the
// subnormal end moves), and the rows a partly filled block holds follow a
// scale that grows by an exact division.
//
// Work: an item is one page of one request, in which the call's new tokens fill
// some rows.  A CTA takes one item and eight of its 2 * Hkv tasks (K or V, head), a
// warp each: it loads up to 16 rows, takes their largest magnitude from the raw
// bits, fixes the scale, rotates K from registers with the sines and cosines the
// CTA shares, rounds and stores.  Longer pages run in groups of 16 rows and read
// their rows a second time (out of L2).  Query rows are taken by further CTAs of
// the same launch, as in append.cu.
//
// 17100 tokens of 9 requests, 32 query and 8 KV heads, D 128 (385 MB, 280 of them
// the queries): 64 us, 6.0 TB/s.  K and V of a head in one warp (128 registers, 16
// warps per SM, for the query rows too) took 73 us.  At 80 registers, for three CTAs
// per SM, eight of the twelve instances spill 8 to 36 bytes.  One token for each of 64
// requests: 4.5 us, a chain of dependent reads (offsets, length, block id, scale).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "append.cuh"
#include "e4m3.cuh"
#include "pdl.cuh"

namespace attn {
namespace {

constexpr int kPageWarps = 8;
constexpr int kGroup = 16;  // rows in registers at a time

// The smallest power of two s >= 2^-100 with amax <= limit * s.
__device__ __forceinline__ float block_scale(float amax, float limit) {
    const float q = amax / limit;
    float s = fmaxf(__uint_as_float(__float_as_uint(q) & 0x7f800000u), kE4m3MinScale);
    while (amax > limit * s) s *= 2.0f;  // at most twice: the quotient was rounded down
    return s > kE4m3MinScale && amax <= limit * (0.5f * s) ? 0.5f * s : s;
}

// Largest finite magnitude of the two 16-bit elements of each word.
template <typename E>
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w) {
    constexpr uint32_t kInf = E::kInfinity;
    const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    return max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u);
}

struct BlockBf16 : RopeBf16 {
    static constexpr uint32_t kInfinity = 0x7f80u;
};
struct BlockF16 : RopeF16 {
    static constexpr uint32_t kInfinity = 0x7c00u;
};

// The rows of one (page, K or V, head) as a warp holds them.
template <typename E, int D, int kLayout>
struct PageRows {
    using R = Rope<E, D, kLayout>;
    static constexpr int kSteps = kGroup / R::kRows;
    typename R::Raw raw[kSteps];

    // Rows 16 g .. of `rows` at x (the warp's token 0 and head), zeros beyond.
    __device__ __forceinline__ void load(const uint8_t* x, long long row_bytes, int g, int rows, int grp,
                                         int at0, int at1) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = g * kGroup + i * R::kRows + grp;
            const uint8_t* at = x + r * row_bytes;
            raw[i] = r < rows ? R::load(at + at0, at + at1) : R::zero();
        }
    }
    // Largest magnitude's bits, both halves of a word apart; infinities and NaN count.
    __device__ __forceinline__ uint32_t magnitude() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            m = __vmaxu2(__vmaxu2(m, raw[i].c0.x & 0x7fff7fffu), raw[i].c1.x & 0x7fff7fffu);
            m = __vmaxu2(__vmaxu2(m, raw[i].c0.y & 0x7fff7fffu), raw[i].c1.y & 0x7fff7fffu);
            m = __vmaxu2(__vmaxu2(m, raw[i].c0.z & 0x7fff7fffu), raw[i].c1.z & 0x7fff7fffu);
            m = __vmaxu2(__vmaxu2(m, raw[i].c0.w & 0x7fff7fffu), raw[i].c1.w & 0x7fff7fffu);
        }
        return m;
    }
    __device__ __forceinline__ uint32_t finite() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            m = max(m, max(finite_magnitude<E>(raw[i].c0.x), finite_magnitude<E>(raw[i].c1.x)));
            m = max(m, max(finite_magnitude<E>(raw[i].c0.y), finite_magnitude<E>(raw[i].c1.y)));
            m = max(m, max(finite_magnitude<E>(raw[i].c0.z), finite_magnitude<E>(raw[i].c1.z)));
            m = max(m, max(finite_magnitude<E>(raw[i].c0.w), finite_magnitude<E>(raw[i].c1.w)));
        }
        return m;
    }
};

// The block's scale for new rows of magnitude amax; the `held` rows it has
// already follow a scale that grows.
template <int D>
__device__ __forceinline__ float settle_scale(float amax, float limit, int held, float* scale_at, uint8_t* block,
                                              int lane) {
    float scale = block_scale(amax, limit);
    if (held > 0) {
        const float old = *scale_at;
        if (scale > old) {
            const float ratio = old / scale;
            for (long long c = lane; c < held * (D / 16ll); c += 32) {
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
    return scale;
}

template <typename R>
__device__ __forceinline__ void store_codes(uint8_t* row, int e0, int e1, typename R::Pairs& v, float inv) {
    R::scale(v, inv);
    float x[8], y[8];
    R::elements(v, x, y);
    *reinterpret_cast<uint2*>(row + e0) =
        make_uint2(e4m3_pack4(x[0], x[1], x[2], x[3]), e4m3_pack4(x[4], x[5], x[6], x[7]));
    *reinterpret_cast<uint2*>(row + e1) =
        make_uint2(e4m3_pack4(y[0], y[1], y[2], y[3]), e4m3_pack4(y[4], y[5], y[6], y[7]));
}

template <typename E, int D, int kLayout>
__global__ void __launch_bounds__(kPageWarps * 32, 3)
append_e4m3_kernel(const AppendParams p) {
    using R = Rope<E, D, kLayout>;
    using Rows = PageRows<E, D, kLayout>;
    __shared__ __align__(16) float s_table[kGroup][D];  // a row's cosines and sines
    __shared__ float s_scratch[R::kScratch ? kPageWarps * R::kScratch : 1];
    static_assert(kGroup >= kPageWarps, "query CTAs take a table row for each warp");
    grid_wait();
    grid_launch_next();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float* scratch = s_scratch + (R::kScratch ? warp * R::kScratch : 0);
    const unsigned kv_blocks = p.items * p.splits;
    if (blockIdx.x >= kv_blocks) {
        const unsigned qb = blockIdx.x - kv_blocks;
        if (qb >= p.q_blocks) {
            append_report(p, qb - p.q_blocks);
            return;
        }
        append_rows<E, D, kLayout>(p, static_cast<int>(qb / p.segs) * kPageWarps + warp, static_cast<int>(qb % p.segs),
                                   s_table[warp], scratch);
        return;
    }
    const int j = lane % R::kLanes, grp = lane / R::kLanes;
    if (R::kScratch) scratch += grp * D;
    const int half = p.table.half;
    const unsigned on = R::turning(half, j);

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
    const int first_task = static_cast<int>(blockIdx.x % p.splits) * kPageWarps, task = first_task + warp;
    const bool active = task < 2 * Hkv, is_v = task >= Hkv, cta_turns = first_task < Hkv && half > 0;
    const int head = is_v ? task - Hkv : task;
    const RopeRows& src = is_v ? p.v : p.k;
    const int at0 = R::first(j, half), at1 = R::second(j, half);  // elements
    const uint8_t* x = static_cast<const uint8_t*>(src.x) + (token0 * src.x_token + head * src.x_head) * E::kBytes;
    const long long row_bytes = src.x_token * E::kBytes;
    const int mine = active ? rows : 0;  // rows this warp loads
    Rows r;
    r.load(x, row_bytes, 0, mine, grp, at0 * E::kBytes, at1 * E::kBytes);
    const int id = append_block(p, b, p.page.quotient(static_cast<int>(page0)));
    const bool write = active && id >= 0;

    uint32_t most = r.magnitude();
    for (int g = 1; g < groups; ++g) {
        r.load(x, row_bytes, g, mine, grp, at0 * E::kBytes, at1 * E::kBytes);
        most = __vmaxu2(most, r.magnitude());
    }
    most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
    if (most >= E::kInfinity) {  // infinities or NaN among them: the finite ones alone
        most = 0;
        for (int g = 0; g < groups; ++g) {
            if (groups > 1) r.load(x, row_bytes, g, mine, grp, at0 * E::kBytes, at1 * E::kBytes);
            most = max(most, r.finite());
        }
        most = __reduce_max_sync(0xffffffffu, most);
    }
    const int64_t slot = (static_cast<int64_t>(id) * 2 + (is_v ? 1 : 0)) * Hkv + head;
    uint8_t* block = p.cache + slot * p.page.size * D;
    float inv = 0.0f;
    if (write)
        inv = 1.0f / settle_scale<D>(E::lo(most), is_v ? kE4m3Max : p.k_limit, r0, p.scales + slot, block, lane);

    // From the last group, which is in registers, to the first.
    for (int g = groups - 1; g >= 0; --g) {
        const int here = min(kGroup, rows - g * kGroup);
        if (cta_turns) {
            if (g != groups - 1) __syncthreads();  // the table of the group before has been read
            for (int i = threadIdx.x; i < here * (D / 2); i += kPageWarps * 32) {
                const int rr = i / (D / 2), token = token0 + g * kGroup + rr;
                rope_entry<D>(p.table, i % (D / 2), p.positions ? p.positions[token] : start + (token - rq.begin),
                              s_table[rr]);
            }
            __syncthreads();
        }
        if (!active) continue;
        if (g != groups - 1) r.load(x, row_bytes, g, mine, grp, at0 * E::kBytes, at1 * E::kBytes);
#pragma unroll
        for (int i = 0; i < Rows::kSteps; ++i) {
            if (i * R::kRows >= here) break;  // the same for the whole warp
            const int in_group = i * R::kRows + grp, rr = g * kGroup + in_group;
            typename R::Pairs v = R::unpack(r.raw[i]);
            if (!is_v && cta_turns) {
                typename R::Coef coef;
                R::coefficients(s_table[in_group], j, coef);
                R::turn(v, coef, on, half, j, s_table[in_group], scratch);
            }
            if (rr >= rows) continue;
            if (!is_v && p.k.y != nullptr) {
                uint8_t* y = static_cast<uint8_t*>(p.k.y) +
                             ((token0 + rr) * p.k.y_token + head * p.k.y_head) * E::kBytes;
                if (cta_turns) R::store(y + at0 * E::kBytes, y + at1 * E::kBytes, v);
                else R::store(y + at0 * E::kBytes, y + at1 * E::kBytes, r.raw[i]);
            }
            if (write) store_codes<R>(block + static_cast<int64_t>(r0 + rr) * D, at0, at1, v, inv);
        }
    }
}

template <typename E, int D>
cudaError_t launch_layout(const AppendParams& p, int layout, unsigned blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent:
            return launch_serial(append_e4m3_kernel<E, D, kRopeAdjacent>, blocks, kPageWarps * 32, 0, st, p);
        case kRopeHalves:
            return launch_serial(append_e4m3_kernel<E, D, kRopeHalves>, blocks, kPageWarps * 32, 0, st, p);
        default:
            return launch_serial(append_e4m3_kernel<E, D, kRopeHalvesOdd>, blocks, kPageWarps * 32, 0, st, p);
    }
}

}  // namespace

cudaError_t launch_append_paged_e4m3(const AppendShape& s, const RopeShape& r, const RopeRows* q,
                                     const RopeRows& k, const RopeRows& v, const LaunchEnv& env,
                                     int* grid_out, int* kernels_launched) {
    AppendParams p = append_params(s, r, q, k, v, env);
    // What a rotation may raise a key's element by; elements that pass through stay.
    const double raise = r.rot_dim > 0 ? 1.4142135623730951 * static_cast<double>(r.magnitude) : 1.0;
    p.k_limit = static_cast<float>(448.0 / (r.rot_dim < r.D ? std::max(raise, 1.0) : raise));
    // Request b's pages are items cu[b] / page + 2 b and on: it touches at most
    // n / page + 2 of them, so the ranges do not meet.
    p.splits = static_cast<unsigned>((2 * k.heads + kPageWarps - 1) / kPageWarps);
    const long long items = s.total / s.page + 2ll * s.B;
    // The query heads' steps as in append.cu.
    const int step_rows = 32 * 16 / r.D;
    p.q_steps = p.steps = (p.q.heads + step_rows - 1) / step_rows;
    p.segs = p.steps > 0 ? append_segments(p, env.num_sms) : 0;
    const long long q_blocks = static_cast<long long>((s.total + kPageWarps - 1) / kPageWarps) * p.segs;
    const long long blocks = items * p.splits + q_blocks + (s.B + kPageWarps * 32 - 1) / (kPageWarps * 32);
    p.q_blocks = static_cast<unsigned>(q_blocks);
    if (items > 0x7fffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.items = static_cast<unsigned>(items);
    const unsigned g = static_cast<unsigned>(blocks);
    const int layout = rope_layout(r.rot_dim, r.interleaved, 2);
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
