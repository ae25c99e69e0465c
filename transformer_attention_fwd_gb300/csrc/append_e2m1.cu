// append_e2m1.cu -- new keys and values into the paged 4-bit cache, with one e4m3 scale
// for each 16 elements of a row (attn_append_paged_e2m1).
//
// Of the 16 elements x of a group (K's after their rotation, in fp32), with the head's
// factor f:  s = max |x| / (6 f) rounded to e4m3, between 2^-9 and 448;  code = x * r
// rounded to e2m1, r = 1 / (s f).  A row depends on nothing but itself: no block's scale
// to settle and no older rows to follow, so the work is the 16-bit append's (append.cu):
// a warp takes one token and a run of its heads.  A lane holds two chunks of eight
// elements of a row, and a group's two chunks meet by shuffles; each of its two lanes settles one of the
// two groups they share.  17100 tokens of 8 KV heads (D 128) take 24 to 27 us (floor by bytes
// 13): 18 M instructions, the groups' exchanges between lanes among them, in 60% of the issue slots,
// which is no limit; the rest waits, mostly for memory, at a third of the warps an SM can hold.
// A step of 64 tokens takes 3.1, a chain of reads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "append.cuh"
#include "e2m1.cuh"
#include "pdl.cuh"

namespace attn {
namespace {

struct RowBf16 : RopeBf16 {
    static constexpr uint32_t kInfinity = 0x7f80u;
};
struct RowF16 : RopeF16 {
    static constexpr uint32_t kInfinity = 0x7c00u;
};

template <typename E, int D, int kLayout>
struct E2m1Rows {
    using R = Rope<E, D, kLayout>;
    static constexpr bool kPlain = false;
    long long row = -1;  // the slot's K row of head 0; negative: the page is left out
    int chunk[2];        // this lane's chunks of eight elements
    int lane[2], slot[2];  // where the other chunk of the group is
    bool next;             // in the next lane, at the same place, for all chunks of the warp

    __device__ __forceinline__ void begin(int j, int half) {
        chunk[0] = R::first(j, half) / 8;
        chunk[1] = R::second(j, half) / 8;
        const int base = (threadIdx.x % 32) / R::kLanes * R::kLanes, hc = half / 8;
        next = kLayout != kRopeHalves || hc == R::kLanes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = chunk[i] ^ 1;
            int l, at;
            if (kLayout != kRopeHalves) {
                l = c % R::kLanes;
                at = c / R::kLanes;
            } else if (c < 2 * hc) {
                l = c < hc ? c : c - hc;
                at = c < hc ? 0 : 1;
            } else {
                l = hc + (c - 2 * hc) / 2;
                at = c & 1;
            }
            lane[i] = base + l;
            slot[i] = at;
        }
    }
    __device__ __forceinline__ void place(const AppendParams& p, int id, int in_page) {
        row = id < 0 ? -1 : static_cast<long long>(id) * 2 * p.k.heads * p.page.size + in_page;
    }

    // Largest finite magnitude of a chunk, or NaN, as fp32 bits: of fp32 values, and of 16-bit
    // ones as they were read (two at a time: their bits are in the order of their magnitudes).
    static __device__ __forceinline__ uint32_t magnitude(const float (&x)[8]) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        if (m != 0x7f800000u) return m;
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
            m = max(m, a < 0x7f800000u ? a : 0u);
        }
        return m;
    }
    static __device__ __forceinline__ uint32_t magnitude(const uint4& c) {
        const uint32_t w[4] = {c.x & 0x7fff7fffu, c.y & 0x7fff7fffu, c.z & 0x7fff7fffu, c.w & 0x7fff7fffu};
        const uint32_t two = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
        uint32_t m = max(two & 0xffffu, two >> 16);
        if (m == E::kInfinity) {
            m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
                m = max(m, max(lo < E::kInfinity ? lo : 0u, hi < E::kInfinity ? hi : 0u));
            }
        }
        return __float_as_uint(E::lo(m));
    }
    // The scale of a group by its magnitude, and what its elements are multiplied by.  The quotient's
    // rounding matters only next to a border of e4m3's: elsewhere a product with the reciprocal,
    // off by at most 2^-22, has the same code on both sides.
    static __device__ __forceinline__ uint32_t scale(uint32_t most, float factor, float over, float& by) {
        const float m = __uint_as_float(most), near = m * over;
        const uint32_t both = e4m3_pack2(fminf(fmaxf(near * (1.0f - 0x1p-21f), kRowScaleMin), kE4m3Max),
                                         fminf(fmaxf(near * (1.0f + 0x1p-21f), kRowScaleMin), kE4m3Max));
        uint32_t code = both & 0xffu;
        if (code != both >> 8) code = e4m3_pack2(fminf(fmaxf(m / (kE2m1Max * factor), kRowScaleMin), kE4m3Max), 0.0f) & 0xffu;
        if (most > 0x7f800000u) code = 0x7fu;  // a NaN makes the scale NaN
        by = 1.0f / (f16_lo_to_f32(e4m3_to_f16x2(code)) * factor);
        return code;
    }
    // By the whole warp; in: this lane's row is one of the call's.  head: V's follow K's.
    __device__ __forceinline__ void store(const AppendParams& p, int head, bool in, const typename R::Raw& v) const {
        store(p, head, in, R::unpack(v), magnitude(v.c0), magnitude(v.c1));
    }
    __device__ __forceinline__ void store(const AppendParams& p, int head, bool in, const typename R::Pairs& v) const {
        float x[8], y[8];
        R::elements(v, x, y);
        store(p, head, in, v, magnitude(x), magnitude(y));
    }

  private:
    __device__ __forceinline__ void store(const AppendParams& p, int head, bool in, typename R::Pairs v, uint32_t m0,
                                          uint32_t m1) const {
        const float factor = p.factors && in ? p.factors[head] : 1.0f;
        float over;  // off by up to 2^-23
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(over) : "f"(kE2m1Max * factor));
        uint32_t code[2];
        float by[2];
        if (next) {  // both groups are shared with the next lane: a lane settles one of them
            m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
            const bool odd = threadIdx.x & 1;
            float own_by;
            const uint32_t own = scale(odd ? m1 : m0, factor, over, own_by);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
            const float other_by = __shfl_xor_sync(0xffffffffu, own_by, 1);
            code[0] = odd ? other : own;
            code[1] = odd ? own : other;
            by[0] = odd ? other_by : own_by;
            by[1] = odd ? own_by : other_by;
        } else {
            const uint32_t m[2] = {m0, m1};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t a = __shfl_sync(0xffffffffu, m0, lane[i]), b = __shfl_sync(0xffffffffu, m1, lane[i]);
                code[i] = scale(max(m[i], slot[i] == 0 ? a : b), factor, over, by[i]);
            }
        }
        if (!in || row < 0) return;
        const uint64_t by0 = f2_pack(by[0], by[0]), by1 = f2_pack(by[1], by[1]);
#pragma unroll
        for (int k = 0; k < R::kP2; ++k) {  // adjacent pairs: both chunks in a and b; else one in each
            const bool second = kLayout == kRopeAdjacent && k >= R::kP2 / 2;
            v.a[k] = f2_mul(v.a[k], second ? by1 : by0);
            v.b[k] = f2_mul(v.b[k], kLayout == kRopeAdjacent ? (second ? by1 : by0) : by1);
        }
        float x[8], y[8];
        R::elements(v, x, y);
        const long long at = row + static_cast<long long>(head) * p.page.size;
        uint8_t* codes = p.cache + at * (D / 2);
        *reinterpret_cast<uint32_t*>(codes + chunk[0] * 4) = e2m1_pack8(x);
        *reinterpret_cast<uint32_t*>(codes + chunk[1] * 4) = e2m1_pack8(y);
        uint8_t* scales = p.row_scales + at * (D / kRowScaleSpan);
        if ((chunk[0] & 1) == 0) scales[chunk[0] / 2] = static_cast<uint8_t>(code[0]);
        if ((chunk[1] & 1) == 0) scales[chunk[1] / 2] = static_cast<uint8_t>(code[1]);
    }
};

// Blocks to an SM by registers: six (17100 tokens of 8 KV heads as they are 23.6 us, with five 24.0; adjacent
// pairs 28.2 and 28.7), but for halves, which spill at six (30.7 and 30.1).
template <typename E, int D, int kLayout>
__global__ void __launch_bounds__(kAppendWarps * 32, kLayout == kRopeHalves ? 5 : 6)
append_e2m1_kernel(const AppendParams p) {
    using R = Rope<E, D, kLayout>;
    __shared__ __align__(16) float s_table[kAppendWarps][D];
    __shared__ float s_scratch[R::kScratch ? kAppendWarps * R::kScratch : 1];
    grid_wait();
    grid_launch_next();
    if (blockIdx.x >= p.token_blocks) {
        if (blockIdx.y == 0) append_report(p, blockIdx.x - p.token_blocks);
        return;
    }
    const int warp = threadIdx.x / 32;
    append_rows<E, D, kLayout, E2m1Rows<E, D, kLayout>>(p, static_cast<int>(blockIdx.x) * kAppendWarps + warp,
                                                        blockIdx.y, s_table[warp], s_scratch + warp * R::kScratch);
}

template <typename E, int D>
cudaError_t launch_layout(const AppendParams& p, int layout, dim3 blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent: return launch_serial(append_e2m1_kernel<E, D, kRopeAdjacent>, blocks, kAppendWarps * 32, 0, st, p);
        case kRopeHalves: return launch_serial(append_e2m1_kernel<E, D, kRopeHalves>, blocks, kAppendWarps * 32, 0, st, p);
        default: return launch_serial(append_e2m1_kernel<E, D, kRopeHalvesOdd>, blocks, kAppendWarps * 32, 0, st, p);
    }
}

}  // namespace

cudaError_t launch_append_paged_e2m1(const AppendShape& s, const RopeShape& r, const RopeRows* q,
                                     const RopeRows& k, const RopeRows& v, const LaunchEnv& env,
                                     int* grid_out, int* kernels_launched) {
    AppendParams p = append_params(s, r, q, k, v, env);
    const int rows = 32 * 16 / r.D;  // Rope<...>::kRows of 16-bit elements
    p.q_steps = (p.q.heads + rows - 1) / rows;
    p.kv_steps = (k.heads + rows - 1) / rows;
    p.steps = p.q_steps + 2 * p.kv_steps;
    const int segs = append_segments(p, env.num_sms);
    if (segs > 65535) return cudaErrorInvalidConfiguration;
    p.token_blocks = static_cast<unsigned>((s.total + kAppendWarps - 1) / kAppendWarps);
    const dim3 g(p.token_blocks + (s.B + kAppendWarps * 32 - 1) / (kAppendWarps * 32), segs);
    const int layout = rope_layout(r.rot_dim, r.interleaved, 2);
    cudaError_t e;
    if (r.dtype == ATTN_F16)
        e = r.D == 64 ? launch_layout<RowF16, 64>(p, layout, g, env.stream)
                      : launch_layout<RowF16, 128>(p, layout, g, env.stream);
    else
        e = r.D == 64 ? launch_layout<RowBf16, 64>(p, layout, g, env.stream)
                      : launch_layout<RowBf16, 128>(p, layout, g, env.stream);
    if (grid_out) *grid_out = static_cast<int>(g.x * g.y);
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
