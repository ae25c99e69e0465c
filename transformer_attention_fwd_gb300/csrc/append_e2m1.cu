// append_e2m1.cu -- new keys and values into the paged 4-bit cache, with one e4m3 scale
// for each 16 elements of a row (attn_append_paged_e2m1).
//
// Of the 16 elements x of a group (K's after their rotation, in fp32), with the head's
// factor f:  s = max |x| / (6 f) rounded to e4m3, between 2^-9 and 448;  code = x * r
// rounded to e2m1, r = 1 / (s f).  A row depends on nothing but itself: no block's scale
// to settle and no older rows to follow, so the work is the 16-bit append's (append.cu):
// a warp takes one token and a run of its heads.  A lane holds two chunks of eight
// elements of a row, and a group's two chunks meet by shuffles.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "append.cuh"
#include "e2m1.cuh"
#include "pdl.cuh"

namespace attn {
namespace {

template <typename E, int D, int kLayout>
struct E2m1Rows {
    using R = Rope<E, D, kLayout>;
    static constexpr bool kPlain = false;
    long long row = -1;  // the slot's K row of head 0; negative: the page is left out
    int chunk[2];        // this lane's chunks of eight elements
    int lane[2], slot[2];  // where the other chunk of the group is

    __device__ __forceinline__ void begin(int j, int half) {
        chunk[0] = R::first(j, half) / 8;
        chunk[1] = R::second(j, half) / 8;
        const int base = (threadIdx.x % 32) / R::kLanes * R::kLanes, hc = half / 8;
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

    // Largest finite magnitude of a chunk, or NaN, as bits.
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
    // By the whole warp; in: this lane's row is one of the call's.  head: V's follow K's.
    __device__ __forceinline__ void store(const AppendParams& p, int head, bool in, const typename R::Pairs& v) const {
        float x[2][8];
        R::elements(v, x[0], x[1]);
        const uint32_t m[2] = {magnitude(x[0]), magnitude(x[1])};
        const long long at = row + static_cast<long long>(head) * p.page.size;
        const float factor = p.factors && in ? p.factors[head] : 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = __shfl_sync(0xffffffffu, m[0], lane[i]), b = __shfl_sync(0xffffffffu, m[1], lane[i]);
            const uint32_t most = max(m[i], slot[i] == 0 ? a : b);
            if (!in || row < 0) continue;
            const float q = fminf(fmaxf(__uint_as_float(most) / (kE2m1Max * factor), kRowScaleMin), kE4m3Max);
            const uint32_t code = most > 0x7f800000u ? 0x7fu : e4m3_pack2(q, 0.0f) & 0xffu;  // a NaN makes the scale NaN
            const float by = 1.0f / (f16_lo_to_f32(e4m3_to_f16x2(code)) * factor);
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = x[i][k] * by;
            *reinterpret_cast<uint32_t*>(p.cache + at * (D / 2) + chunk[i] * 4) = e2m1_pack8(y);
            if ((chunk[i] & 1) == 0) p.row_scales[at * (D / kRowScaleSpan) + chunk[i] / 2] = static_cast<uint8_t>(code);
        }
    }
};

template <typename E, int D, int kLayout>
__global__ void __launch_bounds__(kAppendWarps * 32, 5)
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
        e = r.D == 64 ? launch_layout<RopeF16, 64>(p, layout, g, env.stream)
                      : launch_layout<RopeF16, 128>(p, layout, g, env.stream);
    else
        e = r.D == 64 ? launch_layout<RopeBf16, 64>(p, layout, g, env.stream)
                      : launch_layout<RopeBf16, 128>(p, layout, g, env.stream);
    if (grid_out) *grid_out = static_cast<int>(g.x * g.y);
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
