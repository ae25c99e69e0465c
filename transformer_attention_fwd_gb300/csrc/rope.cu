// rope.cu -- rotary positions of query and key heads, with or without the
// norm of each head, in one pass over the data (attn_rope,
// attn_qk_norm_rope).
//
//   y = R(t) (x * w / sqrt(mean(x^2) + eps)),  R(t): the rotation of rope.cuh
//
// Memory bound: every element is read once and written once, 3 to 7 flops
// between.  One warp takes one token and a run of its heads, kRows of them a
// step; D/16 lanes (fp32: D/8) share a row, two 16-byte chunks each, so a
// warp's accesses cover whole rows.  The sines and cosines belong to the token,
// not to the head: the warp computes each once, into shared memory, and every
// lane keeps those of its pairs in registers for all its heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeUnroll = 2;  // steps a lane has in flight

struct RopeParams {
    RopeRows q, k;
    const void* qw;
    const void* kw;
    const int* positions;
    RopeTable table;
    long long warps;  // tokens * segments
    int T;
    int q_steps, steps, segs, per_seg;  // a token's steps, cut into segments
    float eps;
};

template <typename E, int D, int kLayout, bool kNorm>
__global__ void __launch_bounds__(kRopeWarps * 32, kNorm ? 5 : 6)
rope_kernel(const RopeParams p) {
    using R = Rope<E, D, kLayout, kNorm>;
    __shared__ __align__(16) float s_table[kRopeWarps][D];
    __shared__ float s_scratch[R::kScratch ? kRopeWarps * R::kScratch : 1];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int j = lane % R::kLanes, grp = lane / R::kLanes;
    const long long w = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
    if (w >= p.warps) return;
    const long long token = w / p.segs;
    const int seg = static_cast<int>(w - token * p.segs);
    const long long b = token / p.T, t = token - b * p.T;
    const int half = p.table.half;
    const unsigned on = R::turning(half, j);
    const long long at0 = R::first(j, half) * E::kBytes, at1 = R::second(j, half) * E::kBytes;
    const uint8_t* xq = static_cast<const uint8_t*>(p.q.x) + (b * p.q.x_batch + t * p.q.x_token) * E::kBytes;
    const uint8_t* xk = static_cast<const uint8_t*>(p.k.x) + (b * p.k.x_batch + t * p.k.x_token) * E::kBytes;
    uint8_t* yq = static_cast<uint8_t*>(p.q.y) + (b * p.q.y_batch + t * p.q.y_token) * E::kBytes;
    uint8_t* yk = static_cast<uint8_t*>(p.k.y) + (b * p.k.y_batch + t * p.k.y_token) * E::kBytes;
    float* table = s_table[warp];
    float* scratch = s_scratch + (R::kScratch ? warp * R::kScratch + grp * D : 0);

    const int s0 = seg * p.per_seg, s1 = min(p.steps, s0 + p.per_seg);
    typename R::Coef coef;
    typename R::Pairs weight;  // the odd layout multiplies by it; the others have it in coef
    int coef_of = -1;          // 0: query heads, 1: key heads
    for (int s = s0; s < s1; s += kRopeUnroll) {
        typename R::Raw raw[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const bool is_k = s + u >= p.q_steps;
            const int head = (is_k ? s + u - p.q_steps : s + u) * R::kRows + grp;
            const uint8_t* x = is_k ? xk + head * p.k.x_head * E::kBytes : xq + head * p.q.x_head * E::kBytes;
            raw[u] = s + u < s1 && head < (is_k ? p.k.heads : p.q.heads) ? R::load(x + at0, x + at1) : R::zero();
        }
        if (s == s0) {  // behind the first loads
            rope_fill<D>(p.table, p.positions[token], lane, table);
            if (!kNorm) R::coefficients(table, j, coef);
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (s + u >= s1) break;  // the same for the whole warp
            const bool is_k = s + u >= p.q_steps;
            const int head = (is_k ? s + u - p.q_steps : s + u) * R::kRows + grp;
            typename R::Pairs v = R::unpack(raw[u]);
            float scale = 1.0f;
            if (kNorm) {
                if (coef_of != (is_k ? 1 : 0)) {
                    coef_of = is_k ? 1 : 0;
                    const uint8_t* wrow = static_cast<const uint8_t*>(is_k ? p.kw : p.qw);
                    weight = wrow ? R::unpack(R::load(wrow + at0, wrow + at1)) : R::ones();
                    R::coefficients(table, j, coef, &weight);
                }
                scale = R::rms_scale(v, p.eps);
                if (kLayout == kRopeHalvesOdd) R::multiply(v, weight);
            }
            R::turn(v, coef, on, half, j, table, scratch);
            if (kNorm) R::scale(v, scale);
            uint8_t* y = is_k ? yk + head * p.k.y_head * E::kBytes : yq + head * p.q.y_head * E::kBytes;
            if (head < (is_k ? p.k.heads : p.q.heads)) R::store(y + at0, y + at1, v);
        }
    }
}

template <typename E, int D, int kLayout>
cudaError_t launch_norm(const RopeParams& p, bool norm, unsigned blocks, cudaStream_t st) {
    if (norm) rope_kernel<E, D, kLayout, true><<<blocks, kRopeWarps * 32, 0, st>>>(p);
    else rope_kernel<E, D, kLayout, false><<<blocks, kRopeWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_type(RopeParams p, int D, int layout, bool norm, const LaunchEnv& env, int* grid) {
    const int rows = 32 * 2 * (16 / E::kBytes) / D;  // Rope<...>::kRows
    p.q_steps = (p.q.heads + rows - 1) / rows;
    p.steps = p.q_steps + (p.k.heads + rows - 1) / rows;
    // A token's steps stay in one warp once 32 warps per SM are there without
    // cutting; fewer tokens cut them (a decode step is all latency).
    const long long tokens = p.warps, want = static_cast<long long>(env.num_sms) * 32;
    p.segs = static_cast<int>(std::max<long long>(1, std::min<long long>(p.steps, want / tokens)));
    p.per_seg = (p.steps + p.segs - 1) / p.segs;
    p.segs = (p.steps + p.per_seg - 1) / p.per_seg;
    p.warps = tokens * p.segs;
    const long long blocks = (p.warps + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned g = static_cast<unsigned>(blocks);
    *grid = static_cast<int>(g);
    if (D == 64)
        switch (layout) {
            case kRopeAdjacent: return launch_norm<E, 64, kRopeAdjacent>(p, norm, g, env.stream);
            case kRopeHalves: return launch_norm<E, 64, kRopeHalves>(p, norm, g, env.stream);
            default: return launch_norm<E, 64, kRopeHalvesOdd>(p, norm, g, env.stream);
        }
    switch (layout) {
        case kRopeAdjacent: return launch_norm<E, 128, kRopeAdjacent>(p, norm, g, env.stream);
        case kRopeHalves: return launch_norm<E, 128, kRopeHalves>(p, norm, g, env.stream);
        default: return launch_norm<E, 128, kRopeHalvesOdd>(p, norm, g, env.stream);
    }
}

}  // namespace

int rope_layout(int rot_dim, int interleaved, int bytes) {
    if (interleaved || rot_dim == 0) return kRopeAdjacent;
    return (rot_dim / 2) % (16 / bytes) == 0 ? kRopeHalves : kRopeHalvesOdd;
}

cudaError_t launch_rope(const RopeShape& s, const RopeRows& q, const RopeRows& k, const void* qw,
                        const void* kw, bool norm, float eps, const int* positions,
                        const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.qw = qw;
    p.kw = kw;
    p.positions = positions;
    p.table = RopeTable{s.turns, s.rot_dim / 2, s.magnitude};
    p.T = s.T;
    p.eps = eps;
    p.warps = static_cast<long long>(s.B) * s.T;
    const int layout = rope_layout(s.rot_dim, s.interleaved, s.dtype == ATTN_F32 ? 4 : 2);
    int grid = 0;
    cudaError_t e;
    if (s.dtype == ATTN_F32) e = launch_type<RopeF32>(p, s.D, layout, norm, env, &grid);
    else if (s.dtype == ATTN_F16) e = launch_type<RopeF16>(p, s.D, layout, norm, env, &grid);
    else e = launch_type<RopeBf16>(p, s.D, layout, norm, env, &grid);
    if (grid_out) *grid_out = grid;
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
