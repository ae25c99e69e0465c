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
//
// 8192 tokens, 32 + 8 heads, D 128, bf16 with the norm (168 MB): 28 us, 5.9 TB/s;
// fp32 without it (4099 tokens, 168 MB) 27 us; [8, 12 + 12, 1024, 64] fp16 (50 MB)
// 9.1 us, the launch and the last blocks' tail being 1.5 of them.  A token's sines
// once for each lane and tensor instead of once for each token, and partners
// fetched by shuffles, took 62, 35 and 15 us.  One token: 1.9 us, a launch.
// (At 96 registers the norm's instances for any half spill 8 to 16 bytes.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "pdl.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kRopeWarps = 4;

struct RopeParams {
    RopeRows q, k;
    const void* qw;
    const void* kw;
    const int* positions;
    RopeTable table;
    unsigned tokens, T;
    int q_steps, steps, per_seg;  // a token's steps; grid.y segments of per_seg
    float eps;
};

template <typename E, int D, int kLayout, bool kNorm>
__global__ void __launch_bounds__(kRopeWarps * 32, kNorm ? 5 : 6)
rope_kernel(const RopeParams p) {
    using R = Rope<E, D, kLayout, kNorm>;
    // Steps a lane has in flight: a step's registers are loaded again once unpacked.
    // (8192 tokens: 3 for 2 took the norm from 29.0 to 28.1 us, and the dense fp16
    // rotation from 9.2 to 9.6 us.)
    constexpr int kRopeUnroll = kNorm ? 3 : 2;
    __shared__ __align__(16) float s_table[kRopeWarps][D];
    __shared__ float s_scratch[R::kScratch ? kRopeWarps * R::kScratch : 1];
    grid_wait();
    grid_launch_next();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int j = lane % R::kLanes, grp = lane / R::kLanes;
    const unsigned token = blockIdx.x * kRopeWarps + warp;
    if (token >= p.tokens) return;
    const unsigned b = p.tokens == p.T ? 0u : token / p.T, t = token - b * p.T;
    const int half = p.table.half;
    const unsigned on = R::turning(half, j);
    const int at0 = R::first(j, half) * E::kBytes, to1 = R::second(j, half) * E::kBytes - at0;
    float* table = s_table[warp];
    float* scratch = s_scratch + (R::kScratch ? warp * R::kScratch + grp * D : 0);

    const int s0 = blockIdx.y * p.per_seg, s1 = min(p.steps, s0 + p.per_seg);
    typename R::Coef coef;
    typename R::Pairs weight;  // the odd layout multiplies by it; the others have it in coef
    bool filled = false;
    // Heads h0 + grp, h0 + grp + kRows, .. below h1 of one tensor.
    auto run = [&](const RopeRows& r, const void* w, int h0, int h1) {
        const long long xs = R::kRows * r.x_head * E::kBytes, ys = R::kRows * r.y_head * E::kBytes;
        const uint8_t* x = static_cast<const uint8_t*>(r.x) + at0 +
                           (b * r.x_batch + t * r.x_token + (h0 + grp) * r.x_head) * E::kBytes;
        uint8_t* y = static_cast<uint8_t*>(r.y) + at0 +
                     (b * r.y_batch + t * r.y_token + (h0 + grp) * r.y_head) * E::kBytes;
        typename R::Raw raw[kRopeUnroll];
        auto load = [&](int u, int h) {
            raw[u] = h < h1 ? R::load(x, x + to1) : R::zero();
            x += xs;
        };
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) load(u, h0 + grp + u * R::kRows);
        if (!filled) {  // behind the first loads
            rope_fill<D>(p.table, p.positions[token], lane, table);
            filled = true;
            if (!kNorm) R::coefficients(table, j, coef);
        }
        if (kNorm) {
            const uint8_t* row = static_cast<const uint8_t*>(w) + at0;
            weight = w ? R::unpack(R::load(row, row + to1)) : R::ones();
            R::coefficients(table, j, coef, &weight);
        }
        for (int h = h0 + grp; h - grp < h1; h += kRopeUnroll * R::kRows) {
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u) {
                if (u > 0 && h - grp + u * R::kRows >= h1) break;  // the same for the whole warp
                typename R::Pairs v = R::unpack(raw[u]);
                load(u, h + (kRopeUnroll + u) * R::kRows);
                float scale = 1.0f;
                if (kNorm) {
                    scale = R::rms_scale(v, p.eps);
                    if (kLayout == kRopeHalvesOdd) R::multiply(v, weight);
                }
                R::turn(v, coef, on, half, j, table, scratch);
                if (kNorm) R::scale(v, scale);
                if (h + u * R::kRows < h1) R::store(y, y + to1, v);
                y += ys;
            }
        }
    };
    if (s0 < p.q_steps) run(p.q, p.qw, s0 * R::kRows, min(p.q.heads, s1 * R::kRows));
    if (s1 > p.q_steps)
        run(p.k, p.kw, max(0, s0 - p.q_steps) * R::kRows, min(p.k.heads, (s1 - p.q_steps) * R::kRows));
}

template <typename E, int D, int kLayout>
cudaError_t launch_norm(const RopeParams& p, bool norm, dim3 blocks, cudaStream_t st) {
    return launch_serial(norm ? rope_kernel<E, D, kLayout, true> : rope_kernel<E, D, kLayout, false>, blocks,
                         kRopeWarps * 32, 0, st, p);
}

template <typename E>
cudaError_t launch_type(RopeParams p, int D, int layout, bool norm, const LaunchEnv& env, int* grid) {
    const int rows = 32 * 2 * (16 / E::kBytes) / D;  // Rope<...>::kRows
    p.q_steps = (p.q.heads + rows - 1) / rows;
    p.steps = p.q_steps + (p.k.heads + rows - 1) / rows;
    // A token's steps stay in one warp once 32 warps per SM are there without
    // cutting; fewer tokens cut them (a decode step is all latency).
    const int want = env.num_sms * 32;
    int segs = std::max(1, static_cast<int>(std::min<unsigned>(p.steps, want / p.tokens)));
    p.per_seg = (p.steps + segs - 1) / segs;
    segs = (p.steps + p.per_seg - 1) / p.per_seg;
    if (segs > 65535) return cudaErrorInvalidConfiguration;
    const dim3 g((p.tokens + kRopeWarps - 1) / kRopeWarps, segs);
    *grid = static_cast<int>(g.x * g.y);
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
    p.tokens = static_cast<unsigned>(s.B) * static_cast<unsigned>(s.T);
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
