// rope.cu -- rotary positions of query and key heads, with or without the
// norm of each head, in one pass over the data (attn_rope,
// attn_qk_norm_rope).
//
//   y = R(t) (x * w / sqrt(mean(x^2) + eps)),  R(t): the rotation of rope.cuh
//
// Memory bound: every element is read once and written once, 3 to 7 flops
// between.  One warp takes one token and a run of its heads; D/8 lanes share a
// row, 16 bytes (fp32: 32) each, so a warp access covers 32/(D/8) whole rows.
// The sines and cosines belong to the token, not to the head: a lane computes
// those of its eight elements once and applies them to every head of the run,
// which is as long as the grid stays large enough to fill the GPU.  Halves
// trade whole 8-element chunks between lanes (four shuffles a row); only a
// rotated half that is no multiple of eight elements goes through shared
// memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeUnroll = 4;  // rows a lane has in flight

struct RopeParams {
    RopeRows q, k;
    const void* qw;
    const void* kw;
    const int* positions;
    RopeTable table;
    long long warps;  // tokens * (q segments + k segments)
    int T;
    int q_segs, segs, steps;  // segments of the query heads, of all heads; steps a segment
    float eps;
    int norm;
};

template <typename Row, int D, int kLayout>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / kRopeChunk, kRowsPerStep = 32 / kLanes;
    __shared__ float s_row[kLayout == kRopeHalvesOdd ? kRopeWarps * kRowsPerStep * D : 1];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int sub = lane % kLanes, grp = lane / kLanes;
    const long long w = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
    if (w >= p.warps) return;
    const long long token = w / p.segs;
    int seg = static_cast<int>(w - token * p.segs);
    const bool is_k = seg >= p.q_segs;
    if (is_k) seg -= p.q_segs;
    const RopeRows& r = is_k ? p.k : p.q;
    const long long b = token / p.T, t = token - b * p.T;
    const uint8_t* x = static_cast<const uint8_t*>(r.x) +
                       (b * r.x_batch + t * r.x_token + sub * kRopeChunk) * Row::kBytes;
    uint8_t* y = static_cast<uint8_t*>(r.y) +
                 (b * r.y_batch + t * r.y_token + sub * kRopeChunk) * Row::kBytes;
    const long long xh = r.x_head * Row::kBytes, yh = r.y_head * Row::kBytes;
    const int h0 = seg * p.steps * kRowsPerStep;
    const int h1 = min(r.heads, h0 + p.steps * kRowsPerStep);
    float* row = s_row + (kLayout == kRopeHalvesOdd ? (warp * kRowsPerStep + grp) * D : 0);

    RopeCoef coef;
    bool have = false;
    for (int h = h0; h < h1; h += kRopeUnroll * kRowsPerStep) {
        typename Row::Raw raw[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int head = h + u * kRowsPerStep + grp;
            raw[u] = head < h1 ? Row::load(x + head * xh) : Row::zero();
        }
        if (!have) {  // behind the first loads
            rope_coefficients<Row, kLayout>(p.table, sub * kRopeChunk, p.positions[token],
                                            p.norm ? (is_k ? p.kw : p.qw) : nullptr, coef);
            have = true;
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (h + u * kRowsPerStep >= h1) break;  // the same for the whole warp
            const int head = h + u * kRowsPerStep + grp;
            float v[8], vp[8];
            Row::unpack(raw[u], v);
            rope_exchange<Row, kLayout, D>(raw[u], v, p.table.half, lane, row, vp);
            const float scale = p.norm ? rope_rms_scale<D>(v, p.eps) : 1.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = fmaf(v[e], coef.own[e], vp[e] * coef.other[e]) * scale;
            if (head < h1) Row::store(y + head * yh, v);
        }
    }
}

template <typename Row, int D>
cudaError_t launch_layout(const RopeParams& p, int layout, unsigned blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent: rope_kernel<Row, D, kRopeAdjacent><<<blocks, kRopeWarps * 32, 0, st>>>(p); break;
        case kRopeHalves: rope_kernel<Row, D, kRopeHalves><<<blocks, kRopeWarps * 32, 0, st>>>(p); break;
        default: rope_kernel<Row, D, kRopeHalvesOdd><<<blocks, kRopeWarps * 32, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

template <typename Row>
cudaError_t launch_dim(const RopeParams& p, int D, int layout, unsigned blocks, cudaStream_t st) {
    return D == 64 ? launch_layout<Row, 64>(p, layout, blocks, st)
                   : launch_layout<Row, 128>(p, layout, blocks, st);
}

}  // namespace

int rope_layout(int rot_dim, int interleaved) {
    if (interleaved || rot_dim == 0) return kRopeAdjacent;
    return (rot_dim / 2) % 8 == 0 ? kRopeHalves : kRopeHalvesOdd;
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
    p.norm = norm ? 1 : 0;
    const int rows = 32 / (s.D / kRopeChunk);
    const long long tokens = static_cast<long long>(s.B) * s.T;
    const int q_steps = (q.heads + rows - 1) / rows, k_steps = (k.heads + rows - 1) / rows;
    // Steps a warp takes: one while 32 warps per SM are not reached (a decode
    // step is all latency), then as many as keep that many warps.
    const long long per = tokens * (q_steps + k_steps) / (static_cast<long long>(env.num_sms) * 32);
    p.steps = static_cast<int>(std::max<long long>(1, std::min<long long>(per, std::max(q_steps, k_steps))));
    p.q_segs = (q_steps + p.steps - 1) / p.steps;
    p.segs = p.q_segs + (k_steps + p.steps - 1) / p.steps;
    p.warps = tokens * p.segs;
    const long long blocks = (p.warps + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned g = static_cast<unsigned>(blocks);
    cudaError_t e;
    const int layout = rope_layout(s.rot_dim, s.interleaved);
    if (s.dtype == ATTN_F32) e = launch_dim<RopeF32>(p, s.D, layout, g, env.stream);
    else if (s.dtype == ATTN_F16) e = launch_dim<RopeF16>(p, s.D, layout, g, env.stream);
    else e = launch_dim<RopeBf16>(p, s.D, layout, g, env.stream);
    if (grid_out) *grid_out = static_cast<int>(g);
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
