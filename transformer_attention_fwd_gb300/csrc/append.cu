// append.cu -- new keys and values into the paged 16-bit cache, keys (and the
// queries of the same tokens) rotated on the way (attn_append_paged).
//
// A copy with the rotation of rope.cuh in it, memory bound: q, k and v are
// read once, q and the cache rows written once.  The work split is rope.cu's
// (one warp takes one token and a run of the heads of q, k or v); a warp finds
// its token's request with a 32-way search of the offsets, then the block of
// its slot, while its first rows are on the way.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "append.cuh"

namespace attn {
namespace {

constexpr int kUnroll = 4;  // rows a lane has in flight

template <typename Row, int D, int kLayout>
__global__ void __launch_bounds__(kAppendWarps * 32)
append_kernel(const AppendParams p) {
    constexpr int kLanes = D / kRopeChunk, kRowsPerStep = 32 / kLanes;
    __shared__ float s_row[kLayout == kRopeHalvesOdd ? kAppendWarps * kRowsPerStep * D : 1];
    if (blockIdx.x == gridDim.x - 1) append_report(p);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int sub = lane % kLanes, grp = lane / kLanes;
    const long long w = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
    if (w >= p.warps) return;
    const int token = static_cast<int>(w / p.segs);
    int seg = static_cast<int>(w - static_cast<long long>(token) * p.segs);
    const int kind = seg < p.q_segs ? 0 : (seg < p.q_segs + p.k_segs ? 1 : 2);
    if (kind > 0) seg -= p.q_segs;
    if (kind > 1) seg -= p.k_segs;
    const RopeRows& r = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
    const uint8_t* x = static_cast<const uint8_t*>(r.x) +
                       (token * r.x_token + sub * kRopeChunk) * Row::kBytes;
    const long long xh = r.x_head * Row::kBytes;
    const int h0 = seg * p.steps * kRowsPerStep;
    const int h1 = min(r.heads, h0 + p.steps * kRowsPerStep);
    float* row = s_row + (kLayout == kRopeHalvesOdd ? (warp * kRowsPerStep + grp) * D : 0);

    RopeCoef coef;
    bool have = false;
    uint8_t* y = nullptr;      // the caller's tensor
    uint8_t* cache = nullptr;  // the slot's row of head 0
    long long yh = 0;
    const long long ch = static_cast<long long>(p.page.size) * D * Row::kBytes;
    for (int h = h0; h < h1; h += kUnroll * kRowsPerStep) {
        typename Row::Raw raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int head = h + u * kRowsPerStep + grp;
            raw[u] = head < h1 ? Row::load(x + head * xh) : Row::zero();
        }
        if (!have) {
            int b, slot;
            if (!append_slot(p, token, lane, &b, &slot)) return;  // the whole warp
            if (kind < 2) {
                rope_coefficients<Row, kLayout>(p.table, sub * kRopeChunk,
                                                p.positions ? p.positions[token] : slot, nullptr, coef);
                if (r.y != nullptr) {
                    y = static_cast<uint8_t*>(r.y) + (token * r.y_token + sub * kRopeChunk) * Row::kBytes;
                    yh = r.y_head * Row::kBytes;
                }
            }
            if (kind > 0) {
                int in_page;
                const int id = append_block(p, b, p.page.split(slot, &in_page));
                if (id >= 0)
                    cache = p.cache + ((static_cast<int64_t>(id) * 2 + (kind - 1)) * p.k.heads * p.page.size +
                                       in_page) * D * Row::kBytes + sub * kRopeChunk * Row::kBytes;
            }
            have = true;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h + u * kRowsPerStep >= h1) break;  // the same for the whole warp
            const int head = h + u * kRowsPerStep + grp;
            if (kind == 2) {
                if (head < h1 && cache) Row::store_raw(cache + head * ch, raw[u]);
                continue;
            }
            float v[8], vp[8];
            Row::unpack(raw[u], v);
            rope_exchange<Row, kLayout, D>(raw[u], v, p.table.half, lane, row, vp);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], coef.own[e], vp[e] * coef.other[e]);
            if (head < h1 && y) Row::store(y + head * yh, v);
            if (head < h1 && cache) Row::store(cache + head * ch, v);
        }
    }
}

template <typename Row, int D>
cudaError_t launch_layout(const AppendParams& p, int layout, unsigned blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent: append_kernel<Row, D, kRopeAdjacent><<<blocks, kAppendWarps * 32, 0, st>>>(p); break;
        case kRopeHalves: append_kernel<Row, D, kRopeHalves><<<blocks, kAppendWarps * 32, 0, st>>>(p); break;
        default: append_kernel<Row, D, kRopeHalvesOdd><<<blocks, kAppendWarps * 32, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

AppendParams append_params(const AppendShape& s, const RopeShape& r, const RopeRows* q,
                           const RopeRows& k, const RopeRows& v, const LaunchEnv& env) {
    AppendParams p{};
    if (q) p.q = *q;
    p.k = k;
    p.v = v;
    p.cu = s.cu_seqlens;
    p.lens = s.seq_lens;
    p.positions = s.positions;
    p.block_table = s.block_table;
    p.cache = static_cast<uint8_t*>(s.cache);
    p.scales = s.scales;
    p.status = env.status;
    p.table = RopeTable{r.turns, r.rot_dim / 2, r.magnitude};
    p.page = PageDivider(s.page);
    p.B = s.B;
    p.total = s.total;
    p.max_pages = s.max_pages;
    p.num_blocks = s.num_blocks;
    return p;
}

cudaError_t launch_append_paged(const AppendShape& s, const RopeShape& r, const RopeRows* q,
                                const RopeRows& k, const RopeRows& v, const LaunchEnv& env,
                                int* grid_out, int* kernels_launched) {
    AppendParams p = append_params(s, r, q, k, v, env);
    const int rows = 32 / (r.D / kRopeChunk);
    const int q_steps = (p.q.heads + rows - 1) / rows, kv_steps = (k.heads + rows - 1) / rows;
    // As in rope.cu: one step a warp until 32 warps per SM are there.
    const long long per = static_cast<long long>(s.total) * (q_steps + 2 * kv_steps) /
                          (static_cast<long long>(env.num_sms) * 32);
    p.steps = static_cast<int>(std::max<long long>(1, std::min<long long>(per, std::max(q_steps, kv_steps))));
    p.q_segs = (q_steps + p.steps - 1) / p.steps;
    p.k_segs = (kv_steps + p.steps - 1) / p.steps;
    p.segs = p.q_segs + 2 * p.k_segs;
    p.warps = static_cast<long long>(s.total) * p.segs;
    const long long blocks = (p.warps + kAppendWarps - 1) / kAppendWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned g = static_cast<unsigned>(blocks);
    const int layout = rope_layout(r.rot_dim, r.interleaved);
    cudaError_t e;
    if (r.dtype == ATTN_F16)
        e = r.D == 64 ? launch_layout<RopeF16, 64>(p, layout, g, env.stream)
                      : launch_layout<RopeF16, 128>(p, layout, g, env.stream);
    else
        e = r.D == 64 ? launch_layout<RopeBf16, 64>(p, layout, g, env.stream)
                      : launch_layout<RopeBf16, 128>(p, layout, g, env.stream);
    if (grid_out) *grid_out = static_cast<int>(g);
    if (kernels_launched) *kernels_launched = 1;
    return e;
}

}  // namespace attn
