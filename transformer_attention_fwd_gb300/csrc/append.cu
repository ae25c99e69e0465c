// append.cu -- new keys and values into the paged 16-bit cache, keys (and the
// queries of the same tokens) rotated on the way (attn_append_paged).
//
// A copy with the rotation of rope.cuh in it, memory bound: q, k and v are
// read once, q and the cache rows written once.  The work split is rope.cu's
// (one warp takes one token and a run of its heads of q, k and v); a warp finds
// its token's request with a 32-way search of the offsets, then the block of
// its slot, while its first rows are on the way.
//
// 17100 tokens of 9 requests, 32 query and 8 KV heads, D 128 (420 MB): 66 us,
// 6.4 TB/s.  One token for each of 64 requests: 3.0 us.  80 registers, for 24 warps
// per SM; the instances for halves of whole chunks spill 12 bytes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "append.cuh"
#include "pdl.cuh"

namespace attn {
namespace {

template <typename E, int D, int kLayout>
__global__ void __launch_bounds__(kAppendWarps * 32, 6)
append_kernel(const AppendParams p) {
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
    append_rows<E, D, kLayout>(p, static_cast<int>(blockIdx.x) * kAppendWarps + warp, blockIdx.y, s_table[warp],
                               s_scratch + warp * R::kScratch);
}

template <typename E, int D>
cudaError_t launch_layout(const AppendParams& p, int layout, dim3 blocks, cudaStream_t st) {
    switch (layout) {
        case kRopeAdjacent: return launch_serial(append_kernel<E, D, kRopeAdjacent>, blocks, kAppendWarps * 32, 0, st, p);
        case kRopeHalves: return launch_serial(append_kernel<E, D, kRopeHalves>, blocks, kAppendWarps * 32, 0, st, p);
        default: return launch_serial(append_kernel<E, D, kRopeHalvesOdd>, blocks, kAppendWarps * 32, 0, st, p);
    }
}

}  // namespace

// As in rope.cu: a token's steps are cut while 32 warps per SM are not there.
int append_segments(AppendParams& p, int num_sms) {
    const int segs = std::max(1, std::min(p.steps, num_sms * 32 / p.total));
    p.per_seg = (p.steps + segs - 1) / segs;
    return (p.steps + p.per_seg - 1) / p.per_seg;
}

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
