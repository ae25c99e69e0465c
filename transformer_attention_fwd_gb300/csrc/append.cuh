// append.cuh -- shared by the two paged appends (append.cu: 16-bit cache,
// append_e4m3.cu: 8-bit cache): which request and slot a new token has, and
// the rotation of rows that stay in the caller's strided tensors.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "attn_internal.h"
#include "rope.cuh"

namespace attn {

constexpr int kAppendWarps = 8;

struct AppendParams {
    RopeRows q, k, v;  // packed tokens: the token and head strides only; q.heads = 0 without q
    const int* cu;     // [B + 1] offsets of the new tokens
    const int* lens;   // [B] keys of each request, the new ones among them
    const int* positions;  // [total] or null: a token's position is its slot
    const int* block_table;
    uint8_t* cache;
    float* scales;  // 8-bit cache only
    unsigned* status;
    RopeTable table;
    PageDivider page;
    int B, total, max_pages, num_blocks;
    long long warps;  // 16-bit: tokens * segs; 8-bit: those of the query rows
    int q_segs, k_segs, segs, steps;
    float k_limit;  // 8-bit: largest |K| element a scale of 1 takes
    unsigned items, splits;  // 8-bit: blocks of the K and V pages (see append_e4m3.cu)
};

// The last i in 0 .. n - 1 with value(i) <= target, for non-decreasing values
// (0 if there is none); the warp probes 32 places at a time.
template <typename F>
__device__ __forceinline__ int warp_last_at_most(int n, long long target, int lane, F value) {
    int lo = 0;
    while (n > 1) {
        const int stride = (n + 31) / 32;
        const int at = lane * stride;
        const bool below = at < n && at >= 0 && value(lo + at) <= target;
        const unsigned hits = __ballot_sync(0xffffffffu, below);
        const int count = hits == 0xffffffffu ? 32 : __ffs(~hits) - 1;
        if (count == 0) break;
        lo += (count - 1) * stride;
        n = min(stride, n - (count - 1) * stride);
    }
    return lo;
}

// A request's new tokens; ok: its offsets and length are in range.
struct AppendRequest {
    int begin, end, len;
    bool ok;
};
__device__ __forceinline__ AppendRequest append_request(const AppendParams& p, int b) {
    AppendRequest r;
    r.begin = p.cu[b];
    r.end = p.cu[b + 1];
    r.len = p.lens[b];
    const long long most = static_cast<long long>(p.max_pages) * p.page.size;
    r.ok = r.begin >= 0 && r.begin <= r.end && r.end <= p.total && r.len >= r.end - r.begin &&
           r.len <= most;
    return r;
}

// One CTA reports requests that append_request() drops.
__device__ __forceinline__ void append_report(const AppendParams& p) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x)
        if (!append_request(p, b).ok) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
}

// The request and slot of a new token (by the whole warp); false if no valid
// request has it.
__device__ __forceinline__ bool append_slot(const AppendParams& p, int token, int lane, int* b,
                                            int* slot) {
    *b = warp_last_at_most(p.B, token, lane, [&](int i) { return static_cast<long long>(p.cu[i]); });
    const AppendRequest r = append_request(p, *b);
    *slot = r.len - (r.end - token);
    return r.ok && token >= r.begin && token < r.end;
}

// Block of a request's page, -1 (reported) if its id is outside the pool.
__device__ __forceinline__ int append_block(const AppendParams& p, int b, int page) {
    const int id = p.block_table[static_cast<int64_t>(b) * p.max_pages + page];
    if (id >= 0 && id < p.num_blocks) return id;
    atomicOr(p.status, ATTN_DEV_BAD_INPUT);
    return -1;
}

}  // namespace attn
