// append.cuh -- shared by the two paged appends (append.cu: 16-bit cache,
// append_e4m3.cu: 8-bit cache): which request and slot a new token has, and
// the rotation of rows that stay in the caller's strided tensors.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "attn_internal.h"
#include "rope.cuh"

namespace attn {

constexpr int kAppendWarps = 4;
constexpr int kAppendUnroll = 2;  // steps a lane has in flight

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
    long long warps;  // tokens * segs; 8-bit cache: of the query rows
    int q_steps, kv_steps, steps, segs, per_seg;  // a token's steps, cut into segments
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

// A warp's segment w of the steps of a token: its query heads into q.y, its
// key heads into the cache and k.y, its values into the cache.  With kv_steps =
// 0 the query heads alone.  table: D floats of shared memory, scratch:
// Rope<...>::kScratch.
template <typename E, int D, int kLayout>
__device__ __forceinline__ void append_rows(const AppendParams& p, long long w, float* table, float* scratch) {
    using R = Rope<E, D, kLayout>;
    const int lane = threadIdx.x % 32;
    const int j = lane % R::kLanes, grp = lane / R::kLanes;
    if (w >= p.warps) return;
    const int token = static_cast<int>(w / p.segs);
    const int seg = static_cast<int>(w - static_cast<long long>(token) * p.segs);
    const int half = p.table.half;
    const unsigned on = R::turning(half, j);
    const long long at0 = R::first(j, half) * E::kBytes, at1 = R::second(j, half) * E::kBytes;
    const uint8_t* xq = static_cast<const uint8_t*>(p.q.x) + token * p.q.x_token * E::kBytes;
    const uint8_t* xk = static_cast<const uint8_t*>(p.k.x) + token * p.k.x_token * E::kBytes;
    const uint8_t* xv = static_cast<const uint8_t*>(p.v.x) + token * p.v.x_token * E::kBytes;
    if (R::kScratch) scratch += grp * D;

    // Steps of a token: its query heads, then its key heads, then its values.
    const int s0 = seg * p.per_seg, s1 = min(p.steps, s0 + p.per_seg);
    const int k_end = p.q_steps + p.kv_steps;
    typename R::Coef coef;
    uint8_t* cache = nullptr;  // the slot's K row of head 0; null: the page is left out
    const long long ch = static_cast<long long>(p.page.size) * D * E::kBytes, to_v = p.k.heads * ch;
    for (int s = s0; s < s1; s += kAppendUnroll) {
        typename R::Raw raw[kAppendUnroll];
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int st = s + u;
            const int kind = st < p.q_steps ? 0 : (st < k_end ? 1 : 2);
            const int head = (st - (kind == 0 ? 0 : (kind == 1 ? p.q_steps : k_end))) * R::kRows + grp;
            const uint8_t* x = kind == 0 ? xq + head * p.q.x_head * E::kBytes
                                         : (kind == 1 ? xk + head * p.k.x_head * E::kBytes
                                                      : xv + head * p.v.x_head * E::kBytes);
            raw[u] = st < s1 && head < (kind == 0 ? p.q.heads : p.k.heads) ? R::load(x + at0, x + at1) : R::zero();
        }
        if (s == s0) {  // behind the first loads
            int b, slot;
            if (!append_slot(p, token, lane, &b, &slot)) return;  // the whole warp
            if (s0 < k_end) {
                rope_fill<D>(p.table, p.positions ? p.positions[token] : slot, lane, table);
                R::coefficients(table, j, coef);
            }
            if (s1 > p.q_steps) {
                int in_page;
                const int id = append_block(p, b, p.page.split(slot, &in_page));
                if (id >= 0)
                    cache = p.cache +
                            (static_cast<int64_t>(id) * 2 * p.k.heads * p.page.size + in_page) * D * E::kBytes;
            }
        }
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int st = s + u;
            if (st >= s1) break;  // the same for the whole warp
            const int kind = st < p.q_steps ? 0 : (st < k_end ? 1 : 2);
            const int head = (st - (kind == 0 ? 0 : (kind == 1 ? p.q_steps : k_end))) * R::kRows + grp;
            const bool in = head < (kind == 0 ? p.q.heads : p.k.heads);
            uint8_t* row = cache + head * ch;
            if (kind == 2) {
                if (in && cache) {
                    *reinterpret_cast<uint4*>(row + to_v + at0) = raw[u].c0;
                    *reinterpret_cast<uint4*>(row + to_v + at1) = raw[u].c1;
                }
                continue;
            }
            typename R::Pairs v = R::unpack(raw[u]);
            R::turn(v, coef, on, half, j, table, scratch);
            const RopeRows& r = kind == 0 ? p.q : p.k;
            if (in && r.y) {
                uint8_t* y = static_cast<uint8_t*>(r.y) + (token * r.y_token + head * r.y_head) * E::kBytes;
                R::store(y + at0, y + at1, v);
            }
            if (in && kind == 1 && cache) R::store(row + at0, row + at1, v);
        }
    }
}

}  // namespace attn
