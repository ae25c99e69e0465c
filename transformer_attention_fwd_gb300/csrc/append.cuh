// append.cuh -- shared by the two paged appends (append.cu: 16-bit cache,
// append_e4m3.cu: 8-bit cache): which request and slot a new token has, and
// the rotation of rows that stay in the caller's strided tensors.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "attn_internal.h"
#include "rope.cuh"

namespace attn {

template <int N>
struct Int {
    static constexpr int value = N;
};

constexpr int kAppendWarps = 4;
constexpr int kAppendUnroll = 2;  // steps a lane has in flight (as in rope.cu)

struct AppendParams {
    RopeRows q, k, v;  // packed tokens: the token and head strides only; q.heads = 0 without q
    const int* cu;     // [B + 1] offsets of the new tokens
    const int* lens;   // [B] keys of each request, the new ones among them
    const int* positions;  // [total] or null: a token's position is its slot
    const int* block_table;
    uint8_t* cache;
    float* scales;  // 8-bit cache only
    uint8_t* row_scales;   // 4-bit cache only, and
    const float* factors;  // [2, heads] or null
    unsigned* status;
    RopeTable table;
    PageDivider page;
    int B, total, max_pages, num_blocks;
    int q_steps, kv_steps, steps, per_seg;  // a token's steps; segments of per_seg
    float k_limit;  // 8-bit: largest |K| element a scale of 1 takes
    unsigned items, splits, segs, q_blocks;  // 8-bit cache: see append_e4m3.cu
    unsigned token_blocks;                   // 16-bit cache: those behind them report bad requests
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

// Reporting block `block`: the requests of its threads that append_request() drops.
__device__ __forceinline__ void append_report(const AppendParams& p, unsigned block) {
    const unsigned b = block * blockDim.x + threadIdx.x;
    if (b < static_cast<unsigned>(p.B) && !append_request(p, static_cast<int>(b)).ok)
        atomicOr(p.status, ATTN_DEV_BAD_INPUT);
}

// The request and slot of a new token (by the whole warp); false if no valid
// request has it.  (Offsets out of order may hide a valid one; that is reported.)
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

// Where append_rows() puts a token's K and V rows: into the 16-bit cache, as its own rows are
// stored.  (append_e2m1.cu has the 4-bit cache, whose rows take more.)
struct PlainRows {
    static constexpr bool kPlain = true;
};

// Segment `seg` of a token's steps, by one warp: its query heads into q.y, its key
// heads into the cache and k.y, its values into the cache.  With kv_steps = 0 the
// query heads alone.  table: D floats of shared memory, scratch:
// Rope<...>::kScratch.
template <typename E, int D, int kLayout, class Sink = PlainRows>
__device__ __forceinline__ void append_rows(const AppendParams& p, int token, int seg, float* table, float* scratch) {
    using R = Rope<E, D, kLayout>;
    if (token >= p.total) return;
    const int lane = threadIdx.x % 32;
    const int j = lane % R::kLanes, grp = lane / R::kLanes;
    const int half = p.table.half;
    const unsigned on = R::turning(half, j);
    const int at0 = R::first(j, half) * E::kBytes, to1 = R::second(j, half) * E::kBytes - at0;
    if (R::kScratch) scratch += grp * D;

    const int s0 = seg * p.per_seg, s1 = min(p.steps, s0 + p.per_seg);
    const int k_end = p.q_steps + p.kv_steps;
    typename R::Coef coef;
    uint8_t* cache = nullptr;  // the slot's K row of head 0; null: the page is left out
    const long long head_bytes = static_cast<long long>(p.page.size) * D * E::kBytes;
    Sink sink{};
    if constexpr (!Sink::kPlain) sink.begin(j, half);
    bool found = false, mine = true;
    // The token's request, coefficients and place in the cache, behind the first
    // loads; false if no request has it.
    auto find = [&]() {
        found = true;
        int b, slot;
        mine = append_slot(p, token, lane, &b, &slot);
        if (!mine) return;
        if (s0 < k_end && half > 0) {
            rope_fill<D>(p.table, p.positions ? p.positions[token] : slot, lane, table);
            R::coefficients(table, j, coef);
        }
        if (s1 > p.q_steps) {
            int in_page;
            const int id = append_block(p, b, p.page.split(slot, &in_page));
            if constexpr (!Sink::kPlain) sink.place(p, id, in_page);
            else if (id >= 0)
                cache = p.cache + (static_cast<int64_t>(id) * 2 * p.k.heads * p.page.size + in_page) * D * E::kBytes;
        }
    };
    // Heads h0 + grp, h0 + grp + kRows, .. below h1: of q (kind 0), k (1), v (2).
    auto run = [&](auto kind_tag, const RopeRows& r, int h0, int h1) {
        constexpr int kKind = decltype(kind_tag)::value;
        const long long xs = R::kRows * r.x_head * E::kBytes, ys = R::kRows * r.y_head * E::kBytes;
        const long long cs = R::kRows * head_bytes;
        const uint8_t* x = static_cast<const uint8_t*>(r.x) + at0 + (token * r.x_token + (h0 + grp) * r.x_head) * E::kBytes;
        uint8_t* y = static_cast<uint8_t*>(r.y) + at0 + (token * r.y_token + (h0 + grp) * r.y_head) * E::kBytes;
        long long c = at0 + (h0 + grp + (kKind == 2 ? p.k.heads : 0)) * head_bytes;
        typename R::Raw raw[kAppendUnroll];
        auto load = [&](int u, int h) {
            raw[u] = h < h1 ? R::load(x, x + to1) : R::zero();
            x += xs;
        };
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) load(u, h0 + grp + u * R::kRows);
        if (!found) find();
        if (!mine) return;
        for (int h = h0 + grp; h - grp < h1; h += kAppendUnroll * R::kRows) {
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u) {
                if (u > 0 && h - grp + u * R::kRows >= h1) break;  // the same for the whole warp
                const bool in = h + u * R::kRows < h1;
                if (kKind == 2 || half == 0) {  // copied as they are
                    if (kKind != 2 && in && r.y) R::store(y, y + to1, raw[u]);
                    if constexpr (!Sink::kPlain) {
                        if (kKind != 0) sink.store(p, h + u * R::kRows + (kKind == 2 ? p.k.heads : 0), in, raw[u]);
                    } else {
                        if (kKind != 0 && in && cache) R::store(cache + c, cache + c + to1, raw[u]);
                    }
                    load(u, h + (kAppendUnroll + u) * R::kRows);
                } else {
                    typename R::Pairs v = R::unpack(raw[u]);
                    load(u, h + (kAppendUnroll + u) * R::kRows);
                    R::turn(v, coef, on, half, j, table, scratch);
                    if (in && r.y) R::store(y, y + to1, v);
                    if constexpr (!Sink::kPlain) {
                        if (kKind == 1) sink.store(p, h + u * R::kRows, in, v);
                    } else {
                        if (kKind == 1 && in && cache) R::store(cache + c, cache + c + to1, v);
                    }
                }
                y += ys;
                c += cs;
            }
        }
    };
    if (s0 < p.q_steps) run(Int<0>{}, p.q, s0 * R::kRows, min(p.q.heads, s1 * R::kRows));
    if (p.kv_steps == 0) return;
    if (mine && s0 < k_end && s1 > p.q_steps)
        run(Int<1>{}, p.k, max(0, s0 - p.q_steps) * R::kRows, min(p.k.heads, (s1 - p.q_steps) * R::kRows));
    if (mine && s1 > k_end)
        run(Int<2>{}, p.v, max(0, s0 - k_end) * R::kRows, min(p.v.heads, (s1 - k_end) * R::kRows));
}

}  // namespace attn
