// weights.cuh -- shared by the two kernels that add up attention weights over a paged
// cache's keys (weights.cu, weights_tiles.cu).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "attn_internal.h"
#include "sm100.cuh"

namespace attn {

constexpr float kWeightsLog2e = 1.4426950408889634f;

struct WeightsParams {
    const uint16_t* q;
    long long q_token, q_head;
    const float* lse;
    long long lse_head, lse_token;
    const uint8_t* cache;
    const uint8_t* scales;
    const float* factors;
    const int *block_table, *cu, *lens;
    float* weights;
    unsigned* status;
    PageDivider page;
    int B, total, Hq, Hkv, group, max_pages, num_blocks;
    float scale_log2;
};

// A request's queries and length; ok: both in range.
struct WeightsRequest {
    int begin, end, len;
    bool ok;
};
__device__ __forceinline__ WeightsRequest weights_request(const WeightsParams& p, int b) {
    WeightsRequest r;
    r.begin = p.cu[b];
    r.end = p.cu[b + 1];
    r.len = p.lens[b];
    r.ok = r.begin >= 0 && r.begin <= r.end && r.end <= p.total && r.len >= r.end - r.begin &&
           r.len <= p.max_pages * p.page.size;
    return r;
}

inline WeightsParams weights_params(const WeightsShape& s, const LaunchEnv& env) {
    WeightsParams p{};
    p.q = static_cast<const uint16_t*>(s.q);
    p.q_token = s.q_token;
    p.q_head = s.q_head;
    p.lse = s.lse;
    p.lse_head = s.lse_head;
    p.lse_token = s.lse_token;
    p.cache = static_cast<const uint8_t*>(s.cache);
    p.scales = s.scales;
    p.factors = s.factors;
    p.block_table = s.block_table;
    p.cu = s.cu_seqlens;
    p.lens = s.seq_lens;
    p.weights = s.weights;
    p.status = env.status;
    p.page = PageDivider(s.page);
    p.B = s.B;
    p.total = s.total;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.group = s.Hq / s.Hkv;
    p.max_pages = s.max_pages;
    p.num_blocks = s.num_blocks;
    p.scale_log2 = s.scale * kWeightsLog2e;
    return p;
}

}  // namespace attn
