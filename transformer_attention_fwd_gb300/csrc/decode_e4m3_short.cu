// decode_e4m3_short.cu -- the decode over the 8-bit cache (decode_e4m3.cu) when a
// request's share of the work is small: short contexts and few requests, where
// latency counts and not the balance of the SMs.
//
// A cluster of 1 to 8 CTAs takes one (request, KV head, head chunk) unit, each warp
// of it an equal run of the unit's tiles.  Nothing has to be known of the other
// requests: no prefix of the lengths, no search, no workspace and no second kernel.
// The warps' parts are merged in their CTA, and the CTAs' parts by a cluster
// barrier, after which each CTA adds up some heads out of the others' shared
// memory.  Latency bounds it: length, block ids, tiles, two merges.
//
// 3 requests of up to 1476 keys (12 heads, D 64): 5.4 us against 8.9 for the
// two launches of decode_e4m3.cu, and 5 us of host time against 9.
#include <cuda_runtime.h>

#include "decode_cache_short.cuh"
#include "decode_e4m3.cuh"

namespace attn {

int decode_e4m3_short_ranks(const PagedShape& s, int num_sms) { return decode_short_ranks<E4m3Cache>(s, num_sms); }

cudaError_t launch_decode_e4m3_short(const CacheParams& p, const PagedShape& s, int ranks, const LaunchEnv& env,
                                     int* grid_out) {
    return launch_decode_short<E4m3Cache>(p, s, ranks, env, grid_out);
}

}  // namespace attn
