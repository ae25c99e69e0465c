// decode_e2m1_short.cu -- the decode over the 4-bit cache (decode_e2m1.cu) for short
// contexts and few requests; the work is the 8-bit decode's (decode_e4m3_short.cu).
#include <cuda_runtime.h>

#include "decode_cache_short.cuh"
#include "decode_e2m1.cuh"

namespace attn {

int decode_e2m1_short_ranks(const PagedShape& s, int num_sms) { return decode_short_ranks<E2m1Cache>(s, num_sms); }

cudaError_t launch_decode_e2m1_short(const CacheParams& p, const PagedShape& s, int ranks, const LaunchEnv& env,
                                     int* grid_out) {
    return launch_decode_short<E2m1Cache>(p, s, ranks, env, grid_out);
}

}  // namespace attn
