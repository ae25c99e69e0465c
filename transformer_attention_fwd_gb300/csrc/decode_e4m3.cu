// decode_e4m3.cu -- decode (one query row per (request, head)) over the paged
// 8-bit cache with one scale for each block, K or V, and head
// (attn_fwd_decode_paged_e4m3).
//
//   O = sum_j p_j vs_j v_j / sum_j p_j,  p_j = 2^x_j,
//   x_j = log2(e) * scale * ks_j * (q . k_j)
//
// with k_j, v_j the codes and ks_j, vs_j the scales of key j's block.  HBM bound:
// 2 * D bytes per key and KV head are read once.  Half the bytes of the 16-bit
// cache leave half the time per key, so the products go to the tensor cores
// (mma.sync m16n8k16 in fp16, fp32 sums; the codes convert exactly): S^T = K Q^T
// with 16 keys as rows and eight query heads of their KV head as columns, and
// O^T = V^T P^T with 16 columns of V as rows.  P^T's operand is S^T's result with
// each 8 x 8 block transposed (movmatrix).  The order of a product's inner index
// is free, so K's columns and V's rows are dealt to lanes so that each reads 16
// contiguous bytes.
//
// Two running references.  The sum of the p_j is taken relative to 2^m, m a
// maximum over x_j, in fp32.  What multiplies a code is w_j = p_j vs_j, taken
// relative to 2^mv, mv following a maximum over x_j + log2 vs_j, as two fp16 terms
// with a product each: one alone, 11 bits, made results that are small differences of
// large sums wrong by their own size.  A tile with keys 2^20 or more under the reference
// takes its weights in groups, each relative to its largest, so what light keys add up
// to behind a heavy one with no value is there too.  (The second term costs 1 % at
// 64 x 4096 keys with up to 8 heads per KV head of 128, 8 % of 64, and 15 % with 16
// heads; products in another order, both checks in one vote and the second term made
// behind the first one's products change nothing.)  The result is (sum w_j v_j) / (sum p_j) * 2^(mv - m).  A reference moves
// only when a key exceeds it by 2^kSlack.
//
// Work: all 16-key tiles of all (request, KV head, head chunk) units are laid
// end to end, cut into one equal slice per CTA and that into one per warp.  A
// warp streams its tiles through a ring of its own with 16-byte asynchronous
// copies; nothing in the loop waits for another warp.  Units inside one warp's
// range are written at once; the pieces of the others are merged in the CTA at
// its end, and those that a CTA boundary cuts by the combine kernel.  Two to four
// small CTAs share an SM, as registers allow, so that one's start and end pass
// under the others' streaming (three instead of two, with rings of three tiles
// instead of four, took 3.4 us off below, and 1.1 off the ragged one).  More of them
// than fit at once, to even out the SMs, lost 5 us for each further wave: a start
// costs that much.
//
// 64 requests of 4096 keys, Hq 32, Hkv 8, D 128, 16-token blocks (539 MB): 89.6 us,
// 6.0 TB/s.  Every CTA sums the lengths and finds its place in 2.8 us, the first
// tiles are there after 5.6, the SMs run dry between 75 and 81 us (together they
// stream at 7.2 TB/s; these before the weights' second terms, at 88.6 us), merging
// takes 1 to 2 us and the combine kernel 3.  With 8 query heads per KV head and ragged
// lengths (231 MB) 44.6 us, by the same fixed costs (short contexts, for which they
// are all of the time, are in decode_e4m3_short.cu); at D = 64 101 us for 540 MB.
// With 16 heads per KV head 118 us (D = 128) and 139 us (D = 64): two and three warps
// to a scheduler, each waiting out the latencies of its own instructions (issue active
// 43 and 58 %, tensor pipe 38 and 32 %).
#include <cuda_runtime.h>

#include "decode_cache_long.cuh"
#include "decode_e4m3.cuh"

namespace attn {

size_t decode_e4m3_workspace_bytes(const PagedShape& s, int num_sms) {
    return decode_e4m3_short_ranks(s, num_sms) > 0 ? 0 : decode_long_workspace<E4m3Cache>(s, num_sms);
}

cudaError_t launch_decode_paged_e4m3(const uint16_t* q, const uint8_t* kv, const float* scales,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     uint16_t* o, float* lse, void* ws, const PagedShape& s,
                                     const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    CacheParams p = cache_params<E4m3Cache>(q, kv, block_table, seq_lens, o, lse, s, env);
    p.scales = scales;
    if (const int ranks = decode_e4m3_short_ranks(s, env.num_sms); ranks > 0) {
        *kernels_launched = 1;
        return launch_decode_e4m3_short(p, s, ranks, env, grid_out);
    }
    return launch_decode_long<E4m3Cache>(p, s, ws, env, grid_out, kernels_launched);
}

}  // namespace attn
