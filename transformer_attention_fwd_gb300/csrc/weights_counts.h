// weights_counts.h -- how the sums of attention weights (weights.cu, weights_tiles.cu) are
// cut into work, in integers alone: the same for the host and the device.
#pragma once

#include <cuda_runtime.h>

namespace attn {

constexpr int kWeightsKeyShift = 8;  // log2 of an item's keys
constexpr int kWeightsCols = 128;    // query rows of a tile

// Tokens of a query tile: as many as it has rows for.  0: the kernel that streams the keys
// (weights.cu) takes the call: a group that a tile has no room for; up to eight query rows to a KV
// head, as far as the host can tell (with a step's one token over 64 x 4096 keys tiles took 98 us
// in 16 bits and 152 in 4, that kernel 88 and 47; with 16 rows over 32 x 4096, 53 and 77, that one 63
// and 77); so many tokens that a range, or what follows it, would pass 31 bits.
inline int weights_tile_tokens(int total, int group, int B) {
    if (group > kWeightsCols || static_cast<long long>(total) * group <= 8ll * B || total >= 1 << 30) return 0;
    return kWeightsCols / group;
}

// A request's queries are worked on in ranges of 1 << shift tokens.  One with several has a
// place in the workspace for each range's sums; places are handed out request by request.
// Each request's offsets are checked by themselves, so those of a call may overlap and their
// tokens add up to more than it has: a request whose places would pass the last one is left out.
struct WeightsRanges {
    static constexpr int kMany = 1 << 24;  // more places than there ever are
    int shift;
    int places;
    // Places of a request of n queries.
    __host__ __device__ int of(int n) const {
        return n <= 1 << shift ? 0 : (n + (1 << shift) - 1) >> shift;
    }
    // Places of several requests: up to kMany, so that no number of requests wraps.
    static __host__ __device__ int add(int a, int b) { return a + b < kMany ? a + b : kMany; }
    // Whether a request has its places, the last of which is number `end`, counted from 1.
    __host__ __device__ bool fits(int end) const { return end <= places; }
};

// Two blocks of keys to a range, so that there are items for all SMs (a 4096-token prompt took
// 82 us with one block, 77 with two, 99 with four, 122 with sixteen); more where the partial sums
// would not stay in the L2 (64 MB), or a head's items not fit in 31 bits.
// total: under 2^30 (weights_tile_tokens), so that shift is at most 30.
inline WeightsRanges weights_ranges(int total, int Hkv, long long keys) {
    constexpr double kPartialBytes = 64ll << 20;
    int shift = kWeightsKeyShift + 1;
    while (total >> shift > 0 &&
           (static_cast<double>(2ll * total >> shift) * Hkv * keys * 4 > kPartialBytes ||  // (may pass 64 bits)
            ((keys >> kWeightsKeyShift) + 1) * ((total >> shift) + 1) > 0x3fffffffll))
        ++shift;
    // Requests with more tokens than a range, and as many as the call has in all, have at most
    // 2 n / range of them.
    return WeightsRanges{shift, total <= 1ll << shift ? 0 : static_cast<int>(2ll * total >> shift)};
}

// A request's first query row, of n tokens with `group` rows each, that sees a key of its len ones;
// of a key behind them (a chunk's places end later) n * group, which the host has checked.
__host__ __device__ inline int weights_first_row(int key, int len, int n, int group) {
    const int token = key - (len - n);
    return token <= 0 ? 0 : (token < n ? token : n) * group;
}

// A tile's first column that sees a key: token i of the tile, `group` columns, sees the keys up to
// past + i.  At most an item's keys lie behind past; those far before it, times the group, would wrap.
__host__ __device__ inline int weights_first_column(int key, int past, int group) {
    return key > past ? (key - past) * group : 0;
}

}  // namespace attn
