// evict.cu -- eviction from a paged cache by accumulated attention weight
// (attn_evict_paged, attn_evict_paged_e2m1).
//
// Of a request with more than `keep` keys, each KV head keeps its last `recent` slots and
// the keep - recent heaviest of the others, and the kept rows move to slots 0 .. keep - 1 in
// their order.  Two kernels.  evict_select_kernel, a CTA for each (request, KV head): the
// weights as integers in their order in shared memory, the smallest kept one found digit by
// digit from histograms (radix selection: 11, 11 and 10 bits; once few share the first digit,
// among those alone), then the kept slots and their weights written in order.
// evict_move_kernel: the rows.  A kept row never moves up, so in place is safe if a row is
// read before its slot is written: slots are taken in order, a chunk is read whole before any
// of it is written, and the next chunk is read before that too (its rows lie above every slot
// of this one).  Columns of a row have nothing to do with
// one another: where (request, KV head) pairs are few their columns go to CTAs of their own.
// Where that leaves SMs idle, a cluster of CTAs takes a run of slots, or of rows, each: the
// histograms meet in the first one's shared memory, and a chunk is read by all before any of
// it is written.
//
// Measured: 64 requests of 4096 16-bit keys, 8 KV heads, to 2048: selection 29 us (bound by its
// instructions), move 163 (HBM, 6.2 TB/s).  32 of 8192 4-bit keys to 4096: 27 and 69; the scales'
// rows of 8 bytes leave most of their sectors unused.  One pair of 32000 keys: 43 in all, with
// one CTA for each part 205.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "e2m1.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace attn {
namespace {

struct EvictParams {
    uint8_t* cache;
    uint8_t* scales;
    float* weights;
    const int *block_table, *lens;
    int *new_lens, *kept;
    unsigned* status;
    PageDivider page;
    int B, Hkv, max_pages, num_blocks, keep, recent;
    int held;  // weights a CTA of the first kernel has room for
    bool fours;  // four slots from a multiple of four on are 16 aligned bytes of weights
};

constexpr int kMaxRanks = 8;  // CTAs of a cluster
constexpr int kSelectThreads = 512;  // (256 with five CTAs an SM: 122 us instead of 114 for 32 x 8192 4-bit keys)
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
// Weights in shared memory; of longer requests those behind are read again.  The table's width
// sizes them, whatever the requests' lengths; from some 23,700 on one CTA has an SM to itself.
// (With at most 23,680 there is always room for two: 64 requests of 30,000 4-bit keys, 8 KV heads,
// D 64, took 499 us instead of 516 and 64 of 4096 in tables as wide 89.7 instead of 91.5, but 64 of
// 16,000 304 instead of 294, and 32 of 24,000, which are then read twice, 221 instead of 183.)
constexpr int kMaxHeld = 24576;
constexpr int kPages = 1024;     // pages whose places are
constexpr int kList = 1024;      // keys that share the first digit, if they are so few
constexpr int kFew = 64;         // so few are compared with one another
constexpr int kBatch = 4;        // weights of a thread read at a time

// Integers in the order of the weights: -0 as 0, NaN under everything.
__device__ __forceinline__ uint32_t ordered(uint32_t raw) {
    const uint32_t u = __float_as_uint(__uint_as_float(raw) + 0.0f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The weight of a key (not of -0 and NaN, which are not told apart).
__device__ __forceinline__ uint32_t weight_of(uint32_t key) { return (key & 0x80000000u) ? key ^ 0x80000000u : ~key; }

// The CTAs that share a unit: a cluster.
template <bool kCluster>
struct Team {
    const int ranks, rank;
    __device__ __forceinline__ void sync() const {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // Shared memory of another CTA of the cluster, at this CTA's address.
    static __device__ __forceinline__ uint32_t of(const void* p, int rank) {
        uint32_t r;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
        return r;
    }
    static __device__ __forceinline__ int read(const int* p, int rank) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(of(p, rank)) : "memory");
        return v;
    }
    static __device__ __forceinline__ void write(uint32_t* p, int rank, uint32_t v) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(of(p, rank)), "r"(v) : "memory");
    }
    static __device__ __forceinline__ int add(int* p, int rank, int v) {
        int old;
        asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(of(p, rank)), "r"(v) : "memory");
        return old;
    }
};

// One CTA (which the runtime form costs 4% of a long eviction of many).
template <>
struct Team<false> {
    static constexpr int ranks = 1, rank = 0;
    __device__ __forceinline__ Team(int, int) {}
    __device__ __forceinline__ void sync() const { __syncthreads(); }
    static __device__ __forceinline__ int read(const int* p, int) { return *p; }
    static __device__ __forceinline__ void write(uint32_t* p, int, uint32_t v) { *p = v; }
    static __device__ __forceinline__ int add(int* p, int, int v) { return atomicAdd(p, v); }
};

// A request's slots; len: 0 if out of range (reported by the first kernel), so that it is left out.
struct Slots {
    const EvictParams& p;
    const int* table;
    int len;
    __device__ __forceinline__ Slots(const EvictParams& params, int b, bool report)
        : p(params), table(params.block_table + static_cast<int64_t>(b) * params.max_pages) {
        const int n = p.lens[b], most = p.max_pages * p.page.size;
        len = n < 0 || n > most ? 0 : n;
        if (report && len != n) atomicOr(p.status, ATTN_DEV_BAD_INPUT);
    }
    // Block of a page; -1 (reported) if its id is outside the pool.
    __device__ __forceinline__ int block(int page) const {
        const int id = table[page];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) return id;
        atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        return -1;
    }
};

// What the ranks of a unit agree on, in the first one's shared memory.
struct Agreed {
    int digit, above, found, count, odd;
};

template <bool kCluster>
__global__ void __launch_bounds__(kSelectThreads, 3) evict_select_kernel(const EvictParams p, int all_ranks) {
    extern __shared__ __align__(16) uint32_t s_key[];  // [held], of this rank's slots
    __shared__ __align__(16) int s_bin[kBins];
    __shared__ int64_t s_page[kPages];  // first weight of a page; negative: none
    __shared__ uint32_t s_list[kList];
    __shared__ int s_warp[kSelectWarps][2];
    __shared__ int s_total[2];
    __shared__ Agreed s_agreed;
    grid_wait();
    grid_launch_next();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const Team<kCluster> team{all_ranks, static_cast<int>(blockIdx.x) % all_ranks};
    const int ranks = team.ranks;
    const bool lead = team.rank == 0;
    const long long units = static_cast<long long>(p.B) * p.Hkv;
    for (long long unit = blockIdx.x / ranks; unit < units; unit += gridDim.x / ranks) {
        const int b = static_cast<int>(unit / p.Hkv), hkv = static_cast<int>(unit % p.Hkv);
        const Slots slots(p, b, hkv == 0 && lead && tid == 0);
        int* kept = p.kept + unit * p.keep;
        if (hkv == 0 && lead && tid == 0) p.new_lens[b] = min(slots.len, p.keep);
        if (slots.len <= p.keep) {
            if (lead)
                for (int i = tid; i < p.keep; i += kSelectThreads) kept[i] = i < slots.len ? i : -1;
            continue;
        }
        const int n = slots.len - p.recent, want = p.keep - p.recent;  // candidates, those of them kept
        // This rank's slots, and the candidates and held weights among them.
        constexpr int kStep = 128;
        const int per = ((slots.len + ranks - 1) / ranks + kStep - 1) / kStep * kStep;
        const int lo = static_cast<int>(min(static_cast<long long>(slots.len), static_cast<long long>(team.rank) * per));
        const int hi = lo + min(slots.len - lo, per), last = max(lo, min(hi, n)), held = lo + min(hi - lo, p.held);
        const int pages = p.page.quotient(slots.len - 1) + 1;
        auto page_at = [&](int page) -> int64_t {
            const int id = slots.block(page);
            return id < 0 ? -1 : (static_cast<int64_t>(id) * p.Hkv + hkv) * p.page.size;
        };
        __syncthreads();  // the unit before has been read
        for (int i = tid; i < min(pages, kPages); i += kSelectThreads) s_page[i] = page_at(i);
        for (int i = tid; i < kBins; i += kSelectThreads) s_bin[i] = 0;
        if (tid == 0) s_agreed.count = s_agreed.odd = 0;
        team.sync();
        auto at = [&](int slot) -> float* {
            int row;
            const int page = p.page.split(slot, &row);
            const int64_t first = page < kPages ? s_page[page] : page_at(page);
            return first < 0 ? nullptr : p.weights + first + row;
        };
        auto load = [&](int slot) {  // a weight's bits; of a bad block NaN's
            const float* w = at(slot);
            return w ? __float_as_uint(*w) : 0x7fffffffu;
        };
        // The weights, and the first digit's histogram.
        bool odd = false;
        auto look = [&](int i, uint32_t raw) {  // the key of slot i's weight
            odd |= raw == 0x80000000u || (raw & 0x7fffffffu) > 0x7f800000u;
            const uint32_t k = ordered(raw);
            if (i < n) atomicAdd(&s_bin[k >> 21], 1);
            return k;
        };
        if (p.fours) {  // four at a time, here and at the end: 110 us instead of 114 for 32 x 8192 4-bit keys to 4096
            constexpr int kAhead = 2;
            for (int i0 = lo + 4 * tid; i0 < held; i0 += kAhead * 4 * kSelectThreads) {
                uint4 raw[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const float* from = i0 + u * 4 * kSelectThreads < held ? at(i0 + u * 4 * kSelectThreads) : nullptr;
                    raw[u] = from ? *reinterpret_cast<const uint4*>(from)
                                  : make_uint4(0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 0x7fffffffu);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * 4 * kSelectThreads;
                    if (i >= held) break;
                    uint4 k = raw[u];
                    k.x = look(i, k.x);
                    if (i + 1 < held) k.y = look(i + 1, k.y);
                    if (i + 2 < held) k.z = look(i + 2, k.z);
                    if (i + 3 < held) k.w = look(i + 3, k.w);
                    *reinterpret_cast<uint4*>(s_key + (i - lo)) = k;
                }
            }
        } else {
            for (int i0 = lo + tid; i0 < held; i0 += kBatch * kSelectThreads) {
                uint32_t raw[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    raw[u] = i0 + u * kSelectThreads < held ? load(i0 + u * kSelectThreads) : 0u;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kSelectThreads;
                    if (i < held) s_key[i - lo] = look(i, raw[u]);
                }
            }
        }
        for (int i = held + tid; i < last; i += kSelectThreads) atomicAdd(&s_bin[ordered(load(i)) >> 21], 1);
        if (odd || hi > held) team.add(&s_agreed.odd, 0, 1);  // not all at hand, or not as they are
        // Keys i .. i + 3 (i - lo a multiple of 4; those from `last` on are not to be looked at).
        auto keys = [&](int i) {
            if (i + 3 < held) return *reinterpret_cast<const uint4*>(s_key + (i - lo));
            uint32_t k[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) k[u] = i + u < held ? s_key[i + u - lo] : i + u < last ? ordered(load(i + u)) : 0u;
            return make_uint4(k[0], k[1], k[2], k[3]);
        };

        // The key of the last kept one, from the highest digit on: `left` of those that share
        // the digits so far are kept.
        uint32_t prefix = 0;
        int left = want;
        for (int shift = 32, bits = 11; shift > 0 && want > 0; shift -= bits, bits = shift < 11 ? shift : 11) {
            const int low = shift - bits;
            const uint32_t mask = (1u << bits) - 1;
            bool few = false;  // the first rank goes on alone
            if (shift < 32) {
                for (int i = tid; i < kBins; i += kSelectThreads) s_bin[i] = 0;
                if (shift == 21)  // those with the first digit, if they are few, to the first rank
                    for (int i = lo + 4 * tid; i < last; i += 4 * kSelectThreads) {
                        const uint4 k = keys(i);
                        const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (i + u < last && (v[u] >> 21) == prefix) {
                                const int place = team.add(&s_agreed.count, 0, 1);
                                if (place < kList) team.write(&s_list[place], 0, v[u]);
                            }
                    }
                team.sync();
                const int some = team.read(&s_agreed.count, 0);
                few = some <= kList;
                if (some <= kFew) {  // each counts those over it
                    if (lead && tid < some) {
                        const uint32_t own = s_list[tid];
                        int greater = 0, same = 0;
                        for (int i = 0; i < some; ++i) {
                            greater += s_list[i] > own;
                            same += s_list[i] == own;
                        }
                        if (greater < left && left <= greater + same) {  // the same key and count in each that is it
                            s_agreed.found = static_cast<int>(own);
                            s_agreed.above = greater;
                        }
                    }
                    team.sync();
                    prefix = static_cast<uint32_t>(team.read(&s_agreed.found, 0));
                    left -= team.read(&s_agreed.above, 0);
                    break;
                }
                if (few) {
                    if (lead)
                        for (int i = tid; i < some; i += kSelectThreads)
                            if ((s_list[i] >> shift) == prefix) atomicAdd(&s_bin[s_list[i] >> low & mask], 1);
                } else {
                    for (int i = lo + 4 * tid; i < last; i += 4 * kSelectThreads) {
                        const uint4 k = keys(i);
                        const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (i + u < last && (v[u] >> shift) == prefix) atomicAdd(&s_bin[v[u] >> low & mask], 1);
                    }
                }
            }
            if (ranks > 1 && !few) {  // all histograms into the first rank's
                team.sync();
                if (!lead)
                    for (int i = tid; i < kBins; i += kSelectThreads)
                        if (s_bin[i] > 0) team.add(&s_bin[i], 0, s_bin[i]);
            }
            team.sync();
            if (lead) {
                // Thread i has bins kPer i and on; counts from the top bin down.
                constexpr int kPer = kBins / kSelectThreads;
                int mine[kPer], own = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) own += mine[i] = s_bin[tid * kPer + i];
                int above = own;  // in this and all higher lanes, then warps
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_down_sync(0xffffffffu, above, o);
                    if (lane + o < 32) above += x;
                }
                if (lane == 0) s_warp[warp][0] = above;
                __syncthreads();
                for (int i = warp + 1; i < kSelectWarps; ++i) above += s_warp[i][0];
                above -= own;
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i) {
                    if (above < left && left <= above + mine[i]) {
                        s_agreed.digit = tid * kPer + i;
                        s_agreed.above = above;
                    }
                    above += mine[i];
                }
            }
            team.sync();
            prefix = prefix << bits | static_cast<uint32_t>(team.read(&s_agreed.digit, 0));
            left -= team.read(&s_agreed.above, 0);
        }

        // Kept slots in order: a warp has a run of them, four to a lane at a time, and counts first.
        const int run = (last - lo + kSelectWarps * kStep - 1) / (kSelectWarps * kStep) * kStep;
        const int from = min(last, lo + warp * run), to = min(last, from + run);
        int over = 0, equal = 0;
        for (int i = from + 4 * lane; i < to; i += kStep) {
            const uint4 k = keys(i);
            const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                over += i + u < to && v[u] > prefix;
                equal += i + u < to && v[u] == prefix;
            }
        }
        over = __reduce_add_sync(0xffffffffu, over);
        equal = __reduce_add_sync(0xffffffffu, equal);
        __syncthreads();  // s_warp has been read
        if (lane == 0) {
            s_warp[warp][0] = over;
            s_warp[warp][1] = equal;
        }
        __syncthreads();
        over = equal = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            if (i == warp && lane == 0 && warp == kSelectWarps - 1) {
                s_total[0] = over + s_warp[i][0];
                s_total[1] = equal + s_warp[i][1];
            }
            if (i >= warp) continue;
            over += s_warp[i][0];
            equal += s_warp[i][1];
        }
        team.sync();  // and every rank's weights have been read
        for (int i = 0; i < team.rank; ++i) {
            over += team.read(&s_total[0], i);
            equal += team.read(&s_total[1], i);
        }
        // With all weights at hand they are written as their slots are found.
        const bool whole = team.read(&s_agreed.odd, 0) == 0;
        auto place = [&](int slot, uint32_t raw) {
            float* w = at(slot);
            if (w) *w = __uint_as_float(raw);
        };
        if (want > 0)
            for (int i0 = from; i0 < to; i0 += kStep) {
                const int i = i0 + 4 * lane;
                const uint4 k = i < to ? keys(i) : make_uint4(0, 0, 0, 0);
                const uint32_t v[4] = {k.x, k.y, k.z, k.w};
                int mine = 0;  // over in the low half, equal in the high one
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i + u < to) mine += v[u] > prefix ? 1 : v[u] == prefix ? 1 << 16 : 0;
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                const int all = __shfl_sync(0xffffffffu, incl, 31), before = incl - mine;
                int o = over + (before & 0xffff), e = equal + (before >> 16);  // in front of this lane's
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i + u >= to) break;
                    const bool is_over = v[u] > prefix, is_equal = v[u] == prefix;
                    if (is_over || (is_equal && e < left)) {  // of equal ones the lowest stay
                        const int place_at = o + min(e, left);
                        kept[place_at] = i + u;
                        if (whole) place(place_at, weight_of(v[u]));
                    }
                    o += is_over;
                    e += is_equal;
                }
                over += all & 0xffff;
                equal += all >> 16;
            }
        for (int i = max(n, lo) + tid; i < hi; i += kSelectThreads) {  // the recent ones
            kept[want + i - n] = i;
            if (whole) place(want + i - n, weight_of(s_key[i - lo]));
        }
        if (!whole) {  // the weights follow as the rows do, by the first rank
            team.sync();
            if (lead) {
                for (int i0 = 0; i0 < p.keep; i0 += kSelectThreads) {
                    const int i = i0 + tid;
                    const float* old = i < p.keep ? at(kept[i]) : nullptr;  // null: the row stays too
                    const uint32_t raw = old ? __float_as_uint(*old) : 0u;
                    __syncthreads();
                    if (old) place(i, raw);
                }
            }
            team.sync();
        }
        // Nothing from `keep` on is read again.
        const int gone = max(p.keep, lo);
        if (p.fours) {
#pragma unroll 2
            for (int i = (gone & ~3) + 4 * tid; i < hi; i += 4 * kSelectThreads) {
                float* w = at(i);
                if (!w) continue;
                if (i >= gone && i + 3 < hi) {
                    *reinterpret_cast<uint4*>(w) = make_uint4(0, 0, 0, 0);
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i + u >= gone && i + u < hi) w[u] = 0.0f;
                }
            }
        } else {
#pragma unroll 4
            for (int i = gone + tid; i < hi; i += kSelectThreads) place(i, 0u);
        }
        if (ranks > 1) team.sync();  // the first rank's memory has been read
    }
}

constexpr int kMoveThreads = 256;
// Pieces of a thread in a chunk; two chunks are in flight.  A warp's lanes find the places of a row
// each, so of small rows a chunk has no more.  (Four of those too, two rows to a lane: 3 us less
// for one head of 4000 keys of 16 bits, but 4-bit rows take 10 to 20% longer.)
template <int kPieces>
constexpr int kDepthOf = kPieces < 4 ? kPieces : 4;

// Moves one column range of the kept rows of (request, KV head, K or V): pieces of T, kPieces to a
// row, at byte `first` of rows of row_bytes.  A warp's lanes find the places of its rows of a
// chunk, a row each, and hand them round.
template <typename T, int kPieces, typename Team>
__device__ __forceinline__ void move_rows(const EvictParams& p, uint8_t* base, int row_bytes, int first,
                                          const Slots& slots, const int* kept, int side, int hkv, const Team& team) {
    constexpr int kMoveDepth = kDepthOf<kPieces>;
    constexpr int kStep = 32 / kPieces, kRows = kMoveThreads / kPieces;  // rows of a warp, of the CTA, at a time
    constexpr int kChunk = kRows * kMoveDepth, kOwn = kStep * kMoveDepth;  // rows of the CTA's and the warp's chunk
    static_assert(kOwn <= 32, "a lane a row");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, piece = lane % kPieces;
    // Row `slot` in the pool of rows; negative: none.
    auto row_of = [&](int slot) -> int64_t {
        int row;
        const int id = slots.block(p.page.split(slot, &row));
        return id < 0 ? -1 : ((static_cast<int64_t>(id) * 2 + side) * p.Hkv + hkv) * p.page.size + row;
    };
    auto at = [&](int64_t row) { return reinterpret_cast<T*>(base + row * row_bytes + first) + piece; };
    T v[2][kMoveDepth];
    int64_t to[2][kMoveDepth];  // negative: the row stays, or has no place
    auto load = [&](int i0, T (&x)[kMoveDepth], int64_t (&dst)[kMoveDepth]) {
        const int i = i0 + lane / kStep * kRows + warp * kStep + lane % kStep;
        const int slot = lane < kOwn && i < p.keep ? kept[i] : i;
        int64_t src_row = -1, dst_row = -1;
        if (slot != i) {
            src_row = row_of(slot);
            dst_row = row_of(i);
            if (src_row < 0) dst_row = -1;
        }
#pragma unroll
        for (int u = 0; u < kMoveDepth; ++u) {
            const int r = u * kStep + lane / kPieces;
            const int64_t src = __shfl_sync(0xffffffffu, src_row, r);
            dst[u] = __shfl_sync(0xffffffffu, dst_row, r);
            if (dst[u] >= 0) x[u] = *at(src);
        }
    };
    auto store = [&](const T (&x)[kMoveDepth], const int64_t (&dst)[kMoveDepth]) {
#pragma unroll
        for (int u = 0; u < kMoveDepth; ++u)
            if (dst[u] >= 0) *at(dst[u]) = x[u];
    };
    // Each rank has a chunk of its own of the cluster's.
    const int step = team.ranks * kChunk, own = team.rank * kChunk;
    load(own, v[0], to[0]);
    for (int i0 = 0; i0 < p.keep; i0 += 2 * step) {
        if (i0 + step < p.keep) load(i0 + step + own, v[1], to[1]);
        team.sync();
        store(v[0], to[0]);
        if (i0 + step >= p.keep) break;
        if (i0 + 2 * step < p.keep) load(i0 + 2 * step + own, v[0], to[0]);
        team.sync();
        store(v[1], to[1]);
    }
}

// Block (x, y): unit y of (request, KV head), rank x % ranks of part x / ranks: sides times column
// ranges, then sides of the scales.
template <int kRowBytes, int kScaleBytes, int kRanges, bool kCluster>
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const EvictParams p, int ranks) {
    grid_wait();
    grid_launch_next();
    for (long long unit = blockIdx.y; unit < static_cast<long long>(p.B) * p.Hkv; unit += gridDim.y) {
        const int b = static_cast<int>(unit / p.Hkv), hkv = static_cast<int>(unit % p.Hkv);
        const Slots slots(p, b, false);
        if (slots.len <= p.keep) continue;
        const int* kept = p.kept + unit * p.keep;
        const Team<kCluster> team{ranks, static_cast<int>(blockIdx.x) % ranks};
        const int part = static_cast<int>(blockIdx.x) / team.ranks, side = part % 2;
        constexpr int kBytes = kRowBytes / kRanges;
        if (part < 2 * kRanges)
            move_rows<uint4, kBytes / 16>(p, p.cache, kRowBytes, part / 2 * kBytes, slots, kept, side, hkv, team);
        else if constexpr (kScaleBytes == 8)
            move_rows<uint2, 1>(p, p.scales, 8, 0, slots, kept, side, hkv, team);
        else if constexpr (kScaleBytes == 4)
            move_rows<uint32_t, 1>(p, p.scales, 4, 0, slots, kept, side, hkv, team);
    }
}

// Column ranges of 32 bytes and more, a power of two of them, until there are two CTAs for an SM (64
// pairs of 16000 16-bit keys: 165 us instead of 262 with whole rows, one pair of 32000 46 instead of 97).
template <int kRowBytes, int kScaleBytes, int kRanges = 1>
cudaError_t launch_move(const EvictParams& p, const LaunchEnv& env, int* grid_out) {
    const long long units = static_cast<long long>(p.B) * p.Hkv;
    if constexpr (kRanges * 32 < kRowBytes)
        if (2 * kRanges * units < 2ll * env.num_sms)
            return launch_move<kRowBytes, kScaleBytes, 2 * kRanges>(p, env, grid_out);
    const int parts = 2 * kRanges + (kScaleBytes ? 2 : 0);
    int ranks = 1;
    if constexpr (kRanges * 32 >= kRowBytes)  // until the SMs have two CTAs each, or a rank 512 rows
        while (ranks < kMaxRanks && 2 * ranks * parts * units <= 2ll * env.num_sms && p.keep > 512 * ranks) ranks *= 2;
    const dim3 grid(parts * ranks, static_cast<unsigned>(std::min(units, 65535ll)));
    *grid_out = static_cast<int>(grid.x * grid.y);
    if constexpr (kRanges * 32 >= kRowBytes)
        if (ranks > 1)
            return launch_serial_clusters(evict_move_kernel<kRowBytes, kScaleBytes, kRanges, true>, grid, kMoveThreads,
                                          0, ranks, env.stream, p, ranks);
    return launch_serial(evict_move_kernel<kRowBytes, kScaleBytes, kRanges, false>, grid, kMoveThreads, 0, env.stream,
                         p, 1);
}

}  // namespace

cudaError_t launch_evict_paged(const EvictShape& s, const LaunchEnv& env, int* grid_out, int* kernels_launched) {
    EvictParams p{};
    p.cache = static_cast<uint8_t*>(s.cache);
    p.scales = s.scales;
    p.weights = s.weights;
    p.block_table = s.block_table;
    p.lens = s.seq_lens;
    p.new_lens = s.new_lens;
    p.kept = s.kept;
    p.status = env.status;
    p.page = PageDivider(s.page);
    p.B = s.B;
    p.Hkv = s.Hkv;
    p.max_pages = s.max_pages;
    p.num_blocks = s.num_blocks;
    p.keep = s.keep;
    p.recent = s.recent;
    p.fours = s.page % 4 == 0 && reinterpret_cast<uintptr_t>(s.weights) % 16 == 0;
    static bool attr_set[64] = {};  // device < 64 (device_env)
    cudaError_t e = cudaSuccess;
    if (!attr_set[env.device]) {
        for (auto* kernel : {evict_select_kernel<false>, evict_select_kernel<true>}) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 4);
            if (e != cudaSuccess) return e;
        }
        attr_set[env.device] = true;
    }
    const long long units = static_cast<long long>(s.B) * s.Hkv, keys = static_cast<long long>(s.max_pages) * s.page;
    // With one CTA for each pair 8 pairs of 8000 4-bit keys took 41 us, with clusters 31; 16-bit ones
    // 43 both; at up to 4096 keys clusters lose 2 us, and so they do where SMs have work already.
    int ranks = 1;  // of tables wider than 4096: until the SMs have a CTA each, or a rank 2048 slots
    while (keys > 4096 && ranks < kMaxRanks && 2 * ranks * units <= env.num_sms && keys > 2048 * ranks) ranks *= 2;
    const long long per = ((keys + ranks - 1) / ranks + 127) / 128 * 128;
    p.held = static_cast<int>(std::min<long long>(per, kMaxHeld));
    const long long clusters = std::min(units, 0x7fffffffll / ranks);
    auto* select = ranks > 1 ? evict_select_kernel<true> : evict_select_kernel<false>;
    e = launch_serial_clusters(select, dim3(static_cast<unsigned>(clusters * ranks)), kSelectThreads,
                               static_cast<size_t>(p.held) * 4, ranks, env.stream, p, ranks);
    if (e != cudaSuccess) return e;
    *kernels_launched = 2;
    if (s.scales) return s.D == 64 ? launch_move<32, 4>(p, env, grid_out) : launch_move<64, 8>(p, env, grid_out);
    return s.D == 64 ? launch_move<128, 0>(p, env, grid_out) : launch_move<256, 0>(p, env, grid_out);
}

}  // namespace attn
