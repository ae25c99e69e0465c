// weights_tiles.cu -- attention weights of packed queries added up over the keys of a
// paged cache (weights.cu has the formula), on the 5th-generation tensor cores.
//
// S^T tiles of 128 keys (tensor-memory lanes) by 128 query rows (columns): a thread of
// the sum warps owns a key and adds 2^(x - lse) over the columns, so nothing crosses
// lanes, the probabilities never leave registers and each key's sum has a fixed order.
//
// A work item is 256 keys of one (request, KV head) with the queries that see them, at
// most `range` tokens of them; a CTA per SM walks the items of all requests in a fixed
// order.  A key's sums from several ranges go to a workspace, and a second kernel adds
// them up in order.  Warps:
//   0-15   sums: eight warps take the even query tiles, eight the odd ones; of each eight,
//          four have keys 0-127 of the item and four keys 128-255.  (Eight in all left the
//          tensor cores waiting.)  At an item's end the second eight hand their sums over.
//   16     query tiles by TMA: whole tokens, a KV head's query heads within, read straight
//          out of the caller's tensor (a box of 64 elements x heads x tokens)
//   17     tensor memory, and all MMAs: for each query tile one 128 x 128 x D product for
//          each half of the keys, into one of two accumulators each
//   18     the rows' -lse into shared memory
//   19     the items: their place in the requests takes some 1400 cycles to find, which
//          every warp by itself spent at every item (a window's period was 5800 cycles)
//   20 on  K rows into one of two buffers.  16-bit pages of 8 .. 256 rows (a power of two)
//          by TMA, other 16-bit rows by asynchronous 16-byte copies, 4-bit rows converted in
//          registers (a code times its scale has six significant bits: exact in either
//          16-bit type), by four warps or eight
// Every wait is bounded (sm100.cuh).
//
// What bounds it: a 128 x 128 x 16 product takes 67 cycles and reads 8 KB, all that shared memory
// gives, so the products of a 4096-token prompt (32 + 8 heads, D 128, 4-bit keys) take 65 us (a pair
// of CTAs with half of the queries each would read half), the sums alone 68: their 268 M
// exponentials would take 28 at 32 a clock and SM, but a sum warp reads 32 columns of tensor memory,
// waits, and only then adds.  Both together 77 to 80 (floor by operations 36); windows of 64 tokens
// over 16 requests of 4096 16-bit keys 42 to 46 (floor by bytes 21).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "e2m1.cuh"
#include "pdl.cuh"
#include "prefill_common.cuh"
#include "sm100.cuh"
#include "weights.cuh"
#include "weights_counts.h"

namespace attn {
namespace {

using prefill::desc_advance;
using prefill::kDrainLimitNs;
using prefill::wait_quiet;
using prefill::warp_wait;

constexpr int kKeyShift = kWeightsKeyShift, kKeys = 1 << kKeyShift;  // of an item
constexpr int kHalf = 128;  // keys of an MMA
constexpr int kCols = kWeightsCols;  // query rows of a tile
// Items: the lse warp is four tiles ahead, so four items where they have one tile each (with four
// places windows of 64 tokens over 16 x 4096 4-bit keys took 61.7 us instead of 60.3).
constexpr int kQStages = 3, kKStages = 2, kSBufs = 2, kItems = 5;
constexpr int kSumWarps = 16, kRowWarps = 4;
constexpr int kQWarp = kSumWarps, kMmaWarp = kQWarp + 1, kLseWarp = kMmaWarp + 1, kItemWarp = kLseWarp + 1;
constexpr int kLoadWarp0 = kItemWarp + 1;
// How an item's keys arrive, and the warps for it.
enum KeyLoads { kPages, kRows16, kRows4, kRows4More };
template <int kLoads>
constexpr int kLoadWarps = kLoads == kPages ? 1 : kLoads == kRows4More ? 2 * kRowWarps : kRowWarps;
template <int kLoads>
constexpr int kThreads = (kLoadWarp0 + kLoadWarps<kLoads>) * 32;
constexpr uint32_t kTmemCols = 512;

enum : unsigned {
    SITE_W_K_EMPTY = 48, SITE_W_K_FULL, SITE_W_Q_EMPTY, SITE_W_Q_FULL, SITE_W_L_EMPTY, SITE_W_L_FULL,
    SITE_W_S_EMPTY, SITE_W_S_FULL, SITE_W_X_EMPTY, SITE_W_X_FULL, SITE_W_I_EMPTY,
    SITE_W_I_FULL
};

struct Item {  // b < 0: the end
    int b, hkv, begin, n;
    int len, key0;  // keys of the request; the item's first
    int t0, t1;     // tokens of the item, counted from the request's first query
    int slot;       // of the partial sums; -1: none
};
struct alignas(16) ItemPlace {  // all but the slot
    int4 request, keys;
};

struct Control {
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t q_full[kQStages], q_empty[kQStages];
    uint64_t l_full[kQStages], l_empty[kQStages];
    uint64_t s_full[2][kSBufs], s_empty[2][kSBufs];  // [half of the keys]
    uint64_t x_full[2], x_empty[2];                  // sums handed over
    uint64_t i_full[kItems], i_empty[kItems];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    alignas(16) float nlse[kQStages][kCols];  // -log2(e) lse of a tile's rows; +inf: adds nothing
    float handed[kKeys];
    ItemPlace items[kItems];
    int item_slots[kItems];
    int rows[kQStages];  // of a tile that add something
};

template <int D>
struct Layout {
    static constexpr int kTile = kHalf * D * 2;  // 128 rows: D / 64 boxes of 128 rows x 128 bytes
    static constexpr int kK = 0;
    static constexpr int kQ = kK + kKStages * 2 * kTile;
    static constexpr int kControl = kQ + kQStages * kTile;
    static constexpr int kBytes = kControl + static_cast<int>(sizeof(Control));
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct TilesParams {
    WeightsParams w;
    float* partial;       // [ranges.places, Hkv, keys] sums of ranges, or null: no request has several
    long long keys;       // max_pages * page
    WeightsRanges ranges;
    int tile_tokens;      // tokens of a query tile
    unsigned long long limit_ns;
};

// Blocks of keys that all n queries see, all blocks, and the items of one KV head: block kb has
// range_count() of them.  The last n - ... keys are seen by fewer queries block by block:
// their counts, from the last block on, are floor(j / m) + 1 with m = range / kKeys.
struct Counts {
    int blocks, flat, ranges, shift;  // m = 1 << shift
    __device__ __forceinline__ Counts(const TilesParams& p, int len, int n) : shift(p.ranges.shift - kKeyShift) {
        blocks = (len + kKeys - 1) >> kKeyShift;
        flat = min(blocks, ((len - n) >> kKeyShift) + 1);
        ranges = (n + (1 << p.ranges.shift) - 1) >> p.ranges.shift;
    }
    // Items of the last j blocks.  (Items of a head fit in 31 bits: range_of().)
    __device__ __forceinline__ int tail(int j) const {
        const unsigned a = static_cast<unsigned>(j) >> shift, c = j - (a << shift);
        return j + static_cast<int>(((a * (a - 1) / 2) << shift) + a * c);
    }
    __device__ __forceinline__ int items() const { return flat * ranges + tail(blocks - flat); }
    // Item i: its block and range.
    __device__ __forceinline__ void find(int i, int* kb, int* r) const {
        if (i < flat * ranges) {
            *kb = ranges == 1 ? i : static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(ranges));
            *r = i - *kb * ranges;
            return;
        }
        i -= flat * ranges;
        int lo = 0, hi = blocks - flat - 1;  // the last j with tail(j) <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tail(mid) <= i) lo = mid; else hi = mid - 1;
        }
        *kb = blocks - 1 - lo;
        *r = i - tail(lo);
    }
};

// This CTA's items one after the other, by a whole warp.  32 requests are looked at at a time,
// a lane each.
struct Finder {
    const TilesParams& p;
    const int lane;
    long long next, base = 0, incl = 0, chunk = 0;  // items before the lanes' requests; their prefix; all of them
    int first = -32, begin = 0, n = 0, len = 0, slots = 0, slot_base = 0;
    __device__ __forceinline__ Finder(const TilesParams& params, int lane_id)
        : p(params), lane(lane_id), next(blockIdx.x) {}

    __device__ __forceinline__ void look() {
        base += chunk;
        slot_base = WeightsRanges::add(slot_base, __shfl_sync(0xffffffffu, slots, 31));
        first += 32;
        const int b = first + lane;
        bool ok = true;
        n = 0;
        if (b < p.w.B) {
            const WeightsRequest r = weights_request(p.w, b);
            begin = r.begin;
            n = r.ok ? r.end - r.begin : 0;
            len = r.len;
            ok = r.ok;
        }
        const int own_slots = p.ranges.of(n);
        slots = own_slots;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, slots, o);
            if (lane >= o) slots += x;
        }
        if (own_slots > 0 && !p.ranges.fits(slot_base + slots)) {  // (weights_ranges_kernel leaves it out too)
            n = 0;
            ok = false;
        }
        if (!ok && blockIdx.x == 0) atomicOr(p.w.status, ATTN_DEV_BAD_INPUT);
        incl = n > 0 ? static_cast<long long>(Counts(p, len, n).items()) * p.w.Hkv : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        chunk = __shfl_sync(0xffffffffu, incl, 31);
    }
    __device__ __forceinline__ bool take(Item& it) {
        while (next - base >= chunk) {
            if (first + 32 >= p.w.B) return false;
            look();
        }
        const int at = __popc(__ballot_sync(0xffffffffu, incl <= next - base));  // the request's lane
        const long long before = __shfl_sync(0xffffffffu, incl, max(at - 1, 0));
        const int slots_before = __shfl_sync(0xffffffffu, slots, max(at - 1, 0));
        it.b = first + at;
        it.begin = __shfl_sync(0xffffffffu, begin, at);
        it.n = __shfl_sync(0xffffffffu, n, at);
        it.len = __shfl_sync(0xffffffffu, len, at);
        const Counts c(p, it.len, it.n);
        const long long i = next - base - (at > 0 ? before : 0);
        const int per = c.items();
        it.hkv = (i >> 31) == 0 ? static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(per)) : static_cast<int>(i / per);
        int kb, r;
        c.find(static_cast<int>(i - static_cast<long long>(it.hkv) * per), &kb, &r);
        it.key0 = kb << kKeyShift;
        it.t0 = max(0, it.key0 - (it.len - it.n)) + (r << p.ranges.shift);
        it.t1 = min(it.n, it.t0 + (1 << p.ranges.shift));
        it.slot = c.ranges > 1 ? slot_base + (at > 0 ? slots_before : 0) + r : -1;
        next += gridDim.x;
        return true;
    }
};

// The items as the other warps take them from the item warp; every call by a whole warp.
struct Items {
    Control* ctl;
    const int lane;
    const WaitGuard& g;
    uint32_t i_it = 0;
    __device__ __forceinline__ Items(Control* control, int lane_id, const WaitGuard& guard)
        : ctl(control), lane(lane_id), g(guard) {}
    // kVote: not in the MMA warp (warp_wait says why).
    template <bool kVote = true>
    __device__ __forceinline__ bool take(Item& it) {
        const uint32_t s = i_it % kItems;
        bool ok = warp_wait(&ctl->i_full[s], (i_it / kItems) & 1, g, SITE_W_I_FULL);
        if (kVote) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const int4 x = ctl->items[s].request, y = ctl->items[s].keys;
        it.slot = ctl->item_slots[s];
        it.b = x.x; it.hkv = x.y; it.begin = x.z; it.n = x.w;
        it.len = y.x; it.key0 = y.y; it.t0 = y.z; it.t1 = y.w;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->i_empty[s]);
        ++i_it;
        return it.b >= 0;
    }
};

__device__ void find_items(const TilesParams& p, Control* ctl, int lane, const WaitGuard& g) {
    Finder finder(p, lane);
    bool more = true;
    for (uint32_t i_it = 0; more; ++i_it) {
        Item it{};
        more = finder.take(it);
        if (!more) it.b = -1;
        const uint32_t s = i_it % kItems;
        if (i_it >= kItems &&
            !__all_sync(0xffffffffu, mbar_wait(&ctl->i_empty[s], ((i_it / kItems) & 1) ^ 1, g, SITE_W_I_EMPTY)))
            return;
        if (lane == 0) {
            ctl->items[s].request = make_int4(it.b, it.hkv, it.begin, it.n);
            ctl->items[s].keys = make_int4(it.len, it.key0, it.t0, it.t1);
            ctl->item_slots[s] = it.slot;
            mbar_arrive(&ctl->i_full[s]);
        }
        __syncwarp();
    }
}

// 64 keys of an item for one of four warps: two lanes' worth of slots, looked up ahead.
struct RowIds {
    int64_t row[2];  // of keys lane and lane + 32 in the pool of rows; negative: none
    __device__ __forceinline__ void find(const WeightsParams& p, const Item& it, int first, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = first + lane + 32 * i;
            row[i] = -1;
            if (key >= it.len) continue;
            int in_page;
            const int id = p.block_table[static_cast<int64_t>(it.b) * p.max_pages + p.page.split(key, &in_page)];
            if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks))
                row[i] = (static_cast<int64_t>(id) * 2 * p.Hkv + it.hkv) * p.page.size + in_page;
            else
                atomicOr(p.status, ATTN_DEV_BAD_INPUT);
        }
    }
    // Of key i of the 64.
    __device__ __forceinline__ int64_t of(int i) const {
        const int64_t a = __shfl_sync(0xffffffffu, row[0], i & 31), b = __shfl_sync(0xffffffffu, row[1], i & 31);
        return i < 32 ? a : b;
    }
};

// Byte of 16-byte chunk c of key k in a K buffer: 128-byte rows, swizzled by the row.
template <int D>
__device__ __forceinline__ uint32_t key_chunk(int k, int c) {
    return static_cast<uint32_t>((k / kHalf) * Layout<D>::kTile + (c >> 3) * (kHalf * 128) + (k % kHalf) * 128 +
                                 (((c & 7) ^ (k & 7)) << 4));
}

// Pages by TMA: a box of up to 128 rows x 64 elements.  Rows past the request's last key are
// other slots' or stale: they are lanes that nobody adds up.
template <int D>
__device__ void load_pages(const TilesParams& p, const CUtensorMap* tmK, uint8_t* smem, Control* ctl, int lane,
                           const WaitGuard& g) {
    const int page = p.w.page.size, rows = min(page, kHalf), boxes = kKeys / rows;  // boxes of an item, up to 32
    Items items(ctl, lane, g);
    Item it;
    bool more = items.take(it);
    auto look_up = [&]() {  // this lane's box; -1: none
        const int key = it.key0 + lane * rows;
        return more && lane < boxes && key < it.len
                   ? p.w.block_table[static_cast<int64_t>(it.b) * p.w.max_pages + p.w.page.quotient(key)] : -1;
    };
    int id = look_up();
    uint32_t k_it = 0;
    bool ok = true;
    while (more) {
        const uint32_t s = k_it % kKStages;
        if (k_it >= kKStages) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl->k_empty[s], ((k_it / kKStages) & 1) ^ 1, g, SITE_W_K_EMPTY));
            if (!ok) break;
        }
        const bool have = lane < boxes && it.key0 + lane * rows < it.len;
        const bool good = have && static_cast<unsigned>(id) < static_cast<unsigned>(p.w.num_blocks);
        if (have && !good) atomicOr(p.w.status, ATTN_DEV_BAD_INPUT);
        const unsigned there = __ballot_sync(0xffffffffu, good);
        if (lane == 0)
            mbar_arrive_expect_tx(&ctl->k_full[s], static_cast<uint32_t>(__popc(there)) * rows * D * 2);
        __syncwarp();
        if (good) {
            uint8_t* to = smem + Layout<D>::kK + s * 2 * Layout<D>::kTile + (lane * rows / kHalf) * Layout<D>::kTile +
                          (lane * rows % kHalf) * 128;
            const int slab = id * 2 * p.w.Hkv + it.hkv;  // fits (the host checks)
            const int row = lane * rows % page;          // pages of 256 rows are two boxes
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_3d(to + h * (kHalf * 128), tmK, &ctl->k_full[s], h * 64, row, slab);
        }
        ++k_it;
        more = items.take(it);
        id = look_up();
    }
    // Copies in flight land before the CTA leaves.
    if (lane == 0)
        for (uint32_t i = k_it > kKStages ? k_it - kKStages : 0; i < k_it; ++i)
            wait_quiet(&ctl->k_full[i % kKStages], (i / kKStages) & 1, kDrainLimitNs);
}

template <int D>
__device__ void load_rows16(const TilesParams& p, uint8_t* smem, Control* ctl, int warp, int lane, const WaitGuard& g) {
    constexpr int kPer = D / 8;           // chunks of a row
    constexpr int kRowsPer = 32 / kPer;   // rows of a warp's copy
    const uint32_t buffers = smem_u32(smem + Layout<D>::kK);
    const int c = lane % kPer;
    Items items(ctl, lane, g);
    Item it;
    uint32_t k_it = 0;
    bool waiting = false;  // the copies before have not been handed over
    auto hand_over = [&](uint32_t n) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->k_full[n % kKStages]);
    };
    while (items.take(it)) {
        RowIds ids;
        ids.find(p.w, it, it.key0 + warp * 64, lane);
        const uint32_t s = k_it % kKStages;
        if (k_it >= kKStages) {
            const uint32_t parity = ((k_it / kKStages) & 1) ^ 1;
            if (waiting && !__all_sync(0xffffffffu, mbar_try_wait(&ctl->k_empty[s], parity))) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                hand_over(k_it - 1);
                waiting = false;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&ctl->k_empty[s], parity, g, SITE_W_K_EMPTY))) break;
        }
        const uint32_t to = buffers + s * 2 * Layout<D>::kTile;
#pragma unroll 8
        for (int i = 0; i < 64 / kRowsPer; ++i) {
            const int r = i * kRowsPer + lane / kPer;
            const int64_t row = ids.of(r);
            const uint8_t* src = p.w.cache + (row < 0 ? 0 : row) * (D * 2) + c * 16;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         :: "r"(to + key_chunk<D>(warp * 64 + r, c)), "l"(src), "r"(row < 0 ? 0 : 16) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (waiting) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            hand_over(k_it - 1);
        }
        waiting = true;
        ++k_it;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (waiting) hand_over(k_it - 1);
}

// The next 32 keys' codes are read as a warp's are converted, and the places of those after are
// looked up.
template <int D, bool kF16, int kWarps>
__device__ void load_rows4(const TilesParams& p, uint8_t* smem, Control* ctl, int warp, int lane, const WaitGuard& g) {
    constexpr int kPer = D / 32;         // lanes of a row: 32 elements each
    constexpr int kRowsPer = 32 / kPer;
    constexpr int kSteps = 32 / kRowsPer, kTurns = kKeys / (32 * kWarps);  // of 32 keys a warp, for an item
    uint8_t* buffers = smem + Layout<D>::kK;
    const int part = lane % kPer;
    // Rows of 128 elements: the second half's chunks go out in another order, so that eight
    // lanes' meet no bank twice (key_chunk puts both halves' on the same ones).
    const int swap = part & 2;
    Items items(ctl, lane, g);
    Item it{};
    int turn = 0;  // that is looked up
    auto first = [&](int n) { return (n * kWarps + warp) * 32; };
    auto advance = [&]() {
        if (++turn < kTurns) return true;
        turn = 0;
        return items.take(it);
    };
    auto find = [&]() -> int64_t {  // row of this lane's key in the pool of rows; negative: none
        const int key = it.key0 + first(turn) + lane;
        if (key >= it.len) return -1;
        int in_page;
        const int id = p.w.block_table[static_cast<int64_t>(it.b) * p.w.max_pages + p.w.page.split(key, &in_page)];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.w.num_blocks))
            return (static_cast<int64_t>(id) * 2 * p.w.Hkv + it.hkv) * p.w.page.size + in_page;
        atomicOr(p.w.status, ATTN_DEV_BAD_INPUT);
        return -1;
    };
    uint4 codes[kSteps];
    uint32_t scales[kSteps];
    auto read = [&](int i, int64_t rows) {
        const int64_t row = __shfl_sync(0xffffffffu, rows, i * kRowsPer + lane / kPer);
        codes[i] = make_uint4(0, 0, 0, 0);
        scales[i] = 0;
        if (row >= 0) {
            codes[i] = *reinterpret_cast<const uint4*>(p.w.cache + row * (D / 2) + part * 16);
            scales[i] = *reinterpret_cast<const uint16_t*>(p.w.scales + row * (D / kRowScaleSpan) + part * 2);
        }
    };
    bool more = items.take(it);
    int64_t rows = more ? find() : -1;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) read(i, rows);
    bool next = more && advance();
    rows = next ? find() : -1;
    for (uint32_t n = 0; more; ++n) {
        const uint32_t k_it = n / kTurns, s = k_it % kKStages;
        if (n % kTurns == 0 && k_it >= kKStages &&
            !__all_sync(0xffffffffu, mbar_wait(&ctl->k_empty[s], ((k_it / kKStages) & 1) ^ 1, g, SITE_W_K_EMPTY)))
            return;
        uint8_t* to = buffers + s * 2 * Layout<D>::kTile;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int k = first(n % kTurns) + i * kRowsPer + lane / kPer;
            uint32_t by[2];
            e2m1_scales<kF16>(scales[i], by);
            uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
            if (swap) {
                const uint32_t w0 = w[0], w1 = w[1], by0 = by[0];
                w[0] = w[2]; w[1] = w[3]; by[0] = by[1];
                w[2] = w0; w[3] = w1; by[1] = by0;
            }
            read(i, rows);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[4];
                e2m1_to_f16x8(w[j], v);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = e2m1_times<kF16>(v[x], by[j / 2]);
                *reinterpret_cast<uint4*>(to + key_chunk<D>(k, part * 4 + (j ^ swap))) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        if (n % kTurns == kTurns - 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->k_full[s]);
        }
        more = next;
        next = more && advance();
        rows = next ? find() : -1;
    }
}

template <int D>
__device__ void load_queries(const TilesParams& p, const CUtensorMap* tmQ, uint8_t* smem, Control* ctl, int lane,
                             const WaitGuard& g) {
    const uint32_t bytes = static_cast<uint32_t>(p.tile_tokens * p.w.group) * D * 2;
    Items items(ctl, lane, g);
    Item it;
    uint32_t q_it = 0;
    bool ok = true;
    while (ok && items.take(it)) {
        for (int t = it.t0; t < it.t1; t += p.tile_tokens, ++q_it) {
            const uint32_t s = q_it % kQStages;
            if (q_it >= kQStages) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl->q_empty[s], ((q_it / kQStages) & 1) ^ 1, g, SITE_W_Q_EMPTY));
                if (!ok) break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&ctl->q_full[s], bytes);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(smem + Layout<D>::kQ + s * Layout<D>::kTile + h * (kCols * 128), tmQ, &ctl->q_full[s],
                                h * 64, it.hkv * p.w.group, it.begin + t);
            }
        }
    }
    // Copies in flight land before the CTA leaves (they have, but for an abort elsewhere).
    if (lane == 0)
        for (uint32_t i = q_it > kQStages ? q_it - kQStages : 0; i < q_it; ++i)
            wait_quiet(&ctl->q_full[i % kQStages], (i / kQStages) & 1, kDrainLimitNs);
}

__device__ void load_lse(const TilesParams& p, Control* ctl, int lane, const WaitGuard& g) {
    constexpr int kOwn = kCols / 32;
    const WeightsParams& w = p.w;
    // This lane's rows of a tile: lane, lane + 32, ..
    int token[kOwn];
    long long head_at[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int row = lane + 32 * i;
        token[i] = row / w.group;
        head_at[i] = (row - token[i] * w.group) * w.lse_head;
        if (token[i] >= p.tile_tokens) token[i] = 1 << 30;  // no row
    }
    // The next kAhead tiles' values are on their way in registers (one tile ahead, a tile took the
    // reads' latency: 30 us of a prompt's 77).  A tile's are handed over before the next are asked
    // for, so that a wait for another item holds up nothing that the item before needs.
    constexpr int kAhead = 4;
    Items items(ctl, lane, g);
    Item it{};
    bool more = items.take(it);
    int t = it.t0;
    float v[kAhead][kOwn];
    bool there[kAhead];
    auto ask = [&](float (&x)[kOwn]) -> bool {  // the next tile's values; false: there is none
        if (!more) return false;
        const float* from = w.lse + it.hkv * w.group * w.lse_head + (it.begin + t) * w.lse_token;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) x[i] = token[i] < it.t1 - t ? from[head_at[i] + token[i] * w.lse_token] : -INFINITY;
        t += p.tile_tokens;
        if (t >= it.t1) {
            more = items.take(it);
            t = it.t0;
        }
        return true;
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) there[a] = ask(v[a]);
    uint32_t l_it = 0;
    while (there[0]) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a, ++l_it) {
            if (!there[a]) return;
            const uint32_t s = l_it % kQStages;
            if (l_it >= kQStages &&
                !__all_sync(0xffffffffu, mbar_wait(&ctl->l_empty[s], ((l_it / kQStages) & 1) ^ 1, g, SITE_W_L_EMPTY)))
                return;
            int rows = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const float nl = -v[a][i] * kWeightsLog2e;
                ctl->nlse[s][lane + 32 * i] = nl;
                // A row that saw nothing (-inf) is as no row, whatever its scores are.
                rows += __popc(__ballot_sync(0xffffffffu, nl != INFINITY));
            }
            if (lane == 0) ctl->rows[s] = rows;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->l_full[s]);
            there[a] = ask(v[a]);
        }
    }
}

// S[tmem cols] = keys . queries^T: M = 128, N as idesc has it, K = D in steps of 16.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint64_t kd, uint64_t qd, uint32_t idesc, uint32_t leader) {
    constexpr int kSteps = D / 16;
    uint64_t a[kSteps], b[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const uint32_t off16 = static_cast<uint32_t>(((i / 4) * (kHalf * 128) + (i % 4) * 32) >> 4);
        a[i] = desc_advance(kd, off16);
        b[i] = desc_advance(qd, off16);
    }
    if constexpr (kSteps == 8) mma_bf16_ss_x8(d_tmem, a, b, idesc, 0u, leader);
    else mma_bf16_ss_x4(d_tmem, a, b, idesc, 0u, leader);
}

template <int D, bool kF16>
__device__ void issue_mmas(const TilesParams& p, uint8_t* smem, Control* ctl, uint32_t tmem, int lane,
                           const WaitGuard& g) {
    constexpr uint32_t kTile16 = Layout<D>::kTile >> 4;
    const uint64_t k0 = smem_desc_sw128(smem_u32(smem + Layout<D>::kK), 16, 1024);
    const uint64_t q0 = smem_desc_sw128(smem_u32(smem + Layout<D>::kQ), 16, 1024);
    const uint32_t leader = elect_leader();
    // Columns for a tile's rows, a multiple of 16.
    const int cols = (p.tile_tokens * p.w.group + 15) & ~15;
    const uint32_t idesc = mma_idesc_bf16_f32(kHalf, 16, false, false, kF16) + ((static_cast<uint32_t>(cols) >> 3) - 2u << 17);
    Items items(ctl, lane, g);
    Item it;
    uint32_t k_it = 0, q_it = 0, uses[2][kSBufs] = {};
    bool ok = true;
    while (ok && items.take<false>(it)) {
        const uint32_t ks = k_it % kKStages;
        const int halves = it.key0 + kHalf < it.len ? 2 : 1;
        ok = warp_wait(&ctl->k_full[ks], (k_it / kKStages) & 1, g, SITE_W_K_FULL);
        for (int t = it.t0; ok && t < it.t1; t += p.tile_tokens, ++q_it) {
            const uint32_t qs = q_it % kQStages;
            ok = warp_wait(&ctl->q_full[qs], (q_it / kQStages) & 1, g, SITE_W_Q_FULL);
            const uint32_t buf = q_it & 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!ok || h >= halves) continue;
                const uint32_t used = buf ? uses[h][1] : uses[h][0];
                if (used > 0) ok = warp_wait(&ctl->s_empty[h][buf], (used - 1) & 1, g, SITE_W_S_EMPTY);
                if (!ok) continue;
                tc_fence_after_sync();
                issue_scores<D>(tmem + (h * kSBufs + buf) * kCols, desc_advance(k0, (ks * 2 + h) * kTile16),
                                desc_advance(q0, qs * kTile16), idesc, leader);
                mma_commit(&ctl->s_full[h][buf], leader);
                uses[h][0] += buf ^ 1;
                uses[h][1] += buf;
            }
            mma_commit(&ctl->q_empty[qs], leader);
        }
        mma_commit(&ctl->k_empty[ks], leader);
        ++k_it;
    }
    // Every MMA issued so far is done before tensor memory is released.
    mma_commit(&ctl->drain, leader);
    wait_quiet(&ctl->drain, 0, kDrainLimitNs);
}

// 32 columns of a key: adds 2^(x sc + nl) of all of them.
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const float* nl, uint64_t sc2, uint64_t (&acc)[2]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 l = reinterpret_cast<const float4*>(nl)[i];
        const uint64_t l2[2] = {f2_pack(l.x, l.y), f2_pack(l.z, l.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x, y;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[4 * i + 2 * k]), __uint_as_float(s[4 * i + 2 * k + 1])), sc2, l2[k]),
                      x, y);
            acc[k] = f2_add(acc[k], f2_pack(ex2_approx(x), ex2_approx(y)));
        }
    }
}
// The same of those columns whose bits are set; others may hold anything.
__device__ __forceinline__ float add_some_columns(const uint32_t (&s)[32], const float* nl, float sc, uint32_t bits) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float e = ex2_approx(fmaf(__uint_as_float(s[i]), sc, nl[i]));
        sum += bits >> i & 1 ? e : 0.0f;
    }
    return sum;
}

__device__ void add_up(const TilesParams& p, Control* ctl, uint32_t tmem, int warp, int lane, const WaitGuard& g) {
    const WeightsParams& w = p.w;
    const int set = warp / 8, half = warp / 4 % 2, quarter = warp % 4;
    const uint32_t at = tmem_lane_base(tmem, warp) + (half * kSBufs + set) * kCols;  // the accumulator
    Items items(ctl, lane, g);
    Item it;
    uint32_t l_it = 0, uses = 0, handed = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, g, site)) != 0;
    };
    while (items.take(it)) {
        const int first = it.key0 + half * kHalf, key = first + quarter * 32 + lane;
        if (first >= it.len) {  // no keys in this half: the tiles' rows pass by
            for (int t = it.t0; t < it.t1; t += p.tile_tokens, ++l_it) {
                if ((l_it & 1) != set) continue;
                const uint32_t s = l_it % kQStages;
                if (!wait(&ctl->l_full[s], (l_it / kQStages) & 1, SITE_W_L_FULL)) return;
                if (lane == 0) mbar_arrive(&ctl->l_empty[s]);
            }
            continue;
        }
        // An item of one tile (of a decode step, all are) is one set's alone.
        const bool single = it.t1 - it.t0 <= p.tile_tokens;
        if (single && static_cast<int>(l_it & 1) != set) {
            ++l_it;
            continue;
        }
        int in_page;  // (the id is looked at once the sums are there)
        const int page = w.page.split(min(key, it.len - 1), &in_page);
        const int id = w.block_table[static_cast<int64_t>(it.b) * w.max_pages + page];
        const float sc = w.scale_log2 * (w.factors ? w.factors[it.hkv] : 1.0f);
        const uint64_t sc2 = f2_pack(sc, sc);
        float sum = 0.0f;
        for (int t = it.t0; t < it.t1; t += p.tile_tokens, ++l_it) {
            if ((l_it & 1) != set) continue;
            const uint32_t ls = l_it % kQStages;
            const int valid = min(p.tile_tokens, it.t1 - t) * w.group;
            // Token t sees keys up to len - n + t: this key is seen from column lo on, the warp's
            // first key from lo_warp on.
            const int past = it.len - it.n + t;
            const int lo = weights_first_column(key, past, w.group);
            const int lo_warp = weights_first_column(first + quarter * 32, past, w.group);
            if (!wait(&ctl->l_full[ls], (l_it / kQStages) & 1, SITE_W_L_FULL)) return;
            const bool whole = (first + quarter * 32 + 31 <= past) && (valid & 31) == 0 && ctl->rows[ls] == valid;
            if (!wait(&ctl->s_full[half][set], uses & 1, SITE_W_S_FULL)) return;
            ++uses;
            tc_fence_after_sync();
            const float* nl = ctl->nlse[ls];
            auto read = [&]() {  // the accumulator has been read
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->s_empty[half][set]);
            };
            if (whole) {
                uint64_t acc[2] = {0, 0};
#pragma unroll 1  // (unrolled the loops outgrow the instruction caches: 58 us of a prompt's 124)
                for (int c = 0; c < valid; c += 32) {
                    uint32_t a[32];
                    tmem_ld32(at + c, a);
                    tmem_wait_ld(a);
                    if (c + 32 >= valid) read();
                    add_columns(a, nl + c, sc2, acc);
                }
                float x, y, u, v;
                f2_unpack(acc[0], x, y);
                f2_unpack(acc[1], u, v);
                sum += (x + y) + (u + v);
            } else {
                float part = 0.0f;
#pragma unroll 1
                for (int c = lo_warp & ~31; c < valid; c += 32) {
                    uint32_t a[32];
                    tmem_ld32(at + c, a);
                    tmem_wait_ld(a);
                    const uint32_t bits = __ballot_sync(0xffffffffu, nl[c + lane] != INFINITY);
                    part += add_some_columns(a, nl + c, sc, lo <= c ? bits : lo - c < 32 ? bits & ~0u << (lo - c) : 0u);
                }
                read();
                sum += part;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->l_empty[ls]);
        }
        // The odd tiles' sums to the warps of the even ones.
        const int place = half * kHalf + quarter * 32 + lane;
        if (single) {
        } else if (set == 1) {
            if (handed > 0 && !wait(&ctl->x_empty[half], (handed - 1) & 1, SITE_W_X_EMPTY)) return;
            ctl->handed[place] = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->x_full[half]);
        } else {
            if (!wait(&ctl->x_full[half], handed & 1, SITE_W_X_FULL)) return;
            sum += ctl->handed[place];
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->x_empty[half]);
        }
        handed += !single;
        if ((set == 0 || single) && key < it.len) {
            if (it.slot >= 0)
                p.partial[(static_cast<int64_t>(it.slot) * w.Hkv + it.hkv) * p.keys + key] = sum;
            else if (static_cast<unsigned>(id) < static_cast<unsigned>(w.num_blocks))  // the request's only addition to this key
                atomicAdd(w.weights + (static_cast<int64_t>(id) * w.Hkv + it.hkv) * w.page.size + in_page, sum);
        }
    }
}

template <int D, bool kF16, int kLoads>
__global__ void __launch_bounds__(kThreads<kLoads>, 1)
weights_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ TilesParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle needs it; there is no room for slack
        if (threadIdx.x == 0) atomicOr(p.w.status, ATTN_DEV_BAD_INPUT);
        return;
    }
    Control* ctl = reinterpret_cast<Control*>(smem + Layout<D>::kControl);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&ctl->k_full[i], kLoadWarps<kLoads>);
            mbar_init(&ctl->k_empty[i], 1);
        }
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(&ctl->q_full[i], 1);
            mbar_init(&ctl->q_empty[i], 1);
            mbar_init(&ctl->l_full[i], 1);
            mbar_init(&ctl->l_empty[i], kSumWarps / 2);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&ctl->x_full[h], 4);
            mbar_init(&ctl->x_empty[h], 4);
            for (int i = 0; i < kSBufs; ++i) {
                mbar_init(&ctl->s_full[h][i], 1);
                mbar_init(&ctl->s_empty[h][i], 4);
            }
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ctl->i_full[i], 1);
            mbar_init(&ctl->i_empty[i], kLoadWarp0 - 1 + kLoadWarps<kLoads>);  // all warps but the item warp
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    // Rows of a query tile past its tokens stay zeros.
    for (int i = threadIdx.x; i < kQStages * Layout<D>::kTile / 16; i += kThreads<kLoads>)
        reinterpret_cast<uint4*>(smem + Layout<D>::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == kQWarp && lane == 0) tma_prefetch_desc(&tmQ);
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    const WaitGuard g{p.w.status, &ctl->abort, p.limit_ns};
    grid_wait();
    grid_launch_next();

    if (warp < kSumWarps) {
        add_up(p, ctl, tmem, warp, lane, g);
    } else if (warp == kQWarp) {
        load_queries<D>(p, &tmQ, smem, ctl, lane, g);
    } else if (warp == kMmaWarp) {
        issue_mmas<D, kF16>(p, smem, ctl, tmem, lane, g);
    } else if (warp == kLseWarp) {
        load_lse(p, ctl, lane, g);
    } else if (warp == kItemWarp) {
        find_items(p, ctl, lane, g);
    } else {
        if constexpr (kLoads == kRows4 || kLoads == kRows4More)
            load_rows4<D, kF16, kLoadWarps<kLoads>>(p, smem, ctl, warp - kLoadWarp0, lane, g);
        else if constexpr (kLoads == kRows16) load_rows16<D>(p, smem, ctl, warp - kLoadWarp0, lane, g);
        else load_pages<D>(p, &tmK, smem, ctl, lane, g);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Adds the partial sums of requests with several ranges, in their order.  Block (x, y, z): keys
// of KV heads y, y + gridDim.y, .. of requests z, z + gridDim.z, ..
constexpr int kAddThreads = 256;

__global__ void __launch_bounds__(kAddThreads) weights_ranges_kernel(const __grid_constant__ TilesParams p) {
    __shared__ int s_base[kAddThreads / 32];
    grid_wait();
    grid_launch_next();
    for (int b = blockIdx.z; b < p.w.B; b += gridDim.z) {
        const WeightsRequest r = weights_request(p.w, b);
        const int n = r.ok ? r.end - r.begin : 0;
        const int own = p.ranges.of(n);
        if (own == 0) continue;
        // Slots of the requests before.
        int base = 0;
        for (int i = threadIdx.x; i < b; i += kAddThreads) {
            const WeightsRequest q = weights_request(p.w, i);
            base = WeightsRanges::add(base, p.ranges.of(q.ok ? q.end - q.begin : 0));
        }
        base = WeightsRanges::add(0, __reduce_add_sync(0xffffffffu, base));
        __syncthreads();  // the request before has been read
        if (threadIdx.x % 32 == 0) s_base[threadIdx.x / 32] = base;
        __syncthreads();
        base = 0;
        for (int i = 0; i < kAddThreads / 32; ++i) base += s_base[i];
        if (!p.ranges.fits(base + own)) continue;  // left out and reported
        for (int key = blockIdx.x * kAddThreads + threadIdx.x; key < r.len; key += gridDim.x * kAddThreads) {
            int in_page;
            const int id = p.w.block_table[static_cast<int64_t>(b) * p.w.max_pages + p.w.page.split(key, &in_page)];
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.w.num_blocks)) continue;  // reported
            const int t0 = max(0, (key & -kKeys) - (r.len - n)), ranges = (n - t0 + (1 << p.ranges.shift) - 1) >> p.ranges.shift;
            for (int hkv = blockIdx.y; hkv < p.w.Hkv; hkv += gridDim.y) {
                float sum = 0.0f;
                for (int i = 0; i < ranges; ++i)
                    sum += p.partial[(static_cast<int64_t>(base + i) * p.w.Hkv + hkv) * p.keys + key];
                atomicAdd(p.w.weights + (static_cast<int64_t>(id) * p.w.Hkv + hkv) * p.w.page.size + in_page, sum);
            }
        }
    }
}

WeightsRanges ranges_of(const WeightsShape& s) {
    return weights_ranges(s.total, s.Hkv, static_cast<long long>(s.max_pages) * s.page);
}

template <int D, bool kF16, int kLoads>
cudaError_t launch_tiles(const WeightsMaps& maps, const TilesParams& p, int grid, const LaunchEnv& env) {
    auto* kern = weights_tiles_kernel<D, kF16, kLoads>;
    static bool attr_set[64] = {};  // device < 64 (device_env)
    if (!attr_set[env.device]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[env.device] = true;
    }
    return launch_serial(kern, dim3(grid), kThreads<kLoads>, Layout<D>::kBytes, env.stream, maps.q, maps.k, p);
}

template <int D, int kLoads>
cudaError_t launch_types(const WeightsMaps& maps, const TilesParams& p, bool f16, int grid, const LaunchEnv& env) {
    return f16 ? launch_tiles<D, true, kLoads>(maps, p, grid, env) : launch_tiles<D, false, kLoads>(maps, p, grid, env);
}
template <int D>
cudaError_t launch_loads(const WeightsMaps& maps, const TilesParams& p, bool f16, int loads, int grid, const LaunchEnv& env) {
    if (loads == kRows4) return launch_types<D, kRows4>(maps, p, f16, grid, env);
    if (loads == kRows4More) return launch_types<D, kRows4More>(maps, p, f16, grid, env);
    if (loads == kRows16) return launch_types<D, kRows16>(maps, p, f16, grid, env);
    return launch_types<D, kPages>(maps, p, f16, grid, env);
}

}  // namespace

int weights_tile_tokens(const WeightsShape& s) { return weights_tile_tokens(s.total, s.Hq / s.Hkv, s.B); }

// Pages that boxes cover come by TMA: windows of 64 tokens took 60 us by the warps' copies, 45 so.
int weights_page_rows(const WeightsShape& s) {
    const bool box = s.page >= 8 && s.page <= kKeys && (s.page & (s.page - 1)) == 0;
    const long long slabs = 2ll * s.num_blocks * s.Hkv;
    return !s.scales && box && slabs <= 0x7fffffffll ? std::min(s.page, kHalf) : 0;
}

size_t weights_workspace_bytes(const WeightsShape& s) {
    return 4ull * ranges_of(s).places * s.Hkv * s.max_pages * s.page;
}

cudaError_t launch_weights_tiles(const WeightsShape& s, const WeightsMaps& maps, void* ws, const LaunchEnv& env,
                                 int* grid_out, int* kernels_launched) {
    TilesParams p{};
    p.w = weights_params(s, env);
    p.partial = static_cast<float*>(ws);
    p.keys = static_cast<long long>(s.max_pages) * s.page;
    p.ranges = ranges_of(s);
    p.tile_tokens = weights_tile_tokens(s);
    p.limit_ns = env.wait_limit_ns;
    const int grid = env.num_sms;
    *grid_out = grid;
    *kernels_launched = ws ? 2 : 1;
    // Four warps convert 4-bit rows under the products of many query tiles; where an item has few,
    // eight: 16 rows over 32 x 4096 keys (D 128) 108 us with four, 77 with eight, 512 rows over 16 x 4096
    // 91 and 88, a 4096-token prompt 76 and 79 (eight leave the sums too few registers); D 64, 160
    // rows over 32 x 4096, 82 and 89.
    const bool few = static_cast<long long>(s.total) * p.w.group <= (s.D == 128 ? 4ll : 1ll) * kCols * s.B;
    const int loads = s.scales ? (few ? kRows4More : kRows4) : weights_page_rows(s) > 0 ? kPages : kRows16;
    cudaError_t e = s.D == 64 ? launch_loads<64>(maps, p, s.f16 != 0, loads, grid, env)
                              : launch_loads<128>(maps, p, s.f16 != 0, loads, grid, env);
    if (e != cudaSuccess || !ws) return e;
    const unsigned y = static_cast<unsigned>(std::min(s.Hkv, 65535)), z = static_cast<unsigned>(std::min(s.B, 64));
    const long long want = std::max(1ll, 8ll * env.num_sms / (static_cast<long long>(y) * z));
    const unsigned x = static_cast<unsigned>(std::min(want, (p.keys + kAddThreads - 1) / kAddThreads));
    return launch_serial(weights_ranges_kernel, dim3(x, y, z), kAddThreads, 0, env.stream, p);
}

}  // namespace attn
