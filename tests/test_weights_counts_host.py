"""How the sums of attention weights are cut into work (csrc/weights_counts.h), compiled for
the host and compared with counts that cannot wrap."""
import os
import shutil
import subprocess

import pytest

PROLOGUE = r"""
#include "weights_counts.h"
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>
using namespace attn;
typedef long long ll;
std::mt19937_64 gen(7);
ll uniform(ll lo, ll hi) { return lo + static_cast<ll>(gen() % static_cast<unsigned long long>(hi - lo + 1)); }
// Spread over the logarithm.
ll spread(ll hi) { return std::min(hi, std::max<ll>(1, uniform(1, 1ll << uniform(1, 62 - __builtin_clzll(hi))))); }
"""

PLACES = PROLOGUE + r"""
int main() {
    int left_out = 0, with_places = 0;
    for (int round = 0; round < 3000; ++round) {
        const int total = static_cast<int>(round < 200 ? uniform(1, 3000) : spread(1 << 28));
        const ll keys = total + uniform(0, 5000);
        const WeightsRanges r = weights_ranges(total, static_cast<int>(spread(64)), keys);
        const int B = static_cast<int>(uniform(1, 700));
        const bool ordered = round % 3 == 0;
        std::vector<ll> cu(B + 1);
        for (auto& x : cu) x = round % 3 == 1 ? (uniform(0, 1) ? total : 0) : uniform(-3, total + 3ll);
        if (ordered) {
            for (auto& x : cu) x = std::min<ll>(std::max<ll>(x, 0), total);
            std::sort(cu.begin(), cu.end());
        }
        // As the kernels count: 32 requests at a time, and by 256 threads.
        std::vector<int> own(B);
        for (int b = 0; b < B; ++b) {
            const bool ok = cu[b] >= 0 && cu[b] <= cu[b + 1] && cu[b + 1] <= total;
            own[b] = ok ? r.of(static_cast<int>(cu[b + 1] - cu[b])) : 0;
            const ll n = ok ? cu[b + 1] - cu[b] : 0, ranges = (n + (1ll << r.shift) - 1) >> r.shift;
            if (own[b] != (ranges > 1 ? ranges : 0)) return std::printf("%lld tokens: %d places\n", n, own[b]), 1;
        }
        int base = 0;
        ll exact = 0;
        for (int first = 0; first < B; first += 32) {
            int slots = 0;
            for (int b = first; b < std::min(B, first + 32); ++b) {
                const int before = slots;
                slots += own[b];
                const bool fits = r.fits(base + slots), should = exact + own[b] <= r.places;
                if (own[b] > 0) {
                    ++with_places;
                    left_out += !fits;
                    if (fits != should || (ordered && !fits)) return std::printf("request %d of %d\n", b, B), 1;
                    if (fits && (base + before < 0 || base + before + own[b] > r.places)) return std::printf("place\n"), 1;
                    int parts[256] = {}, sum = 0;
                    for (int i = 0; i < b; ++i) parts[i % 256] = WeightsRanges::add(parts[i % 256], own[i]);
                    for (int w = 0; w < 8; ++w) {
                        int of_warp = 0;
                        for (int i = 0; i < 32; ++i) of_warp += parts[w * 32 + i];
                        sum += WeightsRanges::add(0, of_warp);
                    }
                    if (r.fits(sum + own[b]) != fits || (fits && sum != base + before)) return std::printf("second kernel\n"), 1;
                }
                exact += own[b];
            }
            base = WeightsRanges::add(base, slots);
        }
    }
    // Both kinds came up.
    return left_out > 1000 && with_places - left_out > 1000 ? 0 : (std::printf("%d of %d\n", left_out, with_places), 1);
}
"""

COLUMNS = PROLOGUE + r"""
int main() {
    const ll top = 0x7fffffffll - 1024;
    for (int i = 0; i < 2000000; ++i) {
        const int group = static_cast<int>(uniform(1, 128));
        const ll past = i % 2 ? uniform(0, top) : spread(top);
        // Any earlier key, and those of an item from `past` on.
        const ll key = i % 3 ? uniform(0, past) : std::min(top + 511, past + uniform(0, 511));
        const ll want = std::max<ll>(0, (key - past) * group);
        const int got = weights_first_column(static_cast<int>(key), static_cast<int>(past), group);
        if (got != want) return std::printf("key %lld, past %lld, group %d: %d\n", key, past, group, got), 1;
    }
    return 0;
}
"""

SHIFTS = PROLOGUE + r"""
int main() {
    const ll top = 0x7fffffffll - 1024;
    bool far = false;
    for (int i = 0; i < 300000; ++i) {
        const ll total = i % 2 ? spread(top) : uniform(1, top), Hkv = i % 3 ? 1 : spread(64), group = spread(128);
        if (weights_tile_tokens(static_cast<int>(total), static_cast<int>(group), 1) == 0) continue;
        const ll keys = std::max(total, spread(top));
        const WeightsRanges r = weights_ranges(static_cast<int>(total), static_cast<int>(Hkv), keys);
        far |= r.shift == 30;
        if (r.shift > 30 || 1 << r.shift != 1ll << r.shift || r.places >= WeightsRanges::kMany) return 1;
        // A request of n tokens has its last range's end, and its count of ranges, in 31 bits.
        for (ll n : {1ll, total / 2 + 1, total - 1, total}) {
            if (n < 1) continue;
            const ll ranges = (n + (1ll << r.shift) - 1) >> r.shift;
            if (r.of(static_cast<int>(n)) != (ranges > 1 ? ranges : 0) || ((n - 1) >> r.shift << r.shift) + (1ll << r.shift) > 0x7fffffffll ||
                r.of(static_cast<int>(n)) > r.places)
                return std::printf("%lld of %lld tokens, %lld keys: shift %d\n", n, total, keys, r.shift), 1;
        }
    }
    return far ? 0 : 2;
}
"""

ROWS = PROLOGUE + r"""
int main() {
    const ll top = 0x7fffffffll - 1024;
    for (int i = 0; i < 2000000; ++i) {
        const ll group = spread(1 << 20), most = top / group, n = i % 2 ? most : uniform(1, most);
        const ll len = std::min(top, n + (i % 3 ? uniform(0, top - n) : uniform(0, 40)));
        const ll key = i % 5 ? uniform(0, len - 1) : len - 1 + uniform(0, 31);
        const ll token = std::max<ll>(0, key - (len - n));
        const int got = weights_first_row(static_cast<int>(key), static_cast<int>(len), static_cast<int>(n), static_cast<int>(group));
        if (got != std::min(token, n) * group)
            return std::printf("key %lld of %lld, %lld tokens, group %lld: %d\n", key, len, n, group, got), 1;
    }
    return 0;
}
"""


def run(tmp_path, program):
    from transformer_attention_fwd_gb300 import build
    if not shutil.which("g++"):
        pytest.skip("g++ not found")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    (tmp_path / "w.cpp").write_text(program)
    exe = str(tmp_path / "w")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", build.CSRC, "-isystem",
                    os.path.join(cuda, "include"), str(tmp_path / "w.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_no_place_is_past_those_allocated(tmp_path):
    """Offsets in order or not: a request has places within the workspace or is left out, by
    both kernels alike."""
    run(tmp_path, PLACES)


def test_first_columns_of_long_contexts(tmp_path):
    """Up to 2^31 keys and 128 heads, against 64 bits."""
    run(tmp_path, COLUMNS)


def test_ranges_stay_in_31_bits(tmp_path):
    """Of as many tokens as the tiles take."""
    run(tmp_path, SHIFTS)


def test_first_rows_of_many_heads(tmp_path):
    """As many rows as a call may have, and the places of a chunk behind the last key."""
    run(tmp_path, ROWS)
