"""The page division that the kernels use (csrc/attn_internal.h), compiled for the host and
run over the borders of its divisors and numerators."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "attn_internal.h"
#include <cstdio>
#include <vector>
int main() {
    const long long top = 0x7fffffffll;
    std::vector<long long> sizes;
    for (long long d = 1; d <= 300; ++d) sizes.push_back(d);
    for (int b = 8; b <= 30; ++b)
        for (long long o = -2; o <= 2; ++o) sizes.push_back((1ll << b) + o);
    for (long long d : {641ll, 6700417ll, 1000000007ll, top - 1025, top - 1, top}) sizes.push_back(d);
    unsigned seed = 1;
    for (long long d : sizes) {
        const attn::PageDivider by(static_cast<int>(d));
        std::vector<long long> ns = {0, 1, 2, d - 1, d, d + 1, top - 1, top};
        for (long long q : {1ll, 2ll, 3ll, 1000ll, top / d, top / d - 1, top / (2 * d)})
            for (long long o = -1; o <= 1; ++o) ns.push_back(q * d + o);
        for (int i = 0; i < 2000; ++i) {
            seed = seed * 1664525u + 1013904223u;
            ns.push_back(seed >> 1);
        }
        for (long long n : ns) {
            if (n < 0 || n > top) continue;
            int rest = 0;
            const int q = by.split(static_cast<int>(n), &rest);
            if (q != n / d || rest != n % d) {
                std::printf("%lld / %lld: %d rest %d\n", n, d, q, rest);
                return 1;
            }
        }
    }
    return 0;
}
"""


def test_the_kernels_page_division_is_exact(tmp_path):
    from transformer_attention_fwd_gb300 import build
    if not shutil.which("g++"):
        pytest.skip("g++ not found")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    (tmp_path / "d.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "d")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, "-isystem", os.path.join(cuda, "include"),
                    str(tmp_path / "d.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
