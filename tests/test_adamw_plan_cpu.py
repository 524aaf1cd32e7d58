"""The list step's host-only rules (zero1_adamw_plan.h), compiled with g++."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_adamw_gb300", "csrc")

PARTIALS = r"""
#include <cstdio>
#include <vector>
#include "zero1_adamw_plan.h"
int main() {
    unsigned long long sms, count;
    while (std::scanf("%llu %llu", &sms, &count) == 2) {
        std::vector<uint64_t> first(1, 0);
        for (unsigned long long i = 0, n; i < count; ++i) {
            if (std::scanf("%llu", &n) != 1) return 1;
            first.push_back(first.back() + (n + zero1::kListBlock - 1) / zero1::kListBlock);
        }
        // as a step's launches write them: the highest place that one of them takes
        unsigned cap = zero1::kCaps[2];
        for (int c : zero1::kCaps) if (count <= (unsigned long long)c) { cap = c; break; }
        uint64_t before = 0, launches = 0;
        for (uint64_t i = 0; i < count; i += cap) {
            const uint64_t end = std::min<uint64_t>(i + cap, count);
            const uint32_t grid = zero1::norm_grid(first[end] - first[i], end == count, (int)sms);
            before += grid;
            launches += grid > 0;
        }
        std::printf("%llu %llu %llu\n", (unsigned long long)zero1::norm_partials(first.data(), count, zero1::kCaps[2], (int)sms),
                    (unsigned long long)before, (unsigned long long)launches);
    }
    return 0;
}
"""


def compiled(tmp_path_factory, name, source):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp(name)
    src, exe = d / f"{name}.cpp", d / name
    src.write_text(source)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


@pytest.fixture(scope="module")
def partials(tmp_path_factory):
    exe = compiled(tmp_path_factory, "partials", PARTIALS)

    def run(sizes, sms=152):
        r = subprocess.run([exe], input=f"{sms} {len(sizes)} " + " ".join(map(str, sizes)), capture_output=True, text=True, check=True)
        return tuple(int(v) for v in r.stdout.split())
    return run


@pytest.mark.parametrize("sizes,launches", [
    ([300], 1), ([0, 5, 0], 1), ([1] * 32, 1), ([1] * 33, 1), ([70000] * 257, 1), ([256] * 1600, 1), ([256] * 1601, 2),
    ([300] + [0] * 2000, 2),                       # the last launch has no tensor with entries
    ([6400] * 1600 + [0] * 1600, 2),               # ... after one of 608 partial sums, a multiple of 32
    ([6400] * 1600 + [0], 2),
    ([0] * 1600 + [6400] * 1600, 1),               # ... the first has none
    ([6400] * 1600 + [0] * 1600 + [9], 2), ([6400] * 1600 + [0] * 3200, 2), ([256 * 64] * 1600 + [0] * 1600, 2),
])
@pytest.mark.parametrize("sms", [152, 148, 1])
def test_every_partial_sum_of_the_norm_has_its_place(partials, sizes, launches, sms):
    held, written, n = partials(sizes, sms)
    assert written <= held and n == launches
    assert held == written    # and none is waste
