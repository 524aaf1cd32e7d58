"""The matrix optimizer's rules on sizes (zero1_muon_tiles.h, host-only C++),
compiled with g++ for the tests: which launch a matrix gets, the tile width of
a list, and the rule's estimate of an iteration's time."""
from __future__ import annotations

import functools
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_adamw_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <vector>
#include "zero1_muon_tiles.h"
int main() {
    int sms; unsigned n;
    while (std::scanf("%d %u", &sms, &n) == 2) {
        std::vector<uint32_t> r, c;
        int small = -1;
        for (unsigned i = 0; i < n; ++i) {
            unsigned a, b;
            if (std::scanf("%u %u", &a, &b) != 2) return 1;
            const int q = zero1::small_blocks(std::min(a, b), std::max(a, b));
            if (q >= 0) small = q; else r.push_back(a), c.push_back(b);
        }
        const auto sides = [&](size_t i, uint32_t &a, uint32_t &b) { a = r[i], b = c[i]; };
        uint64_t gram = 0, full = 0;
        const uint32_t t = zero1::tile_columns(r.size(), sides, sms);
        for (size_t i = 0; i < r.size(); ++i) gram += zero1::tiles_of(r[i], c[i], t).gram, full += zero1::tiles_of(r[i], c[i], t).full;
        std::printf("%d %zu %u %.6f %.6f %llu %llu\n", small, r.size(), t, zero1::iteration_us(r.size(), sides, 128, sms / 2),
                    zero1::iteration_us(r.size(), sides, 256, sms / 2), (unsigned long long)gram, (unsigned long long)full);
    }
    return 0;
}
"""


@functools.cache
def driver() -> str:
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    d = tempfile.mkdtemp(prefix="muon_tiles")
    src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
    with open(src, "w") as f:
        f.write(DRIVER)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, src, "-o", exe], check=True)
    return exe


def rules(shapes, sms: int = 152):
    """(log2 of the blocks of the last small matrix or -1, tiled matrices, tile
    columns, estimated us an iteration at 128 and 256 columns, Gram tiles, full tiles)."""
    stdin = f"{sms} {len(shapes)} " + " ".join(f"{r} {c}" for r, c in shapes) + "\n"
    out = subprocess.run([driver()], input=stdin, capture_output=True, text=True, check=True).stdout.split()
    return int(out[0]), int(out[1]), int(out[2]), float(out[3]), float(out[4]), int(out[5]), int(out[6])


def small_blocks(rows: int, cols: int) -> int:
    """Blocks of the single launch that steps this matrix, or 0 if it is tiled."""
    q = rules([(rows, cols)])[0]
    return 1 << q if q >= 0 else 0


def tile_columns(shapes, sms: int = 152) -> int:
    return rules(shapes, sms)[2]
