"""The list step's host-only rules (zero1_adamw_plan.h), compiled with g++."""
from __future__ import annotations

import os
import random
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


STATE = r"""
#include <cstdio>
#include <vector>
#include "zero1_adamw_plan.h"
int main() {
    unsigned long long count, pb, gb, buffers, a, b, c;
    while (std::scanf("%llu %llu %llu %llu", &count, &pb, &gb, &buffers) == 4) {
        std::vector<uint64_t> sizes;
        std::vector<const void *> grads;
        std::vector<void *> params;
        std::vector<zero1::StateBuffer> state;
        for (unsigned long long i = 0; i < count; ++i) {
            if (std::scanf("%llu %llu %llu", &a, &b, &c) != 3) return 1;
            sizes.push_back(a), params.push_back((void *)b), grads.push_back((const void *)c);
        }
        for (unsigned long long i = 0; i < buffers; ++i) {
            if (std::scanf("%llu %llu", &a, &b) != 2) return 1;
            state.push_back({(const void *)a, b});
        }
        int which = -1;
        bool param = false;
        const size_t i = zero1::tensor_in_state({sizes.data(), sizes.size(), grads.data(), params.data(), gb, pb}, state.data(),
                                                (int)buffers, &which, &param);
        if (i == count) std::printf("none\n");
        else std::printf("%zu %d %d\n", i, which, (int)param);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def state(tmp_path_factory):
    exe = compiled(tmp_path_factory, "state", STATE)

    def run(tensors, buffers, pb=2, gb=2):
        words = [len(tensors), pb, gb, len(buffers)] + [v for t in tensors for v in t] + [v for b in buffers for v in b]
        r = subprocess.run([exe], input=" ".join(map(str, words)), capture_output=True, text=True, check=True)
        return r.stdout.strip()
    return run


@pytest.mark.parametrize("tensors,buffers,answer", [
    # (entries, parameter, gradient); (address, bytes): master, m, v, scales
    ([(100, 4096, 8192)], [(16384, 1024), (32768, 1024)], "none"),
    ([(100, 4096, 8192)], [(4296, 1024), (8192 - 1024, 1024)], "none"),        # ends where the other begins
    ([(100, 4096, 8192)], [(4295, 1024), (32768, 1024)], "0 0 1"),
    ([(100, 4096, 8192)], [(16384, 1024), (4096 - 1023, 1024)], "0 1 1"),
    ([(100, 4096, 8192)], [(16384, 1024), (8391, 1)], "0 1 0"),
    ([(100, 4096, 8192)], [(0, 1 << 40), (8000, 4096)], "0 1 0"),              # a buffer that is not there
    ([(0, 0, 0), (0, 16384, 16384), (7, 4096, 16390)], [(16384, 1024)], "2 0 0"),
    ([(0, 16384, 16384)], [(16384, 1024)], "none"),                            # empty tensors share nothing
    ([(1 << 33, 1 << 40, 1 << 45)], [((1 << 40) + (1 << 34) - 1, 16)], "0 0 1"),
])
def test_tensors_that_share_memory_with_the_state(state, tensors, buffers, answer):
    assert state(tensors, buffers) == answer


SHARED = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>
#include "zero1_adamw_plan.h"
static unsigned long long allocations = 0;
void *operator new(std::size_t n) { ++allocations; if (void *p = std::malloc(n)) return p; throw std::bad_alloc(); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
int main() {
    unsigned long long count, pb, gb, a, b, c;
    while (std::scanf("%llu %llu %llu", &count, &pb, &gb) == 3) {
        std::vector<uint64_t> sizes;
        std::vector<const void *> grads;
        std::vector<void *> params;
        for (unsigned long long i = 0; i < count; ++i) {
            if (std::scanf("%llu %llu %llu", &a, &b, &c) != 3) return 1;
            sizes.push_back(a), params.push_back((void *)b), grads.push_back((const void *)c);
        }
        std::vector<zero1::TensorRange> ranges(2 * count);
        const unsigned long long before = allocations;
        const size_t i = zero1::shared_param({sizes.data(), sizes.size(), grads.data(), params.data(), gb, pb}, ranges.data());
        std::printf("%zu %llu\n", i, allocations - before);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def shared(tmp_path_factory):
    exe = compiled(tmp_path_factory, "shared", SHARED)

    def run(lists, pb, gb):
        words = [v for tensors in lists for v in [len(tensors), pb, gb] + [w for t in tensors for w in t]]
        r = subprocess.run([exe], input=" ".join(map(str, words)), capture_output=True, text=True, check=True)
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    return run


@pytest.mark.parametrize("pb,gb", [(2, 2), (4, 2), (2, 4)])
def test_parameters_that_share_memory_are_found_without_allocating(shared, pb, gb):
    """3,000 lists of up to 40 tensors in any order of addresses, empty ones among them, against every pair."""
    rng = random.Random(pb * 10 + gb)
    lists, expected = [], []
    for _ in range(3000):
        count = rng.choice((1, 2, 3, 8, 40))
        room = rng.choice((60, 600, 6000)) * count
        tensors = [(rng.choice((0, 1, 5, 30)), 4 * rng.randrange(room // 4), 4 * rng.randrange(room // 4)) for _ in range(count)]
        if rng.random() < 0.3:    # each in a place of its own, in a random order
            places = rng.sample(range(2 * count), 2 * count)
            tensors = [(n, 128 * places[2 * i], 128 * places[2 * i + 1]) for i, (n, _, _) in enumerate(tensors)]
        every = [(p, p + n * pb, i, True) for i, (n, p, _) in enumerate(tensors) if n]
        every += [(g, g + n * gb, i, False) for i, (n, _, g) in enumerate(tensors) if n]
        guilty = set()
        for x, a in enumerate(every):
            for b in every[x + 1:]:
                if (a[3] or b[3]) and a[0] < b[1] and b[0] < a[1]:
                    guilty |= {r[2] for r in (a, b) if r[3]}
        lists.append(tensors)
        expected.append((count, guilty))
    answers = shared(lists, pb, gb)
    assert len(answers) == len(lists) and {bool(g) for _, g in expected} == {True, False}
    for (i, allocated), (count, guilty) in zip(answers, expected):
        assert allocated == 0
        assert i in guilty if guilty else i == count
