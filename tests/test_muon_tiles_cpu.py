"""The matrix optimizer's rules on sizes against enumeration and against
times measured on GB300."""
from __future__ import annotations

import math

import pytest

from tests.muon_tiles import rules, small_blocks, tile_columns

BLOCK = [(768, 2304), (768, 768), (768, 3072), (3072, 768)]
# (list, us of one iteration measured with tiles of 128 columns, of 256)
MEASURED = [
    ([(768, 768)], 43.7, 61.1), ([(768, 768)] * 3, 46.2, 62.8), ([(768, 768)] * 6, 52.0, 64.5),
    ([(768, 768)] * 9, 61.9, 71.1), ([(768, 768)] * 12, 72.7, 77.0), ([(768, 768)] * 16, 91.5, 86.5),
    ([(768, 768)] * 24, 137.3, 103.0), ([(1031, 257)] * 3, 38.4, 54.4), ([(1031, 257)] * 12, 46.5, 60.9),
    ([(1031, 257)] * 40, 90.1, 91.9), (BLOCK, 80.2, 97.4), (BLOCK * 2, 116.5, 113.9), (BLOCK * 3, 165.8, 134.0),
    (BLOCK * 4, 216.2, 161.4), (BLOCK * 12, 681.5, 462.3), ([(1024, 1024)], 60.4, 82.8), ([(1024, 1024)] * 4, 62.9, 75.4),
    ([(1024, 1024)] * 8, 97.4, 90.2), ([(1536, 1536)], 69.4, 92.2), ([(1792, 1792)], 95.4, 102.6),
    ([(2048, 2048)], 108.8, 113.3), ([(2304, 2304)], 187.1, 152.1), ([(2560, 2560)], 209.6, 168.3),
    ([(3840, 3840)], 613.8, 426.2), ([(4096, 4096)], 712.4, 519.1), ([(4096, 16384)], 2267.3, 1548.8),
    ([(1024, 4096)], 98.2, 111.3), ([(1024, 4096)] * 2, 106.9, 118.2), ([(1024, 4096)] * 4, 160.8, 144.3),
    ([(1280, 5120)], 127.9, 147.1), ([(300, 517)] * 20, 44.5, 56.1), ([(300, 517)] * 40, 63.5, 69.7),
    ([(300, 517)] * 60, 90.6, 86.8), ([(300, 517)] * 80, 118.8, 107.3), ([(300, 517)] * 120, 181.3, 162.8),
    ([(256, 4096)], 65.4, 89.0), ([(256, 16384)], 190.2, 242.9), ([(512, 512)] * 16, 49.5, 56.2),
    ([(512, 512)] * 32, 66.1, 75.7), ([(512, 512)] * 64, 132.9, 101.2), ([(160, 2000)] * 30, 70.1, 74.9),
    ([(160, 2000)] * 80, 149.5, 116.9), ([(2304, 768)] * 8, 112.3, 107.5), ([(130, 130)] * 100, 40.3, 46.5),
    ([(130, 130)] * 300, 119.4, 91.1),
]


@pytest.mark.parametrize("shapes,narrow,wide", MEASURED)
def test_width_is_the_faster_one_measured(shapes, narrow, wide):
    _, tiled, width, t128, t256, _, _ = rules(shapes)
    assert tiled == len(shapes)
    assert width == (128 if narrow <= wide else 256)
    assert abs(math.log(t128 / narrow)) <= math.log(1.28) and abs(math.log(t256 / wide)) <= math.log(1.28)


@pytest.mark.parametrize("s", [1, 17, 128])
def test_single_launch_bounds(s):
    for l, blocks in ((s, 1), (256, 1), (257, 2), (384, 2), (385, 4), (768, 4), (769, 8), (1536, 8), (1537, 0)):
        assert small_blocks(s, l) == blocks and small_blocks(l, s) == blocks
    assert small_blocks(129, 129) == 0


@pytest.mark.parametrize("rows,cols", [(129, 129), (256, 300), (257, 1031), (1031, 257), (513, 770), (2305, 2311), (130, 5000)])
@pytest.mark.parametrize("copies", [1, 400])
def test_tiles_cover_each_product_once(rows, cols, copies):
    _, _, width, _, _, gram, full = rules([(rows, cols)] * copies)
    s = min(rows, cols)
    want = sum(1 for r in range(0, s, 256) for c in range(0, s, width) if c // 256 >= r // 256)
    assert gram == copies * want
    assert full == copies * math.ceil(rows / 256) * math.ceil(cols / width)


def test_fewer_sms_widen_tiles_sooner():
    assert tile_columns([(768, 768)] * 3) == 128 and tile_columns([(768, 768)] * 3, 16) == 256
