"""The shapes of test_gpu_fp8_ragged_tilings.py reach every tile of the FP8 expert products (CPU only)."""
import os
import re

from tests import fp8_ragged_tilings as t

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_grouped_amd", "csrc", "fp8_ragged.hip")


def test_rule_names_the_tiles_that_are_written():
    text = re.sub(r"//.*", "", open(SOURCE).read())
    written = re.findall(r"return launch<OP, E8, OUT32, (\d+), (\d+), \d+, \d+(?:, (\d+))?>", text)
    assert {(int(a), int(b)) for a, b, _ in written} == {t.SMALL, t.LOW, t.MIDDLE, t.LARGE}
    assert {(int(a), int(d or 2)) for a, _, d in written} == {(32, 4), (64, 2), (128, 2), (256, 2)}


def test_shapes_reach_every_tile_with_more_than_one_a_workgroup():
    ahead = {t.SMALL: 4, t.LOW: 2, t.MIDDLE: 2, t.LARGE: 2}
    for tile, n in ahead.items():
        steps = {-(-K // 128) for c, N, K in t.PRODUCTS if t.tile("fwd", sum(c), len(c), N, K) == tile and t.rounds("fwd", c, N, K) > 1}
        assert {1, n, n + 1} <= steps, (tile, steps)
    assert {(t.tile("wgrad", sum(c), len(c), N, K), K % 64 == 0) for c, N, K in t.GRADIENTS} == {(t.MIDDLE, False), (t.LARGE, False), (t.LARGE, True)}
    assert all(t.rounds("wgrad", c, N, K) > 1 for c, N, K in t.GRADIENTS)


def test_expected_tiles():
    assert abs(t.expected_tiles(1000, 1, 32) - 32) < 1e-9 and abs(t.expected_tiles(256, 1, 256) - 1) < 1e-9
    assert 32 * 8.4 < t.expected_tiles(65536, 32, 256) < 32 * 8.6       # 2048 on average: half of the experts have a ninth
