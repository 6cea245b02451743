"""The shapes of test_gpu_fp4_ragged_tilings.py reach every kernel of the 4-bit and ragged products (CPU only)."""
import itertools
import os
import re

import pytest

from tests import fp4_ragged_tilings as t

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_grouped_amd", "csrc")


def _written(name, pattern):
    text = open(os.path.join(CSRC, name)).read()
    return {tuple(int(v) for v in m) for m in re.findall(pattern, re.sub(r"//.*", "", text))}


def _reachable(fmt, group, fp16):
    sizes = (1, 40, 300, 1000, 2000, 7000, 9000, 20000, 33000, 131000)
    dense = [] if fmt == t.W16 else [(R, 0, N, K) for R, N, K in itertools.product(range(1, 66), sizes, (288, 4128))]
    most = 8 if fmt == t.W16 else 64
    grouped = [(R, E, N, K) for E, N, K in itertools.product((1, 3, 9, 16, 40, 65, 256), sizes, (288, 4128))
               for R in {1, E // 2 + 1, *(E * a for a in range(1, most + 1))} if R <= most * E]
    return {t.skinny(fmt, group, fp16, *s) for s in dense + grouped}


def test_rules_name_the_tilings_that_are_written():
    written = _written("skinny.hip", r"launch_tile<W, GROUP, F16, (\d+), (\d+), (\d+), (\d+),")
    assert written
    every = set().union(*(_reachable(f, g, h) for (f, g), h in itertools.product(t.FORMATS + [(t.W16, 128)], (False, True))))
    assert every == written
    assert _written("ragged_gemm.hip", r"launch<OP, F16, OUT32, (\d+), \d+, (\d+), (\d+)>") == {(256, 4, 2), (128, 4, 2), (64, 2, 2)}


@pytest.mark.parametrize("fp16", [False, True])
@pytest.mark.parametrize("fmt,group", t.FORMATS)
def test_shapes_reach_every_4bit_tiling(fmt, group, fp16):
    linear = {t.skinny(fmt, group, fp16, M, 0, N, K) for M, N, K in t.LINEAR}
    experts = {t.skinny(fmt, group, fp16, sum(c), len(c), N, K) for c, N, K in t.EXPERTS}
    assert linear | experts == _reachable(fmt, group, fp16)
    for K in (288, 4128):   # those of experts by themselves, too
        grid = itertools.product((1, 3, 9, 16, 40, 65, 256), (1, 40, 300, 1000, 2000, 7000, 33000), range(1, 65))
        assert {t.skinny(fmt, group, fp16, a * E, E, N, K) for E, N, a in grid} <= experts


def test_shapes_reach_every_16bit_tiling():
    reached = {t.skinny(t.W16, 128, False, sum(c), len(c), N, K) for c, N, K in t.WEIGHTS16}
    assert reached == _reachable(t.W16, 128, False)
    assert all(t.ragged("fwd", sum(c), len(c), N, K) == 0 for c, N, K in t.WEIGHTS16)


def test_shapes_reach_every_ragged_tile():
    reached = {(op, t.ragged(op, sum(c), len(c), N, K)) for op, c, N, K in t.RAGGED}
    assert reached == set(itertools.product(("fwd", "dgrad", "wgrad"), (64, 128, 256)))
