"""tests/fp8_ragged_tilings.py follows the tile rule of csrc/fp8_ragged.hip: the rule's own text, compiled for the host, gives the same tile for
every shape tried (CPU only)."""
import os
import random
import shutil
import subprocess

import pytest

from tests import fp8_ragged_tilings as t

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_grouped_amd", "csrc", "fp8_ragged.hip")

AROUND = """
#include <math.h>
#include <stdint.h>
#include <stdio.h>
typedef void* hipStream_t;
struct Fp8Args { int R, E, N, K; };
enum Fp8Op : int { kFp8Fwd = 0, kFp8Wgrad = 1 };
static int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }
template <int OP, bool E8, bool OUT32, int BM, int BN, int WM, int WN, int D = 2>
int launch(const Fp8Args&, hipStream_t) { return BM * 1000 + BN; }
%s
int main() {
  int op;
  Fp8Args g;
  while (scanf("%%d %%d %%d %%d %%d", &op, &g.R, &g.E, &g.N, &g.K) == 5)
    printf("%%d\\n", op == kFp8Fwd ? run<kFp8Fwd, true, false>(g, 0) : run<kFp8Wgrad, true, false>(g, 0));
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """[(op, R, E, N, K)] -> [(rows, columns)] of the tile, by the source."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    text = open(SOURCE).read()
    text = text[text.index("double expected_tiles("):text.index("bool on4(")]
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(AROUND % text)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(d / "rule"), str(d / "rule.cpp")], check=True)

    def ask(shapes):
        lines = "".join("%d %d %d %d %d\n" % (("fwd", "wgrad").index(s[0]), *s[1:]) for s in shapes)
        out = subprocess.run([str(d / "rule")], input=lines, capture_output=True, text=True, check=True).stdout.split()
        return [divmod(int(v), 1000) for v in out]

    return ask


def test_rule_of_the_source_and_of_the_tests(rule):
    rng = random.Random(1)
    size = lambda lo, hi, step: max(lo, int(lo * (hi / lo) ** rng.random()) // step * step)
    shapes = [(rng.choice(("fwd", "wgrad")), size(1, 100000, 1), size(1, 600, 1), size(8, 8192, 8), size(16, 8192, 16)) for _ in range(4000)]
    for E in (1, 3, 32, 257):                            # both sides of each number of rows an expert
        shapes += [("fwd", n * E + d, E, 4096, 2048) for n in (12, 40) for d in (-1, 0, 1) if n * E + d > 0]
    shapes += [("fwd", sum(c), len(c), N, K) for c, N, K in t.PRODUCTS] + [("wgrad", sum(c), len(c), N, K) for c, N, K in t.GRADIENTS]
    got, want = rule(shapes), [t.tile(*s) for s in shapes]
    wrong = [(s, a, b) for s, a, b in zip(shapes, got, want) if a != b]
    assert len(got) == len(shapes) and not wrong, wrong[:5]
    for op, tiles in (("fwd", {t.SMALL, t.LOW, t.MIDDLE, t.LARGE}), ("wgrad", {t.MIDDLE, t.LARGE})):
        assert {a for s, a in zip(shapes, got) if s[0] == op} == tiles
