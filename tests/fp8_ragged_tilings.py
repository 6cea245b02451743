"""Which tile the FP8 expert products take for a shape, and shapes that reach each of them.

tile() follows the rule in csrc/fp8_ragged.hip; test_fp8_ragged_tilings.py compares it with the instantiations written there and
shows what the shapes below reach, test_gpu_fp8_ragged_tilings.py runs them.
"""
import math

SMALL, LOW, MIDDLE, LARGE = (32, 64), (64, 128), (128, 128), (256, 256)


def _ceil(a, b):
    return -(-a // b)


def expected_tiles(R, E, t):
    """Row tiles of t rows that R rows make over E experts by chance."""
    a = R / E
    sd = math.sqrt(2 * a * (1 - 1 / E)) + 1e-9
    sure = max(0, int((a - 3 * sd) / t))
    n, k = float(sure), sure
    while k * t < a + 3 * sd:
        n += 0.5 * math.erfc((k * t + 0.5 - a) / sd)
        k += 1
    return n * E


def tile(op, R, E, N, K):
    def tiles(t):
        return (expected_tiles(R, E, t[0]) if op == "fwd" else E * _ceil(N, t[0])) * _ceil(N if op == "fwd" else K, t[1])

    if op == "fwd":
        if R <= 12 * E or tiles(SMALL) <= 512:
            return SMALL
        if R <= 40 * E:
            return LOW
    return LARGE if math.ceil(tiles(LARGE) / 256) <= 0.715 * tiles(MIDDLE) / 512 else MIDDLE


def rounds(op, counts, N, K):
    """Tiles for each workgroup that the CUs hold at a time."""
    t = tile(op, sum(counts), len(counts), N, K)
    if op == "fwd":
        n = sum(_ceil(c, t[0]) for c in counts) * _ceil(N, t[1])
    else:
        n = len(counts) * _ceil(N, t[0]) * _ceil(K, t[1])
    return n / (256 if t == LARGE else 512)


# (rows of the experts, N, K), with one step of 128 a tile, as many as are on their way at a time and more
PRODUCTS = ([([9, 0, 3, 14] * 24, 1032, K) for K in (16, 272, 400, 528)] + [([30, 41, 0, 38] * 16, 2056, K) for K in (16, 144, 272)] +
            [([130, 128, 1, 60] * 8, 2056, K) for K in (16, 144, 272)] + [([1000, 1020, 0, 512] * 2, 5000, K) for K in (16, 144, 272)])
GRADIENTS = [([3, 150, 0, 20] * 32, 264, 264), ([3, 150, 0, 300] * 12, 504, 1016), ([3, 150, 0, 300] * 12, 504, 1024)]
