"""Which kernel the 4-bit and ragged products take for a shape, and the shapes that reach each of them.

The functions follow the rules of csrc/skinny.hip and csrc/ragged_gemm.hip; test_fp4_ragged_tilings.py compares them with
the instantiations written there and shows that the shapes below reach every one, test_gpu_fp4_ragged_tilings.py runs them.
"""
W16, FP32, E8M0 = "16-bit", "fp32", "e8m0"
FORMATS = [(FP32, g) for g in (32, 64, 128)] + [(E8M0, g) for g in (32, 64, 128)]


def _ceil(a, b):
    return -(-a // b)


def _cols(M, N, K):
    passes = _ceil(M, 32 if M <= 32 else 64)
    if _ceil(N, 128) * passes >= 128:
        return 128
    return 64 if M > 32 and K > 4096 and _ceil(N, 64) * passes >= 64 else 32


def skinny(fmt, group, fp16, R, E, N, K):
    """(rows of a pass, 16-column tiles of a wave, column waves, K waves); E = 0: one matrix."""
    w16, dense = fmt == W16, E == 0
    mats = 1 if dense else min(R, E)
    rows = R if dense else _ceil(R, E)

    def groups(cols):
        return _ceil(N, cols) * mats

    if not w16 and dense and rows <= 4:
        return (4, 2, 2, 2) if groups(64) >= 512 else (4, 1, 1, 4) if groups(32) < 192 else (4, 1, 2, 2)
    wide = groups(128) >= 1024
    at_once = not w16 and not dense and wide and K < 4096
    if rows <= (8 if dense else 4) and not at_once:
        if wide:
            return (8, 2, 4, 1) if w16 else (8, 1, 4, 1)
        return (8, 2, 2, 2) if groups(64) >= 512 else (8, 1, 1, 4) if groups(32) < 192 else (8, 1, 2, 2)
    if rows <= (16 if dense else 12):
        if wide:
            return (16, 2, 4, 1) if w16 else (16, 4, 2, 2)
        if groups(64) >= 512:
            return (16, 2, 2, 2)
        if groups(32) < 192:
            return (16, 1, 1, 4)
        return (16, 2, 4, 2) if fmt == FP32 and group == 128 and groups(128) >= 128 else (16, 1, 2, 2)
    assert not w16
    if not dense:
        if rows <= 20:
            return (32, 2, 4, 1)
        wave_columns = group == 128 if fmt == FP32 else not fp16 or group == 32
        return (64, 2, 8, 1) if wave_columns else (64, 2, 4, 1)
    cols = _cols(R, N, K)
    if rows <= 32:
        return (32, 2, 4, 2) if cols == 128 else (32, 1, 2, 2)
    return {128: (64, 2, 4, 2), 64: (64, 1, 4, 2), 32: (64, 1, 2, 2)}[cols]


def ragged(op, R, E, N, K):
    """Tile of a ragged product, or 0 where it goes to the kernel above."""
    if op == "fwd" and R <= 8 * E:
        return 0
    cols = N if op == "fwd" else K

    def tiles(t):
        if op == "wgrad":
            return E * _ceil(N, t) * _ceil(K, t)
        return (R // t + (min(E, R) + 1) // 2) * _ceil(cols, t)

    if tiles(256) >= 512 if op == "wgrad" else tiles(256) >= 200 and R >= 112 * E:
        return 256
    return 128 if tiles(128) >= 192 else 64


# 4-bit: (rows or the experts' rows, N, K).  K is a multiple of 128 in the first of two, in the second the scale rows of
# groups of 32 start off whole dwords and the last group of 64 or 128 is short.
LINEAR = [(M, N, K) for N, Ks, Ms in (
    (40, (4224, 4128), (1, 4, 7, 13, 27, 61)),          # few columns
    (7000, (512, 288), (3, 6, 14)), (7000, (4224, 4128), (24, 50)),
    (20000, (512, 288), (11, 31, 63)),
    (33000, (512, 288), (2, 5, 12, 30)),
    (131000, (512, 288), (8, 15)),
) for K in Ks for M in Ms]


def _spread(rows, E, at=(0, 1, -1)):
    """`rows` of E experts, in a few of them: most in the first."""
    c = [0] * E
    c[at[0]] = rows - rows // 3
    c[at[1]] += rows // 3 - 1
    c[at[2]] += 1
    return c


EXPERTS = [(tuple(_spread(R, E)), N, K) for R, E, N, Ks in (
    (20, 9, 72, (512, 288)),        # 3 rows on average: few columns,
    (26, 13, 500, (512, 288)),      # more,
    (160, 40, 1000, (512, 288)),    # many,
    (130, 65, 2040, (4224, 4128)),  # and the most over a long K
    (130, 65, 2040, (512, 288)),    # the most over a short one
    (72, 8, 72, (512, 288)),        # 9 rows on average
    (300, 26, 250, (512, 288)),
    (150, 16, 1020, (512, 288)),
    (420, 40, 1000, (512, 288)),
    (700, 65, 2040, (512, 288)),
    (90, 5, 300, (512, 288)),       # 18 rows
    (200, 4, 330, (512, 288)),      # 50 rows
) for K in Ks]

# 16-bit, few rows an expert: the same kernel
WEIGHTS16 = [(tuple(_spread(R, E)), N, K) for R, E, N, Ks in (
    (20, 9, 72, (512, 264)), (26, 13, 504, (512, 264)), (160, 40, 1000, (512, 264)), (130, 65, 2040, (512, 264)),
    (64, 8, 72, (512, 264)), (208, 26, 248, (512, 264)), (320, 40, 1000, (512, 264)), (520, 65, 2040, (512, 264)),
) for K in Ks]

# ragged products: (op, experts' rows, N, K)
RAGGED = [(op, c, N, K) for op, c, N, K in (
    ("fwd", (700, 0, 1300, 513, 1), 5128, 136), ("dgrad", (700, 0, 1300, 513, 1), 136, 5128), ("wgrad", (200, 0, 97, 64, 1), 2600, 2568),
    ("fwd", (300, 0, 129, 1, 70), 4000, 200), ("fwd", (1, 640, 0, 60), 3208, 64),
    ("dgrad", (300, 0, 129, 1, 70), 200, 4000), ("dgrad", (1, 640, 0, 60), 64, 3208),
    ("wgrad", (100, 0, 65, 1), 1000, 1032), ("wgrad", (700, 3), 1288, 1304),
    ("fwd", (64, 0, 65, 1), 136, 72), ("dgrad", (64, 0, 65, 1), 72, 136), ("wgrad", (64, 0, 65, 1), 136, 72))]
