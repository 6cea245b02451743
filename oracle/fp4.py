"""4-bit (OCP e2m1) weights with group scales, in numpy binary64.

code = sign << 3 | index, value LEVELS[index]; two codes per byte, even column in the low half.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(y):
    """Nearest code of y (float64), ties to the even code, saturating, sign kept."""
    y = np.asarray(y, np.float64)
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    a = np.abs(y)
    idx = np.zeros(y.shape, np.uint8)
    for i, b in enumerate(mid):                  # between index i and i + 1; a tie goes to the even one
        idx += ((a > b) | ((a == b) & (i % 2 == 1))).astype(np.uint8)
    return idx | (np.signbit(y).astype(np.uint8) << 3)


def decode(codes):
    c = np.asarray(codes)
    v = LEVELS[c & 7]
    return np.where(c >= 8, -v, v)


def pack(codes):
    c = np.asarray(codes, np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(q):
    q = np.asarray(q, np.uint8)
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def scale_values(scale):
    """Scales as float64: fp32 ones as they are, E8M0 bytes as 2^(c - 127) with 255 = NaN."""
    scale = np.asarray(scale)
    if scale.dtype != np.uint8:
        return scale.astype(np.float64)
    return np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int32) - 127))


def quant_groups(w, group, e8m0):
    """w float32 [..., K] -> (packed codes, scales fp32 or E8M0 bytes).  Groups that hold NaN or
    infinities get a NaN scale (their codes mean nothing)."""
    w = np.asarray(w, np.float32)
    K = w.shape[-1]
    G = -(-K // group)
    p = np.zeros((*w.shape[:-1], G * group), np.float32)
    p[..., :K] = w
    p = p.reshape(*w.shape[:-1], G, group)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(p).max(-1)
        bad = ~np.isfinite(p).all(-1)
        safe = np.where(bad | (amax == 0), np.float32(6.0), amax)
        if e8m0:
            ex = np.clip(np.frexp(safe.astype(np.float64))[1] - 3, -127, 127)
            ex = np.where(amax == 0, 0, ex)
            scale = np.where(bad, 255, ex + 127).astype(np.uint8)
            y = np.ldexp(p.astype(np.float64), -ex[..., None])
        else:
            s = np.where(amax == 0, np.float32(1), safe / np.float32(6)).astype(np.float32)
            scale = np.where(bad, np.float32(np.nan), s)
            y = (p / s[..., None]).astype(np.float64)         # IEEE fp32 quotient
        codes = encode(np.where(np.isfinite(y), y, 0.0))
    return pack(codes.reshape(*w.shape[:-1], G * group)[..., :K]), scale


def dequant_groups(q, scale, group):
    """float64 values, unrounded."""
    v = decode(unpack(q))
    s = np.repeat(scale_values(scale), group, -1)[..., :v.shape[-1]]
    return v * s
