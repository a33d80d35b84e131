"""Plain 64-bit definitions of a cache in 8 bits and of token log probabilities, in numpy. Shares no code with the library."""
import numpy as np

LIMITS = {"bf16": (-124, 119), "fp16": (-15, 7)}  # exponents of a scale


def _table():
    """What each e4m3 code stands for: 1 sign, 4 exponent (bias 7), 3 fraction bits; no infinities, S.1111.111 is NaN."""
    v = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else -x if c >> 7 else x
    return v


CODES = _table()
_POSITIVE = CODES[:127]  # 0 .. 448, rising; a code's number is its place


def encode(x):
    """The nearest code, ties to the even one; past 448 it is 448."""
    m = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, m), 1, 126)
    lo = hi - 1
    below, above = m - _POSITIVE[lo], _POSITIVE[hi] - m
    c = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def power(byte, dtype):
    """2^(byte - 127), the exponent kept within the type's limits; 255 is NaN."""
    lo, hi = LIMITS[dtype]
    return np.where(np.asarray(byte) == 255, np.nan, 2.0 ** np.clip(np.asarray(byte).astype(int) - 127, lo, hi))


def scale_byte(top, dtype):
    """The least exponent whose 448-fold reaches top, within the limits, biased."""
    lo, hi = LIMITS[dtype]
    if not np.isfinite(top):
        return 255
    e = lo
    while e < hi and 448.0 * 2.0 ** e < top:
        e += 1
    return e + 127


def decode(code, byte, dtype, block):
    """code uint8 [..., slots, D], byte uint8 [..., blocks] -> float64 [..., slots, D]"""
    at = np.arange(code.shape[-2]) // block
    return CODES[code] * power(byte[..., at], dtype)[..., None]


def logprobs(x, temperature):
    """l = x / t - log(sum(exp(x / t))) and the entropy, of rows of float64."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = x / temperature
        top = z.max(-1, keepdims=True)
        shifted = np.where(np.isneginf(top), -np.inf, z - top)
        p = np.exp(shifted)
        total = p.sum(-1, keepdims=True)
        l = np.where(total == 0, -np.inf, shifted - np.log(total))
        h = -np.where(np.exp(l) == 0, 0.0, np.exp(l) * l).sum(-1)
    bad = np.isnan(x).any(-1) | np.isposinf(x).any(-1)
    l[bad], h[bad] = np.nan, np.nan
    return l, h


def best(x, K):
    """Ids of the K largest, ties to the lower id, NaN above all."""
    return np.argsort(np.where(np.isnan(x), -np.inf, -np.where(np.isnan(x), 0, x)) - 0.0, axis=-1, kind="stable")[..., :K] \
        if not np.isposinf(x).any() else _best_slow(x, K)


def _best_slow(x, K):
    out = np.empty(x.shape[:-1] + (K,), np.int64)
    for i in np.ndindex(*x.shape[:-1]):
        out[i] = sorted(range(x.shape[-1]), key=lambda j: (0 if np.isnan(x[i][j]) else 1, 0 if np.isnan(x[i][j]) else -x[i][j], j))[:K]
    return out
