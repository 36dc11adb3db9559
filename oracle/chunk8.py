"""CPU definitions of the cache held in 8 bits and of the calls on it, in Python integers
and numpy float64.  Test infrastructure like the rest of this package: no code is shared with
the CUDA path."""
import math

import numpy as np

LEAST = -124  # the smallest exponent that is written

# the value of every code: sign, four bits of exponent (bias 7), three of mantissa; 0x7f, 0xff NaN
VALUES = np.array([(-1.0) ** (c >> 7) * (math.nan if c & 0x7f == 0x7f else
                                         (c & 7) * 2.0 ** -9 if c & 0x78 == 0 else
                                         (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
                   for c in range(256)])
_UP = VALUES[:127]  # 0 to 448, ascending


def encode(x):
    """Codes of the nearest values, ties to the even code; what is not finite becomes 0x7f."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    a = np.where(ok, np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(_UP, a), 1, 126)
    lo = hi - 1
    up, down = _UP[hi] - a, a - _UP[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(ok, code | (np.signbit(x) << 7), 0x7f).astype(np.uint8)


def factor(scale):
    """The factor of each scale byte."""
    s = np.asarray(scale, np.float64)
    return np.where(s == 255, np.nan, 2.0 ** (s - 127))


def exponent(a):
    """The least e >= LEAST with a <= 448 * 2^e."""
    e = LEAST
    while a > 448.0 * 2.0 ** e:
        e += 1
    return e


def values(codes, scales, block):
    """float64 values of a pool [..., P, hd] with scales [..., P / block]."""
    return VALUES[codes] * np.repeat(factor(scales), block, -1)[..., None]


def quantise(pool, block):
    """A pool of values as (codes, scales), every block scaled by its largest finite value."""
    *lead, P, hd = pool.shape
    x = pool.reshape(*lead, P // block, block, hd)
    a = np.abs(np.where(np.isfinite(x), x, 0.0)).max((-1, -2))
    scales = (np.vectorize(exponent)(a) + 127).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        codes = encode(x / factor(scales)[..., None, None])
    return codes.reshape(pool.shape), scales


def runs(pos, page, slot, block, P, NP):
    """[first row, end, page, block in the page] of the rows that are placed, and the status bits
    (8: a page or slot outside the pool, 128: more rows than slots)."""
    flags, out, t, n = 0, [], 0, len(pos)

    def of(i):
        if pos[i] < 0 or page[i] < 0:
            return None
        if page[i] >= NP or not 0 <= slot[i] < P:
            return "bad"
        return int(page[i]), int(slot[i]) // block

    while t < n:
        b = of(t)
        if b is None or b == "bad":
            flags |= 8 if b == "bad" else 0
            t += 1
            continue
        end = t + 1
        while end < n and of(end) == b:
            end += 1
        if end - t > block:
            flags |= 128
        out.append((t, min(end, t + block), *b))
        t = end
    return out, flags
