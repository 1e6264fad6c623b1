"""One AdamW step, with states in 32 bits or in 8 (oracle side, float64).

Test infrastructure only (see ``oracle/__init__.py``).

    m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
    p = p (1 - lr wd) - lr (m / (1 - b1^T)) / (sqrt(v / (1 - b2^T)) + eps)

An 8-bit state holds m and sqrt(v) as e4m3 codes against a power of two per 128 entries,
rounded at random by 16 bits of Philox4x32-10.

Pins (``tests/test_oracle_training.py``): a worked first step; with a constant gradient the step
is lr whatever its size; weight decay alone; Philox4x32-10 against its published answers;
codes against the values of e4m3; the mean of many random roundings is the value.
"""

import numpy as np

BLOCK = 128


def step(p, g, m, v, T, lr, b1=0.9, b2=0.999, eps=1e-8, wd=0.01):
    """(p, m, v) after step T."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * wd) - lr * (m / (1 - b1 ** T)) / (np.sqrt(v / (1 - b2 ** T)) + eps)
    return p, m, v


def code_value(code):
    """The value of an e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    code = np.asarray(code, dtype=np.int64)
    e, f = (code >> 3) & 15, code & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(float) - 10))
    return np.where(code & 128, -mag, mag)


def scales(x):
    """Per 128 entries the power of two that takes their largest magnitude into [128, 256)."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = np.append(x, np.zeros(-len(x) % BLOCK)).reshape(-1, BLOCK).max(1)
    return np.maximum(2.0 ** (np.frexp(x)[1] - 8.0), 2.0 ** -126)


def philox4x32(key, counter):
    """Four output words (SC'11, table 2) of arrays of key (2) and counter (4) words."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k = [int(w) for w in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def random16(seed, n, T, tensor, first=0):
    """The 16-bit random numbers of entries first..first+n-1: (for m, for v)."""
    i = np.arange(n, dtype=np.uint64) + np.uint64(first)
    b = i // np.uint64(4)
    zero = np.zeros(n, dtype=np.uint64)
    w = philox4x32((seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF),
                   (b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), zero + np.uint64(T), zero + np.uint64(tensor)))
    w = np.choose((i % np.uint64(4)).astype(int), w)
    return (w & np.uint64(0xFFFF)).astype(np.int64), (w >> np.uint64(16)).astype(np.int64)


def encode(x, random, root=False, s=None):
    """(codes, scales, margin) of x: rounded up where the fraction left over and random / 2^16
    reach 1; the margin is how far their sum is from that, or x from a code that a number next to
    it would be rounded from, a code's spacing being 1."""
    x = np.asarray(x, dtype=np.float64)
    s = scales(x) if s is None else s
    y = np.abs(x) / np.repeat(s, BLOCK)[:len(x)]
    e = np.where(y > 0, np.maximum(np.frexp(y)[1] - 1, -6), -6)
    units = y * 2.0 ** (3.0 - e)                    # of the code's spacing
    whole = np.floor(units)
    total = (units - whole) + random / 65536.0
    up = whole + (total >= 1.0)
    code = np.where(e == -6, up, up + (e + 6) * 8.0).astype(np.int64)
    if root:
        code = np.where((x > 0) & (code < 1), 1, code)
    margin = np.minimum(np.abs(total - 1.0), np.maximum(units - whole, random / 65536.0))
    return code | np.where(x < 0, 128, 0), s, margin
