"""AdamW, its 8-bit moments and the global gradient norm in float64, from
their definitions (AdamW: Loshchilov & Hutter, "Decoupled Weight Decay
Regularization").

The 8-bit formats: blocks of 256 elements share a power of two; the first
moment is held as sign and e4m3, the root of the second as unsigned e4m4.
Rounding takes 16 random bits u: |x| in units of its last place becomes
floor(|x| + u / 2^16).
"""

import numpy as np

BLOCK = 256
M_FORMAT = (3, -6, 448.0)     # mantissa bits, exponent of the smallest normal number, largest number
V_FORMAT = (4, 0, 31744.0)
BF16_FORMAT = (7, -126, None)
_WEYL, _A, _B, _C = 0x9E3779B9, 0x6A09E667, 0xBB67AE85, 0x3C6EF373
_MASK = 0xFFFFFFFF


def _key(words):
    x = 0
    for w in words:
        x ^= int(w) & _MASK
        x ^= x >> 16
        x = x * _A & _MASK
        x ^= x >> 16
        x = x * _B & _MASK
        x ^= x >> 15
        x = (x + _WEYL) & _MASK
    return x


def draws(seed, step, tensor, index):
    """(m, v, parameter) random 16-bit integers of the elements `index`."""
    index = np.asarray(index, dtype=np.uint64)
    high = index >> np.uint64(32)
    key = np.zeros(index.shape, dtype=np.uint64)
    for h in np.unique(high):
        key[high == h] = _key((seed & _MASK, seed >> 32, step, tensor, h))
    mask = np.uint64(_MASK)
    x = ((index & mask) * np.uint64(_WEYL) + key) & mask
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(_A)) & mask
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(_B)) & mask
    x = x ^ (x >> np.uint64(16))
    return x >> np.uint64(16), x & np.uint64(0xFFFF), ((x * np.uint64(_C)) & mask) >> np.uint64(16)


def on_grid(x, fmt, u=None):
    """|x| on the format's numbers, of unlimited range above; u: 16-bit
    integers, or None for nearest, ties to even."""
    mantissa, lowest, _ = fmt
    x = np.abs(np.asarray(x, dtype=np.float64))
    e = np.maximum(np.frexp(x)[1] - 1, lowest) - mantissa
    q = np.ldexp(x, -e)
    q = np.rint(q) if u is None else np.floor(q + np.asarray(u, dtype=np.float64) / 65536.0)
    return np.ldexp(q, e)


def block_exponents(x, fmt):
    """Exponent of each block's scale: the least power of two that brings the
    block's maximum within the format, -126 at least."""
    x = np.abs(np.asarray(x, dtype=np.float64)).ravel()
    x = np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK).max(1)
    f, e = np.frexp(x / fmt[2])
    e = np.where(f == 0.5, e - 1, e)
    return np.where(x > 0, np.maximum(e, -126), -126)


def held(x, fmt, exponents, u=None):
    """Signed values that x is held as, with the given block exponents."""
    x = np.asarray(x, dtype=np.float64).ravel()
    s = np.repeat(np.asarray(exponents), BLOCK)[:len(x)]
    q = on_grid(np.ldexp(x, -s), fmt, u)
    if fmt is V_FORMAT:  # never rounded away
        q = np.where(x > 0, np.maximum(q, 2.0 ** (fmt[1] - fmt[0])), q)
    return np.copysign(np.ldexp(q, s), x)


def decode(codes, scales, fmt):
    """Values of 8-bit codes and scale bytes."""
    codes = np.asarray(codes).astype(np.int64).ravel()
    mantissa, lowest, _ = fmt
    sign = np.ones(len(codes))
    if fmt is M_FORMAT:
        sign = np.where(codes & 128, -1.0, 1.0)
        codes = codes & 127
    e, f = codes >> mantissa, codes & ((1 << mantissa) - 1)
    y = np.where(e > 0, np.ldexp(1.0 + f / 2.0 ** mantissa, e - 1 + lowest), np.ldexp(f / 2.0 ** mantissa, lowest))
    s = np.repeat(np.asarray(scales).astype(np.int64).ravel(), BLOCK)[:len(codes)]
    return np.where(s == 0, 0.0, sign * np.ldexp(y, s - 127))


def step(p, g, m, v, t, beta1, beta2, eps, lr, weight_decay, coef=1.0):
    """One AdamW step; returns (p, m, v), nothing rounded."""
    g = coef * g
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    m_hat, v_hat = m / (1.0 - beta1 ** t), v / (1.0 - beta2 ** t)
    return p - lr * (m_hat / (np.sqrt(v_hat) + eps) + weight_decay * p), m, v


def norm_and_coef(grads, max_norm, inv_scale):
    n = inv_scale * np.sqrt(np.sum([np.sum(np.square(np.asarray(g, dtype=np.float64))) for g in grads]))
    return n, inv_scale * min(1.0, max_norm / n) if n > 0 else inv_scale
