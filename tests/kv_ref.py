"""The paged 4-bit key/value cache in plain 64-bit arithmetic, on the CPU: what
its bytes stand for, and attention over it token by token.  Shares nothing with
the library."""
import math

import numpy as np

BLOCK = {"nvfp4": 16, "mxfp4": 32}
LATTICE = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def scale_values(fmt, byte):
    b = byte.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    b = b & 127
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, np.ldexp(1 + m / 8.0, e - 7))
    return np.where(b == 127, np.nan, v)


def row_values(fmt, codes, scales, g=1.0):
    """[..., bytes] codes and [..., blocks] scales -> [..., 2 * bytes] float64."""
    x = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = np.repeat(scale_values(fmt, scales), BLOCK[fmt], axis=-1)
    return LATTICE[x] * s * (float(g) if fmt == "nvfp4" else 1.0)


def hadamard128():
    h = np.array([[1.0]])
    for _ in range(7):
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(128)


def rotate(x):
    return (x.reshape(*x.shape[:-1], -1, 128) @ hadamard128()).reshape(x.shape)


def tokens_of(fmt, codes, scales, g, table_row, n, page):
    """Values [n, heads, dim] of a sequence's first n tokens; planes [pages, heads, page, bytes]."""
    heads, dim = codes.shape[1], codes.shape[3] * 2
    out = np.zeros((n, heads, dim))
    for t in range(n):
        p = int(table_row[t // page])
        if 0 <= p < codes.shape[0]:
            out[t] = row_values(fmt, codes[p, :, t % page], scales[p, :, t % page], g)
    return out


def attention(q, k, v, scale, causal=True, window=0):
    """q [m, q_heads, dim], k and v [n, heads, dim] -> out [m, q_heads, dim], lse [m, q_heads], float64.
    Only the tokens a query sees are looked at."""
    m, q_heads, dim = q.shape
    n, heads = k.shape[0], k.shape[1]
    out, lse = np.zeros((m, q_heads, dim)), np.full((m, q_heads), -np.inf)
    for i in range(m):
        last = min(n - m + i, n - 1) if causal else n - 1
        first = max(0, n - m + i - window + 1) if window else 0
        if last < first:
            continue
        for h in range(q_heads):
            kk, vv = k[first:last + 1, h * heads // q_heads], v[first:last + 1, h * heads // q_heads]
            with np.errstate(invalid="ignore"):
                s = (kk @ q[i, h]) * scale
                top = s.max()
                p = np.exp(s - top)
                out[i, h] = (p @ vv) / p.sum()
                lse[i, h] = top + np.log(p.sum())
    return out, lse
