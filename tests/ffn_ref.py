"""Linear layers over 4-bit weights, the gated pair, the norm and their
gradients in plain 64-bit arithmetic on the CPU.  Shares nothing with the
library."""
import numpy as np

from kv_ref import BLOCK, row_values  # noqa: F401  (what codes and scales stand for)


def e4m3_values(codes):
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, np.ldexp(1 + m / 8.0, e - 7))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


def mxfp8_values(codes, scales):
    s = scales.astype(np.int64)
    s = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return e4m3_values(codes) * np.repeat(s, 32, axis=-1)


E4M3_GRID = e4m3_values(np.arange(127, dtype=np.uint8))


def mxfp8_of(y):
    """(codes, scales) of float64 rows: scale 2^(floor(log2 of the block's largest) - 8), nearest element, ties to the
    even code, past 448 to 448; a block that is not finite has the NaN scale and zero codes."""
    b = y.reshape(*y.shape[:-1], -1, 32)
    most = np.abs(b).max(-1)
    bad = ~np.isfinite(most)
    _, e = np.frexp(np.where(bad | (most == 0), 256.0, most))
    e = np.maximum(e - 1 - 8, -127)
    q = np.abs(np.where(bad[..., None], 0.0, b)) / np.ldexp(1.0, e)[..., None]
    mid = (E4M3_GRID[1:] + E4M3_GRID[:-1]) / 2
    lo, hi = np.searchsorted(mid, q, side="left"), np.searchsorted(mid, q, side="right")
    code = np.where(lo % 2 == 0, lo, hi) | (np.signbit(b) & ~bad[..., None]) << 7
    scale = np.where(bad, 255, np.where(most == 0, 127, e + 127))
    return code.reshape(y.shape).astype(np.uint8), scale.astype(np.uint8)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def gated(g, u):
    return g * sigmoid(g) * u


def gated_grad(dh, g, u):
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def rms_norm(s, w, eps):
    """(y, r) of float64 rows."""
    r = 1 / np.sqrt(np.square(s).mean(-1) + eps)
    return s * r[:, None] * w, r


def rms_norm_grad(dy, s, w, eps):
    """(dx, dw) from y_i = s_i r w_i, dr / ds_j = -r^3 s_j / d."""
    r = 1 / np.sqrt(np.square(s).mean(-1) + eps)
    along = (dy * w * s).sum(-1) * r ** 3 / s.shape[1]
    return dy * w * r[:, None] - s * along[:, None], (dy * s * r[:, None]).sum(0)
