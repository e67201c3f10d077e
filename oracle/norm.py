"""Layer norm and dropout with a residual for the oracle, in 64 bits. Test
infrastructure only (see the package docstring).

Keep mask of the elementwise dropout: element e (row-major) is kept iff word
(e mod 4) of Philox4x32-10(counter = (floor(e / 4) mod 2^32, floor(e / 2^34),
0, 1), key = (seed mod 2^32, seed >> 32)) is >= round(p * 2^32).
"""
import numpy as np

from .philox import keep_threshold, philox4x32_10


def element_keep_mask(n, seed, p_drop, first=0):
    """Boolean [n]: elements first .. first + n - 1."""
    e = np.arange(first, first + n, dtype=np.uint64)
    c = e >> np.uint64(2)
    seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    words = philox4x32_10(c & np.uint64(0xFFFFFFFF), c >> np.uint64(32), 0, 1, seed & 0xFFFFFFFF,
                          seed >> 32)
    words = [np.broadcast_to(w, (n,)) for w in words]
    w = np.choose((e & np.uint64(3)).astype(np.int64), words)
    return w >= np.uint32(keep_threshold(p_drop))


def dropout(x, p_drop, seed):
    """x Z / (1 - p) for the float32 value of p_drop."""
    x = np.asarray(x, dtype=np.float64)
    if p_drop == 0:
        return x.copy()
    keep = element_keep_mask(x.size, seed, p_drop).reshape(x.shape)
    return np.where(keep, x, 0.0) / (1.0 - float(np.float32(p_drop)))


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) over the rows of x [rows, C]."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) for stored statistics."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)
