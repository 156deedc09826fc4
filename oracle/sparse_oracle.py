"""Float64 definitions of the sparse layer's operators, in numpy.

Dropout (Philox4x32-10 of Salmon, Moraes, Dror and Shaw, 2011), layer norm with
dropout and residual and its backward, routing to experts, 8-bit floating rows.
It shares no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

MASK = 0xFFFFFFFF
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}     # exponent of the smallest normal number


# ------------------------------------------------------------------ dropout
def philox(counter, key):
    """One block of Philox4x32-10: four 32-bit words from a counter of four and a key of two (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & MASK, (p0 >> 32) ^ c[3] ^ k[1], p0 & MASK]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return c


def drop_threshold(p):
    return int(np.rint(float(np.float32(p)) * 65536.0))


def keep(rows, cols, p, seed, offset, row0=0):
    """Which elements are kept, bool [rows, cols]."""
    t = drop_threshold(p)
    n = -(-cols // 8)
    r = np.repeat(np.arange(row0, row0 + rows, dtype=np.uint64), n)
    g = np.tile(np.arange(n, dtype=np.uint64), rows)
    sh, lo = np.uint64(32), np.uint64(MASK)
    c = [g | (r >> sh) << np.uint64(24), r & lo, np.full(rows * n, offset & MASK, np.uint64),
         np.full(rows * n, offset >> 32, np.uint64)]
    k = [seed & MASK, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & lo, (p0 >> sh) ^ c[3] ^ np.uint64(k[1]), p0 & lo]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    bits = np.empty((rows * n, 8), np.uint64)
    for i, w in enumerate(c):
        bits[:, 2 * i], bits[:, 2 * i + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    return (bits.reshape(rows, n * 8)[:, :cols] >= t)


def drop_factor(rows, cols, p, seed, offset):
    t = drop_threshold(p)
    if t >= 65536:
        return np.zeros((rows, cols))
    return keep(rows, cols, p, seed, offset) * (65536.0 / (65536 - t))


# ------------------------------------------------------------------ layer norm
def layer_norm(h, gamma, beta, eps):
    mean = h.mean(-1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[:, None]
    y = y if gamma is None else y * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_backward(dy, dh, h, mean, rstd, gamma):
    xh = (h - mean[:, None]) * rstd[:, None]
    t = dy if gamma is None else dy * gamma
    dr = rstd[:, None] * (t - t.mean(-1, keepdims=True) - xh * (t * xh).mean(-1, keepdims=True))
    return (dr if dh is None else dr + dh), (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------ routing
def expert_sort(expert, experts):
    """offsets [E+1], position (as expert), source [slots]: a loop over the slots."""
    flat = np.asarray(expert).reshape(-1)
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(s)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
    source = np.full(flat.size, -1, np.int32)
    order = np.array([s for v in lists for s in v], np.int32)
    source[: order.size] = order
    position = np.full(flat.size, -1, np.int32)
    position[order] = np.arange(order.size)
    return offsets, position.reshape(np.asarray(expert).shape), source


def combine(position, weight, y):
    out = np.zeros((position.shape[0], y.shape[1]))
    for j in range(position.shape[1]):
        at = position[:, j]
        live = at >= 0
        w = 1.0 if weight is None else weight[live, j : j + 1]
        out[live] += w * y[at[live]]
    return out


def combine_backward(position, weight, dout, y):
    """dy (rows without a source are NaN) and dweight."""
    dy, dw = np.full(y.shape, np.nan), np.zeros(position.shape)
    for j in range(position.shape[1]):
        live = position[:, j] >= 0
        at = position[live, j]
        dy[at] = (1.0 if weight is None else weight[live, j : j + 1]) * dout[live]
        dw[live, j] = (dout[live] * y[at]).sum(-1)
    return dy, dw


# ------------------------------------------------------------------ 8-bit floating rows
def block_exp(amax, fmt):
    """Exponent byte of blocks whose largest magnitudes are amax (finite), found by search."""
    amax = np.asarray(amax, np.float64)
    e = np.zeros(amax.shape, np.int64)
    for b in range(254, -1, -1):       # the smallest that holds the block
        e[amax <= LARGEST[fmt] * 2.0 ** (b - 127)] = b
    return e


def to_f8(v, fmt):
    """v rounded to the format's values, ties to even (|v| <= its largest)."""
    v = np.asarray(v, np.float64)
    _, k = np.frexp(np.where(v == 0, 1.0, v))
    step = 2.0 ** (np.maximum(k - 1, LOWEST[fmt]) - MANTISSA[fmt])
    return np.where(v == 0, v, np.rint(v / step) * step)


def quant_rows(x, fmt):
    """x [R, C] -> the values kept [R, P] and exponent bytes [R, P / 128]; blocks with infinities or NaN: 0 and 255."""
    R, C = x.shape
    P = -(-C // 128) * 128
    b = np.zeros((R, P))
    b[:, :C] = x
    b = b.reshape(R, P // 128, 128)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = np.where(bad, 255, block_exp(np.abs(b).max(-1), fmt))
    q = to_f8(b * 2.0 ** (127.0 - np.where(bad, 127, e))[..., None], fmt)
    return q.reshape(R, P), e


def row_values(q, e, cols):
    """What 8-bit rows stand for."""
    step = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return (q.reshape(q.shape[0], e.shape[1], 128) * step[..., None]).reshape(q.shape)[:, :cols]


def round_rows(x, fmt):
    return row_values(*quant_rows(x, fmt), x.shape[1])
