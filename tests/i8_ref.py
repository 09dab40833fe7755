"""Plain definitions of 8-bit integer rows and of the rows of experts, for their tests.
numpy only; shares no code with the library."""
import numpy as np


def pitch(cols):
    return -(-cols // 16) * 16


def pack(x):
    """(codes, scales) of a float64 matrix whose values a float holds: int8 rows of the packed
    layout and float32 scales."""
    rows, cols = x.shape
    m = np.abs(x).max(axis=1, initial=0.0)
    bad = ~np.isfinite(m)
    m = np.where(bad, 0, m)
    y = np.where(bad[:, None], 0, x) * 127
    m1 = np.where(m > 0, m, 1)[:, None]
    low = np.floor(y / m1)
    twice = 2 * (y - low * m1)  # exact: at most 24 + 8 bits
    up = (twice > m1) | ((twice == m1) & (low % 2 != 0))
    codes = np.zeros((rows, pitch(cols)), np.int8)
    codes[:, :cols] = np.where(m[:, None] > 0, low + up, 0)
    scales = m.astype(np.float32) / np.float32(127)
    with np.errstate(over="ignore"):  # the largest rows' scales are rounded down, so that 127 of them are finite
        scales = np.where(np.isinf(scales * np.float32(127)), np.nextafter(scales, np.float32(0)), scales)
    return codes, np.where(bad, np.float32(np.nan), scales)


def unpack(codes, scales, cols):
    """float32 values: the products, rounded once."""
    return codes[:, :cols].astype(np.float32) * scales[:, None]


def product(a, sa, b, sb):
    """float32 results of the product of codes: the exact sum rounded to a float, times the
    smaller scale, times the larger one."""
    with np.errstate(over="ignore", invalid="ignore"):
        sums = (a.astype(np.int64) @ b.astype(np.int64).T).astype(np.float32)
        x, y = np.broadcast_to(sa[:, None], sums.shape), np.broadcast_to(sb[None], sums.shape)
        less = np.abs(x) < np.abs(y)
        return sums * np.where(less, x, y) * np.where(less, y, x)


def order(ids, experts):
    """(order, offsets) of ids, those out of range behind the last expert's."""
    key = np.where((ids < 0) | (ids >= experts), experts, ids)
    return np.argsort(key, kind="stable"), np.searchsorted(np.sort(key), np.arange(experts + 1))


def grouped_product(a, b, offsets, y):
    """y with the rows of each expert overwritten; b [experts, outs, ins]."""
    y = y.copy()
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        y[rows] = a[rows] @ b[e].T
    return y


def grouped_wgrad(dy, x, offsets):
    return np.stack([dy[offsets[e]:offsets[e + 1]].T @ x[offsets[e]:offsets[e + 1]] for e in range(len(offsets) - 1)])
