"""Plain 64-bit definitions of the language-model operators, for their tests: element
tables, packing by search in them, and the formulas.  numpy only; shares no code with
the library."""
import numpy as np

E4M3, E2M1 = 0, 1
_E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])
_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = {E4M3: _E4M3, E2M1: _E2M1}
TOP = {E4M3: 119, E2M1: 125}
LOW = -117


def blocks(cols):
    return -(-cols // 32)


def pitch(cols, fmt):
    return blocks(cols) * (32 if fmt == E4M3 else 16)


def scale_pitch(cols):
    return -(-blocks(cols) // 4) * 4


def pack(x, fmt):
    """(codes, scales) of a float64 matrix, as uint8 matrices of the packed layout."""
    rows, cols = x.shape
    v = TABLE[fmt]
    b = np.zeros((rows, blocks(cols) * 32))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    top = np.abs(b).max(axis=2)
    bad = ~np.isfinite(top)
    exps = np.arange(LOW, TOP[fmt] + 1)
    at = np.minimum(np.searchsorted(v[-1] * 2.0 ** exps.astype(float), np.where(bad, 0, top)), len(exps) - 1)
    s = exps[at]
    y = np.where(bad[..., None], 0, b) / 2.0 ** s[..., None].astype(float)
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(y)
    k = np.searchsorted(mid, a)  # a value on a border stays below it
    tie = (k < len(mid)) & (mid[np.minimum(k, len(mid) - 1)] == a) & (k % 2 == 1)
    k = np.where(bad[..., None], 0, k + tie).reshape(rows, -1)
    sign = (np.signbit(y) & ~bad[..., None]).reshape(rows, -1)
    if fmt == E4M3:
        codes = (k + 128 * sign).astype(np.uint8)
    else:
        n = (k + 8 * sign).astype(np.uint8)
        codes = n[:, 0::2] | (n[:, 1::2] << 4)
    scales = np.zeros((rows, scale_pitch(cols)), np.uint8)
    scales[:, : s.shape[1]] = np.where(bad, 255, s + 127)
    return codes, scales


def unpack(codes, scales, cols, fmt):
    """float64 values of codes and scales."""
    v = TABLE[fmt]
    if fmt == E4M3:
        k = codes & 127
        y = np.where(k == 127, np.nan, v[np.minimum(k, 126)]) * np.where(codes & 128, -1.0, 1.0)
    else:
        n = np.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1)
        y = v[n & 7] * np.where(n & 8, -1.0, 1.0)
    s = scales[:, : blocks(cols)].astype(float)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return (y.reshape(len(y), -1, 32) * f[..., None]).reshape(len(y), -1)[:, :cols]


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def swiglu_backward(dh, g, u):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def embedding_grad(dout, ids, n_rows, scale, padding):
    """(gradient, sums of magnitudes, tokens per row) in float64."""
    g, m, n = np.zeros((n_rows, dout.shape[1])), np.zeros((n_rows, dout.shape[1])), np.zeros(n_rows, int)
    keep = (ids >= 0) & (ids < n_rows) & (ids != padding)
    np.add.at(g, ids[keep], dout[keep])
    np.add.at(m, ids[keep], np.abs(dout[keep]))
    np.add.at(n, ids[keep], 1)
    return g * scale, m * abs(scale), n
