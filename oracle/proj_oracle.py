"""Plain fp64 definitions of the operators around the halves of the layer (NumPy; shares nothing with the HIP code).

norm: the residual's addition and the RMS norm of each row.  e4m3: the nearest E4M3 value.  quantise: rows with one
scale per 128 columns.  fp8_product: rows by weights with scales.  lora: each token's adapter beside a base.
"""
import numpy as np

BLOCK = 128
TOP = 448.0
TINY = 2.0 ** -126


def norm(x, residual, weight, eps):
    """(h, y) of fp64 rows."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, y if weight is None else y * np.asarray(weight, np.float64)


def e4m3(v):
    """The nearest E4M3 value, ties to the even one, for |v| < 464."""
    v = np.asarray(v, np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -30))), -6.0)
    step = 2.0 ** (e - 3)
    return np.clip(np.round(v / step) * step, -TOP, TOP)


def decode(b):
    """E4M3 bytes -> values (0x7F and 0xFF: NaN)."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def encode(v):
    """E4M3 values -> bytes."""
    table = decode(np.arange(127))
    b = np.searchsorted(table, np.abs(v))
    assert np.array_equal(table[b], np.abs(v))
    return (b + 128 * np.signbit(v)).astype(np.uint8)


def quantise(v, rows):
    """Values [a, b] -> (bytes, scales [ceil(a / rows), ceil(b / 128)] fp32): one scale per rows x 128 block."""
    a, b = v.shape
    s = np.zeros((-(-a // rows), -(-b // BLOCK)), np.float32)
    q = np.zeros((a, b), np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(j * BLOCK, (j + 1) * BLOCK))
            s[i, j] = max(np.max(np.abs(v[at])) / TOP, TINY)
            q[at] = encode(e4m3(v[at] / s[i, j]))
    return q, s


def spread(s, rows, a, b):
    """Scales of rows x 128 blocks to every element of [a, b]."""
    return np.repeat(np.repeat(np.asarray(s, np.float64), rows, 0)[:a], BLOCK, 1)[:, :b]


def fp8_product(x, xs, w, ws):
    """(y, sum of |x w|, sum over groups of 8 columns of the largest |x| times the largest |w|) of bytes and scales."""
    xv, wv = decode(x) * spread(xs, 1, *x.shape), decode(w) * spread(ws, BLOCK, *w.shape)
    xm, wm = (np.max(np.abs(t).reshape(t.shape[0], -1, 8), axis=2) for t in (xv, wv))
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T, xm @ wm.T


def lora(x, base, ids, a, b, ranks, scales):
    """(out, per output: sum of |s v B|, sum of |s| sum|x A| |B|) with a [n, R, K], b [n, N, R]."""
    out = np.array(base, np.float64)
    mag, deep = np.zeros_like(out), np.zeros_like(out)
    for t, i in enumerate(ids):
        if 0 <= i < len(a):
            r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
            s = 1.0 if scales is None else float(scales[i])
            ar, br = np.asarray(a[i, :r], np.float64), np.asarray(b[i, :, :r], np.float64)
            v = ar @ x[t]
            out[t] += s * (br @ v)
            mag[t] = abs(s) * (np.abs(br) @ np.abs(v))
            deep[t] = abs(s) * (np.abs(br) @ (np.abs(ar) @ np.abs(x[t])))
    return out, mag, deep
