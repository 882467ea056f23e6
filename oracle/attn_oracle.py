"""Plain fp64 definitions of the attention operators (NumPy; shares nothing with the HIP code).

norm_rope: RMS norm of a head row, then rotation of its first dims by the
position.  attend: softmax attention of the last rows of a sequence over its
visible keys, causal, optionally a window with a few first keys that stay
visible.  place / store / load: where a token sits in the paged cache.
"""
import math

import numpy as np


def rope_table(n_positions, rotary, base=10000.0):
    """[n_positions, rotary] fp32: cosines, then sines, of position * base^(-2i / rotary)."""
    ang = np.arange(n_positions, dtype=np.float64)[:, None] * \
        base ** (-np.arange(0, rotary, 2, dtype=np.float64) / max(rotary, 1))[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def norm_rope(x, w, eps, table_row, interleaved):
    """x [..., D] fp64, w [D] or None, table_row [..., R] (cosines, sines)."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    R = table_row.shape[-1]
    if not R:
        return y
    h = R // 2
    c, s = np.asarray(table_row[..., :h], np.float64), np.asarray(table_row[..., h:], np.float64)
    i = np.arange(h)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    out = y.copy()
    out[..., ia] = y[..., ia] * c - y[..., ib] * s
    out[..., ib] = y[..., ib] * c + y[..., ia] * s
    return out


def visible(n, m, window, sinks):
    """[m, n] bool: which of n keys the last m positions see (positions may be negative)."""
    p = np.arange(n - m, n)[:, None]
    k = np.arange(n)[None, :]
    see = k <= p
    if window:
        see &= (p - k < window) | (k < sinks)
    return see


def attend(q, k, v, scale, window, sinks):
    """q [m, H, D], k and v [n, K, D] -> (out [m, H, D], sum of weights times |v|, largest scale * sum |q||k|)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    m, H, D = q.shape
    n, K = k.shape[0], k.shape[1]
    out, mag, big = np.zeros((m, H, D)), np.zeros((m, H, D)), 0.0
    see = visible(n, m, window, sinks)
    if not see.any():
        return out, mag, big
    for h in range(H):
        kk, vv = k[:, h // (H // K)], v[:, h // (H // K)]
        s = np.where(see, q[:, h] @ kk.T * scale, -math.inf)
        top = np.max(s, axis=1, keepdims=True)
        e = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        tot = np.sum(e, axis=1, keepdims=True)
        w = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
        out[:, h] = w @ vv
        mag[:, h] = w @ np.abs(vv)
        big = max(big, float(np.max(np.where(see, np.abs(q[:, h]) @ np.abs(kk).T * scale, 0.0))))
    return out, mag, big


def place(token, page_row, page_size):
    """(page, place in the page) of a sequence's token."""
    return page_row[token // page_size], token % page_size


def store(k_cache, v_cache, page, at, k_row, v_row):
    """One token's rows [K, D] into k_cache [P, K, D/8, page, 8] and v_cache [P, K, page/8, D, 8]."""
    K, D = k_row.shape
    k_cache[page, :, :, at, :] = k_row.reshape(K, D // 8, 8)
    v_cache[page, :, at // 8, :, at % 8] = v_row


def load(k_cache, v_cache, page, at):
    K, D = k_cache.shape[1], k_cache.shape[2] * 8
    return k_cache[page, :, :, at, :].reshape(K, D), v_cache[page, :, at // 8, :, at % 8]
