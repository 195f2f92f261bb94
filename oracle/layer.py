"""Oracle of the operators between the linears: RMS norm, rotary positions, attention over the cache.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Everything here is float64 from the definitions; nothing is rounded except where the definition
stores a rounded value (codes, fp16 scales).  Callers give values (float64 arrays), not bits.
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """(y, h): h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, per row, unrounded."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rho = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return h * rho * np.asarray(weight, np.float64), h


def norm_heads(x, weight, eps):
    """RMS norm of every head row of x [T, H, D] (weight None: x), unrounded."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    rho = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + np.float64(np.float32(eps)))
    return x * rho * np.asarray(weight, np.float64)


def rope(x, positions, inv_freq, factor=1.0, interleaved=False, axes=None):
    """Rotary positions on the first 2 * len(inv_freq) channels of x [T, H, D], unrounded; with axes,
    frequency i takes its position from row axes[i] of positions [n, T]."""
    x = np.asarray(x, np.float64)
    n = len(inv_freq)
    positions = np.asarray(positions, np.float64)
    at = positions[:, None] if axes is None else positions[np.asarray(axes)].T
    ang = at * np.asarray(inv_freq, np.float64)[None, :]
    c, s = factor * np.cos(ang)[:, None, :], factor * np.sin(ang)[:, None, :]
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    out = x.copy()
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    return out


def slots_of(table_row, length, page_size, pool):
    """Cache entries of a sequence's tokens; -1 where the page is outside the pool."""
    t = np.arange(length)
    page = np.asarray(table_row, np.int64)[t // page_size]
    ok = (page >= 0) & (page < pool // page_size)
    return np.where(ok, page * page_size + t % page_size, -1)


def kv_attention(q, k, v, block_table, seq_lens, page_size, q_start=None, scale=None, causal=True, window=0):
    """(out [T, Hq, D], lse [T, Hq], written [T], spread [T, Hq, D]) of q over cache values k, v
    [pool, Hk, D]: softmax attention of each sequence's last query tokens.  Rows that see nothing give 0 and
    -inf; `written` marks the rows that belong to a sequence; `spread` is sum_t p_t |v_t|, which error
    bounds scale with."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    T, Hq, D = q.shape
    pool, Hk, _ = k.shape
    B = len(seq_lens)
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    starts = np.arange(B + 1) if q_start is None else np.asarray(q_start)
    out, spread = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((T, Hq), -np.inf)
    written = np.zeros(T, bool)
    for b in range(B):
        L, lo, hi = int(seq_lens[b]), int(starts[b]), int(starts[b + 1])
        nq = hi - lo
        written[lo:hi] = True
        slot = slots_of(block_table[b], L, page_size, pool)
        for i in range(nq):
            p = L - nq + i
            t = np.arange(L)
            see = slot >= 0
            if causal:
                see &= t <= p
            if window:
                see &= t > p - window
            at = slot[see]
            if at.size == 0:
                continue
            for h in range(Hq):
                s = scale * (k[at, h // G] @ q[lo + i, h])
                m = s.max()
                w = np.exp(s - m)
                lse[lo + i, h] = m + np.log(w.sum())
                w /= w.sum()
                out[lo + i, h] = w @ v[at, h // G]
                spread[lo + i, h] = w @ np.abs(v[at, h // G])
    return out, lse, written, spread
