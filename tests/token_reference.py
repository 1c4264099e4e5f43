"""Plain 64-bit forms of the operators that fill the cache and attend to it
with many tokens a request, written from their definitions."""
from __future__ import annotations

import numpy as np

from tests.cache_reference import D, G, S, bf16_to_f64


def turned(x, weight, eps, inv_freq, axis, positions, interleaved=False, scale=1.0):
    """(rows, sizes) of rows x [T][H][d] fp64 after norm and rotation; sizes [T][H][d] are |a| + |b| of an element's pair
    (its own magnitude where it is not rotated), what the arithmetic's errors are relative to.  positions [axes][T]."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight if weight is not None else x.copy()
    size = np.abs(y)
    for i, (f, a) in enumerate(zip(inv_freq, axis)):
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
        t = (positions[a].astype(np.float64) * f)[:, None]
        u, v = y[..., first].copy(), y[..., second].copy()
        y[..., first], y[..., second] = scale * (u * np.cos(t) - v * np.sin(t)), scale * (v * np.cos(t) + u * np.sin(t))
        size[..., first] = size[..., second] = abs(scale) * (np.abs(u) + np.abs(v))
    return y, size


def request_rows(token_starts, seq_lens, max_pages):
    """(request, row, index in the request) of every row whose request takes part in an append."""
    for r, L in enumerate(int(x) for x in seq_lens):
        lo, hi = int(token_starts[r]), int(token_starts[r + 1])
        if hi - lo <= L <= max_pages * S:
            for i in range(hi - lo):
                yield r, lo + i, L - (hi - lo) + i


def attend_chunk(q, k, v, table, seq_lens, token_starts, scale, causal, num_pages=None):
    """(out [T][Hq][d], sizes) in fp64 of bf16 bit patterns; sizes are sum w |v|.  Rows of no request are NaN."""
    T, Hq = q.shape[:2]
    P, H = k.shape[:2]
    num_pages = P if num_pages is None else num_pages
    out, size = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    qd = bf16_to_f64(q)
    for r, L in enumerate(int(x) for x in seq_lens):
        L = min(max(L, 0), table.shape[1] * S)
        lo, hi = int(token_starts[r]), int(token_starts[r + 1])
        t = np.arange(L)
        page = table[r, t // S]
        there = (page >= 0) & (page < num_pages)
        for j in range(H):
            ks, vs = (bf16_to_f64(x[np.where(there, page, 0), j, t % S]) for x in (k, v))
            for i in range(hi - lo):
                vis = L - (hi - lo) + i + 1 if causal else L
                use = there & (t < vis)
                o, z = out[lo + i, j * G:(j + 1) * G], size[lo + i, j * G:(j + 1) * G]
                o[:], z[:] = 0.0, 0.0
                if not use.any():
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = qd[lo + i, j * G:(j + 1) * G] @ ks[use].T * scale
                    e = np.exp(s - s.max(1, keepdims=True))
                    w = e / e.sum(1, keepdims=True)
                    o[:], z[:] = w @ vs[use], w @ np.abs(vs[use])
    return out, size
