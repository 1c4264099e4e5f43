"""Plain 64-bit forms of the cache operators, written from their definitions:
shared-prefix attention with the own tokens' weights, and eviction."""
from __future__ import annotations

import numpy as np

S, D, G = 16, 128, 4


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def tokens_of(pool, pages, j, n):
    """The first n tokens of head j of the listed physical pages, [n][d] fp64; ids outside the pool drop their tokens."""
    rows = []
    for i, p in enumerate(pages):
        if i * S >= n:
            break
        if 0 <= p < pool.shape[0]:
            rows.append(pool[p, j, :min(S, n - i * S)])
    return bf16_to_f64(np.concatenate(rows)) if rows else np.zeros((0, D))


def attend_shared(q, k, v, prefix_table, prefix_lens, group_starts, lists, lengths, seq_lens, scale, weights=None):
    """(out [B][Hq][d], |v|-weighted scale of each output, weights) in fp64; weights starts from `weights`."""
    B, Hq = q.shape[:2]
    H = Hq // G
    out, size = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    w = None if weights is None else weights.astype(np.float64).copy()
    qd = bf16_to_f64(q)
    for r in range(B):
        g = next((g for g in range(len(prefix_lens)) if group_starts[g] <= r < group_starts[g + 1]), None)
        for j in range(H):
            ln = int(lengths[r, j])
            own = lists[r, j, :ln]
            tail = int(seq_lens[r]) % S
            n = ln * S - (S - tail if ln and tail else 0)
            ks, vs = tokens_of(k, own, j, n), tokens_of(v, own, j, n)
            n_own = len(ks)
            if g is not None and prefix_lens[g] > 0:
                ks = np.concatenate([ks, tokens_of(k, prefix_table[g], j, int(prefix_lens[g]))])
                vs = np.concatenate([vs, tokens_of(v, prefix_table[g], j, int(prefix_lens[g]))])
            if not len(ks):
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                s = qd[r, j * G:(j + 1) * G] @ ks.T * scale
                e = np.exp(s - s.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
                out[r, j * G:(j + 1) * G] = p @ vs
                size[r, j * G:(j + 1) * G] = p @ np.abs(vs)
            if w is not None:
                at = 0
                for i, pid in enumerate(own):
                    t = min(S, n - i * S)
                    if 0 <= pid < k.shape[0]:
                        w[pid, j, :t] += p[:, at:at + t].sum(0)
                        at += t
    return out, size, w


def evict(k, v, weights, positions, table, seq_lens, budget, sinks, recent, num_pages=None):
    """In-place eviction on host copies; returns (new_lens, pages whose keys changed per head as (page, head))."""
    P, H = weights.shape[:2]
    num_pages = P if num_pages is None else num_pages
    new, renewed = [], []
    for r, n in enumerate(int(x) for x in seq_lens):
        n = min(max(n, 0), table.shape[1] * S)
        m = min(n, budget)
        pages = table[r, :-(-n // S)]
        if n > m and (np.any(pages < 0) or np.any(pages >= num_pages)):
            new.append(n)
            continue
        new.append(m)
        if n <= m:
            continue
        pg, sl = pages[np.arange(n) // S].astype(np.int64), np.arange(n) % S
        for j in range(H):
            w, pos = weights[pg, j, sl], positions[pg, j, sl].astype(np.int64)
            unset = np.flatnonzero(pos < 0)
            if len(unset):
                pos[unset] = pos.max() + 1 + unset - unset[0] if pos.max() >= 0 else unset - unset[0]
            protected = (pos < sinks) | (pos > pos.max() - recent)
            order = sorted(range(n), key=lambda t: (0 if protected[t] else 1,
                                                    0.0 if protected[t] else
                                                    (np.inf if np.isnan(w[t]) else -float(w[t])),
                                                    np.isnan(w[t]) and not protected[t], t))
            keep = np.zeros(n, bool)
            keep[order[:m]] = True
            holes, movers = np.flatnonzero(~keep[:m]), m + np.flatnonzero(keep[m:])
            assert len(holes) == len(movers)
            for a, b in zip(holes, movers):
                k[pg[a], j, sl[a]] = k[pg[b], j, sl[b]]
                v[pg[a], j, sl[a]] = v[pg[b], j, sl[b]]
                w[a], pos[a] = w[b], pos[b]
            w[m:], pos[m:] = 0.0, -1
            weights[pg, j, sl], positions[pg, j, sl] = w, pos
            renewed += [(int(table[r, p]), j) for p in np.unique(holes // S) if p < m // S]
    return np.asarray(new, np.int32), renewed
