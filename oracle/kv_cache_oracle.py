"""The paged KV cache operators in plain 64-bit numpy -- TEST INFRASTRUCTURE.

Written from the definitions in include/peagle_cache.h, request by request;
shares no code with the library.  Pools are float64 arrays [num_blocks, H,
16, D] (for e4m3 pools: the codes' values, the scales apart)."""

from __future__ import annotations

import numpy as np

PAGE = 16


def rotate(x, pos, theta):
    """Rotate-half RoPE of x [..., D] at positions pos [...]."""
    x = np.asarray(x, np.float64)
    if not theta:
        return x.copy()
    half = x.shape[-1] // 2
    freq = float(theta) ** (-np.arange(half) / half)
    ang = np.asarray(pos, np.float64)[..., None] * freq
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., :half], x[..., half:]
    return np.concatenate((a * c - b * s, b * c + a * s), axis=-1)


def slot(table, b, p):
    return int(table[b][p // PAGE]), p % PAGE


def gather(pool, table, b, lo, n):
    """Rows lo .. n - 1 of request b, [n - lo, H, D]."""
    return np.stack([pool[blk, :, off] for blk, off in (slot(table, b, p) for p in range(lo, n))])


def append(k_pool, v_pool, scores, k, v, pos, req, table, theta):
    """Writes into the pools; returns the written (block, offset) of each row
    (None for padding)."""
    out = []
    for t in range(len(pos)):
        if pos[t] < 0:
            out.append(None)
            continue
        blk, off = slot(table, int(req[t]), int(pos[t]))
        k_pool[blk, :, off] = rotate(k[t], np.full(k.shape[1], pos[t]), theta)
        v_pool[blk, :, off] = v[t]
        if scores is not None:
            scores[blk, :, off] = 0.0
        out.append((blk, off))
    return out


class Decoded:
    """out [B, Hq, D], lse [B, Hq], weights per request [H, n] at positions
    lo .. n - 1, and what the tolerances need: spread = sum_j p_j |v_j|
    (like out), zabs = the largest sum_i |scale q_i k_i| of the row [B, Hq],
    vmax, peak = 1 / (largest weight) [B, Hq]."""


def decode(k_pool, v_pool, q, table, lens, window=0, scale=None):
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    H = k_pool.shape[1]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    r = Decoded()
    r.out, r.spread = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    r.lse, r.zabs, r.vmax = np.full((B, Hq), -np.inf), np.zeros((B, Hq)), np.zeros((B, Hq))
    r.peak = np.ones((B, Hq))
    r.lo, r.weights = [], []
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        r.lo.append(lo)
        w = np.zeros((H, max(0, n - lo)))
        r.weights.append(w)
        if n <= lo:
            continue
        K, V = gather(k_pool, table, b, lo, n), gather(v_pool, table, b, lo, n)
        for h in range(Hq):
            kh, vh = K[:, h // G], V[:, h // G]
            z = scale * (kh @ q[b, h])
            top = z.max()
            if top == -np.inf:
                continue
            e = np.exp(z - top)
            total = e.sum()
            p = e / total
            r.out[b, h] = p @ vh
            r.spread[b, h] = p @ np.abs(vh)
            r.lse[b, h] = top + np.log(total)
            r.zabs[b, h] = (abs(scale) * np.abs(kh) @ np.abs(q[b, h])).max()
            r.vmax[b, h] = np.abs(vh).max()
            r.peak[b, h] = 1.0 / p.max()
            w[h // G] += p
    return r


def keep(scores, budget, sinks, recent):
    """Positions that stay of a row with these scores [n]."""
    n = len(scores)
    if n <= budget:
        return np.arange(n)
    z = np.asarray(scores, np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    mid = list(range(sinks, n - recent))
    mid.sort(key=lambda p: (-z[p], p))
    return np.array(sorted(list(range(sinks)) + mid[:budget - sinks - recent]
                           + list(range(n - recent, n))), dtype=np.int64)


def evict(k_pool, v_pool, scores, table, lens, budget, sinks, recent, theta, dst_table=None):
    """One layer; returns (kept [B, H, budget], new_lens, and copies of the
    pools and scores after the trim)."""
    B, H = len(lens), k_pool.shape[1]
    k2, v2, s2 = k_pool.copy(), v_pool.copy(), scores.copy()
    kept = np.full((B, H, budget), -1, np.int64)
    new = np.minimum(lens, budget)
    dst = table if dst_table is None else dst_table
    for b in range(B):
        n, m = int(lens[b]), int(new[b])
        for h in range(H):
            row = np.array([scores[blk, h, off] for blk, off in
                            (slot(table, b, p) for p in range(n))])
            kept[b, h, :m] = keep(row, budget, sinks, recent)
            for j in range(m):
                p = int(kept[b, h, j])
                sb, so = slot(table, b, p)
                db, do = slot(dst, b, j)
                x = k_pool[sb, h, so]
                k2[db, h, do] = rotate(x, j - p, theta) if p != j else x
                v2[db, h, do] = v_pool[sb, h, so]
                s2[db, h, do] = scores[sb, h, so]
            end = -(-m // PAGE) * PAGE
            if dst_table is None:
                end = max(end, n)
            for j in range(m, end):
                db, do = slot(dst, b, j)
                s2[db, h, do] = 0.0
    return kept, new, k2, v2, s2
