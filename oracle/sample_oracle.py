"""Sampling, draft verification and 4-bit weights in plain numpy -- TEST
INFRASTRUCTURE.

Written from the definitions in include/peagle_sample.h and include/
peagle_w4.h, row by row, with Python's whole numbers; shares no code with the
library.  The exponentials e (fp32) are an argument, so that the decisions,
which are on whole numbers, can be checked exactly."""

from __future__ import annotations

import math
from dataclasses import dataclass, field
from typing import Dict, List

import numpy as np

ONE = 2 ** 31
MOST = np.finfo(np.float32).max


def clean(x):
    """Logits as the definition takes them, float32."""
    x = np.asarray(x, np.float32).copy()
    x[np.isnan(x)] = -np.inf
    x[x == np.inf] = MOST
    return x + np.float32(0)


def inverse(temperature):
    """(1 / temperature in fp32, greedy)."""
    t = np.float32(temperature)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(1) / t
    if not t > 0 or np.isinf(inv):
        return np.float32(0), True
    return inv, False


def exps(x, temperature):
    """e_i of a row in numpy's fp32 (other exponentials may be off by a step)."""
    x = clean(x)
    inv, _ = inverse(temperature)
    if x.max() == -np.inf:
        return np.zeros_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(((x - x.max()) * inv).astype(np.float32))
    return np.where(np.isnan(e), np.float32(0), e).astype(np.float32)


def weights(e):
    """Whole numbers of 2^-31, ties to even."""
    return [int(v) for v in np.rint(np.asarray(e, np.float64) * ONE)]


@dataclass
class Dist:
    kept: List[int] = field(default_factory=list)     # ids, in their order
    w: Dict[int, int] = field(default_factory=dict)    # kept weights by id
    total: int = 0
    cut: float = -math.inf
    cut_token: int = 0
    max: float = -math.inf


def dist(x, e, top_k=0, top_p=1.0, min_p=0.0, greedy=False) -> Dist:
    x = clean(x)
    V = len(x)
    w = weights(e)
    w = [0 if x[i] == -np.inf else w[i] for i in range(V)]
    mp = np.float32(0) if np.isnan(min_p) else np.float32(min(np.float32(min_p), 1))
    order = sorted((i for i in range(V) if w[i] > 0), key=lambda i: (-float(x[i]), i))
    positive = len(order)
    ok = [i for i in order if np.float32(e[i]) >= mp]
    ok = ok[:1] if greedy else ok[:top_k] if top_k > 0 else ok
    if np.float32(top_p) < 1:
        limit = float(np.float32(top_p)) * float(sum(w[i] for i in ok))
        before, take = 0, []
        for i in ok:
            if take and not float(before) < limit:
                break
            take.append(i)
            before += w[i]
        ok = take
    d = Dist(max=float(x.max()), cut_token=V - 1)
    d.kept, d.w = ok, {i: w[i] for i in ok}
    d.total = sum(d.w.values())
    if len(ok) < positive:
        d.cut, d.cut_token = float(x[ok[-1]]), ok[-1]
    return d


def draw(w: Dict[int, int], u) -> int:
    """Token of the place floor(u total) in the order of the ids; -1: none."""
    total = sum(w.values())
    if total == 0:
        return -1
    at = float(np.float32(u)) * float(total)
    at = 0 if math.isnan(at) else int(min(max(math.floor(at), 0), total - 1))
    run = 0
    for i in sorted(w):
        run += w[i]
        if run > at:
            return i
    raise AssertionError


def verify(rows: List[Dist], window, accept_u, u, draft_rows: List[Dist] | None = None):
    """One request: rows [n] the target's distributions, window [n] the
    tokens (the first is not a draft), draft_rows [n - 1].  Returns the
    accepted drafts and the token after them."""
    for j in range(len(rows) - 1):
        P, d, a = rows[j], int(window[j + 1]), float(np.float32(accept_u[j]))
        w = P.w.get(d, 0)
        if draft_rows is None:
            if w > 0 and (w == P.total or a * float(P.total) < float(w)):
                continue
            return j, draw({i: v for i, v in P.w.items() if i != d}, u)
        Q = draft_rows[j]
        if a * float(Q.w.get(d, 0)) * float(P.total) < float(w) * float(Q.total):
            continue
        if P.total == 0:
            return j, -1
        ap = np.float32(ONE / float(P.total))
        aq = np.float32(ONE / float(Q.total)) if Q.total else np.float32(0)
        p = {i: np.float32(v) * ap for i, v in P.w.items()}
        more = {i: int(np.rint(max(np.float32(v - np.float32(Q.w.get(i, 0)) * aq), 0)))
                for i, v in p.items()}
        if sum(more.values()) == 0:
            more = {i: int(np.rint(v)) for i, v in p.items()}
        return j, draw(more, u)
    return len(rows) - 1, draw(rows[-1].w, u)


def w4_matrix(codes, scales, k, group):
    """[n, k] in 64 bits from codes [n, (k + 1) // 2] and scales (float)."""
    n = codes.shape[0]
    c = np.empty((n, codes.shape[1] * 2), np.float64)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    return (c[:, :k] - 8) * np.repeat(np.asarray(scales, np.float64), group, axis=1)[:, :k]


def bf16(x):
    """Nearest bf16 (ties to even) of float32 values, as float32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32)


def w4_quantize(w, group):
    """Codes [n, k] and scales [n, ceil(k / group)] (bf16 values)."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    G = -(-k // group)
    scales = np.zeros((n, G), np.float32)
    codes = np.full((n, k), 8, np.int64)
    for g in range(G):
        part = w[:, g * group:(g + 1) * group]
        s = bf16(np.abs(part).max(1) / np.float32(7))
        scales[:, g] = s
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.rint((part / s[:, None]).astype(np.float32))
        codes[:, g * group:(g + 1) * group] = 8 + np.where(s[:, None] > 0, np.clip(q, -8, 7), 0)
    return codes, scales
