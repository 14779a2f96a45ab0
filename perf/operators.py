"""The paged KV cache operators, as they are measured.

Three operators that work on one paged pool layout, [num_blocks, kv heads, 16
positions, head_dim], with block tables and lengths per request:

  append  rotary embedding of new tokens' q and k at their positions, and the
          write of k and v into the requests' pages (16 bits, or e4m3 codes)
  decode  attention of one new token per request over its pages (grouped
          heads, optional window), with the log-sum-exp of each row and, where
          asked, each position's attention weight added to the pool's scores
  evict   the positions of a cache that are kept by accumulated weight (the
          first ones, the last ones, the heaviest of the rest, per kv head),
          written in order to fresh pages, keys rotated to their new positions

`own` selects the plain form (torch, 32 bits) or the framework's calls.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a single user's next token: the smallest call, all latency
        dict(name="append-b1", op="append", reqs=1, rows=1, ctx_lo=100, ctx_hi=100, lens_seed=1,
             heads=64, kv_heads=8, dim=64, dtype="bf16", theta=1.5e5),
        # a serving batch's next tokens into an 8-bit cache
        dict(name="append-b64-e4m3", op="append", reqs=64, rows=64, ctx_lo=1, ctx_hi=250,
             lens_seed=2, heads=64, kv_heads=8, dim=64, dtype="e4m3", theta=1.5e5),
        # prompt chunks of four requests prefilled together
        dict(name="append-chunks", op="append", reqs=4, rows=2048, ctx_lo=1, ctx_hi=700,
             lens_seed=3, heads=32, kv_heads=4, dim=128, dtype="bf16", theta=1e6),
        # the debug-precision drafter's single short request
        dict(name="decode-tiny-f32", op="decode", reqs=1, lens="uniform", lo=68, hi=68,
             lens_seed=4, heads=4, kv_heads=4, dim=64, dtype="f32", window=0, scores=False),
        # one user at a few thousand tokens: split over the length or idle
        dict(name="decode-b1", op="decode", reqs=1, lens="uniform", lo=4096, hi=4096,
             lens_seed=5, heads=64, kv_heads=8, dim=64, dtype="bf16", window=0, scores=False),
        # a full serving batch with the long-tailed lengths of chat traffic
        dict(name="decode-b64", op="decode", reqs=64, lens="lognormal", lo=1, hi=20000,
             lens_seed=6, heads=64, kv_heads=8, dim=64, dtype="bf16", window=0, scores=False),
        # the same traffic with 8-bit pools, collecting weights for eviction
        dict(name="decode-b64-e4m3-scores", op="decode", reqs=64, lens="lognormal", lo=1,
             hi=20000, lens_seed=7, heads=64, kv_heads=8, dim=64, dtype="e4m3", window=0,
             scores=True),
        # wider heads, fewer requests, long contexts, collecting weights
        dict(name="decode-b16-scores", op="decode", reqs=16, lens="uniform", lo=1024, hi=16384,
             lens_seed=8, heads=32, kv_heads=4, dim=128, dtype="bf16", window=0, scores=True),
        # an unfilled slot, a first token and odd lengths in one padded batch,
        # five heads a group, a sliding window
        dict(name="decode-ragged-window", op="decode", reqs=33, lens="ragged", lo=0, hi=3001,
             lens_seed=9, heads=10, kv_heads=2, dim=128, dtype="bf16", window=1000,
             scores=False),
        # one long request trimmed to a quarter in the drafter's four layers
        dict(name="evict-b1", op="evict", layers=4, reqs=1, lens="uniform", lo=4096, hi=4096,
             lens_seed=10, kv_heads=8, dim=64, dtype="bf16", budget=1024, sinks=4, recent=256,
             theta=1.5e5),
        # a whole serving batch trimmed at once
        dict(name="evict-b64", op="evict", layers=4, reqs=64, lens="lognormal", lo=1, hi=20000,
             lens_seed=11, kv_heads=8, dim=64, dtype="bf16", budget=2048, sinks=4, recent=512,
             theta=1.5e5),
        # 8-bit pools, an odd budget, no first positions kept
        dict(name="evict-b16-e4m3", op="evict", layers=4, reqs=16, lens="uniform", lo=1024,
             hi=16384, lens_seed=12, kv_heads=4, dim=128, dtype="e4m3", budget=1501, sinks=0,
             recent=333, theta=1e6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "evict"))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 5, 7, 8, 12, 16))
    dtype = rng.choice(("bf16", "bf16", "e4m3", "f32"))
    theta = rng.choice((1e4, 1.5e5, 1e6))
    base = dict(op=op, lens_seed=rng.randrange(1 << 20), kv_heads=kv_heads, dim=dim, dtype=dtype)
    size = {"bf16": 2, "e4m3": 1, "f32": 4}[dtype]
    if op == "append":
        reqs = _log_int(rng, 1, 128)
        rows = reqs if rng.random() < 0.5 else max(reqs, _log_int(rng, 1, 3000))
        return dict(base, reqs=reqs, rows=rows, ctx_lo=0, ctx_hi=_log_int(rng, 1, 600),
                    heads=heads, theta=theta)
    # at most about half of the largest listed case's bytes in K and V
    keys = int(300e6 / (2 * kv_heads * dim * size))
    reqs = _log_int(rng, 1, 128)
    hi = max(1, min(_log_int(rng, 1, 60000), keys // reqs))
    lens = rng.choice(("uniform", "ragged"))
    base.update(reqs=reqs, lens=lens, lo=0 if lens == "ragged" else max(1, hi // 8), hi=hi)
    if op == "decode":
        return dict(base, heads=heads, window=rng.choice((0, 0, _log_int(rng, 1, 4000))),
                    scores=rng.random() < 0.5)
    budget = _log_int(rng, 1, 4000)
    sinks = min(budget, rng.choice((0, 1, 4, 17)))
    recent = rng.randint(0, budget - sinks)
    return dict(base, layers=rng.choice((1, 2, 4)), budget=budget, sinks=sinks, recent=recent,
                theta=rng.choice((0.0, theta)))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lens(case):
    """The requests' lengths: part of the case, not of the seed."""
    rng = np.random.default_rng(case["lens_seed"])
    n = case["reqs"]
    if case["op"] == "append":
        return rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=n)
    lo, hi = case["lo"], case["hi"]
    if case["lens"] == "lognormal":
        return np.clip(np.exp(rng.normal(math.log(3891.0), 0.7966, size=n)), max(lo, 1),
                       hi).astype(np.int64)
    out = rng.integers(lo, hi + 1, size=n)
    if case["lens"] == "ragged":
        edge = np.minimum(np.array([0, 1, 15, 16, 17, 31, 33, hi]), hi)
        out[:min(n, len(edge))] = edge[:n]
    return out


def _rows_of(case):
    """append: each row's request and position (every request's new rows
    follow its cached ones)."""
    n, rows = case["reqs"], case["rows"]
    req = np.sort(np.arange(rows) % n)
    first = np.searchsorted(req, np.arange(n))
    pos = _lens(case)[req] + np.arange(rows) - first[req]
    return req, pos


def _table(lens, rng, extra=0):
    """A block table over randomly ordered pages (entries that no position
    reaches hold -1), and the number of pages, `extra` of them unused."""
    pages = -(-lens // PAGE)
    total = int(pages.sum()) + extra
    order = rng.permutation(total)
    table = np.full((len(lens), max(1, int(pages.max()))), -1, dtype=np.int32)
    at = np.arange(table.shape[1])[None, :] < pages[:, None]
    table[at] = order[:int(pages.sum())]
    return table, order[int(pages.sum()):], max(1, total)


def _normal(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale
    if dtype == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, case["lens_seed"]])
    op, dt, H, D = case["op"], case["dtype"], case["kv_heads"], case["dim"]
    act = "f32" if dt == "f32" else "bf16"
    s = dict(case=case)
    s["scales"] = (0.02 + 0.01 * (seed % 5), 0.03) if dt == "e4m3" else (1.0, 1.0)
    unit = 50.0 if dt == "e4m3" else 1.0       # codes that stand for about N(0, 1)
    if op == "append":
        lens = _lens(case)
        req, pos = _rows_of(case)
        table, _, blocks = _table(lens + np.bincount(req, minlength=case["reqs"]), rng)
        s["req"], s["pos"], s["table"] = _i32(req), _i32(pos), _i32(table)
        T, Hq = case["rows"], case["heads"]
        qkv = _normal((T, Hq + 2 * H, D), act, g)   # one fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.empty(T, Hq, D, dtype=qkv.dtype, device="cuda")
        layers = 1
    else:
        lens = _lens(case)
        layers = case.get("layers", 1)
        fresh = -(-np.minimum(lens, case["budget"]) // PAGE) if op == "evict" else 0 * lens
        table, spare, blocks = _table(lens, rng, int(fresh.sum()))
        s["table"], s["lens"] = _i32(table), _i32(lens)
    s["k_pool"] = _normal((layers, blocks, H, PAGE, D), dt, g, unit)
    s["v_pool"] = _normal((layers, blocks, H, PAGE, D), dt, g, unit)
    s["scores"] = None
    if op == "decode":
        s["q"] = _normal((case["reqs"], case["heads"], D), act, g, 2.0)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["reqs"], case["heads"], device="cuda")
        if case["scores"]:
            s["scores"] = torch.rand((layers, blocks, H, PAGE), generator=g, device="cuda")
    if op == "evict":
        # accumulated weights: long-tailed, a third of the positions never hit
        w = torch.randn((layers, blocks, H, PAGE), generator=g, device="cuda")
        hit = torch.rand(w.shape, generator=g, device="cuda") > 0.33
        s["scores"] = torch.where(hit, torch.exp(1.5 * w), torch.zeros_like(w))
        dst = np.full((case["reqs"], max(1, int(fresh.max()))), -1, dtype=np.int32)
        dst[np.arange(dst.shape[1])[None, :] < fresh[:, None]] = spare
        s["dst"] = _i32(dst)
        s["kept"] = torch.empty(layers, case["reqs"], H, case["budget"], dtype=torch.int32,
                                device="cuda")
        s["new_lens"] = torch.empty(case["reqs"], dtype=torch.int32, device="cuda")
    if own:      # the handle of each layer's pool, which a program keeps
        from speculative_drafting_expand_gb300 import KvPool
        s["pools"] = [KvPool(s["k_pool"][i], s["v_pool"][i],
                             None if s["scores"] is None else s["scores"][i], *s["scales"])
                      for i in range(layers)]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(pool, scale):
    if pool.dtype == torch.uint8:
        return pool.view(torch.float8_e4m3fn).float() * scale
    return pool.float()


def _store(x, like, scale):
    """32-bit values as the pool holds them, rounded once."""
    if like.dtype == torch.uint8:
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(like.dtype)


def _as_values(pool):
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _rotate(x, pos, theta):
    """x [..., D] at positions pos [...]: pairs (i, i + D / 2) turned by
    pos * theta^(-2 i / D); the angle in 64 bits."""
    if not theta:
        return x
    half = x.shape[-1] // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    ang = pos.double().unsqueeze(-1) * torch.pow(torch.tensor(theta, dtype=torch.float64,
                                                              device=x.device), -i / half)
    c, sn = torch.cos(ang).float(), torch.sin(ang).float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * c - b * sn, b * c + a * sn), dim=-1)


def _plain_append(s):
    c = s["case"]
    pos, req = s["pos"].long(), s["req"].long()
    block = s["table"].long()[req, pos // PAGE]
    q = _rotate(s["q"].float(), pos[:, None], c["theta"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), pos[:, None], c["theta"])
    s["k_pool"][0][block, :, pos % PAGE] = _store(k, s["k_pool"], s["scales"][0])
    s["v_pool"][0][block, :, pos % PAGE] = _store(s["v"].float(), s["v_pool"], s["scales"][1])
    return dict(q=q, k=_as_values(s["k_pool"]), v=_as_values(s["v_pool"]))


def _plain_decode(s):
    c = s["case"]
    B, Hq, H, D = c["reqs"], c["heads"], c["kv_heads"], c["dim"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * PAGE
    at = torch.arange(n, device="cuda")
    lens = s["lens"].long()[:, None]
    on = (at < lens) & (at >= lens - (c["window"] or n))
    kv = [_values(p[0], x)[table].transpose(1, 2).reshape(B, H, n, D)
          for p, x in ((s["k_pool"], s["scales"][0]), (s["v_pool"], s["scales"][1]))]
    q = s["q"].float().view(B, H, Hq // H, D)
    z = torch.matmul(q, kv[0].transpose(2, 3)) * D ** -0.5
    z = z.masked_fill(~on[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv[1]) / total.clamp(min=1e-38)
    out = dict(out=out.view(B, Hq, D).to(s["q"].dtype),
               lse=(top + torch.log(total)).view(B, Hq))
    if s["scores"] is not None:
        w = (p / total.clamp(min=1e-38)).sum(2)                      # [B, H, n]
        w = w.view(B, H, -1, PAGE).transpose(1, 2).reshape(-1, H, PAGE)
        s["scores"][0].index_add_(0, table.reshape(-1), w)
        out["scores"] = s["scores"]
    return out


def _plain_evict(s):
    c = s["case"]
    L, B, H, D, N = c["layers"], c["reqs"], c["kv_heads"], c["dim"], c["budget"]
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * PAGE
    at = torch.arange(n, device="cuda")
    lens = s["lens"].long()[:, None]
    z = s["scores"][:, table].transpose(2, 3).reshape(L, B, H, n)
    # 2: kept whatever their weight, 1: by weight, 0: not in the cache
    cls = (at < lens).long() + ((at < lens) & ((at < c["sinks"]) | (at >= lens - c["recent"])
                                               | (lens <= N))).long()
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices
    cls = cls[None, :, None].expand(L, B, H, n)
    by = torch.sort(cls.gather(-1, order), dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, by)[..., :N]
    new = lens.clamp(max=N)
    j = torch.arange(order.shape[-1], device="cuda")
    kept = torch.where(j < new[:, None], order, n).sort(-1).values     # [L, B, H, <= N]
    live = kept < n
    kept = torch.where(live, kept, torch.zeros_like(kept))
    head = torch.arange(H, device="cuda")[:, None]
    layer = torch.arange(L, device="cuda")[:, None, None, None]
    req = torch.arange(B, device="cuda")[:, None, None]
    src = ((layer * s["k_pool"].shape[1] + table[req, kept // PAGE]) * H + head) * PAGE + kept % PAGE
    dst = s["dst"].long()[req, (j // PAGE).clamp(max=s["dst"].shape[1] - 1)].clamp(min=0)
    dst = ((layer * s["k_pool"].shape[1] + dst) * H + head) * PAGE + j % PAGE
    src, dst = src[live], dst.expand_as(kept)[live]
    turn = (j - kept)[live]
    kp, vp, sp = s["k_pool"].view(-1, D), s["v_pool"].view(-1, D), s["scores"].view(-1)
    if c["theta"]:
        moved = _store(_rotate(_values(kp[src], 1.0), turn, c["theta"]), kp, 1.0)
        kp[dst] = torch.where(turn[:, None] == 0, kp[src], moved)
    else:
        kp[dst] = kp[src]
    vp[dst] = vp[src]
    # the rest of the last fresh page starts without weight
    rest = torch.arange(s["dst"].shape[1] * PAGE, device="cuda")
    end = -(-new // PAGE) * PAGE
    rest_on = (rest >= new) & (rest < end)
    page = s["dst"].long().clamp(min=0).repeat_interleave(PAGE, 1)
    where = (page[:, None] * H + head) * PAGE + rest % PAGE
    where = (layer * s["k_pool"].shape[1] * H * PAGE + where)[rest_on[None, :, None].expand(L, B, H, -1)]
    moved = sp[src]
    sp[where] = 0.0
    sp[dst] = moved
    full = torch.full((L, B, H, N), -1, dtype=torch.int32, device="cuda")
    full[..., :kept.shape[-1]] = torch.where(live, kept, torch.full_like(kept, -1)).int()
    return dict(kept=full, lens=new[:, 0].int(), k=_as_values(s["k_pool"]),
                v=_as_values(s["v_pool"]), scores=s["scores"])


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[c["op"]](s)
    import speculative_drafting_expand_gb300 as pe
    if c["op"] == "append":
        pe.pe_kv_append(s["pools"][0], s["q"], s["k"], s["v"], s["pos"], s["table"], c["theta"],
                        req=s["req"], q_out=s["q_out"])
        return dict(q=s["q_out"], k=_as_values(s["k_pool"]), v=_as_values(s["v_pool"]))
    if c["op"] == "decode":
        pe.pe_attn_decode(s["pools"][0], s["q"], s["table"], s["lens"], window=c["window"],
                          accumulate=c["scores"], out=s["out"], lse=s["lse"])
        out = dict(out=s["out"], lse=s["lse"])
        if c["scores"]:
            out["scores"] = s["scores"]
        return out
    pe.pe_kv_evict(s["pools"], s["table"], s["lens"], c["budget"], c["sinks"], c["recent"],
                   rope_theta=c["theta"], dst_table=s["dst"], kept=s["kept"],
                   new_lens=s["new_lens"])
    return dict(kept=s["kept"], lens=s["new_lens"], k=_as_values(s["k_pool"]),
                v=_as_values(s["v_pool"]), scores=s["scores"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "e4m3": 1, "f32": 4}[case["dtype"]]
    act = 4 if case["dtype"] == "f32" else 2
    H, D = case["kv_heads"], case["dim"]
    lens = _lens(case)
    if case["op"] == "append":
        T, Hq = case["rows"], case["heads"]
        return dict(bytes=T * ((2 * Hq + 2 * H) * D * act + 2 * H * D * size + 12),
                    flops=3 * T * (Hq + H) * D)
    if case["op"] == "decode":
        B, Hq = case["reqs"], case["heads"]
        seen = np.minimum(lens, case["window"] or lens)
        keys = int(seen.sum())
        return dict(bytes=2 * keys * H * D * size + B * Hq * (2 * D * act + 4) + 4 * B
                    + int((-(-seen // PAGE)).sum()) * 4
                    + (8 * keys * H if case["scores"] else 0),
                    flops=4 * keys * Hq * D)
    # evict: every score once; each kept row of K and V read and written once,
    # with its score and its place in the list
    kept = int(np.minimum(lens, case["budget"]).sum())
    L = case["layers"]
    return dict(bytes=L * H * (int(lens.sum()) * 4 + kept * (4 * D * size + 8)),
                flops=3 * L * H * kept * D if case["theta"] else 0)


# ---------------------------------------------------------------------------
# the definition, in 64 bits, request by request
# ---------------------------------------------------------------------------

def _slot_rows(table_row, n):
    """Pool rows (block, offset) of positions 0 .. n - 1 of one request."""
    i = np.arange(n)
    t = np.asarray(table_row)
    return torch.from_numpy(t[i // PAGE].astype(np.int64)).cuda(), torch.from_numpy(i % PAGE).cuda()


def _turn64(x, pos, theta):
    """Complex rotation of the pairs (i, i + D / 2) of x (64 bits)."""
    half = x.shape[-1] // 2
    freq = torch.from_numpy(float(theta) ** (-np.arange(half) * 2.0 / (2 * half))).cuda()
    z = torch.complex(x[..., :half], x[..., half:])
    z = z * torch.polar(torch.ones_like(pos[..., None] * freq), pos[..., None] * freq)
    return torch.cat((z.real, z.imag), dim=-1)


def _held(pool, scale=1.0):
    return (pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool).double() * scale


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    H, D, theta = case["kv_heads"], case["dim"], case.get("theta", 0.0)
    table = s["table"].cpu().numpy()
    if case["op"] == "append":
        req, pos = _rows_of(case)
        ks, vs = s["scales"]
        p = torch.from_numpy(pos.astype(np.float64)).cuda()[:, None]
        k, v = _held(s["k_pool"]), _held(s["v_pool"])
        block = torch.from_numpy(table[req, pos // PAGE].astype(np.int64)).cuda()
        off = torch.from_numpy(pos % PAGE).cuda()
        lim = 448.0 if case["dtype"] == "e4m3" else math.inf
        k[0][block, :, off] = (_turn64(s["k"].double(), p, theta) / ks).clamp(-lim, lim)
        v[0][block, :, off] = (s["v"].double() / vs).clamp(-lim, lim)
        return dict(q=_turn64(s["q"].double(), p, theta), k=k, v=v)
    lens = _lens(case)
    if case["op"] == "decode":
        B, Hq = case["reqs"], case["heads"]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        acc = None if s["scores"] is None else s["scores"].double()
        for b in range(B):
            n = int(lens[b])
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            blk, off = (t[lo:] for t in _slot_rows(table[b], n))
            keys = _held(s["k_pool"][0][blk, :, off], s["scales"][0])     # [n, H, D]
            vals = _held(s["v_pool"][0][blk, :, off], s["scales"][1])
            q = s["q"][b].double().reshape(H, Hq // H, D)
            z = torch.einsum("hgd,nhd->hgn", q, keys) / math.sqrt(D)
            lse[b] = torch.logsumexp(z, -1).reshape(Hq)
            w = torch.softmax(z, -1)
            out[b] = torch.einsum("hgn,nhd->hgd", w, vals).reshape(Hq, D)
            if acc is not None:
                acc[0][blk, :, off] += w.sum(1).transpose(0, 1)
        r = dict(out=out, lse=lse)
        if acc is not None:
            r["scores"] = acc
        return r
    # evict: kept positions by a sort of (weight, position) pairs on the host
    if int(lens.sum()) * H * case["layers"] > 30_000_000:
        return None
    N, sinks, recent = case["budget"], case["sinks"], case["recent"]
    dst = s["dst"].cpu().numpy()
    k, v, w = _held(s["k_pool"]), _held(s["v_pool"]), s["scores"].double()
    kept_all = np.full((case["layers"], case["reqs"], H, N), -1, dtype=np.int32)
    for layer in range(case["layers"]):
        for b in range(case["reqs"]):
            n = int(lens[b])
            m = min(n, N)
            if n == 0:
                continue
            blk, off = _slot_rows(table[b], n)
            z = s["scores"][layer][blk, :, off].cpu().numpy()             # [n, H]
            rows = []
            for h in range(H):
                if n <= N:
                    rows.append(np.arange(n))
                    continue
                mid = np.arange(sinks, n - recent)
                best = mid[np.lexsort((mid, -z[mid, h].astype(np.float64)))[:N - sinks - recent]]
                rows.append(np.sort(np.concatenate((np.arange(sinks), best,
                                                    np.arange(n - recent, n)))))
            rows = np.stack(rows, 1)                                      # [m, H]
            kept_all[layer, b, :, :m] = rows.T
            at = torch.from_numpy(rows).cuda()
            dblk, doff = _slot_rows(dst[b], m)
            hh = torch.arange(H, device="cuda")
            keys = _held(s["k_pool"][layer][blk[at], hh, off[at]])
            if theta:
                shift = (torch.arange(m, device="cuda")[:, None] - at).double()
                keys = torch.where(shift[..., None] == 0, keys, _turn64(keys, shift, theta))
                if case["dtype"] == "e4m3":
                    keys = keys.clamp(-448, 448)
            k[layer][dblk, :, doff] = keys
            v[layer][dblk, :, doff] = _held(s["v_pool"][layer][blk[at], hh, off[at]])
            end = -(-m // PAGE) * PAGE
            zb, zo = _slot_rows(dst[b], end)
            w[layer][zb[m:], :, zo[m:]] = 0.0
            w[layer][dblk, :, doff] = s["scores"][layer][blk[at], hh, off[at]].double()
    return dict(kept=None, lens=None, k=k, v=v, scores=w)
