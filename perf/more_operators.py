"""The operators between a hidden row and the next drafting step, as they are
measured.

  w4       a few rows times a matrix of 4-bit weights with a scale for each
           group of inputs: the LM head or a projection of a quantised drafter
  sample   a token for each row of logits, from one given random number:
           temperature, top-k, min-p, top-p, then the inverse of the
           distribution function in the order of the token ids
  verify   the drafts of each request against the target's distributions by
           rejection sampling: how many are accepted and the token that
           follows them, which the next drafting step starts from

The distributions are held as whole numbers: token i of a row has the weight
rint(2^31 exp((x_i - max) / T)), the exponential in 32 bits, so that every sum
is exact and no order of additions can change a token.

`own` selects the plain form (torch, 32 bits) or the framework's calls.
"""

import math

import numpy as np
import torch

own = False

ONE = 2.0 ** 31
MOST = float(np.finfo(np.float32).max)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one row through the drafter's QKV projection: all latency
        dict(name="w4-qkv-b1", op="w4", rows=1, n=5120, k=2880, group=32, dtype="bf16",
             out="bf16"),
        # a single user's LM head: 290 MB of codes for one row
        dict(name="w4-head-b1", op="w4", rows=1, n=201088, k=2880, group=32, dtype="bf16",
             out="f32"),
        # the eight sampled rows of one request's drafting step
        dict(name="w4-head-k8", op="w4", rows=8, n=151936, k=2048, group=128, dtype="bf16",
             out="f32"),
        # a down projection at a batch of sixteen
        dict(name="w4-down-b16", op="w4", rows=16, n=2880, k=7680, group=64, dtype="bf16",
             out="bf16"),
        # the debug precision, a ragged last group and a ragged last tile
        dict(name="w4-odd-f32", op="w4", rows=5, n=1021, k=777, group=32, dtype="f32", out="f32"),
        # a single user's next token
        dict(name="sample-b1", op="sample", rows=1, vocab=201088, dtype="f32", filters="usual",
             masked=0.0, par_seed=1),
        # a vocabulary that is no multiple of anything, 16-bit logits, half of
        # the tokens ruled out by a grammar
        dict(name="sample-odd-bf16", op="sample", rows=33, vocab=50257, dtype="bf16",
             filters="mixed", masked=0.5, par_seed=2),
        # all drafts of a serving batch by temperature alone
        dict(name="sample-b64-k7", op="sample", rows=448, vocab=201088, dtype="f32",
             filters="none", masked=0.0, par_seed=3),
        # a batch whose users each set something else
        dict(name="sample-b128-mixed", op="sample", rows=128, vocab=151936, dtype="f32",
             filters="mixed", masked=0.0, par_seed=4),
        # one request's seven greedy drafts
        dict(name="verify-b1-k7", op="verify", reqs=1, drafts=7, ragged=False, vocab=201088,
             dtype="f32", filters="usual", sampled=False, par_seed=5),
        # a serving batch whose drafts were sampled
        dict(name="verify-b64-k7-sampled", op="verify", reqs=64, drafts=7, ragged=False,
             vocab=201088, dtype="f32", filters="mixed", sampled=True, par_seed=6),
        # windows of different lengths, requests without drafts among them
        dict(name="verify-ragged-bf16", op="verify", reqs=16, drafts=8, ragged=True, vocab=151936,
             dtype="bf16", filters="mixed", sampled=False, par_seed=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("w4", "sample", "verify"))
    if op == "w4":
        n = _log_int(rng, 16, 200000)
        k = _log_int(rng, 16, 9000)
        k = max(16, min(k, 500_000_000 // n))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return dict(op=op, rows=_log_int(rng, 1, 32 if dtype == "bf16" else 8), n=n, k=k,
                    group=rng.choice((32, 64, 128)), dtype=dtype,
                    out="f32" if dtype == "f32" else rng.choice(("bf16", "f32")))
    vocab = _log_int(rng, 8, 262144)
    base = dict(op=op, vocab=vocab, dtype=rng.choice(("f32", "f32", "bf16")),
                filters=rng.choice(("none", "usual", "mixed")), par_seed=rng.randrange(1 << 20))
    if op == "sample":
        rows = min(_log_int(rng, 1, 512), max(1, 80_000_000 // vocab))
        return dict(base, rows=rows, masked=rng.choice((0.0, 0.0, 0.3, 0.9)))
    drafts = rng.randint(1, 15)
    reqs = min(_log_int(rng, 1, 128), max(1, 80_000_000 // (vocab * (drafts + 1))))
    return dict(base, reqs=reqs, drafts=drafts, ragged=rng.random() < 0.5,
                sampled=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _params(case, n):
    """What the users set: temperature, top-k, top-p and min-p of each row (of
    each request); part of the case, not of the seed.  None: not set."""
    rng = np.random.default_rng(case["par_seed"])
    temp = rng.uniform(0.6, 1.2, n).astype(np.float32)
    if case["filters"] == "none":
        return temp, None, None, None
    k = np.full(n, 50, np.int32)
    p = np.full(n, 0.9, np.float32)
    mp = np.zeros(n, np.float32)
    if case["filters"] == "mixed":
        kind = rng.integers(0, 6, n)      # greedy, nothing, k, p, min-p, everything
        temp[kind == 0] = 0.0
        k = np.where((kind == 2) | (kind == 5), rng.choice([1, 5, 40, 200, 2000], n), 0)
        p = np.where((kind == 3) | (kind == 5), rng.uniform(0.5, 0.99, n), 1.0)
        mp = np.where((kind == 4) | (kind == 5), rng.choice([0.001, 0.02, 0.1], n), 0.0)
    return temp, k.astype(np.int32), p.astype(np.float32), mp.astype(np.float32)


def _windows(case):
    """First row of every request's window (its drafts and the row before)."""
    n = np.full(case["reqs"], case["drafts"] + 1)
    if case["ragged"]:
        n = np.random.default_rng(case["par_seed"] + 1).integers(1, case["drafts"] + 2,
                                                                 case["reqs"])
    return np.concatenate(([0], np.cumsum(n)))


def _logits(rows, vocab, g):
    """A bulk of unlikely tokens and a few likely ones."""
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 2.2
    at = torch.randint(vocab, (rows, 48), generator=g, device="cuda")
    up = torch.rand(rows, 48, generator=g, device="cuda") ** 2 * 14.0
    return x.scatter_reduce_(1, at, up, "amax")      # in any order the same


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "w4":
        n, k, group = case["n"], case["k"], case["group"]
        s["codes"] = torch.randint(256, (n, (k + 1) // 2), generator=g, device="cuda",
                                   dtype=torch.uint8)
        scales = torch.rand(n, -(-k // group), generator=g, device="cuda") * 0.01 + 0.002
        s["scales"] = scales.to(torch.bfloat16)
        s["x"] = torch.randn(case["rows"], k, generator=g, device="cuda").to(_type(case["dtype"]))
        s["y"] = torch.empty(case["rows"], n, dtype=_type(case["out"]), device="cuda")
        if own:        # the weights as the program keeps them
            from speculative_drafting_expand_gb300 import W4Weight
            s["w"] = W4Weight(s["codes"], s["scales"], k, group)
        return s
    V = case["vocab"]
    if case["op"] == "sample":
        x = _logits(case["rows"], V, g)
        if case["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < case["masked"],
                           -math.inf)
            if case["rows"] > 8:
                x[5] = -math.inf           # a grammar that allows nothing
        s["x"] = x.to(_type(case["dtype"]))
        s["par"] = [_cuda(a) for a in _params(case, case["rows"])]
        s["u"] = torch.rand(case["rows"], generator=g, device="cuda")
        return s
    cu = _windows(case)
    B, T = case["reqs"], int(cu[-1])
    par = [_cuda(a) for a in _params(case, B)]
    x = _logits(T, V, g)
    s["cu"] = _cuda(cu.astype(np.int32))
    s["par"] = par
    req = np.repeat(np.arange(B), np.diff(cu))
    inner = _cuda(np.setdiff1d(np.arange(T), cu[1:] - 1))     # rows that judge a draft
    s["ids"] = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    s["draft_x"] = s["draft_dist"] = None
    if len(inner):
        # the drafter's logits are the target's with an error of their own
        d = x[inner] + torch.randn(len(inner), V, generator=g, device="cuda") * 0.7
        if case["sampled"]:
            of = _cuda(req)[inner]
            d = d.to(_type(case["dtype"]))
            dist, tok, _ = _plain_dist(d, *[None if a is None else a[of] for a in par],
                                       torch.rand(len(inner), generator=g, device="cuda"))
            s["draft_x"], s["draft_dist"] = d, dist
        else:
            tok = d.argmax(1).int()
        s["ids"][inner + 1] = tok
    elif case["sampled"]:
        s["draft_x"] = torch.empty(0, V, dtype=_type(case["dtype"]), device="cuda")
        s["draft_dist"] = torch.empty(0, 8, dtype=torch.int32, device="cuda")
    s["x"] = x.to(_type(case["dtype"]))
    s["accept_u"] = torch.rand(T, generator=g, device="cuda")
    s["u"] = torch.rand(B, generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _plain_w4(s):
    k, group = s["case"]["k"], s["case"]["group"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).flatten(1)[:, :k].float() - 8.0
    w = codes * s["scales"].float().repeat_interleave(group, 1)[:, :k]
    return torch.matmul(s["x"].float(), w.t()).to(s["y"].dtype)


def _clean(x):
    return torch.nan_to_num(x.float(), nan=-math.inf, posinf=MOST, neginf=-math.inf)


def _inverse(temp):
    """1 / T, and the rows that take the largest logit (T not above 0)."""
    inv = 1.0 / temp
    greedy = ~(temp > 0) | torch.isinf(inv)
    return torch.where(greedy, torch.zeros_like(inv), inv), greedy


def _weights(x, top, inv):
    """exp((x - top) / T) in 32 bits, and the weights, whole numbers."""
    y = torch.exp((x - top) * inv)
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y)
    return y, torch.round(y * ONE).long()


def _pick(w, total, u):
    """The first token whose cumulated weight is above u times the total."""
    at = (u.double() * total.double()).long()
    at = torch.minimum(at, total - 1)
    tok = (torch.cumsum(w, 1) <= at[:, None]).sum(1)
    return torch.where(total > 0, tok, torch.full_like(tok, -1)).int()


def _bits(x):
    return x.float().contiguous().view(torch.int32)


def _kept(logits, temp, k, p, mp):
    """Every row's largest logit, 1 / T, last kept logit and token, and the
    weights of the kept tokens (others 0)."""
    x = _clean(logits)
    R, V = x.shape
    dev = x.device
    temp = torch.ones(R, device=dev) if temp is None else temp
    inv, greedy = _inverse(temp)
    top = x.amax(1) + 0.0
    y, w = _weights(x, top[:, None], inv[:, None])
    k = torch.zeros(R, dtype=torch.int32, device=dev) if k is None else k
    k = torch.where(k > 0, k, torch.full_like(k, V))
    k = torch.where(greedy, torch.ones_like(k), k)
    p = torch.ones(R, device=dev) if p is None else p
    p = torch.where(p < 1, p, torch.full_like(p, math.inf)).double()
    mp = torch.zeros(R, device=dev) if mp is None else mp
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(V, device=dev)
    ok = (ws > 0) & (y.gather(1, order) >= mp[:, None].clamp(max=1.0)) & (rank < k[:, None])
    ws = ws * ok
    before = torch.cumsum(ws, 1) - ws
    total = ws.sum(1).double()
    ok &= (before.double() < (p * total)[:, None]) | (rank == 0)
    n = ok.sum(1)
    every = n == (w > 0).sum(1)
    last = (n - 1).clamp(min=0)[:, None]
    cut = torch.where(every, torch.full_like(top, -math.inf), xs.gather(1, last)[:, 0] + 0.0)
    cut_token = torch.where(every, torch.full_like(n, V - 1), order.gather(1, last)[:, 0])
    keep = torch.zeros_like(ok).scatter_(1, order, ok)
    return top, inv, cut, cut_token.int(), w * keep


def _dist(top, inv, cut, cut_token, total, token):
    halves = total.contiguous().view(torch.int32).view(-1, 2)
    return torch.stack((_bits(top), _bits(inv), _bits(cut), cut_token, halves[:, 0], halves[:, 1],
                        token, torch.zeros_like(token)), 1)


def _logprob(x, token, top, inv, total):
    """ln of the token's share (-inf: no such token)."""
    at = token.long().clamp(min=0)[:, None]
    z = (_clean(x.gather(1, at))[:, 0] - top) * inv
    r = (z.double() - torch.log(total.double() / ONE)).float()
    return torch.where((token >= 0) & (total > 0), r, torch.full_like(r, -math.inf))


def _plain_dist(logits, temp, k, p, mp, u):
    top, inv, cut, cut_token, w = _kept(logits, temp, k, p, mp)
    total = w.sum(1)
    token = _pick(w, total, u)
    return (_dist(top, inv, cut, cut_token, total, token), token,
            _logprob(logits, token, top, inv, total))


def _plain_sample(s):
    dist, token, logprob = _plain_dist(s["x"], *s["par"], s["u"])
    return dict(tokens=token, logprobs=logprob, dist=dist)


def _of_dist(x, dist):
    """The kept weights of rows of logits that the records `dist` describe."""
    x = _clean(x)
    f = dist.view(torch.float32)
    w = _weights(x, f[:, 0:1], f[:, 1:2])[1]
    at = torch.arange(x.shape[1], device=x.device)
    keep = (x > f[:, 2:3]) | ((x == f[:, 2:3]) & (at <= dist[:, 3:4]))
    return w * keep


def _total(dist):
    return dist[:, 4:6].contiguous().view(torch.int64)[:, 0]


def _plain_verify(s):
    cu = s["cu"].long()
    x, ids = s["x"], s["ids"].long()
    T = len(x)
    B = len(cu) - 1
    row = torch.arange(T, device=x.device)
    req = torch.searchsorted(cu, row, right=True) - 1
    top, inv, cut, cut_token, w = _kept(x, *[None if a is None else a[req] for a in s["par"]])
    total = w.sum(1)
    inner = row + 1 < cu[req + 1]
    draft = torch.where(inner, ids[(row + 1).clamp(max=T - 1)], torch.full_like(ids, -1))
    at = draft.clamp(min=0)[:, None]
    wd = w.gather(1, at)[:, 0]
    u = s["accept_u"].double()
    if s["draft_x"] is None:
        ok = u * total.double() < wd.double()
        ok = (wd > 0) & (ok | (wd == total))
        # without the draft (column 0 of a row that judges none stays as it is)
        left = w.scatter(1, at, torch.where(inner, torch.zeros_like(wd), w[:, 0])[:, None])
        token = _pick(left, left.sum(1), s["u"][req])
    else:
        d = (row - req).clamp(max=max(0, len(s["draft_x"]) - 1))     # a row's draft
        if len(s["draft_x"]):
            dist = s["draft_dist"][d]
            xd = _clean(s["draft_x"][d, draft.clamp(min=0)][:, None])
            f = dist.view(torch.float32)
            qd = _weights(xd, f[:, 0:1], f[:, 1:2])[1][:, 0]
            there = (xd[:, 0] > f[:, 2]) | ((xd[:, 0] == f[:, 2]) & (draft <= dist[:, 3]))
            qd = torch.where(there, qd, torch.zeros_like(qd))
            ok = u * qd.double() * total.double() < wd.double() * _total(dist).double()
        else:
            ok = torch.zeros_like(inner)
        token = _pick(w, total, s["u"][req])
        token = torch.where(inner, torch.full_like(token, -1), token)
    ok &= inner
    # accepted: the drafts before a request's first rejection
    bad = torch.where(ok, torch.full_like(row, T), row)
    first = torch.full((B,), T, device=x.device).scatter_reduce_(0, req, bad, "amin")
    accepted = first - cu[:-1]
    nxt = token[first]
    if s["draft_x"] is not None and len(s["draft_x"]):
        # rejected: from what the target has more of than the drafter
        wt, di = w[first], d[first]
        p = wt.float() * (ONE / total[first].double()).float()[:, None]
        q = _of_dist(s["draft_x"][di], s["draft_dist"][di])
        q = q.float() * (ONE / _total(s["draft_dist"][di]).double()).float()[:, None]
        r = torch.round((p - q).clamp(min=0.0)).long()
        r = torch.where((r.sum(1) > 0)[:, None], r, torch.round(p).long())
        nxt = torch.where(inner[first], _pick(r, r.sum(1), s["u"]), nxt)
    follow = torch.where(row < first[req], draft, nxt.long()[req]).int()
    lp = _logprob(x, follow, top, inv, total)
    value = _clean(x.gather(1, follow.long().clamp(min=0)[:, None]))[:, 0]
    there = (value > cut) | ((value == cut) & (follow <= cut_token))
    lp = torch.where(there, lp, torch.full_like(lp, -math.inf))
    lp = torch.where(row <= first[req], lp, torch.zeros_like(lp))
    return dict(accepted=accepted.int(), tokens=nxt, logprobs=lp,
                dist=_dist(top, inv, cut, cut_token, total, token))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"w4": _plain_w4, "sample": _plain_sample, "verify": _plain_verify}[op](s)
    import speculative_drafting_expand_gb300 as pe
    if op == "w4":
        return pe.pe_w4_linear(s["w"], s["x"], out=s["y"])
    temp, k, p, mp = s["par"]
    if op == "sample":
        tokens, logprobs, dist = pe.pe_sample(s["x"], s["u"], temperature=temp, top_k=k, top_p=p,
                                              min_p=mp)
        return dict(tokens=tokens, logprobs=logprobs, dist=dist)
    accepted, tokens, logprobs, dist = pe.pe_verify(
        s["x"], s["ids"], s["cu"], s["accept_u"], s["u"], temperature=temp, top_k=k, top_p=p,
        min_p=mp, draft_logits=s["draft_x"], draft_dist=s["draft_dist"])
    return dict(accepted=accepted, tokens=tokens, logprobs=logprobs, dist=dist)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "w4":
        R, n, k = case["rows"], case["n"], case["k"]
        return dict(bytes=n * k / 2 + 2 * n * -(-k // case["group"]) + R * k * size[case["dtype"]]
                    + R * n * size[case["out"]], flops=2 * R * n * k)
    V, e = case["vocab"], size[case["dtype"]]
    if case["op"] == "sample":
        R = case["rows"]
        return dict(bytes=R * (V * e + 4 * 5 + 40), flops=3 * R * V)
    # the target's rows, and of sampled drafts the row that is rejected
    B, T = case["reqs"], int(_windows(case)[-1])
    rows = T + (B if case["sampled"] and T > B else 0)
    return dict(bytes=rows * V * e + T * 44 + B * 32, flops=3 * rows * V)


# ---------------------------------------------------------------------------
# the definition, in 64 bits, row by row
# ---------------------------------------------------------------------------

class _Row:
    """The distribution of one row: which tokens are kept goes by the weights
    (whole numbers), probabilities are of the 64-bit exponentials."""

    def __init__(self, logits, temp, k, p, mp):
        x = logits.double()
        x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x).clamp(max=MOST)
        self.V, self.n = len(x), 0
        m = float(x.max())
        if m == -math.inf:
            return
        greedy = not temp > 0
        inv = np.float32(0) if greedy else np.float32(1) / np.float32(temp)
        e = torch.exp((x.float() - np.float32(m)) * float(inv))
        w = torch.round(e.double() * ONE).long()
        w[x == -math.inf] = 0
        on = torch.nonzero((w > 0) & (e >= min(mp, 1.0)))[:, 0]
        on = on[torch.sort(x[on], descending=True, stable=True).indices]
        on = on[:1 if greedy else k if k > 0 else self.V]
        if p < 1:
            run = torch.cumsum(w[on], 0)
            on = on[:max(1, int((run - w[on] < float(np.float32(p)) * float(run[-1])).sum()))]
        self.n = len(on)
        self.ids = torch.sort(on).values
        self.w = w[self.ids]
        self.run = torch.cumsum(self.w, 0)
        self.total = int(self.run[-1])
        z = (x[self.ids] - m) * (0.0 if greedy else 1.0 / float(np.float32(temp)))
        self.logp = z - torch.logsumexp(z, 0)

    def at(self, token):
        """Place of a token among the kept ones, or None."""
        if not self.n:
            return None
        i = int(torch.searchsorted(self.ids, token))
        return i if i < self.n and int(self.ids[i]) == token else None

    def weight(self, token):
        i = self.at(token)
        return 0 if i is None else int(self.w[i])

    def log(self, token):
        i = self.at(token)
        return -math.inf if i is None else float(self.logp[i])


def _invert(ids, w, u):
    run = torch.cumsum(w, 0)
    at = min(int(np.float64(u) * float(run[-1])), int(run[-1]) - 1)
    return int(ids[int(torch.searchsorted(run, at, right=True))])


def _row_params(s, n):
    temp, k, p, mp = [None if a is None else a.cpu().numpy() for a in s["par"]]
    return [(1.0 if temp is None else temp[i], 0 if k is None else int(k[i]),
             1.0 if p is None else p[i], 0.0 if mp is None else float(mp[i])) for i in range(n)]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "w4":
        k, group = case["k"], case["group"]
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for lo in range(0, k, group):
            hi = min(lo + group, k)
            j = torch.arange(lo, hi, device="cuda")
            nibble = (s["codes"][:, j // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15
            part = s["x"][:, lo:hi].double() @ (nibble.double() - 8.0).t()
            y += part * s["scales"][:, lo // group].double()
        return y
    if case["op"] == "sample":
        u = s["u"].cpu().numpy()
        out = []
        for i, par in enumerate(_row_params(s, case["rows"])):
            r = _Row(s["x"][i], *par)
            out.append(r.log(_invert(r.ids, r.w, u[i])) if r.n else -math.inf)
        return dict(tokens=None, logprobs=torch.tensor(out, dtype=torch.float64, device="cuda"),
                    dist=None)
    cu, ids = s["cu"].cpu().numpy(), s["ids"].cpu().numpy()
    au, u = s["accept_u"].cpu().numpy().astype(np.float64), s["u"].cpu().numpy()
    lp = np.zeros(int(cu[-1]))
    for b, par in enumerate(_row_params(s, case["reqs"])):
        for t in range(int(cu[b]), int(cu[b + 1])):
            r = _Row(s["x"][t], *par)
            if t + 1 == cu[b + 1]:
                lp[t] = r.log(_invert(r.ids, r.w, u[b]))
                break
            d = int(ids[t + 1])
            w, t_all = r.weight(d), float(r.total)
            if s["draft_x"] is None:
                if w == r.total or au[t] * t_all < float(w):
                    lp[t] = r.log(d)
                    continue
                on = r.ids != d
                lp[t] = r.log(_invert(r.ids[on], r.w[on], u[b]))
                break
            q = _Row(s["draft_x"][t - b], *par)
            if au[t] * float(q.weight(d)) * t_all < float(w) * float(q.total):
                lp[t] = r.log(d)
                continue
            share = torch.zeros(case["vocab"], device="cuda")
            share[r.ids] = r.w.float() * float(np.float32(ONE / t_all))
            kept = share.clone()
            share[q.ids] -= q.w.float() * float(np.float32(ONE / float(q.total)))
            share = torch.round(share.clamp(min=0)).long()
            if int(share.sum()) == 0:
                share = torch.round(kept).long()
            lp[t] = r.log(_invert(torch.arange(case["vocab"]), share, u[b]))
            break
    return dict(accepted=None, tokens=None, dist=None,
                logprobs=torch.from_numpy(lp).cuda())
