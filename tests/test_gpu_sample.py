"""Sampling and draft verification (include/peagle_sample.h) on a GPU.

Decisions are on whole numbers, so tokens, cuts, totals and accepted counts
are compared exactly with the oracle's, which gets the fp32 exponentials from
torch on the same GPU (elementary fp32 exp of the same argument).  Against 64
bits (u = 2^-24): z = (x - max) / T has three roundings, 3 u |z|; the exponential
2 u (CUDA's bound is one step) and the weight's grid 2^-32 a token: the total is
right to sum_i e_i (3 |z_i| + 2) u + n 2^-32, and ln of it to that over the
total; logprobs add 3 u |z| and half a step of fp32."""

import math

import numpy as np
import pytest

from oracle import sample_oracle as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F = np.float32


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _exps(torch, x, temp):
    """torch's fp32 exponentials of every row, on the GPU."""
    x = S.clean(x)
    t = torch.from_numpy(x).cuda()
    inv = torch.from_numpy(np.array([S.inverse(v)[0] for v in temp], F)).cuda()
    e = torch.exp((t - t.amax(1, keepdim=True)) * inv[:, None])
    return torch.nan_to_num(e, nan=0.0).cpu().numpy()


def _dists(torch, x, temp, k, p, mp):
    e = _exps(torch, x, temp)
    return [S.dist(x[i], e[i], k[i], p[i], mp[i], S.inverse(temp[i])[1]) for i in range(len(x))]


def _cuda(torch, a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def _filters(rng, n):
    """Every kind of filter, one row after another."""
    temp, k = np.full(n, 0.9, F), np.zeros(n, np.int32)
    p, mp = np.ones(n, F), np.zeros(n, F)
    for i in range(n):
        kind = i % 10
        temp[i] = rng.uniform(0.3, 2.0)
        if kind == 1:
            temp[i] = [0.0, -1.0, np.nan, 1e-40][i // 10 % 4]
        if kind in (2, 5, 7):
            k[i] = [1, 2, 7, 50, 1000][i // 10 % 5]
        if kind in (3, 5, 6):
            p[i] = [0.9, 0.3, 0.999, 0.0, 1e-6][i // 10 % 5]
        if kind in (4, 6, 7):
            mp[i] = [0.05, 0.5, 1.0, 1e-5, 3.0][i // 10 % 5]
        if kind == 8:
            temp[i], k[i] = [np.inf, 1e30, 50.0][i // 10 % 3], [0, 3][i // 10 % 2]
        if kind == 9:
            p[i], mp[i], k[i] = np.nan, np.nan, -4
    return temp, k, p, mp


def _logits(rng, rows, V, kind):
    x = rng.normal(size=(rows, V)).astype(F) * 3
    if kind == "peaked":
        x[np.arange(rows), rng.integers(0, V, rows)] += 12
    if kind == "equal":
        x[:] = 1.5
    if kind == "few":                   # a handful of values, many ties
        x = np.round(x / 2).astype(F) * 2
    if kind == "near":                  # neighbours in fp32
        x = (F(8) + rng.integers(0, 40, (rows, V)).astype(F) * F(2.0 ** -20)).astype(F)
    if kind == "masked":
        x[rng.random((rows, V)) < 0.7] = -np.inf
        x[0] = -np.inf
    if kind == "special":
        x.flat[rng.integers(0, x.size, max(1, x.size // 5))] = np.nan
        x.flat[rng.integers(0, x.size, max(1, x.size // 50))] = np.inf
        x.flat[rng.integers(0, x.size, max(1, x.size // 5))] = -np.inf
        x.flat[rng.integers(0, x.size, max(1, x.size // 10))] = -0.0
        x[0] = np.nan
    if kind == "huge":
        x *= F(1e37)
    return x


def _check_rows(torch, x, par, u, tokens, logprobs, dist, ref=None):
    ref = ref or _dists(torch, x, *par)
    tokens, dist = tokens.cpu().numpy(), dist.cpu().numpy()
    f = dist.view(F)
    lp = logprobs.cpu().numpy().astype(np.float64)
    for i, d in enumerate(ref):
        who = (i, [a[i] for a in par])
        assert int(np.int64(dist[i, 4:6].copy().view(np.int64)[0])) == d.total, who
        assert f[i, 0] == d.max and f[i, 1] == S.inverse(par[0][i])[0], who
        assert f[i, 2] == F(d.cut) and dist[i, 3] == d.cut_token, (who, f[i, 2], dist[i, 3], d.cut)
        assert dist[i, 7] == 0 and dist[i, 6] == tokens[i], who
        want = S.draw(d.w, u[i])
        assert tokens[i] == want, (who, tokens[i], want)
        if want < 0:
            assert lp[i] == -math.inf
            continue
        inv, greedy = S.inverse(par[0][i])
        c = S.clean(x[i]).astype(np.float64)
        ids = np.array(sorted(d.kept))
        z = (c[ids] - c.max()) * (0.0 if greedy else 1 / np.float64(par[0][i]))
        e = np.exp(z)
        off = (e * (3 * np.abs(z) + 2)).sum() * U + len(ids) * 2.0 ** -32
        assert abs(d.total / S.ONE - e.sum()) <= off
        zt = z[list(ids).index(want)]
        assert abs(lp[i] - (zt - math.log(e.sum()))) <= \
            off / e.sum() + 3 * U * abs(zt) + U * abs(lp[i]) + 2.0 ** -40


def _sample(B, torch, x, par, u, dt="f32", **kw):
    t = _cuda(torch, x).to(torch.float32 if dt == "f32" else torch.bfloat16)
    temp, k, p, mp = [_cuda(torch, a) for a in par]
    return t, B.pe_sample(t, _cuda(torch, u, F), temperature=temp, top_k=k, top_p=p, min_p=mp, **kw)


@pytest.mark.parametrize("V", [1, 2, 5, 31, 257, 1024, 3001, 20000])
@pytest.mark.parametrize("kind", ["plain", "peaked", "equal", "few", "near", "masked", "special",
                                  "huge"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_against_the_definition(V, kind, dt):
    torch, B = _lib()
    rng = np.random.default_rng([V, len(kind)])
    rows = 50 if V <= 3001 else 20
    x = _logits(rng, rows, V, kind)
    par = _filters(rng, rows)
    u = rng.random(rows).astype(F)
    u[:6] = [0.0, 0.99999994, 1.0, -1.0, np.nan, 0.5]
    t, got = _sample(B, torch, x, par, u, dt)
    _check_rows(torch, t.float().cpu().numpy(), par, u, *got)


@pytest.mark.parametrize("rows,V", [(1, 201088), (3, 151936), (40, 50257), (160, 8191), (700, 130)])
def test_sizes_that_spread_differently(rows, V):
    torch, B = _lib()
    rng = np.random.default_rng([rows, V])
    x = _logits(rng, rows, V, "peaked")
    par = [a[:rows] for a in _filters(rng, max(rows, 10))]
    if rows == 1:
        par = [np.array([v], a.dtype) for v, a in zip((0.8, 50, 0.9, 0.0), par)]
    u = rng.random(rows).astype(F)
    t, got = _sample(B, torch, x, par, u)
    _check_rows(torch, x, par, u, *got)


def test_no_filters_and_u_sweeps_the_row():
    """Without filters; u over a grid of the cumulated weights' borders."""
    torch, B = _lib()
    rng = np.random.default_rng(2)
    V = 600
    row = rng.normal(size=V).astype(F)
    d = _dists(torch, row[None], [1.0], [0], [1.0], [0.0])[0]
    run = np.cumsum([d.w[i] for i in range(V)]) / d.total
    u = np.concatenate([run, np.nextafter(run.astype(F), F(0)), np.nextafter(run.astype(F), F(2))])
    u = np.clip(u, 0, 0.99999994).astype(F)
    x = torch.from_numpy(row).cuda().expand(len(u), V)          # stride 0 is no row stride
    with pytest.raises(B.PeError):
        B.pe_sample(x, torch.from_numpy(u).cuda())
    tokens, _, dist = B.pe_sample(x.contiguous(), torch.from_numpy(u).cuda())
    assert tokens.cpu().tolist() == [S.draw(d.w, v) for v in u]
    assert (dist[:, 3] == V - 1).all() and (dist[:, 2].view(torch.float32) == -math.inf).all()


@pytest.mark.parametrize("dt,V", [("f32", 1003), ("bf16", 1003), ("bf16", 64), ("f32", 4)])
def test_rows_anywhere_in_memory(dt, V):
    """Strided and misaligned rows; what lies beside them is not read as theirs."""
    torch, B = _lib()
    rng = np.random.default_rng(V)
    rows = 30
    t = torch.float32 if dt == "f32" else torch.bfloat16
    par = _filters(rng, rows)
    u = rng.random(rows).astype(F)
    temp, k, p, mp = [_cuda(torch, a) for a in par]
    for off in (0, 1, 2, 5):
        for pad in (0, 1, 7):
            wide = torch.full((rows, V + off + pad), float("inf"), dtype=t, device="cuda")
            x = _cuda(torch, _logits(rng, rows, V, "plain")).to(t)
            view = wide[:, off:off + V]
            view.copy_(x)
            got = B.pe_sample(view, _cuda(torch, u), temperature=temp, top_k=k, top_p=p, min_p=mp)
            _check_rows(torch, x.float().cpu().numpy(), par, u, *got)


def _windows(rng, B, most, ragged=True):
    n = rng.integers(1, most + 2, B) if ragged else np.full(B, most + 1)
    return np.concatenate(([0], np.cumsum(n)))


def _verify_case(torch, rng, cu, V, dt, sampled, kind="plain"):
    """Target rows, windows and drafts; of sampled drafts also the drafter's
    rows and their records, by pe_sample."""
    T, n = int(cu[-1]), len(cu) - 1
    td = torch.float32 if dt == "f32" else torch.bfloat16
    x = _cuda(torch, _logits(rng, T, V, kind)).to(td)
    par = [a[:n] for a in _filters(rng, max(n, 10))]
    ids = rng.integers(0, V, T).astype(np.int32)
    req = np.repeat(np.arange(n), np.diff(cu))
    inner = np.setdiff1d(np.arange(T), cu[1:] - 1)
    dx = None
    if len(inner):
        d = x[_cuda(torch, inner)].float() + torch.from_numpy(
            rng.normal(size=(len(inner), V)).astype(F)).cuda()
        dx = d.to(td)
        ids[inner + 1] = dx.float().argmax(1).int().cpu().numpy()
    return x, par, ids, req, inner, (dx if sampled else None)


@pytest.mark.parametrize("B,most,V", [(1, 7, 5000), (1, 0, 100), (6, 4, 33), (30, 3, 257),
                                      (12, 15, 1000), (3, 40, 70)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("kind", ["plain", "peaked", "few", "masked", "special"])
def test_verify_against_the_definition(B, most, V, dt, sampled, kind):
    torch, L = _lib()
    rng = np.random.default_rng([B, most, V, sampled])
    cu = _windows(rng, B, most, ragged=B > 1)
    T = int(cu[-1])
    x, par, ids, req, inner, dx = _verify_case(torch, rng, cu, V, dt, sampled, kind)
    dev = [_cuda(torch, a) for a in par]
    au, u = rng.random(T).astype(F), rng.random(B).astype(F)
    au[::3] *= F(0.2)
    kw, drafts = {}, []
    if sampled:
        of = torch.from_numpy(req[inner]).cuda()
        if dx is None:
            dx = torch.empty(0, V, dtype=x.dtype, device="cuda")
            dd = torch.empty(0, 8, dtype=torch.int32, device="cuda")
        else:
            tok, _, dd = L.pe_sample(dx, torch.rand(len(inner), device="cuda"),
                                     *[a[of].contiguous() for a in dev])
            tok = tok.cpu().numpy()
            ids[inner + 1] = np.where(tok < 0, 0, tok)
            drafts = _dists(torch, dx.float().cpu().numpy(), *[a[req[inner]] for a in par])
        kw = dict(draft_logits=dx, draft_dist=dd)
    ids[rng.integers(0, T, 1)] = V + 3 if kind == "few" else ids[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, tok, lp, dist = L.pe_verify(x, _cuda(torch, ids), _cuda(torch, cu, np.int32),
                                     _cuda(torch, au), _cuda(torch, u), *dev, err=err, **kw)
    host = x.float().cpu().numpy()
    ref = _dists(torch, host, *[a[req] for a in par])
    lp, dist = lp.cpu().numpy().astype(np.float64), dist.cpu().numpy()
    bad = False
    for b in range(B):
        w = range(int(cu[b]), int(cu[b + 1]))
        Q = [drafts[t - b] for t in w[:-1]] if sampled else None
        want = S.verify([ref[t] for t in w], ids[list(w)], au[list(w)], u[b], Q)
        assert (int(acc[b]), int(tok[b])) == want, (b, want)
        bad |= any(not 0 <= ids[t] < V for t in w[1:])
        for j, t in enumerate(w):
            d = ref[t]
            assert dist[t, 4:6].copy().view(np.int64)[0] == d.total
            assert dist[t].view(F)[2] == F(d.cut) and dist[t, 3] == d.cut_token
            if j > want[0]:
                assert lp[t] == 0
                continue
            follow = int(ids[t + 1]) if j < want[0] else want[1]
            if d.w.get(follow, 0) == 0:
                assert lp[t] == -math.inf
            else:
                # the exponential to 2 u, its weight to half of 1, ln's own rounding
                assert abs(lp[t] - math.log(d.w[follow] / d.total)) <= \
                    4 * U + 1 / d.w[follow] + U * abs(lp[t])
    code = int(err)
    assert code in ((0, L.PE_DEV_BAD_TOKEN) if bad else (0,))


def test_verify_bad_windows():
    """Empty, reversed and outside windows: recorded, answered with (0, -1),
    and the sound ones beside them are right; rows of no window stay."""
    torch, L = _lib()
    rng = np.random.default_rng(4)
    V, T = 90, 9
    x = torch.randn(T, V, device="cuda")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    for cu, good in (([0, 3, 3, 6], (0, 2)), ([-2, 3, 5, 7], (1, 2)), ([0, 4, 7, 12], (0, 1))):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dist = torch.full((T, 8), 77, dtype=torch.int32, device="cuda")
        lp = torch.full((T,), 5.0, device="cuda")
        au, u = torch.rand(T, device="cuda"), torch.rand(3, device="cuda")
        acc, tok, _, _ = L.pe_verify(x, ids, _cuda(torch, cu, np.int32), au, u, dist=dist,
                                     logprobs=lp, err=err)
        assert int(err) == L.PE_DEV_BAD_ROW
        rows = [t for b in good for t in range(cu[b], cu[b + 1])]
        rest = [t for t in range(T) if t not in rows]
        assert (dist[rest] == 77).all() and (lp[rest] == 5.0).all()
        for b in range(3):
            if b not in good:
                assert (int(acc[b]), int(tok[b])) == (0, -1)
                continue
            one = slice(cu[b], cu[b + 1])
            a1, t1, l1, d1 = L.pe_verify(
                x[one], ids[one], _cuda(torch, [0, cu[b + 1] - cu[b]], np.int32),
                au[one].contiguous(), u[b:b + 1].contiguous())
            assert int(a1) == int(acc[b]) and int(t1) == int(tok[b])
            assert torch.equal(d1, dist[one]) and torch.equal(l1, lp[one])


def test_streams_graphs_and_given_outputs():
    torch, B = _lib()
    x = torch.randn(7, 3000, device="cuda") * 3
    u = torch.rand(7, device="cuda")
    k = torch.full((7,), 40, dtype=torch.int32, device="cuda")
    want = B.pe_sample(x, u, top_k=k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = B.pe_sample(x, u, top_k=k, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    cu = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
    ids = torch.randint(3000, (7,), dtype=torch.int32, device="cuda")
    au = torch.rand(7, device="cuda")
    vout = [torch.empty_like(t) for t in B.pe_verify(x, ids, cu, au, u[:2].contiguous())]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pe_sample(x, u, top_k=k, tokens=out[0], logprobs=out[1], dist=out[2])
        B.pe_verify(x, ids, cu, au, u[:2].contiguous(), num_accepted=vout[0],
                    sampled_ids=vout[1], logprobs=vout[2], dist=vout[3])
    for _ in range(3):
        x.copy_(torch.randn(7, 3000, device="cuda") * 3)
        u.copy_(torch.rand(7, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, B.pe_sample(x, u, top_k=k)))
        assert all(torch.equal(a, b) for a, b in
                   zip(vout, B.pe_verify(x, ids, cu, au, u[:2].contiguous())))


def test_largest_vocabulary_and_offsets_past_32_bits():
    torch, B = _lib()
    V = 393216
    x = torch.randn(3, V, device="cuda")
    p = torch.full((3,), 0.95, device="cuda")
    u = torch.tensor([0.1, 0.5, 0.97], device="cuda")
    par = (np.ones(3, F), np.zeros(3, np.int32), np.full(3, 0.95, F), np.zeros(3, F))
    got = B.pe_sample(x, u, top_p=p)
    _check_rows(torch, x.cpu().numpy(), par, u.cpu().numpy(), *got)
    # rows 2^31 elements apart
    far = torch.empty((1 << 31) + 1000, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((2, 1000), (1 << 31, 1))
    rows.copy_(x[:2, :1000])
    a = B.pe_sample(rows, u[:2].contiguous())
    b = B.pe_sample(rows.contiguous(), u[:2].contiguous())
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_a_drafting_step_goes_on_from_what_verification_returns():
    """Hidden rows -> 4-bit LM head -> sampled drafts -> target logits ->
    verification -> the next pe_expand_batch."""
    torch, B = _lib()
    from synthetic import workloads as W
    from tests import gpu_helpers as G
    shape = W.small_shape("chain", d=256, n_layers=1, n_heads=4, n_kv_heads=2, head_dim=64,
                          ffn=256, vocab=777)
    rng = np.random.default_rng(0)
    nreq, K = 3, 4
    head = torch.randn(shape.vocab, shape.d, device="cuda") * 0.2
    w4 = B.W4Weight.quantize(head, 32)
    hidden = torch.randn(nreq * K, shape.d, device="cuda").bfloat16()
    logits = B.pe_w4_linear(w4, hidden, out_dtype=torch.float32)
    temp = torch.tensor([0.8, 0.0, 1.2], device="cuda")
    drafts, _, dd = B.pe_sample(logits, torch.rand(nreq * K, device="cuda"),
                                temperature=temp.repeat_interleave(K))
    cu = torch.arange(0, nreq * (K + 1) + 1, K + 1, dtype=torch.int32, device="cuda")
    T = nreq * (K + 1)
    ids = torch.zeros(nreq, K + 1, dtype=torch.int32, device="cuda")
    ids[:, 0] = 5
    ids[:, 1:] = drafts.view(nreq, K)
    target = torch.randn(nreq, K + 1, shape.vocab, device="cuda")
    target[:, :K] = logits.view(nreq, K, -1) + 0.2 * target[:, :K]
    target = target.view(T, -1)
    acc, nxt, lp, dist = B.pe_verify(target, ids.view(-1), cu, torch.rand(T, device="cuda"),
                                     torch.rand(nreq, device="cuda"), temperature=temp,
                                     draft_logits=logits, draft_dist=dd)
    assert ((acc >= 0) & (acc <= K)).all() and ((nxt >= 0) & (nxt < shape.vocab)).all()
    best = target[5:10].argmax(1)
    j = int(acc[1])                      # the greedy request
    assert int(nxt[1]) == int(best[j])
    assert all(int(ids[1, i + 1]) == int(best[i]) for i in range(j))
    # the next step's expansion, from the library's own accepted counts and tokens
    import oracle as O
    from tests.test_gpu_expand import _expand_drafter
    n, a_host, s_host = K + 1, acc.cpu().numpy(), nxt.cpu().numpy()
    wl = W.custom("chain", 91, shape, K, [100] * nreq, [n] * nreq, a_host.tolist())
    inp = W.make_step_inputs(wl)
    dr, _ = _expand_drafter(shape, wl.T_out, nreq)
    st = G.DeviceStep(wl, inp, [], [])
    ex = B.Expanded(wl.T_out, wl.T, nreq, K, shape.hidden3, shape.dtype)
    B.pe_expand_batch(dr, K, ids.view(-1), st.target_pos, cu, acc, nxt, st.block_table,
                      inp.num_blocks, st.target_hidden, ex)
    torch.cuda.synchronize()
    assert B.pe_get_device_error(dr) == 0
    ref = O.expand_batch(K, ids.view(-1).cpu().numpy(), inp.target_pos, cu.cpu().numpy(), a_host,
                         s_host, inp.block_table, shape.page_size, shape.mask_token_id)
    G.check_expand(ex, ref, wl.T)


def test_memory_freed_before_another_stream_has_read_it():
    torch, B = _lib()
    V = 5000
    x, u, k = torch.randn(6, V, device="cuda") * 3, torch.rand(6, device="cuda"), \
        torch.full((6,), 30, dtype=torch.int32, device="cuda")
    want = B.pe_sample(x, u, top_k=k)
    copies = [t.clone() for t in (x, u, k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # 50 ms in which the copies are freed
    got = B.pe_sample(copies[0], copies[1], top_k=copies[2], stream=side)
    del copies
    other = [torch.full_like(t, 7) for t in (x, u, k) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 7).all()) for t in other)


def test_two_host_threads_with_vocabularies_of_different_sizes():
    torch, B = _lib()
    from concurrent.futures import ThreadPoolExecutor

    def work(V):
        x, u = torch.randn(5, V, device="cuda") * 3, torch.rand(5, device="cuda")
        cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
        ids = torch.randint(V, (5,), dtype=torch.int32, device="cuda")
        y = torch.randn(4, V, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())

        def both():
            d = B.pe_sample(y, u[1:].contiguous(), stream=stream)
            return d + B.pe_verify(x, ids, cu, u, u[:1].contiguous(), draft_logits=y,
                                   draft_dist=d[2], stream=stream)

        first = both()
        rest = [both() for _ in range(100)]
        stream.synchronize()
        return all(torch.equal(a, b) for r in rest for a, b in zip(r, first))

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, (400, 200000)))
