"""Which windows pe_verify judges (include/peagle_sample.h): those that are not
empty, lie within [0, T) and are contradicted by no other entry of cu_in.  What
the other windows hold changes no answer, and nothing is read that the call did
not write."""

import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def sound(cu, T):
    """The windows that are judged, from the rule in words."""
    n = len(cu) - 1
    return [0 <= cu[r] < cu[r + 1] <= T and all(c <= cu[r] for c in cu[:r])
            and all(c >= cu[r + 1] for c in cu[r + 2:]) for r in range(n)]


def _inputs(torch, T, V):
    g = torch.Generator(device="cuda").manual_seed(T * V)
    x = torch.randn(T, V, generator=g, device="cuda") * 2
    ids = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    au = torch.rand(T, generator=g, device="cuda") * 0.3
    return x, ids, au


def _alone(torch, L, x, ids, au, u, w0, w1):
    out = L.pe_verify(x[w0:w1], ids[w0:w1], torch.tensor([0, w1 - w0], dtype=torch.int32,
                                                         device="cuda"),
                      au[w0:w1].contiguous(), torch.full((1,), u, device="cuda"))
    return [t.cpu() for t in out]


def _check(torch, L, x, ids, au, u, arrays):
    """Every array of window starts in a call of its own, whose results lie on
    memory full of other numbers; sound windows as if they were alone."""
    T = len(x)
    got = []
    for cu in arrays:
        n = len(cu) - 1
        out = (torch.full((n,), 55, dtype=torch.int32, device="cuda"),
               torch.full((n,), 66, dtype=torch.int32, device="cuda"),
               torch.full((T,), 5.0, device="cuda"),
               torch.full((T, 8), 77, dtype=torch.int32, device="cuda"))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.pe_verify(x, ids, torch.tensor(cu, dtype=torch.int32, device="cuda"), au,
                    torch.full((n,), u, device="cuda"), num_accepted=out[0], sampled_ids=out[1],
                    logprobs=out[2], dist=out[3], err=err)
        got.append(out + (err,))
    alone = {}
    for cu, out in zip(arrays, got):
        acc, tok, lp, dist, err = [t.cpu() for t in out]
        good = sound(cu, T)
        assert int(err) == (0 if all(good) else L.PE_DEV_BAD_ROW), cu
        free = np.ones(T, bool)
        for r, ok in enumerate(good):
            if not ok:
                assert (int(acc[r]), int(tok[r])) == (0, -1), (cu, r)
                continue
            w = (cu[r], cu[r + 1])
            if w not in alone:
                alone[w] = _alone(torch, L, x, ids, au, u, *w)
            a, t, l, d = alone[w]
            assert int(acc[r]) == int(a) and int(tok[r]) == int(t), (cu, r)
            assert torch.equal(lp[w[0]:w[1]], l) and torch.equal(dist[w[0]:w[1]], d), (cu, r)
            free[w[0]:w[1]] = False
        assert (lp.numpy()[free] == 5.0).all() and (dist.numpy()[free] == 77).all(), cu


def test_windows_behind_descending_entries():
    torch, L = _lib()
    x, ids, au = _inputs(torch, 3, 9)
    _check(torch, L, x, ids, au, 0.6, [[1, 1, 0, 3], [2, 1, 0, 3], [0, 3, 1, 3], [5, 0, 3, 3]])
    # four requests (at least as many rows)
    x, ids, au = _inputs(torch, 4, 9)
    _check(torch, L, x, ids, au, 0.6, [[0, 2, 100, 2, 3], [0, 1, -7, 1, 3], [0, 1, 2, 3, 4]])


@pytest.mark.parametrize("n", [1, 2, 3])
def test_every_array_of_starts(n):
    torch, L = _lib()
    T = 4 if n < 3 else 3
    x, ids, au = _inputs(torch, T, 9)
    _check(torch, L, x, ids, au, 0.35, [list(c) for c in
                                        itertools.product(range(-1, T + 2), repeat=n + 1)])


@pytest.mark.parametrize("n", [400, 1000])
def test_many_windows_with_one_entry_out_of_place(n):
    """More entries than a CTA has threads; the displaced one spoils only what
    it contradicts."""
    torch, L = _lib()
    T = 2 * n
    x, ids, au = _inputs(torch, T, 17)
    arrays = []
    for place, value in ((n // 2, 0), (n // 2, T), (n - 3, n - 50), (3, 41), (n, -1), (0, 9)):
        cu = list(range(0, T + 1, 2))
        cu[place] = value
        arrays.append(cu)
    _check(torch, L, x, ids, au, 0.8, arrays)


def test_filters_are_the_windows_own_beside_bad_ones():
    """Request 2 is greedy; its rows never take another request's filters."""
    torch, L = _lib()
    x, ids, au = _inputs(torch, 6, 50)
    temp = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda")
    cu = torch.tensor([0, 0, 0, 4, 6], dtype=torch.int32, device="cuda")
    ids[1:4] = x[:3].argmax(1).int()
    acc, tok, _, dist = L.pe_verify(x, ids, cu, au, torch.full((4,), 0.999, device="cuda"), temp)
    assert acc.cpu().tolist()[:3] == [0, 0, 3] and tok.cpu().tolist()[:2] == [-1, -1]
    assert int(tok[2]) == int(x[3].argmax()) and (dist[:4, 1] == 0).all()


@pytest.mark.parametrize("n,T", [(1, 4), (2, 4), (3, 3), (3, 4)])
def test_sampled_drafts_have_rows_of_the_drafter(n, T):
    """A window whose drafts have no rows of the drafter is a bad one; the rows
    of the others are those of the rule, whatever windows lie before."""
    torch, L = _lib()
    V = 9
    x, ids, au = _inputs(torch, T, V)
    g = torch.Generator(device="cuda").manual_seed(3)
    dx = x + torch.randn(T, V, generator=g, device="cuda")
    tok, _, dd = L.pe_sample(dx, torch.rand(T, generator=g, device="cuda"))
    ids[1:] = tok[:-1]
    cases, got = [], []
    for cu in itertools.product(range(-1, T + 2) if n < 3 else range(0, T + 1), repeat=n + 1):
        out = (torch.full((n,), 55, dtype=torch.int32, device="cuda"),
               torch.full((n,), 66, dtype=torch.int32, device="cuda"),
               torch.full((T,), 5.0, device="cuda"),
               torch.full((T, 8), 77, dtype=torch.int32, device="cuda"),
               torch.zeros(1, dtype=torch.int32, device="cuda"))
        L.pe_verify(x, ids, torch.tensor(cu, dtype=torch.int32, device="cuda"), au,
                    torch.full((n,), 0.6, device="cuda"), draft_logits=dx[:T - n],
                    draft_dist=dd[:T - n], num_accepted=out[0], sampled_ids=out[1],
                    logprobs=out[2], dist=out[3], err=out[4])
        cases.append(cu)
        got.append(out)
    alone = {}
    for cu, out in zip(cases, got):
        acc, tok, lp, dist, err = [t.cpu() for t in out]
        good = [ok and (cu[r + 1] - cu[r] == 1 or (cu[r] >= r and cu[r + 1] - 2 - r < T - n))
                for r, ok in enumerate(sound(cu, T))]
        assert int(err) == (0 if all(good) else L.PE_DEV_BAD_ROW), cu
        free = np.ones(T, bool)
        for r, ok in enumerate(good):
            if not ok:
                assert (int(acc[r]), int(tok[r])) == (0, -1), (cu, r)
                continue
            w = (cu[r], cu[r + 1], r)
            if w not in alone:
                one, of = slice(*w[:2]), slice(max(w[0] - r, 0), max(w[0] - r, 0) + w[1] - w[0] - 1)
                alone[w] = [t.cpu() for t in L.pe_verify(
                    x[one], ids[one], torch.tensor([0, w[1] - w[0]], dtype=torch.int32,
                                                   device="cuda"),
                    au[one].contiguous(), torch.full((1,), 0.6, device="cuda"),
                    draft_logits=dx[of], draft_dist=dd[of])]
            a, t, l, d = alone[w]
            assert int(acc[r]) == int(a) and int(tok[r]) == int(t), (cu, r)
            assert torch.equal(lp[w[0]:w[1]], l) and torch.equal(dist[w[0]:w[1]], d), (cu, r)
            free[w[0]:w[1]] = False
        assert (lp.numpy()[free] == 5.0).all() and (dist.numpy()[free] == 77).all(), cu
