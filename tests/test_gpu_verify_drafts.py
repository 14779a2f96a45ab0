"""Which drafts pe_verify accepts and records at the ends of its rules
(include/peagle_sample.h)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("accept_u", [-1.0, -1e-30, -float("inf"), 0.0, float("nan")])
def test_a_draft_without_probability_is_never_accepted(sampled, accept_u):
    """Whatever accept_u is; the draft is what the target's top-k leaves out and
    the drafter's does not."""
    torch, L = _lib()
    V = 40
    x = torch.zeros(2, V, device="cuda")
    x[:, :5] = torch.arange(5, 0, -1, device="cuda").float()
    k = torch.tensor([3], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    kw = {}
    if sampled:
        d = torch.zeros(1, V, device="cuda")
        _, _, dd = L.pe_sample(d, torch.tensor([0.1], device="cuda"))
        kw = dict(draft_logits=d, draft_dist=dd)
    acc, tok, _, _ = L.pe_verify(x, ids, torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                                 torch.full((2,), accept_u, device="cuda"),
                                 torch.tensor([0.5], device="cuda"), top_k=k, **kw)
    assert int(acc) == 0 and 0 <= int(tok) < 3


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("bad", [-1, 40, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("place", [1, 2, 31, 32, 33, 34, 64, 65, 70])
def test_drafts_of_no_token_are_recorded_wherever_they_are(sampled, bad, place):
    """A window of 70 drafts.  At the first place the bad one is judged and
    rejected; elsewhere the first draft, which has no probability, is."""
    torch, L = _lib()
    V, T = 40, 71
    x = torch.zeros(T, V, device="cuda")
    x[:, 7] = float("-inf")
    ids = torch.full((T,), 3, dtype=torch.int32, device="cuda")
    ids[1] = 7
    kw = {}
    if sampled:
        d = torch.zeros(T - 1, V, device="cuda")
        kw = dict(draft_logits=d, draft_dist=L.pe_sample(
            d, torch.rand(T - 1, device="cuda"))[2])
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    au, u = torch.full((T,), 0.5, device="cuda"), torch.tensor([0.5], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sound = L.pe_verify(x, ids, cu, au, u, err=err, **kw)
    assert int(err) == 0 and int(sound[0]) == 0
    ids[place] = bad
    got = L.pe_verify(x, ids, cu, au, u, err=err, **kw)
    assert int(err) == L.PE_DEV_BAD_TOKEN
    # 39 equal tokens: the place of u = 0.5 is in the twentieth, and id 7 is none
    assert int(got[0]) == 0 and int(got[1]) == 20
    assert int(sound[1]) == 20
    ids[place] = 3
    ids[1] = 3
    err.zero_()
    L.pe_verify(x, ids, cu, au, u, err=err, **kw)
    assert int(err) == 0
