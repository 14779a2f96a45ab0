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
