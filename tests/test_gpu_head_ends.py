"""Verification at the largest vocabulary, and the operators between a hidden row
and the next step in two captured graphs that run at once."""

import numpy as np
import pytest

from oracle import sample_oracle as S

pytestmark = pytest.mark.gpu
F = np.float32


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _dist(torch, x, **f):
    """The oracle's distribution of a row, from torch's fp32 exponentials."""
    t = x.float()
    e = torch.exp(t - t.max()).cpu().numpy()
    return S.dist(t.cpu().numpy(), e, **f)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_sampled_drafts_of_the_largest_vocabulary(dt, off):
    """All of a cluster's shared memory holds the weights of the draw, with a row
    that starts in the middle of 16 bytes too."""
    torch, L = _lib()
    V = 393216
    g = torch.Generator(device="cuda").manual_seed(5)
    td = torch.float32 if dt == "f32" else torch.bfloat16
    x = (torch.randn(2, V + off, generator=g, device="cuda") * 2).to(td)[:, off:]
    d = (x[:1].float() + torch.randn(1, V, generator=g, device="cuda")).to(td)
    tok, _, dd = L.pe_sample(d, torch.rand(1, generator=g, device="cuda"))
    ids = torch.tensor([0, int(tok)], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    P, Q, last = [_dist(torch, r) for r in (x[0], d[0], x[1])]
    for au in (0.0, 0.99999994):
        for u in (0.0, 0.3, 0.99999994):
            got = L.pe_verify(x, ids, cu, torch.full((2,), au, device="cuda"),
                              torch.full((1,), u, device="cuda"), draft_logits=d, draft_dist=dd)
            want = S.verify([P, last], ids.tolist(), [F(au)] * 2, F(u), [Q])
            assert (int(got[0]), int(got[1])) == want, (au, u)


def test_two_graphs_at_once():
    torch, L = _lib()
    g = torch.Generator(device="cuda").manual_seed(6)
    n, k, K, R = 20000, 512, 3, 8
    w = L.W4Weight.quantize(torch.randn(n, k, generator=g, device="cuda") * 0.1, 64)
    cu = torch.arange(0, R * (K + 1) + 1, K + 1, dtype=torch.int32, device="cuda")
    topk = torch.randint(1, 400, (R,), generator=g, device="cuda", dtype=torch.int32)
    topp = torch.rand(R, generator=g, device="cuda") * 0.5 + 0.5

    def inputs():
        return dict(h=torch.randn(R * K, k, generator=g, device="cuda").bfloat16(),
                    t=torch.randn(R * (K + 1), n, generator=g, device="cuda") * 2,
                    ud=torch.rand(R * K, generator=g, device="cuda"),
                    au=torch.rand(R * (K + 1), generator=g, device="cuda"),
                    u=torch.rand(R, generator=g, device="cuda"))

    def step(s):
        logits = L.pe_w4_linear(w, s["h"], out_dtype=torch.float32)
        f = dict(top_k=topk, top_p=topp)
        tok, lp, dd = L.pe_sample(logits, s["ud"],
                                  **{a: b.repeat_interleave(K) for a, b in f.items()})
        ids = torch.cat((torch.zeros(R, 1, dtype=torch.int32, device="cuda"), tok.view(R, K)), 1)
        return (logits, tok, lp, dd) + L.pe_verify(s["t"], ids.view(-1), cu, s["au"], s["u"], **f,
                                                   draft_logits=logits, draft_dist=dd)

    state = [inputs(), inputs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in state:
            step(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in state:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(s))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s in state:
            for a, b in inputs().items():
                s[a].copy_(b)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for s, o in zip(state, outs):
            assert all(torch.equal(a, b) for a, b in zip(o, step(s)))
