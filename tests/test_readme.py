"""The README's examples: every Python block compiles, and the one from hidden
rows to the next step runs and keeps each request's filters."""

import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _blocks():
    text = open(os.path.join(ROOT, "README.md")).read()
    return re.findall(r"^```python\n(.*?)^```", text, re.M | re.S)


def test_python_blocks_compile():
    blocks = _blocks()
    assert len(blocks) >= 2
    for b in blocks:
        compile(b, "README.md", "exec")


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_from_hidden_rows_to_the_next_step(seed):
    import torch
    import oracle as O
    from speculative_drafting_expand_gb300 import binding as L
    from synthetic import workloads as W
    from tests import gpu_helpers as G
    from tests.test_gpu_expand import _expand_drafter
    block, = [b for b in _blocks() if "pe_verify" in b]
    shape = W.small_shape("readme", d=256, n_layers=1, n_heads=4, n_kv_heads=2, head_dim=64,
                          ffn=256, vocab=777)
    B, K = 4, 3
    T, n = B * (K + 1), K + 1
    torch.manual_seed(seed)
    rand = lambda *s: torch.rand(*s, device="cuda")
    # (the step's own inputs; the accepted counts that it assumes are not used)
    wl = W.custom("readme", 92, shape, K, [100] * B, [n] * B, [K] * B)
    inp = W.make_step_inputs(wl)
    dr, _ = _expand_drafter(shape, wl.T_out, B)
    st = G.DeviceStep(wl, inp, [], [])
    ex = L.Expanded(wl.T_out, wl.T, B, K, shape.hidden3, shape.dtype)
    ns = dict(torch=torch, B=B, K=K, lm_head=torch.randn(shape.vocab, shape.d, device="cuda") * 0.2,
              hidden=torch.randn(B * K, shape.d, device="cuda").bfloat16(),
              temperature=torch.full((B,), 1.0, device="cuda"),
              top_k=torch.tensor([1, 5, 1, 5], dtype=torch.int32, device="cuda"),
              top_p=torch.tensor([1.0, 0.5, 0.9, 1.0], device="cuda"),
              min_p=torch.tensor([0.0, 0.1, 0.0, 0.9], device="cuda"),
              u_draft=rand(B * K), accept_u=rand(T), u=rand(B),
              last_token=torch.full((B,), 5, dtype=torch.int32, device="cuda"),
              cu_in=torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda"),
              target_logits=torch.randn(T, shape.vocab, device="cuda") * 3,
              drafter=dr, target_pos=st.target_pos, block_table=st.block_table,
              num_blocks=inp.num_blocks, target_hidden=st.target_hidden, expanded=ex)
    exec(compile(block, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    acc, tok = ns["accepted"].cpu().numpy(), ns["sampled"].cpu().numpy()
    drafts = ns["drafts"].view(B, K).cpu().numpy()
    x, y = ns["target_logits"].view(B, n, -1), ns["logits"].view(B, K, -1)
    for b in range(B):
        k = int(ns["top_k"][b])
        for i in range(K):         # drafts are of the drafter's first k, accepted ones of both
            assert drafts[b, i] in y[b, i].topk(k).indices.tolist()
            assert i >= acc[b] or drafts[b, i] in x[b, i].topk(k).indices.tolist()
        assert tok[b] in x[b, acc[b]].topk(k).indices.tolist()
    ref = O.expand_batch(K, ns["ids"].cpu().numpy(), inp.target_pos, ns["cu_in"].cpu().numpy(),
                         acc, tok, inp.block_table, shape.page_size, shape.mask_token_id)
    assert L.pe_get_device_error(dr) == 0
    G.check_expand(ex, ref, wl.T)
    assert np.array_equal(ns["ids"].view(B, n)[:, 1:].cpu().numpy(), drafts)
