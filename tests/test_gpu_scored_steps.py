"""Drafting steps that collect scores (pe_set_kv_scores) on streams of their
own, beside other work, and with block tables that grow."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

CONTEXTS, K = [1500, 700], 4


def _setup(dtype="bf16", n_heads=8, n_kv_heads=2):
    import dataclasses
    from synthetic import workloads as W
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    shape = W.small_shape("scored-steps", d=512, n_layers=2, n_heads=n_heads,
                          n_kv_heads=n_kv_heads, head_dim=64, ffn=1024, vocab=4096)
    shape = dataclasses.replace(shape, dtype=dtype)
    wl = W.custom("scored-steps", 94, shape, K, CONTEXTS, [K + 1, K + 1], [K, 1])
    inp = W.make_step_inputs(wl)
    return B, wl, inp, W.make_weights(shape, wl.config_id, gains=wl.gains), W.make_kv_cache(wl, inp)


def _step_inputs(wl, inp, cache, width):
    """Device inputs whose block table has `width` columns."""
    import torch
    from tests import gpu_helpers as G
    st = G.DeviceStep(wl, inp, *cache)
    more = width - st.block_table.shape[1]
    assert more >= 0
    st.block_table = torch.nn.functional.pad(st.block_table, (0, more), value=-1).contiguous()
    return st


def _scores(inp, n_kv_heads=2):
    import torch
    rng = np.random.default_rng(51)
    return [torch.from_numpy(rng.random((inp.num_blocks, n_kv_heads, 16)).astype(np.float32)).cuda()
            for _ in range(2)]


@pytest.mark.parametrize("collect", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_steps_on_a_side_stream_beside_queued_work(dtype, collect):
    """A handle's first steps, on a non-blocking stream, with wider tables
    from step to step and work queued on the default stream: what the step
    allocates is cleared before the step reads it and not again later, so
    every result is that of the same steps on an idle device, bit for bit."""
    import torch
    from tests import gpu_helpers as G
    B, wl, inp, w, cache = _setup(dtype)
    narrow = np.asarray(inp.block_table).shape[1]
    got = []
    for side in (None, torch.cuda.Stream()):
        dr = G.make_drafter(wl.shape, w, wl.T_out, wl.B)
        scores = _scores(inp)
        steps = [_step_inputs(wl, inp, cache, narrow + extra) for extra in (0, 64, 700)]
        torch.cuda.synchronize()
        results = []
        for st in steps:
            if side is not None:
                torch.cuda._sleep(100_000_000)      # about 50 ms on the default stream
            with torch.cuda.stream(side):           # None: the current one
                if collect:
                    B.pe_set_kv_scores(dr, scores)
                res = G.run_step(dr, st)            # waits for the whole device
            assert res["err"] == 0
            results += [res["tokens"], res["logits"], res["out_hidden"], *st.kc, *st.vc]
            results += [s.clone() for s in scores]
        dr.close()
        got.append(results)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))


def test_a_table_that_widens_step_by_step_keeps_memory_bounded():
    """The room for the scores' logits at least doubles when it grows, so
    that all of it stays below twice the last (here below 4 times what the
    widest table wants), however many steps widen the table."""
    import torch
    from tests import gpu_helpers as G
    B, wl, inp, w, cache = _setup()
    narrow = np.asarray(inp.block_table).shape[1]
    widths = [narrow + 25 * i for i in range(80)]
    want = B.pe_attn_decode_workspace(wl.B, 8, 2, 64, widths[-1])
    used = []
    for collect in (False, True):
        dr = G.make_drafter(wl.shape, w, wl.T_out, wl.B)
        B.pe_set_kv_scores(dr, _scores(inp) if collect else None)
        st = _step_inputs(wl, inp, cache, widths[0])
        assert G.run_step(dr, st)["err"] == 0
        tables = [_step_inputs(wl, inp, cache, x).block_table for x in widths]
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        held = torch.cuda.memory_reserved()
        for t in tables:
            st.block_table = t
            assert G.run_step(dr, st, want_logits=False)["err"] == 0
        used.append(before - torch.cuda.mem_get_info()[0] - (torch.cuda.memory_reserved() - held))
        dr.close()
    assert used[1] - used[0] <= 4 * want + (8 << 20), (used, want)


def test_room_for_logits_only_where_they_are_kept():
    """Logits are kept where one tile holds all query heads of a kv head; more
    heads ask for no room for them."""
    from speculative_drafting_expand_gb300 import binding as B
    for heads, kv_heads in ((17, 1), (40, 1), (96, 4)):
        for dim in (64, 128):
            assert B.pe_attn_decode_workspace(3, heads, kv_heads, dim, 50) == \
                B.pe_attn_decode_workspace(3, heads, kv_heads, dim)
    for heads in (1, 8, 9, 16):
        assert B.pe_attn_decode_workspace(3, heads, 1, 64, 50) - \
            B.pe_attn_decode_workspace(3, heads, 1, 64) == 3 * 50 * 16 * (16 if heads > 8 else 8) * 4
