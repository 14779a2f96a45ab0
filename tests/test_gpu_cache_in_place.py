"""Trims in place of whole serving batches, where a (layer, request, kv head)
has one or two CTAs: the moved rows against the definition."""

import numpy as np
import pytest

from oracle import kv_cache_oracle as C
from tests.test_gpu_cache import Cache, _check_evict, _host, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("e4m3", 64), ("e4m3", 128),
                                  ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("H,share", [(13, 0.4), (32, 0.4), (32, 0.9)])
def test_batches_trimmed_in_place(dt, D, H, share):
    """Four requests of which three are trimmed, over several rounds of rows;
    52 rows have two CTAs each on 152 SMs, 128 have one.  `share` of the
    positions stay, so that rows move far or hardly at all."""
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    rng = np.random.default_rng(H + D)
    lens = [1433, 1600, 47, 1017]
    budget = int(1000 * share)
    c = Cache(rng, lens, H, D, dt)
    before = _host(c.k), _host(c.v), _host(c.scores)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new = B.pe_kv_evict([c.pool], c.t, _i32(lens), budget, 4, 100, rope_theta=1e4, err=err)
    assert int(err) == 0
    ref = C.evict(*before, c.table, np.array(lens), budget, 4, 100, 1e4)
    _check_evict(c, before, ref, dt, 1e4, kept, new)
