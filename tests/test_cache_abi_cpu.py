"""The paged KV cache operators' C ABI without a GPU: exports, struct layout,
and every refusal that the host makes before it touches the device."""

import ctypes
import os
import re
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "peagle_cache.h")


@pytest.fixture(scope="module")
def B():
    from speculative_drafting_expand_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    binding.lib()
    return binding


def test_library_exports_every_declared_symbol(B):
    fns = sorted(set(re.findall(r"^(?:pe_status|int64_t)\s+(pe_\w+)\(", open(HEADER).read(), re.M)))
    assert set(fns) == set(B.CACHE_EXPORTED)
    assert all(hasattr(B.lib(), f) for f in fns)


def test_pool_layout_and_enumerators_match_the_header(B):
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "peagle_cache.h"
    int main(void) {
      printf("%zu %zu %zu %zu %d %d %d %d %d %d\n", sizeof(pe_kv_pool),
             offsetof(pe_kv_pool, num_blocks), offsetof(pe_kv_pool, dtype),
             offsetof(pe_kv_pool, v_scale), PE_KV_BF16, PE_KV_F32, PE_KV_E4M3,
             PE_DEV_BAD_BLOCK, PE_DEV_BAD_POSITION, PE_DEV_BAD_ROW);
      return 0;
    }
    """
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    P = B.pe_kv_pool
    assert got == [ctypes.sizeof(P), P.num_blocks.offset, P.dtype.offset, P.v_scale.offset,
                   B.PE_KV_BF16, B.PE_KV_F32, B.PE_KV_E4M3, B.PE_DEV_BAD_BLOCK,
                   B.PE_DEV_BAD_POSITION, B.PE_DEV_BAD_ROW]


# host addresses stand in for device pointers: a refused call reads none
BASE = 1 << 20


def _pool(B, **change):
    f = dict(k=BASE, v=BASE, scores=BASE, num_blocks=4, n_kv_heads=2, head_dim=64, dtype=0,
             k_scale=1.0, v_scale=1.0)
    f.update(change)
    return B.pe_kv_pool(*(f[n] for n, _ in B.pe_kv_pool._fields_))


BAD_POOLS = [(dict(k=0), 1), (dict(v=0), 1), (dict(k=BASE + 8), 1), (dict(scores=BASE + 4), 1),
             (dict(num_blocks=0), 1), (dict(n_kv_heads=0), 1), (dict(dtype=3), 1),
             (dict(dtype=2, k_scale=0.0), 1), (dict(dtype=2, v_scale=float("nan")), 1),
             (dict(dtype=2, v_scale=float("inf")), 1), (dict(head_dim=96), 2),
             (dict(head_dim=256), 2)]


def _append(B, pool=None, change=()):
    f = dict(T=3, B=3, n_heads=4, theta=1e4, q=BASE, qs=256, k=BASE, ks=128, v=BASE, vs=128,
             pos=BASE, req=BASE, table=BASE, stride=2, out=BASE, os=256, err=0, stream=0)
    f.update(change)
    pool = pool or _pool(B)
    return B.lib().pe_kv_append(ctypes.byref(pool), *f.values())


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 1), (dict(B=0), 1), (dict(req=0, T=2), 1), (dict(n_heads=3), 1),
    (dict(n_heads=0), 1), (dict(theta=-1.0), 1), (dict(theta=float("inf")), 1), (dict(q=0), 1),
    (dict(out=0), 1), (dict(qs=255), 1), (dict(qs=260), 1), (dict(ks=64), 1), (dict(vs=120), 1),
    (dict(k=0), 1), (dict(v=BASE + 2), 1), (dict(pos=0), 1), (dict(table=0), 1),
    (dict(stride=0), 1), (dict(os=64), 1)])
def test_append_refusals(B, change, status):
    assert _append(B, change=change) == status


def _decode(B, pool=None, change=()):
    f = dict(B=3, n_heads=4, scale=0.1, q=BASE, qs=256, table=BASE, stride=2, lens=BASE,
             window=0, out=BASE + 4096, os=256, lse=0, acc=0, ws=BASE, bytes=1 << 40, err=0, stream=0)
    f.update(change)
    pool = pool or _pool(B)
    return B.lib().pe_attn_decode(ctypes.byref(pool), *f.values())


@pytest.mark.parametrize("change,status", [
    (dict(B=0), 1), (dict(n_heads=3), 1), (dict(n_heads=0), 1), (dict(scale=float("nan")), 1),
    (dict(q=0), 1), (dict(q=BASE + 8), 1), (dict(qs=128), 1), (dict(qs=257), 1),
    (dict(table=0), 1), (dict(stride=0), 1), (dict(lens=0), 1), (dict(window=-1), 1),
    (dict(out=0), 1), (dict(out=BASE), 1), (dict(os=128), 1), (dict(ws=0), 1), (dict(ws=BASE + 8), 1),
    (dict(bytes=0), 1), (dict(stride=1 << 28), 2)])
def test_decode_refusals(B, change, status):
    assert _decode(B, change=change) == status


def test_decode_accumulate_needs_scores(B):
    assert _decode(B, _pool(B, scores=0), dict(acc=1)) == 1


def test_workspace_sizes(B):
    f = B.lib().pe_attn_decode_workspace
    assert f(0, 4, 2, 64, 0) == 0 and f(1, 3, 2, 64, 0) == 0 and f(1, 4, 2, 80, 0) == 0
    assert f(1, 4, 0, 64, 0) == 0 and f(1, 4, 2, 64, -1) == 0


def _evict(B, pools=None, change=()):
    f = dict(n=1, B=3, table=BASE, stride=2, lens=BASE, budget=8, sinks=2, recent=4, theta=1e4,
             dst=0, dstride=0, kept=BASE, new=BASE + 64, err=0, stream=0)
    f.update(change)
    pools = pools or [_pool(B)]
    arr = (B.pe_kv_pool * len(pools))(*pools)
    v = list(f.values())
    return B.lib().pe_kv_evict(v[0], arr, *v[1:])


@pytest.mark.parametrize("change,status", [
    (dict(n=0), 1), (dict(n=65), 1), (dict(B=0), 1), (dict(table=0), 1), (dict(stride=0), 1),
    (dict(lens=0), 1), (dict(budget=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1),
    (dict(sinks=5), 1), (dict(theta=-2.0), 1), (dict(theta=float("nan")), 1),
    (dict(dst=BASE, dstride=0), 1), (dict(kept=0), 1), (dict(new=0), 1), (dict(new=BASE), 1),
    (dict(budget=1 << 30), 2), (dict(sinks=2**31 - 1, recent=2**31 - 1), 1)])
def test_evict_refusals(B, change, status):
    assert _evict(B, change=change) == status


def test_evict_pools_must_agree_and_have_scores(B):
    assert _evict(B, [_pool(B, scores=0)]) == 1
    for change in (dict(n_kv_heads=4), dict(head_dim=128), dict(dtype=1)):
        assert _evict(B, [_pool(B), _pool(B, **change)], dict(n=2)) == 1


@pytest.mark.parametrize("change,status", BAD_POOLS)
def test_bad_pools_are_refused_by_every_operator(B, change, status):
    pool = _pool(B, **change)
    assert _append(B, pool) == status
    assert _decode(B, pool) == status
    assert _evict(B, [pool]) == status


def test_null_pool(B):
    assert B.lib().pe_set_kv_scores(None, None) == 1
    assert B.lib().pe_kv_append(None, *([1] * 3), 0.0, *([None, 0] * 3), None, None, None, 1,
                                None, 0, None, None) == 1
    assert B.lib().pe_kv_evict(1, None, 1, None, 1, None, 1, 0, 0, 0.0, None, 0, None, None,
                               None, None) == 1


def test_python_refusals(B):
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    s = torch.zeros(4, 2, 16)
    for bad in ((k[:, :, :8], k[:, :, :8]), (k, k.float()), (k, k[:2]), (k.half(), k.half()),
                (k.transpose(0, 1), k.transpose(0, 1))):
        with pytest.raises(ValueError):
            B.KvPool(*bad)
    with pytest.raises(ValueError):
        B.KvPool(k, k, s[:2])
    with pytest.raises(ValueError):
        B.KvPool(k, k, s.double())
    pool = B.KvPool(k, k, s)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    lse = torch.empty(3, 4)
    ws = torch.empty(64, dtype=torch.uint8)
    cases = [dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
             dict(table=table.long()), dict(table=table[:2]), dict(lens=lens[:2]),
             dict(table=torch.zeros(3, 4, dtype=torch.int32)[:, :2]), dict(lens=lens.long()),
             dict(out=out[:2]), dict(lse=lse.double()), dict(window=1 << 32)]
    for c in cases:
        a = dict(q=q, table=table, lens=lens, out=out, lse=lse, window=0)
        a.update(c)
        with pytest.raises(ValueError):
            B.pe_attn_decode(pool, a["q"], a["table"], a["lens"], window=a["window"], out=a["out"],
                             lse=a["lse"], workspace=ws)
    # good shapes, but no GPU tensor
    with pytest.raises(ValueError, match="GPU"):
        B.pe_attn_decode(pool, q, table, lens, out=out, lse=lse, workspace=ws)
    with pytest.raises(ValueError, match="GPU"):
        B.pe_kv_append(pool, q, q[:, :2], q[:, 2:], lens, table, 1e4)
    with pytest.raises(ValueError, match="GPU"):
        B.pe_kv_evict([pool], table, lens, 8)
    with pytest.raises(ValueError):
        B.pe_kv_append(pool, None, q[:, :2], q[:, 2:], lens, table, q_out=q)
    with pytest.raises(ValueError):
        B.pe_kv_evict([], table, lens, 8)
    with pytest.raises(ValueError):
        B.pe_kv_evict([pool], table, lens, 0)
    with pytest.raises(ValueError):
        B.pe_kv_evict([pool], table, lens, 8, sinks=1 << 33)
    with pytest.raises(ValueError):
        B.pe_kv_evict([pool], table, lens, 8, kept=torch.zeros(1, 3, 2, 7, dtype=torch.int32))
