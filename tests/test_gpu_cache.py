"""The paged KV cache operators (include/peagle_cache.h) on a GPU against
their 64-bit definitions (oracle/kv_cache_oracle.py), on the values that the
GPU tensors hold.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  logit     a sum of D products in fp32, in any order, truncated or rounded:
            e_z = (2 D + 8) u sum_i |scale q_i k_i|
  weight    e_w = 2 e_z + 2^-20 + 2 n u + 2^-16: the logits of numerator and
            sum, the exponentials (2^-22 each, a few rescalings), a sum of n
            terms, and weights that may be rounded to a pair of 16-bit numbers
  output    e_w sum_j p_j |v_j| + half a step of its type (bf16 2^-8, fp32 u,
            relative); pairs of fp16 (e4m3 pools) end at 2^-25 of the largest
            weight, which adds 2^-24 n max|v| p_max
  lse       e_z + 2 n u + 2^-20 + 4 u |lse|
  scores    the sum of e_w p over the query heads, and u |score|
  rotation  cos and sin to 2^-22 (angle 2^-24 of half a turn, its sine to a
            few u), two products and a sum: 2^-21 (|a| + |b|), then half a
            step of the type (e4m3: 2^-4 relative, 2^-10 below the normals)
"""

import numpy as np
import pytest

from oracle import kv_cache_oracle as C
from oracle.fp8_kv import E4M3_TABLE, e4m3_encode

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U, "e4m3": 2.0 ** -4}
NAN_CODE = 0x7F


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _act(dt):
    import torch
    return torch.float32 if dt == "f32" else torch.bfloat16


def _make(rng, shape, dt, sd=1.0):
    """Device tensor of N(0, sd) values (e4m3: codes)."""
    import torch
    x = rng.normal(size=shape) * sd
    if dt == "e4m3":
        return torch.from_numpy(e4m3_encode(x)).cuda()
    return torch.from_numpy(x.astype(np.float32)).to(_act(dt)).cuda()


def _host(t):
    """The values a tensor holds, in 64 bits (uint8: e4m3 codes)."""
    import torch
    t = t.detach().cpu()
    return E4M3_TABLE[t.numpy()] if t.dtype == torch.uint8 else t.double().numpy()


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _pages(rng, lens, spare=3, width=None):
    """Block table (unused entries -1) over a random order of pages."""
    n = [-(-int(x) // 16) for x in lens]
    order = rng.permutation(sum(n) + spare)
    t = np.full((len(lens), width or max(1, max(n))), -1, np.int64)
    at = 0
    for b, m in enumerate(n):
        t[b, :m] = order[at:at + m]
        at += m
    return t, order[at:], sum(n) + spare


class Cache:
    """A layer's pools with NaN in every slot that no request holds."""

    def __init__(self, rng, lens, H, D, dt, spare=3, width=None, sd=1.0, k_scale=0.5, v_scale=2.0,
                 scores=True):
        torch, B = _lib()
        self.table, self.spare, nb = _pages(rng, lens, spare, width)
        self.k, self.v = _make(rng, (nb, H, 16, D), dt, sd), _make(rng, (nb, H, 16, D), dt)
        used = np.zeros((nb, 16), bool)
        for b, n in enumerate(lens):
            for p in range(int(n)):
                used[self.table[b][p // 16], p % 16] = True
        hole = torch.from_numpy(~used).cuda()[:, None, :, None].expand(self.k.shape)
        for t in (self.k, self.v):
            t[hole] = NAN_CODE if dt == "e4m3" else float("nan")
        self.scores = torch.from_numpy(rng.random((nb, H, 16)).astype(np.float32)).cuda() \
            if scores else None
        self.dt, self.ks, self.vs = dt, k_scale, v_scale
        self.pool = B.KvPool(self.k, self.v, self.scores, k_scale, v_scale)
        self.t = _i32(self.table)

    def values(self):
        ks, vs = (self.ks, self.vs) if self.dt == "e4m3" else (1.0, 1.0)
        return _host(self.k) * np.float64(np.float32(ks)), _host(self.v) * np.float64(np.float32(vs))


def _check_decode(ref, lens, dt, D, out, lse, scores0=None, scores=None, table=None, rows=None):
    n = np.asarray(lens, np.float64)[:, None]
    ez = (2 * D + 8) * U * ref.zabs
    ew = 2 * ez + 2.0 ** -20 + 2 * n * U + 2.0 ** -16
    tol = ew[..., None] * ref.spread + HALF["f32" if dt == "f32" else "bf16"] * np.abs(ref.out)
    if dt == "e4m3":
        tol = tol + (2.0 ** -24 * n * ref.vmax / ref.peak)[..., None]
    got = _host(out)
    rows = range(len(lens)) if rows is None else rows
    for b in rows:
        assert np.all(np.abs(got[b] - ref.out[b]) <= tol[b]), \
            (b, np.max(np.abs(got[b] - ref.out[b]) / np.maximum(tol[b], 1e-30)))
    got = _host(lse)
    tol = ez + 2 * n * U + 2.0 ** -20 + 4 * U * np.abs(np.where(np.isfinite(ref.lse), ref.lse, 0))
    for b in rows:
        same = np.isneginf(ref.lse[b])
        assert np.array_equal(np.isneginf(got[b]), same)
        assert np.all(np.abs(got[b][~same] - ref.lse[b][~same]) <= tol[b][~same]), b
    if scores is None:
        return
    want, tol = _host(scores0), np.zeros(scores0.shape)
    H = want.shape[1]
    G = ez.shape[1] // H
    for b in rows:
        w, lo = ref.weights[b], ref.lo[b]
        e = ew[b].reshape(H, G).max(1)
        for i in range(w.shape[1]):
            blk, off = C.slot(table, b, lo + i)
            want[blk, :, off] += w[:, i]
            tol[blk, :, off] += e * w[:, i] + U * (w[:, i] + np.abs(want[blk, :, off]))
    assert np.all(np.abs(_host(scores) - want) <= tol)


LENS = [[0, 1, 15, 16, 17, 33, 100], [257], [1024, 3, 0, 511, 48], [2], [0, 0]]
HEADS = [(1, 1), (2, 3), (4, 5), (2, 8), (1, 12), (3, 16), (1, 20), (1, 40)]


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", HEADS)
def test_decode_head_layouts(dt, D, H, G):
    torch, B = _lib()
    rng = np.random.default_rng(H * 100 + G + D)
    lens = LENS[(H + G) % 3]
    c = Cache(rng, lens, H, D, dt)
    q = _make(rng, (len(lens), H * G, D), "f32" if dt == "f32" else "bf16", 2.0)
    before = c.scores.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), accumulate=True, err=err)
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens)
    assert int(err) == 0
    _check_decode(ref, lens, dt, D, out, lse, before, c.scores, c.table)


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000])
@pytest.mark.parametrize("lens", LENS)
def test_decode_lengths_and_windows(dt, window, lens):
    torch, B = _lib()
    D, H, G = 64, 2, 4
    rng = np.random.default_rng(window + len(lens))
    c = Cache(rng, lens, H, D, dt, width=80)
    # pages wholly before the window may be anything, and their ids too
    table = c.table.copy()
    for b, n in enumerate(lens):
        table[b, :max(0, n - window) // 16] = -7
    q = _make(rng, (len(lens), H * G, D), "f32" if dt == "f32" else "bf16", 2.0)
    before = c.scores.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = B.pe_attn_decode(c.pool, q, _i32(table), _i32(lens), window=window,
                                accumulate=True, err=err)
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens, window)
    assert int(err) == 0
    _check_decode(ref, lens, dt, D, out, lse, before, c.scores, c.table)


@pytest.mark.parametrize("dt,D,H,G,lens", [
    ("bf16", 64, 8, 8, [9001, 17, 4096]), ("e4m3", 128, 2, 5, [12345]),
    ("f32", 64, 2, 4, [5003, 1]), ("bf16", 128, 1, 16, [20011]), ("e4m3", 64, 4, 8, [6000, 6001])])
def test_decode_long_lengths(dt, D, H, G, lens):
    torch, B = _lib()
    rng = np.random.default_rng(77)
    c = Cache(rng, lens, H, D, dt)
    q = _make(rng, (len(lens), H * G, D), "f32" if dt == "f32" else "bf16", 2.0)
    before = c.scores.clone()
    out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), accumulate=True)
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens)
    _check_decode(ref, lens, dt, D, out, lse, before, c.scores, c.table)


@pytest.mark.parametrize("dt,D,G", [("bf16", 64, 8), ("e4m3", 64, 3), ("f32", 64, 8), ("f32", 128, 3),
                                    ("bf16", 128, 12), ("e4m3", 128, 16)])
def test_decode_scores_from_kept_and_repeated_logits(dt, D, G):
    """A workspace with room for the logits of none, some (odd numbers of
    pages, inside an item) or all pages gives the same scores."""
    torch, B = _lib()
    rng = np.random.default_rng(14)
    lens, H = [333, 0, 16, 70], 2
    c = Cache(rng, lens, H, D, dt)
    q = _make(rng, (4, H * G, D), "f32" if dt == "f32" else "bf16", 2.0)
    least = B.pe_attn_decode_workspace(4, H * G, H, D)
    most = B.pe_attn_decode_workspace(4, H * G, H, D, c.t.shape[1])
    assert most - least == 4 * c.t.shape[1] * H * 16 * (16 if G > 8 else 8) * 4
    before = c.scores.clone()
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens)
    for size in (least, least + 512, least + 7 * 1024, least + 40 * 1024 + 16, most):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # NaN, if it were read
        c.scores.copy_(before)
        out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), accumulate=True, workspace=ws)
        _check_decode(ref, lens, dt, D, out, lse, before, c.scores, c.table)


def test_decode_many_short_requests():
    torch, B = _lib()
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 40, size=3000).tolist()
    c = Cache(rng, lens, 2, 64, "bf16")
    q = _make(rng, (3000, 4, 64), "bf16", 2.0)
    before = c.scores.clone()
    out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), accumulate=True)
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens)
    _check_decode(ref, lens, "bf16", 64, out, lse, before, c.scores, c.table)


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("scale", [0.7, -0.7, 0.0])
def test_decode_strided_rows_scale_and_sharp_logits(dt, scale):
    """q as a slice of a fused projection's output, out as a slice of a wider
    buffer (whose other elements stay), a scale of its own, logits in the
    hundreds."""
    torch, B = _lib()
    D, H, G, lens = 64, 2, 4, [300, 31]
    rng = np.random.default_rng(3)
    c = Cache(rng, lens, H, D, dt, sd=3.0)
    act = "f32" if dt == "f32" else "bf16"
    qkv = _make(rng, (2, H * G + 2 * H, D), act, 3.0)
    q = qkv[:, :H * G]
    wide = torch.full((2, H * G + 4, D), 7.0, dtype=_act(dt), device="cuda")
    out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), scale=scale, out=wide[:, 2:2 + H * G])
    kv = c.values()
    ref = C.decode(np.nan_to_num(kv[0]), np.nan_to_num(kv[1]), _host(q), c.table, lens, 
                   scale=float(np.float32(scale)))
    _check_decode(ref, lens, dt, D, out, lse)
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, -2:] == 7).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_infinities_and_nan(dt):
    """A key of -inf logit gets no weight; a NaN inside a request stays in
    it; a row whose logits are all -inf gives 0 and -inf."""
    torch, B = _lib()
    D, lens = 64, [40, 40, 20]
    rng = np.random.default_rng(4)
    c = Cache(rng, lens, 1, D, dt)
    q = _make(rng, (3, 2, D), dt, 1.0)
    q[:, :, 0] = 1.0
    blk, off = C.slot(c.table, 0, 21)
    c.k[blk, 0, off, 0] = float("-inf")
    blk, off = C.slot(c.table, 1, 5)
    c.v[blk, 0, off, 3] = float("nan")
    for p in range(20):
        blk, off = C.slot(c.table, 2, p)
        c.k[blk, 0, off, 0] = float("-inf")
    before = c.scores.clone()
    out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(lens), accumulate=True)
    k, v = c.values()
    k, v = np.where(np.isnan(k), 0, k), np.nan_to_num(v)
    ref = C.decode(np.where(np.isneginf(k), -1e30, k), v, _host(q), c.table, lens)
    ref.zabs[0] = (np.abs(np.where(np.isinf(k), 0, k)).max() * np.abs(_host(q)).max() * D) / 8
    _check_decode(ref, lens, dt, D, out, lse, rows=[0])
    got = _host(out)
    assert np.isnan(got[1, :, 3]).all() and np.isfinite(np.delete(got[1], 3, axis=1)).all()
    assert not got[2].any() and np.isneginf(_host(lse)[2]).all()
    grew = _host(c.scores) - _host(before)
    assert np.isfinite(grew).all()
    for p in range(20):
        blk, off = C.slot(c.table, 2, p)
        assert grew[blk, 0, off] == 0
    blk, off = C.slot(c.table, 0, 21)
    assert grew[blk, 0, off] == 0


def test_decode_bad_lengths_and_pages_are_recorded():
    torch, B = _lib()
    D, lens = 64, [40, 64, 30]
    rng = np.random.default_rng(5)
    c = Cache(rng, lens, 2, D, "bf16", width=4)
    q = _make(rng, (3, 4, D), "bf16")
    kv = [np.nan_to_num(x) for x in c.values()]
    for given, used, code in (([40, 65, 30], [40, 64, 30], B.PE_DEV_BAD_POSITION),
                              ([40, -1, 30], [40, 0, 30], B.PE_DEV_BAD_POSITION)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = B.pe_attn_decode(c.pool, q, c.t, _i32(given), err=err)
        assert int(err) == code
        _check_decode(C.decode(*kv, _host(q), c.table, used), used, "bf16", D, out, lse)
    # request 1's second page is no page: its positions are left out
    for bad in (-1, c.pool.num_blocks, 1 << 30):
        table = c.table.copy()
        table[1, 1] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        before = c.scores.clone()
        out, lse = B.pe_attn_decode(c.pool, q, _i32(table), _i32(lens), accumulate=True, err=err)
        assert int(err) == B.PE_DEV_BAD_BLOCK
        short = c.table.copy()
        short[1] = [c.table[1, 0], c.table[1, 2], c.table[1, 3], -1]
        less = [40, 48, 30]
        ref = C.decode(*kv, _host(q), short, less)
        _check_decode(ref, less, "bf16", D, out, lse, before, c.scores, short)
        # without a place to record it
        out2, _ = B.pe_attn_decode(c.pool, q, _i32(table), _i32(lens))
        assert torch.equal(out, out2)


def test_decode_requests_sharing_pages():
    """Two requests of one call with a common prefix: both attend it, and its
    scores grow by both."""
    torch, B = _lib()
    rng = np.random.default_rng(6)
    lens = [50, 40]
    c = Cache(rng, lens, 1, 64, "bf16")
    table = c.table.copy()
    table[1, :2] = table[0, :2]
    q = _make(rng, (2, 8, 64), "bf16")
    before = c.scores.clone()
    out, lse = B.pe_attn_decode(c.pool, q, _i32(table), _i32(lens), accumulate=True)
    kv = [np.nan_to_num(x) for x in c.values()]
    _check_decode(C.decode(*kv, _host(q), table, lens), lens, "bf16", 64, out, lse, before,
                  c.scores, table)


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
def test_decode_offsets_past_32_bits(dt):
    """Pages whose element offsets do not fit 31 (and byte offsets 32) bits."""
    torch, B = _lib()
    H, D = 8, 128
    nb = (1 << 31) // (H * 16 * D) + 40
    td = {"bf16": torch.bfloat16, "e4m3": torch.uint8, "f32": torch.float32}[dt]
    k = torch.zeros(nb, H, 16, D, dtype=td, device="cuda")
    v = torch.zeros(nb, H, 16, D, dtype=td, device="cuda")
    s = torch.zeros(nb, H, 16, device="cuda")
    rng = np.random.default_rng(8)
    lens = [70]
    table = np.array([[nb - 1, nb - 17, nb - 3, 0, nb - 30]])
    idx = torch.from_numpy(table[0]).cuda()
    k[idx], v[idx] = _make(rng, (5, H, 16, D), dt), _make(rng, (5, H, 16, D), dt)
    pool = B.KvPool(k, v, s)
    q = _make(rng, (1, 16, D), "f32" if dt == "f32" else "bf16")
    out, lse = B.pe_attn_decode(pool, q, _i32(table), _i32(lens), accumulate=True)
    small = np.arange(5)[None]
    ref = C.decode(_host(k[idx]), _host(v[idx]), _host(q), small, lens)
    _check_decode(ref, lens, dt, D, out, lse, torch.zeros_like(s[idx]), s[idx], small)
    # and a trim whose pages lie there
    dst = np.array([[nb - 2, nb - 5]])
    kept, new = B.pe_kv_evict([pool], _i32(table), _i32(lens), 20, 1, 3, dst_table=_i32(dst))
    want = C.keep(np.concatenate([_host(s[i])[2] for i in table[0]])[:70], 20, 1, 3)
    assert kept[0, 0, 2].tolist() == want.tolist()
    assert torch.equal(k[nb - 5, 2, 3], k[table[0, want[19] // 16], 2, want[19] % 16])
    del k, v, s, pool
    torch.cuda.empty_cache()


def test_decode_is_deterministic_and_replays_in_graphs():
    """Two captured graphs on different inputs, replayed in turn, and eager
    calls between, all give the eager results bit for bit."""
    torch, B = _lib()
    rng = np.random.default_rng(10)
    state = []
    for lens in ([700, 33, 0, 4000], [1, 900, 80, 2500]):
        c = Cache(rng, lens, 4, 64, "bf16")
        q = _make(rng, (4, 32, 64), "bf16", 2.0)
        n = _i32(lens)
        want = B.pe_attn_decode(c.pool, q, c.t, n)
        out, lse = torch.empty_like(q), torch.empty(4, 32, device="cuda")
        state.append((c, q, n, want, out, lse))
    graphs = []
    for c, q, n, _, out, lse in state:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.pe_attn_decode(c.pool, q, c.t, n, out=out, lse=lse)
        graphs.append(g)
    for turn in range(3):
        for g, (c, q, n, want, out, lse) in zip(graphs, state):
            out.zero_(), lse.zero_()
            g.replay()
            again = B.pe_attn_decode(c.pool, q, c.t, n)
            torch.cuda.synchronize()
            for a, b, w in zip((out, lse), again, want):
                assert torch.equal(a, w) and torch.equal(b, w)
    # the lengths and the table are read at replay
    c, q, n, _, out, lse = state[0]
    n.copy_(_i32([650, 0, 0, 3999]))
    want = B.pe_attn_decode(c.pool, q, c.t, n)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_calls_on_another_stream():
    torch, B = _lib()
    rng = np.random.default_rng(11)
    lens = [5000, 1200]
    c = Cache(rng, lens, 4, 64, "bf16")
    q, n = _make(rng, (2, 32, 64), "bf16", 2.0), _i32(lens)
    want = B.pe_attn_decode(c.pool, q, c.t, n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):        # both streams at once, a workspace each
        outs.append(B.pe_attn_decode(c.pool, q, c.t, n, stream=side))
        outs.append(B.pe_attn_decode(c.pool, q, c.t, n))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


def test_streams_and_captures_have_workspaces_of_their_own():
    """Eager calls on two streams at once, beside replays of a graph captured
    on one of them, larger and smaller calls in turn."""
    torch, B = _lib()
    rng = np.random.default_rng(12)
    jobs = []
    for D, lens in ((64, [6000, 900]), (128, [20, 4001, 7, 0])):
        c = Cache(rng, lens, 4, D, "bf16")
        q, n = _make(rng, (len(lens), 32, D), "bf16", 2.0), _i32(lens)
        jobs.append((c, q, n, B.pe_attn_decode(c.pool, q, c.t, n)))
    c, q, n, want = jobs[0]
    out, lse = torch.empty_like(q), torch.empty(2, 32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pe_attn_decode(c.pool, q, c.t, n, out=out, lse=lse)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for turn in range(12):
        g.replay()
        for side in sides:
            with torch.cuda.stream(side):
                for c, q, n, w in (jobs, jobs[::-1])[turn % 2]:
                    got.append((B.pe_attn_decode(c.pool, q, c.t, n), w))
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for (o, l), (wo, wl) in got:
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_threads_on_one_stream():
    """Two host threads that share a stream: neither call's launches fall
    between the other's."""
    import threading
    torch, B = _lib()
    rng = np.random.default_rng(13)
    jobs = []
    for lens in ([3000, 2999], [700, 5000]):
        c = Cache(rng, lens, 4, 64, "bf16")
        q, n = _make(rng, (2, 32, 64), "bf16", 2.0), _i32(lens)
        jobs.append((c, q, n, B.pe_attn_decode(c.pool, q, c.t, n)))
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        c, q, n, _ = jobs[i]
        for _ in range(200):
            got[i].append(B.pe_attn_decode(c.pool, q, c.t, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 200
        assert all(torch.equal(o, jobs[i][3][0]) and torch.equal(l, jobs[i][3][1])
                   for o, l in got[i])


# ------------------------------------------------------------------ append

def _rot_tol(x, dt):
    """Per element of a rotated row x [..., D] (its input values)."""
    half = x.shape[-1] // 2
    s = np.abs(x[..., :half]) + np.abs(x[..., half:])
    return 2.0 ** -21 * np.concatenate((s, s), axis=-1)


def _round_ok(got, want, err, dt):
    """got is `want` (known to within err) rounded to dt."""
    if dt == "e4m3":
        want = np.clip(want, -448, 448)
        return np.all(np.abs(got - want) <= err + np.maximum(HALF[dt] * (np.abs(want) + err), 2.0 ** -10))
    return np.all(np.abs(got - want) <= err + HALF[dt] * (np.abs(want) + err))


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("theta", [0.0, 1e4, 1.5e5])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 8), (5, 3)])
def test_append_rows(dt, D, theta, H, G):
    torch, B = _lib()
    rng = np.random.default_rng(int(theta) + D + H)
    lens = [40, 17, 100]
    c = Cache(rng, lens, H, D, dt, width=8)
    act = "f32" if dt == "f32" else "bf16"
    req = np.array([2, 0, 1, 0, 2, 1, 0])
    pos = np.array([99, 0, 16, 39, 5, -1, 15])
    T = len(req)
    qkv = _make(rng, (T, H * G + 2 * H, D), act)
    q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
    k0, v0, s0 = c.k.clone(), c.v.clone(), c.scores.clone()
    q_out = torch.full((T, H * G, D), 7.0, dtype=_act(dt), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.pe_kv_append(c.pool, q, k, v, _i32(pos), c.t, theta, req=_i32(req), q_out=q_out, err=err)
    assert got is q_out and int(err) == 0
    live = pos >= 0
    qh = _host(q)
    want = C.rotate(qh, np.repeat(pos[:, None], H * G, 1), theta)
    assert _round_ok(_host(q_out)[live], want[live], _rot_tol(qh, act)[live] * bool(theta), act)
    assert bool((q_out[torch.from_numpy(~live).cuda()] == 7).all())
    kh, vh = _host(k), _host(v)
    kw = C.rotate(kh, np.repeat(pos[:, None], H, 1), theta)
    ks, vs = (c.ks, c.vs) if dt == "e4m3" else (1.0, 1.0)
    gk, gv, gs = _host(c.k), _host(c.v), _host(c.scores)
    touched = np.zeros(gk.shape[:3], bool)
    for t in range(T):
        if not live[t]:
            continue
        blk, off = C.slot(c.table, req[t], pos[t])
        touched[blk, :, off] = True
        assert _round_ok(gk[blk, :, off], kw[t] / ks, _rot_tol(kh[t], act) / ks * bool(theta), dt)
        assert _round_ok(gv[blk, :, off], vh[t] / vs, 0.0, dt)
        assert not gs[blk, :, off].any()
    for new, old in ((c.k, k0), (c.v, v0), (c.scores, s0)):
        keep = torch.from_numpy(~touched).cuda()
        a, b = new[keep], old[keep]
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_append_far_positions_in_place_and_without_q():
    """Angles at positions in the millions, q rotated in place, one row a
    request (no req), pools without scores."""
    torch, B = _lib()
    rng = np.random.default_rng(21)
    H, D, theta = 2, 64, 1e6
    nb = 8
    pos = np.array([3_000_017, 2_000_000])
    table = np.full((2, 187502), -1, np.int32)
    table[0, pos[0] // 16], table[1, pos[1] // 16] = 5, 2
    k = torch.zeros(nb, H, 16, D, device="cuda")
    v = torch.zeros_like(k)
    pool = B.KvPool(k, v)
    q = _make(rng, (2, 4, D), "f32")
    kn, vn = _make(rng, (2, H, D), "f32"), _make(rng, (2, H, D), "f32")
    qh = _host(q)
    assert B.pe_kv_append(pool, q, kn, vn, _i32(pos), _i32(table), theta, q_out=q) is q
    want = C.rotate(qh, np.repeat(pos[:, None], 4, 1), theta)
    # the 64-bit angle of the oracle itself is off by pos 2^-53 rad
    assert _round_ok(_host(q), want, _rot_tol(qh, "f32"), "f32")
    wk = C.rotate(_host(kn), np.repeat(pos[:, None], H, 1), theta)
    assert _round_ok(_host(k)[5, :, 1], wk[0], _rot_tol(_host(kn), "f32")[0], "f32")
    assert _round_ok(_host(k)[2, :, 0], wk[1], _rot_tol(_host(kn), "f32")[1], "f32")
    k.zero_()
    assert B.pe_kv_append(pool, None, kn, vn, _i32(pos), _i32(table), 0.0) is None
    assert torch.equal(k[5, :, 1], kn[0]) and torch.equal(v[2, :, 0], vn[1])


def test_append_device_errors():
    torch, B = _lib()
    rng = np.random.default_rng(22)
    c = Cache(rng, [20, 20], 2, 64, "bf16", width=2)
    rows = _make(rng, (2, 8, 64), "bf16")
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    table = c.table.copy()
    table[1, 1] = 10 ** 6
    for req, pos, code in (([0, 2], [19, 3], B.PE_DEV_BAD_ROW), ([0, -1], [19, 3], B.PE_DEV_BAD_ROW),
                           ([0, 1], [19, 32], B.PE_DEV_BAD_POSITION),
                           ([0, 1], [19, 17], B.PE_DEV_BAD_BLOCK)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k0 = c.k.clone()
        out = B.pe_kv_append(c.pool, q, k, v, _i32(pos), _i32(table), 0.0, req=_i32(req), err=err)
        assert int(err) == code
        assert torch.equal(out, q)                       # theta 0: q as it is, errors or not
        blk, off = C.slot(table, 0, 19)
        assert torch.equal(c.k[blk, :, off], k[0])
        k0[blk, :, off] = k[0]
        assert torch.equal(c.k.view(torch.uint8), k0.view(torch.uint8))


def test_append_saturates_e4m3():
    torch, B = _lib()
    c = Cache(np.random.default_rng(23), [1], 1, 64, "e4m3", k_scale=1.0, v_scale=1.0)
    k = torch.full((1, 1, 64), 1e6, dtype=torch.bfloat16, device="cuda")
    B.pe_kv_append(c.pool, None, k, -k, _i32([0]), c.t, 0.0)
    blk, off = C.slot(c.table, 0, 0)
    assert (_host(c.k)[blk, 0, off] == 448).all() and (_host(c.v)[blk, 0, off] == -448).all()


# ------------------------------------------------------------------- evict

def _check_evict(c, before, ref, dt, theta, kept, new, layer=0):
    """Pools after the call against the oracle's."""
    rk, rn, k2, v2, s2 = ref
    assert np.array_equal(kept[layer].cpu().numpy(), rk)
    assert np.array_equal(new.cpu().numpy(), rn)
    k0, v0, s0 = before
    assert np.array_equal(_host(c.v), v2, equal_nan=True)
    assert np.array_equal(_host(c.scores), s2)
    got = _host(c.k)
    same = (k2 == k0) | (np.isnan(k2) & np.isnan(k0))
    if not theta:
        assert np.array_equal(got, k2, equal_nan=True)
        return
    # a rotated key's error goes with its pair's size
    half = k2.shape[-1] // 2
    r = np.sqrt(k2[..., :half] ** 2 + k2[..., half:] ** 2)
    err = 2.0 ** -20 * np.concatenate((r, r), axis=-1)
    fin = ~np.isnan(k2)
    assert np.array_equal(np.isnan(got), ~fin)
    assert _round_ok(got[fin & ~same], k2[fin & ~same], err[fin & ~same], dt)
    rows = same.all(-1)
    assert np.array_equal(got[rows], k0[rows], equal_nan=True)


EVICT = [  # lens, budget, sinks, recent
    ([100, 20, 64, 0, 1], 32, 4, 8), ([300], 1, 0, 0), ([300, 299], 1, 1, 0), ([300], 1, 0, 1),
    ([257, 90], 90, 40, 50), ([1000, 17], 333, 3, 100), ([50, 60], 64, 4, 4), ([1200], 700, 0, 0)]


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 1)])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(dt, D, H, fresh, case):
    torch, B = _lib()
    lens, budget, sinks, recent = EVICT[case]
    theta = 0.0 if case in (2, 4) else 1e4
    rng = np.random.default_rng(case * 10 + H)
    need = sum(-(-min(n, budget) // 16) for n in lens)
    c = Cache(rng, lens, H, D, dt, spare=need + 2)
    # many equal scores, some of them zero, minus zero, NaN or -inf
    s = np.round(rng.random(c.scores.shape) * 8) / 4
    s[rng.random(s.shape) < 0.1] = -0.0
    s[rng.random(s.shape) < 0.03] = np.nan
    s[rng.random(s.shape) < 0.03] = -np.inf
    c.scores.copy_(torch.from_numpy(s.astype(np.float32)))
    s = np.where(np.isnan(s), -1e30, s)          # the oracle's copy: no NaN to compare
    nanmask = torch.isnan(c.scores)
    dst = None
    if fresh:
        dst = np.full((len(lens), max(1, -(-budget // 16))), -1, np.int64)
        at = 0
        for b, n in enumerate(lens):
            m = -(-min(n, budget) // 16)
            dst[b, :m] = c.spare[at:at + m]
            at += m
    before = _host(c.k), _host(c.v), s
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new = B.pe_kv_evict([c.pool], c.t, _i32(lens), budget, sinks, recent, rope_theta=theta,
                              dst_table=None if dst is None else _i32(dst), err=err)
    assert int(err) == 0
    ref = C.evict(before[0], before[1], np.where(nanmask.cpu().numpy(), np.nan, s), c.table,
                  np.array(lens), budget, sinks, recent, theta, dst)
    ref = ref[:4] + (np.nan_to_num(ref[4], nan=-1e30, neginf=-np.inf),)
    c.scores[torch.isnan(c.scores)] = -1e30
    ref[4][:] = np.float32(ref[4])
    _check_evict(c, before, ref, dt, theta, kept, new)


@pytest.mark.parametrize("n,budget", [(70_001, 65_537), (70_001, 900), (40_000, 20_000),
                                      (120_000, 5_000)])
@pytest.mark.parametrize("fresh", [False, True])
def test_evict_long_rows(n, budget, fresh):
    torch, B = _lib()
    rng = np.random.default_rng(31)
    c = Cache(rng, [n], 1, 64, "bf16", spare=-(-budget // 16))
    dst = c.spare[None, :] if fresh else None
    before = _host(c.k), _host(c.v), _host(c.scores)
    kept, new = B.pe_kv_evict([c.pool], c.t, _i32([n]), budget, 5, 700 if budget > 800 else 1,
                              rope_theta=1e4, dst_table=None if dst is None else _i32(dst))
    ref = C.evict(*before, c.table, np.array([n]), budget, 5, 700, 1e4, dst)
    _check_evict(c, before, ref, "bf16", 1e4, kept, new)


def test_evict_long_rows_of_equal_scores():
    """Ties that cross what the shared memory holds at once, alone on the
    device and beside other rows."""
    torch, B = _lib()
    for lens, H in (([60_000], 1), ([30_000, 100] * 20, 4)):
        c = Cache(np.random.default_rng(37), lens, H, 64, "f32")
        s = np.zeros(tuple(c.scores.shape), np.float32)
        s[::3] = 0.25
        c.scores.copy_(torch.from_numpy(s))
        before = _host(c.scores)
        n = lens[0]
        kept, new = B.pe_kv_evict([c.pool], c.t, _i32(lens), n - 7_000, 3, 11)
        for b in (0, len(lens) - 2 if len(lens) > 1 else 0):
            row = np.concatenate([before[c.table[b, i], 0] for i in range(-(-n // 16))])[:n]
            want = C.keep(row, n - 7_000, 3, 11)
            assert np.array_equal(kept[0, b, 0].cpu().numpy(), want)


def test_evict_into_its_own_table_is_in_place():
    torch, B = _lib()
    lens, got = [900, 30], []
    for own_table in (False, True):
        c = Cache(np.random.default_rng(36), lens, 8, 64, "bf16")
        r = B.pe_kv_evict([c.pool], c.t, _i32(lens), 500, 4, 100, 1e4,
                          dst_table=c.t if own_table else None)
        got.append((*r, c.k, c.v, c.scores))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))


@pytest.mark.parametrize("fresh", [False, True])
def test_evict_layers_at_once(fresh):
    """Five layers with their own scores (and pool sizes) in one call equal
    five calls of one."""
    torch, B = _lib()
    rng = np.random.default_rng(32)
    lens = [400, 33, 150]
    caches = []
    for extra in range(5):
        r2 = np.random.default_rng(33)           # the same block table
        c = Cache(r2, lens, 2, 64, "bf16", spare=30)
        k = torch.cat((c.k, c.k[:extra])).contiguous()
        v = torch.cat((c.v, c.v[:extra])).contiguous()
        s = torch.from_numpy(rng.random(k.shape[:3]).astype(np.float32)).cuda()
        caches.append((k, v, s, c))
    c = caches[0][3]
    dst = _i32(np.stack([c.spare[i * 6:i * 6 + 6] for i in range(3)])) if fresh else None
    args = (c.t, _i32(lens), 90, 4, 20, 1e4, dst)
    one = [[x.clone() for x in y[:3]] for y in caches]
    got = [B.pe_kv_evict([B.KvPool(*y)], *args) for y in one]
    kept, new = B.pe_kv_evict([B.KvPool(*y[:3]) for y in caches], *args)
    for l in range(5):
        assert torch.equal(kept[l], got[l][0][0]) and torch.equal(new, got[l][1])
        for a, b in zip(caches[l][:3], one[l]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_evict_device_errors():
    torch, B = _lib()
    rng = np.random.default_rng(34)
    lens = [80, 80]
    for what in ("length", "source", "narrow", "destination"):
        c = Cache(rng, lens, 2, 64, "bf16", spare=10)
        table, dst, given = c.table.copy(), np.stack((c.spare[:3], c.spare[3:6])), list(lens)
        code = B.PE_DEV_BAD_BLOCK
        if what == "length":
            given[1], code = -5, B.PE_DEV_BAD_POSITION
        elif what == "source":
            table[1, 2] = -1
        elif what == "narrow":
            dst, code = dst[:, :2], B.PE_DEV_BAD_POSITION
        else:
            dst[1, 1] = 1 << 20
        before = _host(c.k), _host(c.v), _host(c.scores)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kept, new = B.pe_kv_evict([c.pool], _i32(table), _i32(given), 40, 4, 8, rope_theta=1e4,
                                  dst_table=_i32(dst), err=err)
        assert int(err) == code, what
        # request 0 is trimmed as ever where it has room
        ref = C.evict(*before, c.table, np.array([80, 0]), 40, 4, 8, 1e4,
                      np.concatenate((dst[:, :2], np.stack((c.spare[2:3], c.spare[5:6]))), 1))
        assert np.array_equal(kept[0, 0].cpu().numpy(), ref[0][0])
        for j in range(32 if what == "narrow" else 40):
            blk, off = C.slot(dst, 0, j)
            assert np.array_equal(_host(c.v)[blk, :, off], ref[3][blk, :, off])
        if what == "length":
            assert new.tolist() == [40, 0] and (kept[0, 1] == -1).all()
        if what == "source":      # a bad page's positions go last
            assert not np.isin(np.arange(32, 48), kept[0, 1].cpu().numpy()).any()


def test_evict_replays_in_a_graph():
    torch, B = _lib()
    rng = np.random.default_rng(35)
    lens = [500, 40]
    c = Cache(rng, lens, 2, 64, "e4m3", spare=12)
    dst = _i32(np.stack((c.spare[:6], c.spare[6:12])))
    n = _i32(lens)
    kept, new = B.pe_kv_evict([c.pool], c.t, n, 96, 4, 16, 1e4, dst)
    want = [x.clone() for x in (kept, new, c.k, c.v, c.scores)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pe_kv_evict([c.pool], c.t, n, 96, 4, 16, 1e4, dst, kept=kept, new_lens=new)
    for b, m in enumerate(new.tolist()):          # every slot that the call writes
        for j in range(m):
            blk, off = C.slot(dst.tolist(), b, j)
            c.k[blk, :, off], c.v[blk, :, off] = 0, 0
    kept.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((kept, new, c.k, c.v, c.scores), want):
        assert torch.equal(a, b)


# ------------------------------------------------- the operators as used

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_loop_with_trims(dt):
    """Append, attend with scores, trim when the budget is passed, go on: each
    step against the oracle on the cache that the GPU holds."""
    torch, B = _lib()
    rng = np.random.default_rng(40)
    H, G, D, theta, budget = 2, 4, 64, 1e4, 48
    lens = np.array([45, 3, 60])
    c = Cache(rng, lens, H, D, dt, width=6, spare=18)
    free = list(c.spare)
    for b in range(3):
        for i in range(6):
            if c.table[b, i] < 0:
                c.table[b, i] = free.pop()
    c.t.copy_(torch.from_numpy(c.table))
    act = "f32" if dt == "f32" else "bf16"
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = _i32(lens)
    for step in range(12):
        rows = _make(rng, (3, H * G + 2 * H, D), act)
        q = B.pe_kv_append(c.pool, rows[:, :H * G], rows[:, H * G:H * G + H], rows[:, H * G + H:],
                           n, c.t, theta, err=err)
        n = n + 1
        before = c.scores.clone()
        out, lse = B.pe_attn_decode(c.pool, q, c.t, n, accumulate=True, err=err)
        host = n.cpu().numpy()
        kv = [np.nan_to_num(x) for x in c.values()]
        _check_decode(C.decode(*kv, _host(q), c.table, host), host, dt, D, out, lse, before,
                      c.scores, c.table)
        if step % 4 == 3:
            state = _host(c.k), _host(c.v), _host(c.scores)
            kept, new = B.pe_kv_evict([c.pool], c.t, n, budget, 2, 16, theta, err=err)
            ref = C.evict(*state, c.table, host, budget, 2, 16, theta)
            _check_evict(c, state, ref, dt, theta, kept, new)
            n = new.clone()
    assert int(err) == 0 and int(n.max()) <= budget


def test_drafting_step_on_a_trimmed_cache():
    """A drafter's pools trimmed in all layers, then a drafting step that goes
    on at the shorter length, against the drafting oracle on the same cache."""
    import oracle as O
    from synthetic import workloads as W
    from tests import gpu_helpers as G
    torch, B = _lib()
    shape = W.small_shape("small-bf16", d=512, n_layers=2, n_heads=8, n_kv_heads=2, head_dim=64,
                          ffn=1024, vocab=4096)
    wl = W.custom("trimmed", 91, shape, 4, [300, 90], [5, 5], [4, 2])
    inp = W.make_step_inputs(wl)
    w = W.make_weights(shape, wl.config_id, gains=wl.gains)
    kc, vc = W.make_kv_cache(wl, inp)
    st = G.DeviceStep(wl, inp, kc, vc)
    first = st.target_pos[st.cu_in[:-1].long()]       # the window starts where the cache ends
    lens = (first + 1).int()                          # cached positions 0 .. first
    pools = [B.KvPool(k, v, torch.rand(k.shape[:3], device="cuda")) for k, v in zip(st.kc, st.vc)]
    kept, new = B.pe_kv_evict(pools, st.block_table, lens, 100, 4, 32, rope_theta=shape.rope_theta)
    # the step's window moves with the cache
    shift = (lens - new).cpu().numpy()
    T = int(inp.cu_in[-1])
    r = np.searchsorted(np.asarray(inp.cu_in)[1:], np.arange(T), side="right")
    inp.target_pos = (np.asarray(inp.target_pos) - shift[r]).astype(np.int32)
    st.target_pos.copy_(torch.from_numpy(inp.target_pos))
    kc2, vc2 = [B.to_host(k) for k in st.kc], [B.to_host(v) for v in st.vc]
    dr = G.make_drafter(shape, w, max(wl.T_out, wl.B * wl.K), wl.B)
    res = G.run_step(dr, st)
    assert res["err"] == 0
    ref = O.draft_step(shape, w, wl.K, inp, kc2, vc2, requests=[0, 1])
    got = G.f64(B.to_host(res["out_hidden"]), shape.dtype)
    assert np.abs(got - ref.out_hidden).max() <= 2e-2 * np.abs(ref.out_hidden).max()
    dr.close()


@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16-128", "e4m3"])
@pytest.mark.parametrize("K", [1, 4])
def test_drafting_step_collects_scores(kind, K, monkeypatch):
    """With pe_set_kv_scores the step's results are the same bit for bit, and
    each layer's scores grow by the next-token rows' weights.  The pipeline
    before a layer's logits is right to TOL of their size (the drafting
    suite's rule), so a weight is right to a factor exp(4 TOL max|z|)."""
    import oracle as O
    from oracle import fp8_kv as F
    from oracle import peagle_oracle as PO
    from synthetic import workloads as W
    from tests import gpu_helpers as G
    torch, B = _lib()
    dt = "f32" if kind == "f32" else "bf16"
    tol = 1e-4 if kind == "f32" else 2e-2
    dh = 128 if kind == "bf16-128" else 64
    shape = W.small_shape("scored-" + kind, d=512, n_layers=2, n_heads=8, n_kv_heads=2,
                          head_dim=dh, ffn=1024, vocab=4096)
    if dt == "f32":
        import dataclasses
        shape = dataclasses.replace(shape, dtype="f32")
    wl = W.custom("scored", 92, shape, K, [300, 40, 1, 129], [K + 1, K + 1, K + 1, 1],
                  [K, 0, min(1, K), 0])
    inp = W.make_step_inputs(wl)
    w = W.make_weights(shape, wl.config_id, gains=wl.gains)
    kc, vc = W.make_kv_cache(wl, inp)
    scales = None
    if kind == "e4m3":
        scales = [(0.05, 0.05)] * 2
        kc = [F.quantize(O.to_f64(k, dt), 0.05) for k in kc]
        vc = [F.quantize(O.to_f64(v, dt), 0.05) for v in vc]
    dr = G.make_drafter(shape, w, max(wl.T_out, wl.B * K), wl.B)
    if scales:
        B.pe_set_kv_cache_fp8(dr, [0.05] * 2, [0.05] * 2)
    rng = np.random.default_rng(50)
    start = [torch.from_numpy(rng.random(tuple(kc[0].shape[:3])).astype(np.float32)).cuda()
             for _ in range(2)]
    scores = [x.clone() for x in start]
    results = []
    for collect in (False, True, False):
        B.pe_set_kv_scores(dr, scores if collect else None)
        st = G.DeviceStep(wl, inp, kc, vc)
        res = G.run_step(dr, st)
        assert res["err"] == 0
        results.append((res["tokens"], res["out_hidden"], res["logits"], *st.kc, *st.vc))
    for other in results[1:]:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(results[0], other))

    calls = []
    plain = PO.attention_one_row

    def recording(q, k_seq, v_seq, P):
        z = np.stack([k_seq[:P + 1, h // (q.shape[0] // k_seq.shape[1])] @ q[h]
                      for h in range(q.shape[0])]) / np.sqrt(q.shape[1])
        calls.append((P, z))
        return plain(q, k_seq, v_seq, P)

    monkeypatch.setattr(PO, "attention_one_row", recording)
    O.draft_step(shape, w, K, inp, kc, vc, kv_scales=scales)
    a = np.asarray(inp.num_accepted)
    per_layer = int((a + K).sum())            # rows 0..a and the K - 1 MASK rows
    assert len(calls) == 2 * per_layer
    for l in range(2):
        want, tols = _host(start[l]), np.zeros(start[l].shape)
        at = l * per_layer
        for r in range(wl.B):
            P, z = calls[at + int(a[r])]      # the row that follows the accepted ones
            at += int(a[r]) + K
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            e = np.expm1(4 * tol * np.abs(z).max())
            for i in range(P + 1):
                blk, off = C.slot(inp.block_table, r, i)
                wt = p[:, i].reshape(2, -1).sum(1)
                want[blk, :, off] += wt
                tols[blk, :, off] += e * wt + 2.0 ** -20 * (1 + np.abs(want[blk, :, off]))
        got = _host(scores[l])
        assert np.all(np.abs(got - want) <= tols)
        grew = got - _host(start[l])
        for r in range(wl.B):                 # all of a row's weight is there
            P = int(inp.target_pos[inp.cu_in[r]]) + int(a[r]) + 1
            g = sum(grew[blk, :, off] for blk, off in
                    (C.slot(inp.block_table, r, i) for i in range(P + 1)))
            assert np.all(np.abs(g - 4) <= 4 * 2.0 ** -18 + (P + 1) * 2.0 ** -23)
    dr.close()


def test_score_collecting_refusals():
    from synthetic import workloads as W
    from tests import gpu_helpers as G
    torch, B = _lib()
    shape = W.small_shape("small-bf16", d=512, n_layers=2, n_heads=8, n_kv_heads=2, head_dim=64,
                          ffn=1024, vocab=4096)
    wl = W.custom("refused", 93, shape, 4, [30], [5], [4])
    inp = W.make_step_inputs(wl)
    w = W.make_weights(shape, wl.config_id, gains=wl.gains)
    dr = G.make_drafter(shape, w, wl.T_out, 1)
    ok = torch.zeros(inp.num_blocks, 2, 16, device="cuda")
    for bad in ([ok], [ok, ok.double()], [ok, ok[:, :1]], [ok, ok.cpu()], [ok, ok.transpose(1, 2)]):
        with pytest.raises(ValueError):
            B.pe_set_kv_scores(dr, bad)
    with pytest.raises(B.PeError):
        B.pe_set_kv_scores(dr, [ok, torch.zeros(2 * 16 * 4 + 1, device="cuda")[1:].view(4, 2, 16)])
    small = torch.zeros(inp.num_blocks - 1, 2, 16, device="cuda")
    B.pe_set_kv_scores(dr, [ok, small])
    kc, vc = W.make_kv_cache(wl, inp)
    with pytest.raises(ValueError):
        G.run_step(dr, G.DeviceStep(wl, inp, kc, vc))
    dr.close()
