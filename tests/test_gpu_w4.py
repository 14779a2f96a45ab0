"""Products with 4-bit weights (include/peagle_w4.h) on a GPU against the
64-bit product of the same values.

Tolerance, from the arithmetic (u = 2^-24, S = sum_j |x_j w_j|): products of
bf16 numbers are exact in fp32; a group's products are summed in fp32 in any
order, each addition rounded or truncated (2 u at most): 2 group u S; each
group's sum is scaled and added (2 roundings), partial results of at most 64
warps are added: (2 groups + 64) u S.  fp32 x: three fp16 parts leave less
than u |x| of what is within 2^-14 of its row's largest (less, 2^-38 of that,
vanishes beside the 64 u S), and three times the additions.  y: half a step of its type."""

import numpy as np
import pytest

from oracle import sample_oracle as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _type(torch, name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _weight(torch, B, rng, n, k, group):
    codes = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    scales = torch.from_numpy((rng.random((n, -(-k // group))) * 0.02 + 0.001).astype(np.float32)
                              ).to(torch.bfloat16)
    w = B.W4Weight(torch.from_numpy(codes).cuda(), scales.cuda(), k, group)
    return w, S.w4_matrix(codes, scales.double().numpy(), k, group)


def _check(y, x, w, group, xt, yt):
    x = x.double().cpu().numpy()
    k = x.shape[1]
    want = x @ w.T
    s = np.abs(x) @ np.abs(w).T
    parts = 3 if xt == "f32" else 1
    tol = (2 * parts * min(group, k) + 2 * -(-k // group) + 64 + 2) * U * s + HALF[yt] * np.abs(want)
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / np.maximum(tol, 1e-30))


SIZES = [(1, 1, 1), (1, 16, 64), (1, 17, 65), (2, 1, 4096), (1, 5120, 2880), (8, 300, 129),
         (9, 33, 640), (16, 2880, 960), (17, 100, 2049), (32, 513, 96), (33, 70, 320), (70, 31, 33),
         (1, 40000, 128), (24, 2880, 7680), (3, 64, 16384)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_against_64_bits(rows, n, k, group, xt, yt):
    torch, B = _lib()
    rng = np.random.default_rng([rows, n, k, group])
    w, m = _weight(torch, B, rng, n, k, group)
    x = torch.from_numpy(rng.normal(size=(rows, k)).astype(np.float32)).to(_type(torch, xt)).cuda()
    y = B.pe_w4_linear(w, x, out_dtype=_type(torch, yt))
    assert y.dtype == _type(torch, yt) and tuple(y.shape) == (rows, n)
    _check(y, x, m, group, xt, yt)
    again = B.pe_w4_linear(w, x, out_dtype=_type(torch, yt))
    assert torch.equal(y, again)


def test_every_code_and_place_comes_back():
    """One-hot rows read the matrix out column by column, exactly."""
    torch, B = _lib()
    rng = np.random.default_rng(3)
    for n, k, group in ((19, 70, 32), (16, 200, 128)):
        w, m = _weight(torch, B, rng, n, k, group)
        y = B.pe_w4_linear(w, torch.eye(k, device="cuda"))
        assert np.array_equal(y.double().cpu().numpy().T, m)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_strides_offsets_and_untouched_columns(xt):
    torch, B = _lib()
    rng = np.random.default_rng(5)
    n, k, rows = 50, 130, 5
    w, m = _weight(torch, B, rng, n, k, 64)
    wide = torch.from_numpy(rng.normal(size=(rows, k + 9)).astype(np.float32)).to(
        _type(torch, xt)).cuda()
    out = torch.full((rows, n + 7), 7.0, device="cuda")
    for off in (0, 1, 3, 8):
        x = wide[:, off:off + k]
        y = out[:, 3:3 + n]
        B.pe_w4_linear(w, x, out=y)
        _check(y, x, m, 64, xt, "f32")
        assert (out[:, :3] == 7).all() and (out[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_rows_of_any_magnitude(xt):
    """A power of two on a row is one on its results, from the smallest normal
    numbers to the largest; and a row's small elements count beside large
    ones: right to 2^-38 of the largest (fp32: or 2^-24 of themselves)."""
    torch, B = _lib()
    rng = np.random.default_rng(12)
    n, k = 40, 300
    w, m = _weight(torch, B, rng, n, k, 32)
    base = torch.from_numpy(rng.uniform(0.5, 1.0, k).astype(np.float32)).to(_type(torch, xt)).cuda()
    p = torch.tensor([-119, -101, -60, -14, 0, 1, 15, 16, 61, 100, 118], device="cuda")
    x = (base.float()[None] * torch.exp2(p.double())[:, None].float()).to(_type(torch, xt))
    y = B.pe_w4_linear(w, x, out_dtype=torch.float32).double()
    back = y * torch.exp2(-p.double())[:, None]
    i0 = int((p == 0).nonzero())
    # odd powers meet another even one: the same sums, on another grid of fp16
    assert torch.equal(back[0::1][p % 2 == 0], back[i0].expand(int((p % 2 == 0).sum()), n))
    for r in range(len(p)):
        _check(back[r][None], base.double()[None], m, 32, xt, "f32")
    x = torch.from_numpy((rng.normal(size=(3, k)) * np.exp2(-rng.integers(0, 45, (3, k)))).astype(
        np.float32)).to(_type(torch, xt)).cuda()
    y = B.pe_w4_linear(w, x, out_dtype=torch.float32).double().cpu().numpy()
    xd = x.double().cpu().numpy()
    s = np.abs(xd) @ np.abs(m).T
    grid = 2.0 ** -38 * np.abs(xd).max(1)[:, None] * np.abs(m).sum(1)[None]
    parts = 3 if xt == "f32" else 1
    assert (np.abs(y - xd @ m.T) <= (2 * parts * 32 + 2 * 10 + 67) * U * s + grid).all()


def test_values_of_other_rows_do_not_matter():
    """A row of infinities or NaN leaves the others as they are."""
    torch, B = _lib()
    rng = np.random.default_rng(6)
    w, m = _weight(torch, B, rng, 40, 200, 32)
    x = torch.from_numpy(rng.normal(size=(11, 200)).astype(np.float32)).bfloat16().cuda()
    want = B.pe_w4_linear(w, x, out_dtype=torch.float32)
    x[3] = float("nan")
    x[10, 5] = float("inf")
    got = B.pe_w4_linear(w, x, out_dtype=torch.float32)
    rest = [i for i in range(11) if i not in (3, 10)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[3]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,group", [(5, 33, 32), (40, 200, 64), (17, 384, 128), (3, 1, 32)])
def test_quantize(dt, n, k, group):
    torch, B = _lib()
    rng = np.random.default_rng([n, k])
    wt = torch.from_numpy(rng.normal(size=(n, k + 3)).astype(np.float32)).to(_type(torch, dt)).cuda()
    wt[0, :group] = 0
    part = wt[:, 2:2 + k]
    w = B.W4Weight.quantize(part, group)
    codes, scales = S.w4_quantize(part.float().cpu().numpy(), group)
    m = (codes - 8) * np.repeat(scales.astype(np.float64), group, 1)[:, :k]
    y = B.pe_w4_linear(w, torch.eye(k, device="cuda"))
    assert np.array_equal(y.double().cpu().numpy().T, m)


def test_other_streams_and_graphs():
    torch, B = _lib()
    rng = np.random.default_rng(8)
    w, m = _weight(torch, B, rng, 300, 640, 32)
    x = torch.from_numpy(rng.normal(size=(4, 640)).astype(np.float32)).bfloat16().cuda()
    want = B.pe_w4_linear(w, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = B.pe_w4_linear(w, x, stream=side)
    with torch.cuda.stream(side):
        b = B.pe_w4_linear(w, x)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(g):
        B.pe_w4_linear(w, x, out=out)
    for _ in range(2):
        x.copy_(torch.randn(4, 640, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, B.pe_w4_linear(w, x))


def test_large_offsets():
    """Codes past 2^31 bytes: n k / 2 = 2.4 GB, read at both ends."""
    torch, B = _lib()
    n, k = 1 << 21, 2304
    codes = torch.full((n, k // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n, k // 128, dtype=torch.bfloat16, device="cuda")
    codes[0], codes[-1], codes[n // 2 + 5] = 0x99, 0xAA, 0x77
    w = B.W4Weight(codes, scales, k, 128)
    del codes, scales
    y = B.pe_w4_linear(w, torch.ones(1, k, dtype=torch.bfloat16, device="cuda"),
                       out_dtype=torch.float32)[0]
    assert y[0] == k and y[-1] == 2 * k and y[n // 2 + 5] == -k
    assert int((y != 0).sum()) == 3


def test_memory_freed_before_another_stream_has_read_it():
    torch, B = _lib()
    rng = np.random.default_rng(9)
    n, k = 512, 1024
    codes = torch.from_numpy(rng.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    scales = torch.rand(n, k // 32, device="cuda").bfloat16()
    weight = torch.randn(n, k, device="cuda")
    x = torch.randn(3, k, device="cuda")
    want = B.pe_w4_linear(B.W4Weight(codes, scales, k, 32), x)
    want_q = B.pe_w4_linear(B.W4Weight.quantize(weight), x)
    copies = [t.clone() for t in (codes, scales, weight, x, x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # 50 ms in which the copies are freed
    w = B.W4Weight(copies[0], copies[1], k, 32, stream=side)
    q = B.W4Weight.quantize(copies[2], stream=side)
    y = B.pe_w4_linear(w, copies[3], stream=side)
    yq = B.pe_w4_linear(q, copies[4], stream=side)
    del copies, w, q
    other = [torch.full_like(t, 7) for t in (codes, scales, weight, x, x) for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(yq, want_q)
    assert all(bool((t == 7).all()) for t in other)


def test_two_host_threads_with_matrices_of_different_sizes():
    torch, B = _lib()
    from concurrent.futures import ThreadPoolExecutor

    def work(seed):
        rng = np.random.default_rng(seed)
        w, _ = _weight(torch, B, rng, 256, 4096 if seed else 320, 32)
        x = torch.from_numpy(rng.normal(size=(8, w.k)).astype(np.float32)).cuda()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        first = B.pe_w4_linear(w, x, stream=stream)
        rest = [B.pe_w4_linear(w, x, stream=stream) for _ in range(300)]
        stream.synchronize()
        return all(torch.equal(first, y) for y in rest)

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, (0, 1)))


@pytest.mark.parametrize("rows", [1, 2, 7, 33])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("k,group", [(1 << 17, 32), (1 << 17, 128), ((1 << 17) - 77, 64)])
def test_longest_rows(rows, xt, k, group):
    torch, B = _lib()
    rng = np.random.default_rng([rows, k, group])
    w, m = _weight(torch, B, rng, 35, k, group)
    x = torch.from_numpy(rng.normal(size=(rows, k)).astype(np.float32)).to(_type(torch, xt)).cuda()
    _check(B.pe_w4_linear(w, x, out_dtype=torch.float32), x, m, group, xt, "f32")
