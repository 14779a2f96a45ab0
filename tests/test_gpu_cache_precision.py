"""Where pe_attn_decode could lose what its types hold: weights far below the
largest, and queries near the ends of bf16's range, beside e4m3 pools."""

import numpy as np
import pytest

from oracle import kv_cache_oracle as C
from oracle.fp8_kv import e4m3_encode

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _pools(k, v, k_scale=1.0):
    """One request's rows k, v [n, D] (values that e4m3 holds) in pages."""
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    n, D = k.shape
    pages = -(-n // 16)
    pools = []
    for x in (k, v):
        codes = np.zeros((pages * 16, D), np.uint8)
        codes[:n] = e4m3_encode(x)
        pools.append(torch.from_numpy(codes.reshape(pages, 1, 16, D)).cuda())
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    return B, B.KvPool(*pools, None, k_scale, 1.0), table


@pytest.mark.parametrize("heads", [1, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below", [10, 14, 16, 18, 20, 24])
def test_e4m3_weights_far_below_the_largest(D, heads, below):
    """One position holds (almost) all the weight and a value of 0, 31 others
    e^-below of it each and a value of 1: the output is their weights' sum.

    Tolerance: a weight is a pair of fp16 numbers whose step is at most 2^-24
    of 2^12 times the largest weight's 1, so off by at most 2^-37 each, or
    2^-17 of itself for larger ones; the logits are exact here (products of
    small whole numbers), their scaling to units of ln 2 is off by 3 u of it,
    twice, and the exponential by 2^-21; then half a step of bf16."""
    import torch
    n = 32
    k, v = np.zeros((n, D)), np.ones((n, D))
    k[5, 3], v[5] = below, 0.0
    B, pool, table = _pools(k, v)
    q = torch.zeros(1, heads, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 3] = 1.0
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = B.pe_attn_decode(pool, q, table, lens, scale=1.0)
    small = (n - 1) * np.exp(-float(below))
    want = small / (1 + small)
    got = out.double().cpu().numpy()
    exact = (n - 1) * 2.0 ** -37 + want * (2.0 ** -17 + 6 * U * below * np.log2(np.e) + 2.0 ** -20)
    assert np.all(np.abs(got - want) <= exact + 2.0 ** -8 * (want + exact))
    ref = below + np.log1p(small)
    assert np.all(np.abs(lse.double().cpu().numpy() - ref) <= 2.0 ** -20 + 8 * U * ref)


@pytest.mark.parametrize("heads", [1, 9])
@pytest.mark.parametrize("q_size,scale", [
    (2.0 ** -120, 2.0 ** -32), (2.0 ** -126, 2.0 ** -100), (2.0 ** -126, 2.0 ** 120),
    (2.0 ** -130, 2.0 ** 126), (2.0 ** 126, 2.0 ** -126), (2.0 ** 127, 2.0 ** -127),
    (2.0 ** 120, 2.0 ** -120), (1.0, 1.0)])
def test_e4m3_queries_near_the_ends_of_the_range(heads, q_size, scale):
    """q and the scale at opposite (or the same) ends of fp32's range, over a
    page that the request does not fill: logits are their product's.

    Tolerance: q is a power of two and k whole numbers below 16, so sums are
    exact; scale and factor are rounded a few times (8 u of the logit), the
    exponentials and pairs of weights as above."""
    import torch
    n, D = 21, 64
    rng = np.random.default_rng(60)
    k = rng.integers(-3, 4, size=(n, D)).astype(np.float64)
    v = rng.integers(-8, 9, size=(n, D)).astype(np.float64)
    B, pool, table = _pools(k, v)
    signs = rng.choice((-1.0, 1.0), size=(1, heads, D)) * (np.arange(D) < 5)
    q = torch.from_numpy((signs * q_size).astype(np.float32)).to(torch.bfloat16).cuda()
    assert np.array_equal(q.double().cpu().numpy(), signs * q_size)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = B.pe_attn_decode(pool, q, table, lens, scale=scale)
    z = np.einsum("hd,nd->hn", signs[0] * q_size, k) * scale
    p = np.exp(z - z.max(1, keepdims=True))
    lse_want = z.max(1) + np.log(p.sum(1))
    p /= p.sum(1, keepdims=True)
    want, spread = p @ v, p @ np.abs(v)
    ez = 8 * U * np.abs(z).max(1)
    tol = (2 * ez + 2.0 ** -16)[:, None] * spread + 2.0 ** -8 * np.abs(want) + n * 2.0 ** -37 * 8
    assert np.all(np.abs(out.double().cpu().numpy()[0] - want) <= tol)
    tol = ez + 2.0 ** -19 + 8 * U * np.abs(lse_want)
    assert np.all(np.abs(lse.double().cpu().numpy()[0] - lse_want) <= tol)


@pytest.mark.parametrize("dt", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [1, 12])
@pytest.mark.parametrize("logit", [2.0 ** -30, 2.0 ** -12, 2.0 ** -3, 37.0])
def test_lse_of_one_position_is_its_logit(dt, heads, logit):
    """The sum is one exponential of 0, whose logarithm is 0: what is left is
    the logit, times log2 e and ln 2 in fp32 (6 half steps)."""
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    D = 64
    act = torch.float32 if dt == "f32" else torch.bfloat16
    k = torch.zeros(1, 1, 16, D, dtype=act, device="cuda")
    k[0, 0, 0, 7] = 1.0
    if dt == "e4m3":
        k = k.float().to(torch.float8_e4m3fn)
    q = torch.zeros(1, heads, D, dtype=act, device="cuda")
    q[:, :, 7] = logit
    table, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [1]))
    out, lse = B.pe_attn_decode(B.KvPool(k, k.clone()), q, table, lens, scale=1.0)
    assert np.all(np.abs(lse.double().cpu().numpy() - logit) <= 6 * U * logit)
    want = torch.zeros_like(q)
    want[:, :, 7] = 1.0
    assert torch.equal(out, want)
