"""Products with 4-bit weights over the whole range of their scales: every bf16
scale is accepted, so every result that fp32 has room for has to come out.

Tolerance as in tests/test_gpu_w4.py (u = 2^-24, S = sum_j |x_j w_j|): 2 group u S
for a group's additions (three times that for the parts of fp32 x), (2 groups +
64) u S for scales and partial results, half a step of y's type.  Results whose S
is below 2^-100 are not looked at: past that fp32 itself runs out."""

import numpy as np
import pytest

from oracle import sample_oracle as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _type(torch, name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _weight(torch, B, rng, n, k, group, power, codes=None):
    """Scales of [1, 2) 2^power (a number, or one for each of [n, groups])."""
    if codes is None:
        codes = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    scales = np.ldexp(1 + rng.integers(0, 128, (n, -(-k // group))) / 128, power)
    scales = torch.from_numpy(scales).to(torch.bfloat16)
    w = B.W4Weight(torch.from_numpy(codes).cuda(), scales.cuda(), k, group)
    return w, S.w4_matrix(codes, scales.double().numpy(), k, group)


def _check(got, x, m, group, xt, yt, least=0):
    got, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    want, s = x @ m.T, np.abs(x) @ np.abs(m).T
    k, parts = x.shape[1], 3 if xt == "f32" else 1
    tol = (2 * parts * min(group, k) + 2 * -(-k // group) + 66) * U * s + HALF[yt] * np.abs(want)
    look = (s < 2.0 ** 126) & (s > 2.0 ** -100)
    assert look.sum() >= least
    assert np.isfinite(got[look]).all()
    assert (np.abs(got - want)[look] <= tol[look]).all()


@pytest.mark.parametrize("n,k", [(40, 300), (1000, 2049), (17, 128), (3000, 64)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt,yt", TYPES)
def test_scales_of_any_magnitude(n, k, group, xt, yt):
    torch, B = _lib()
    rng = np.random.default_rng([n, k, group])
    powers = np.array([-119, -100, -60, -20, -1, 0, 15, 40, 61, 100, 115])
    base = rng.uniform(0.5, 1.0, (len(powers), k))
    x = torch.from_numpy(np.ldexp(base, powers[:, None]).astype(np.float32))
    x = x.to(_type(torch, xt)).cuda()
    for power in (-133, -126, -70, 70, 100, 106, 110, 120, 127):
        w, m = _weight(torch, B, rng, n, k, group, power)
        for r in range(1 if n > 100 else 3):       # up to 33 rows: one to four column tiles
            rows = x.repeat(3, 1)[:(11, 1, 33)[r]]
            y = B.pe_w4_linear(w, rows, out_dtype=_type(torch, yt))
            _check(y, rows, m, group, xt, yt)
            again = B.pe_w4_linear(w, rows, out_dtype=_type(torch, yt))
            assert torch.equal(y.nan_to_num(nan=3e38), again.nan_to_num(nan=3e38))


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("px,ps", [(-100, 110), (0, 108), (0, 110), (-20, 127), (10, 104)])
def test_one_group_of_one_row(xt, yt, px, ps):
    """The result is finite, and every element is looked at."""
    torch, B = _lib()
    x = torch.full((1, 32), 2.0 ** px, dtype=_type(torch, xt), device="cuda")
    w, m = _weight(torch, B, np.random.default_rng(ps), 16, 32, 32, ps,
                   np.full((16, 16), 0xFF, np.uint8))
    y = B.pe_w4_linear(w, x, out_dtype=_type(torch, yt))
    _check(y, x, m, 32, xt, yt, least=16)


@pytest.mark.parametrize("xt,yt", TYPES)
def test_a_few_large_scales_among_usual_ones(xt, yt):
    """Rows of weights without one are bit for bit what they are alone; rows of x
    with infinities or NaN stay such."""
    torch, B = _lib()
    rng = np.random.default_rng(1)
    n, k, group = 200, 1500, 64
    power = np.full((n, -(-k // group)), -6)
    power[rng.integers(0, n, 30), rng.integers(0, power.shape[1], 30)] = 112
    codes = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    w, m = _weight(torch, B, np.random.default_rng(2), n, k, group, power, codes)
    usual, _ = _weight(torch, B, np.random.default_rng(2), n, k, group, -6, codes)
    x = torch.from_numpy(rng.normal(size=(6, k)).astype(np.float32)).to(_type(torch, xt)).cuda()
    x[4, 7], x[5, 900] = float("inf"), float("nan")
    y = B.pe_w4_linear(w, x, out_dtype=_type(torch, yt))
    _check(y[:4], x[:4], m, group, xt, yt, least=4 * n)
    assert not torch.isfinite(y[4:]).any()
    rest = torch.from_numpy((power < 0).all(1)).cuda()
    want = B.pe_w4_linear(usual, x, out_dtype=_type(torch, yt))
    assert torch.equal(y[:4, rest], want[:4, rest])


@pytest.mark.parametrize("xt,yt", TYPES)
def test_results_past_the_range_are_infinite(xt, yt):
    torch, B = _lib()
    w, m = _weight(torch, B, np.random.default_rng(0), 20, 96, 32, 127,
                   np.full((20, 48), 0x1F, np.uint8))
    x = torch.ones(2, 96, dtype=_type(torch, xt), device="cuda")
    x[:, 1::2] = 0
    x[1] *= -1
    y = B.pe_w4_linear(w, x, out_dtype=_type(torch, yt))
    assert (y[0] == float("inf")).all() and (y[1] == -float("inf")).all()
