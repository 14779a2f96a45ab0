"""How exactly pe_w4_linear holds x (include/peagle_w4.h): to 2^-38 of the
largest element of its row, and exactly down to 2^-30 of that in bf16, to 2^-14 in
fp32.

Weights are 0 but for one input of each output, whose weight is 1 or another power
of two, so an output is one element of x as the product holds it; a sum of its
parts has no more bits than the element, and every step of it is exact."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _lib():
    import torch
    from speculative_drafting_expand_gb300 import binding as B
    B.lib()
    return torch, B


def _picks(torch, B, k, group, power):
    """Output i is 2^power times input i."""
    codes = np.full((k, (k + 1) // 2), 0x88, np.uint8)
    i = np.arange(k)
    codes[i, i // 2] ^= (np.where(i % 2, 0x10, 0x01)).astype(np.uint8)       # 8 -> 9
    scales = torch.full((k, -(-k // group)), 2.0 ** power, dtype=torch.bfloat16, device="cuda")
    return B.W4Weight(torch.from_numpy(codes).cuda(), scales, k, group)


def _full(rng, shape, dt):
    """[1, 1.5) with all the bits of the type, either sign."""
    bits = 7 if dt == "bf16" else 23
    m = 1 + rng.integers(0, 1 << (bits - 1), shape) / 2.0 ** bits
    return m * np.where(rng.random(shape) < 0.5, -1, 1)


def _x(torch, a, dt):
    x = torch.from_numpy(a.astype(np.float32)).cuda()
    return x if dt == "f32" else x.bfloat16()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k,group", [(40, 32), (333, 64), (1000, 128)])
@pytest.mark.parametrize("rows", [1, 8, 16, 32, 40])
def test_every_bit_of_elements_of_one_size(dt, k, group, rows):
    torch, B = _lib()
    rng = np.random.default_rng([k, rows])
    x = _x(torch, _full(rng, (rows, k), dt) * 2.0 ** rng.integers(-60, 60, (rows, 1)), dt)
    for power in (0, -3, 5):
        y = B.pe_w4_linear(_picks(torch, B, k, group, power), x, out_dtype=torch.float32)
        assert torch.equal(y, x.float() * 2.0 ** power)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k,group", [(40, 32), (333, 64), (2000, 128)])
def test_small_elements_beside_a_large_one(dt, k, group):
    """The first input has the row's largest element, the others are 2^-p of it,
    p from 1 to 46; each output is held to the bound."""
    torch, B = _lib()
    rng = np.random.default_rng(k)
    p = rng.integers(1, 47, (24, k))
    a = _full(rng, (24, k), dt) * 2.0 ** -p
    a[:, 0] = _full(rng, 24, dt)
    a *= 2.0 ** rng.integers(-30, 30, (24, 1))
    x = _x(torch, a, dt)
    y = B.pe_w4_linear(_picks(torch, B, k, group, 0), x, out_dtype=torch.float32)
    xd, yd = x.double().cpu().numpy(), y.double().cpu().numpy()
    part = np.abs(xd) / np.abs(xd).max(1, keepdims=True)
    off = np.abs(yd - xd) / np.abs(xd).max(1, keepdims=True)
    exact = part >= (2.0 ** -30 if dt == "bf16" else 2.0 ** -14)
    assert exact.any() and (~exact).any()
    assert (off[exact] == 0).all()
    assert (off <= 2.0 ** -38).all()
