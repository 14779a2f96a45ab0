"""The sampling and verification oracle against hand-worked cases and the
theorem that makes rejection sampling right."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import sample_oracle as S


def _row(x, t=1.0, **f):
    _, greedy = S.inverse(t)
    return S.dist(x, S.exps(x, t), greedy=greedy, **f)


def test_hand_worked_row():
    # probabilities 8, 4, 2, 2 of 16 at ids 2, 0, 1, 3
    x = np.log(np.array([4, 2, 8, 2], np.float32)).astype(np.float32)
    e = np.array([0.5, 0.25, 1.0, 0.25], np.float32)
    d = S.dist(x, e)
    assert d.kept == [2, 0, 1, 3] and d.total == 4 * 2 ** 30 and d.cut == -math.inf
    assert [S.draw(d.w, u) for u in (0.0, 0.2499, 0.25, 0.374, 0.375, 0.874, 0.875, 0.999)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    assert S.dist(x, e, top_k=3).kept == [2, 0, 1]          # the lower id of the equal ones
    assert S.dist(x, e, top_k=3).cut_token == 1
    assert S.dist(x, e, top_p=0.5).kept == [2]              # 8/16 before the second: not below 0.5
    assert S.dist(x, e, top_p=0.51).kept == [2, 0]
    assert S.dist(x, e, min_p=0.5).kept == [2, 0]
    assert S.dist(x, e, min_p=2.0).kept == [2]
    # of the three kept by top-k (14 of 16), 12/14 come before the third
    assert S.dist(x, e, top_k=3, top_p=0.85).kept == [2, 0]
    assert S.dist(x, e, top_k=3, top_p=0.86).kept == [2, 0, 1]


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), 1e-45])
def test_greedy_is_the_first_largest(t):
    d = _row([1.0, 3.0, 3.0, -2.0], t)
    assert d.kept == [1] and d.total == 2 ** 31


def test_special_logits():
    assert _row([-np.inf, np.nan]).total == 0 and S.draw({}, 0.5) == -1
    d = _row([np.nan, np.inf, 1.0])
    assert d.kept == [1]
    assert set(_row([0.0, -np.inf, 5.0], np.inf).kept) == {0, 2}      # uniform over the finite


@pytest.mark.parametrize("seed,filters", [(0, {}), (1, dict(top_k=3)), (2, dict(top_p=0.8)),
                                          (3, dict(min_p=0.2, top_k=4))])
def test_greedy_drafts_keep_the_target_distribution(seed, filters):
    """P(output = i) = P(d)[i = d] + (1 - P(d)) P(i) / (1 - P(d)): the target's,
    whatever the draft; integrated over a grid of both numbers."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=6).astype(np.float32) * 1.5
    d = _row(x, **filters)
    last = _row(rng.normal(size=6).astype(np.float32))
    draft = int(rng.integers(6))
    n = 2048
    got = np.zeros(6)
    accepted = 0
    for i in range(n):
        a, tok = S.verify([d, last], [0, draft], [i / n], 0.0)
        accepted += a
    p = {i: w / d.total for i, w in d.w.items()}
    assert abs(accepted / n - p.get(draft, 0)) <= 1 / n
    if p.get(draft, 0) < 1:
        for i in range(n):
            a, tok = S.verify([d, last], [0, draft], [0.9999999], i / n)
            got[tok] += 1 - p.get(draft, 0)
        got /= n
        if draft in p:
            got[draft] += p[draft]
        assert np.allclose(got, [p.get(i, 0) for i in range(6)], atol=2 / n)


def test_sampled_drafts_keep_the_target_distribution():
    """sum_d Q(d) [min(1, P/Q)(d) at d + (1 - min(1, P/Q)(d)) R] = P with R the
    normalised max(P - Q, 0), by the oracle's own acceptance and residual."""
    rng = np.random.default_rng(7)
    P = _row(rng.normal(size=5).astype(np.float32))
    Q = _row(rng.normal(size=5).astype(np.float32), top_k=4)
    last = _row(np.zeros(5, np.float32))
    n = 1024
    out = np.zeros(5)
    for d in Q.kept:
        q = Q.w[d] / Q.total
        acc = sum(S.verify([P, last], [0, d], [i / n], 0.0, [Q])[0] for i in range(n)) / n
        assert abs(acc - min(1.0, (P.w[d] / P.total) / q)) <= 1 / n
        out[d] += q * acc
        if acc < 1:
            for i in range(n):
                a, tok = S.verify([P, last], [0, d], [0.9999999], i / n, [Q])
                assert a == 0
                out[tok] += q * (1 - acc) / n
    assert np.allclose(out, [P.w[i] / P.total for i in range(5)], atol=8 / n)


def test_equal_distributions_accept_every_draft():
    P = _row([0.5, 1.5, -1.0])
    for d in range(3):
        assert S.verify([P, P], [0, d], [0.99999994, 0.0], 0.5, [P])[0] == 1


def test_bad_draft_is_rejected():
    P = _row([0.0, 0.0])
    assert S.verify([P, P], [0, 9], [0.0, 0.0], 0.75) == (0, 1)


def test_weights_are_whole_numbers_of_the_largest():
    e = np.array([1.0, 2.0 ** -31, 2.0 ** -32, 0.75 * 2.0 ** -31], np.float32)
    assert S.weights(e) == [2 ** 31, 1, 0, 1]
    assert Fraction(S.weights(np.float32([1 / 3]))[0], 2 ** 31) == Fraction(float(np.float32(1 / 3)))


def test_w4_matrix_and_quantizer():
    codes = np.array([[0x21, 0x0F]], np.uint8)           # 1, 2, 15, (0)
    assert np.array_equal(S.w4_matrix(codes, [[2.0]], 3, 32), [[-14.0, -12.0, 14.0]])
    rng = np.random.default_rng(0)
    w = rng.normal(size=(3, 70)).astype(np.float32)
    w[1, :32] = 0
    c, s = S.w4_quantize(w, 32)
    assert s.shape == (3, 3) and s[1, 0] == 0 and (c[1, :32] == 8).all()
    assert c.min() >= 0 and c.max() <= 15
    back = (c - 8) * np.repeat(s, 32, 1)[:, :70]
    # half a scale, and the scale's own rounding (2^-8) on at most 7 of them
    assert (np.abs(back - w) <= np.repeat(s, 32, 1)[:, :70] * (0.5 + 7 * 2.0 ** -8)).all()
