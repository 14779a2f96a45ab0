"""The 64-bit definitions of the paged KV cache operators, against hand-worked
values and their own invariants."""

import numpy as np

from oracle import kv_cache_oracle as C


def _pool(rng, blocks, H, D):
    return rng.normal(size=(blocks, H, 16, D))


def test_rotation_is_a_group_and_keeps_relative_scores():
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=8), rng.normal(size=8)
    r = C.rotate(C.rotate(x, 7, 1e4), -3, 1e4)
    assert np.allclose(r, C.rotate(x, 4, 1e4), atol=1e-14)
    a = C.rotate(x, 100, 1e4) @ C.rotate(y, 90, 1e4)
    assert np.isclose(a, C.rotate(x, 17, 1e4) @ C.rotate(y, 7, 1e4))
    # one pair by a quarter turn: (1, 0) -> (0, 1)
    assert np.allclose(C.rotate(np.array([1.0, 0.0]), np.pi / 2, 1e4), [0.0, 1.0])


def test_keep_worked_example():
    s = [9.0, 0.0, 3.0, 3.0, -0.0, np.nan, 5.0, 0.0, 1.0, 2.0]
    # first one, last two, and three of positions 1..7: 6 (5.0), 2 and 3 (3.0)
    assert C.keep(s, 6, 1, 2).tolist() == [0, 2, 3, 6, 8, 9]
    # equal scores go to the lowest position: one of the zeros, 1 before 4
    assert C.keep(s, 7, 1, 2).tolist() == [0, 1, 2, 3, 6, 8, 9]
    # a NaN is the last to stay
    assert 5 not in C.keep(s, 9, 1, 2)
    assert C.keep(s, 10, 1, 2).tolist() == list(range(10))


def test_decode_against_a_dense_softmax_and_window():
    rng = np.random.default_rng(1)
    H, D, Hq = 2, 8, 6
    k, v = _pool(rng, 6, H, D), _pool(rng, 6, H, D)
    table = np.array([[4, 1, 3], [0, 5, 2]])
    q = rng.normal(size=(2, Hq, D))
    r = C.decode(k, v, q, table, [37, 5], window=10)
    K = np.concatenate([k[t] for t in table[0]], axis=1)[:, 27:37]
    V = np.concatenate([v[t] for t in table[0]], axis=1)[:, 27:37]
    for h in range(Hq):
        z = K[h // 3] @ q[0, h] / np.sqrt(D)
        p = np.exp(z) / np.exp(z).sum()
        assert np.allclose(r.out[0, h], p @ V[h // 3])
        assert np.isclose(r.lse[0, h], np.log(np.exp(z).sum()))
    assert np.allclose(sum(w.sum() for w in r.weights), 2 * Hq)
    empty = C.decode(k, v, q, table, [0, 0])
    assert not empty.out.any() and np.all(empty.lse == -np.inf)


def test_evicted_cache_attends_like_the_kept_positions():
    """Scores of a trimmed cache at its new last position equal those of the
    kept keys rotated there from scratch."""
    rng = np.random.default_rng(2)
    H, D, n, N = 1, 8, 40, 12
    raw = rng.normal(size=(n, D))
    k, v, s = np.zeros((4, H, 16, D)), _pool(rng, 4, H, D), rng.random((4, H, 16))
    table = np.array([[2, 0, 3]])
    for p in range(n):
        b, o = C.slot(table, 0, p)
        k[b, 0, o] = C.rotate(raw[p], p, 1e4)
    kept, new, k2, v2, s2 = C.evict(k, v, s, table, np.array([n]), N, 2, 4, 1e4)
    assert new[0] == N
    got = C.gather(k2, table, 0, 0, N)[:, 0]
    want = np.stack([C.rotate(raw[p], j, 1e4) for j, p in enumerate(kept[0, 0])])
    assert np.allclose(got, want, atol=1e-13)
    # scores past the kept ones are cleared, nothing else is touched
    assert all(s2[C.slot(table, 0, j)[0], 0, j % 16] == 0 for j in range(N, n))
    assert np.array_equal(k2[1], k[1]) and np.array_equal(v2[1], v[1])


def test_append_writes_the_slot_of_the_position():
    k, v, s = np.zeros((3, 1, 16, 4)), np.zeros((3, 1, 16, 4)), np.ones((3, 1, 16))
    table = np.array([[2, 0]])
    where = C.append(k, v, s, np.ones((2, 1, 4)), np.full((2, 1, 4), 2.0), [17, -1], [0, 0],
                     table, 0.0)
    assert where == [(0, 1), None]
    assert k[0, 0, 1].tolist() == [1, 1, 1, 1] and k.sum() == 4 and v.sum() == 8
    assert s[0, 0, 1] == 0 and s.sum() == 47
