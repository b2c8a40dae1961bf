"""CPU pins of the sampling oracle: closed forms, the filters' order and ties,
and that sampled verification keeps the sampled distribution (by integrating
over its uniform numbers, without sampling)."""
import itertools

import numpy as np
import pytest

from oracle import sampling as sp


def test_distribution_closed_forms():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    assert np.allclose(sp.distribution(l), [0.25, 1.0, 0.5, 0.25])
    assert np.allclose(sp.distribution(l, temperature=0.5), [1 / 16, 1.0, 0.25, 1 / 16])
    assert np.flatnonzero(sp.distribution(l, top_k=3)).tolist() == [0, 1, 2]       # tie to the lower index
    assert np.flatnonzero(sp.distribution(l, top_p=0.5)).tolist() == [1]           # 4 of 8 reaches a half
    assert np.flatnonzero(sp.distribution(l, top_p=0.51)).tolist() == [1, 2]
    assert np.flatnonzero(sp.distribution(l, top_k=2, top_p=0.7)).tolist() == [1, 2]   # of the two left, 4 / 6 < 0.7
    assert np.flatnonzero(sp.distribution(l, top_p=0.0)).tolist() == [1]
    assert np.flatnonzero(sp.distribution(np.array([0.0, 2.0, 2.0]), min_p=1.0)).tolist() == [1, 2]
    assert np.flatnonzero(sp.distribution(l, temperature=0.0)).tolist() == [1]
    assert sp.distribution(np.full(3, -np.inf)).sum() == 0


def test_pick_is_the_inverse_of_the_cumulative_sum():
    w = np.array([0.0, 1.0, 0.0, 2.0, 1.0])
    assert [sp.pick(w, u) for u in (0.0, 0.24, 0.25, 0.74, 0.75, 0.99)] == [1, 1, 3, 3, 4, 4]
    assert sp.pick(np.zeros(3), 0.5) == -1


@pytest.mark.parametrize("certain", [True, False])
def test_verification_keeps_the_distribution(certain):
    """Over a grid of uniform numbers, and over the draft's own distribution, the first committed token
    appears with probability p_0: each grid cell's error is at most its width."""
    g = np.random.default_rng(3)
    V, K, N = 4, 1, 256
    l = g.standard_normal((1, K + 1, V))
    p = sp.distribution(l[0, 0])
    p /= p.sum()
    q = np.zeros(V)
    q[1] = 1.0
    if not certain:
        q = g.random(V)
        q /= q.sum()
    got = np.zeros(V)
    grid = (np.arange(N) + 0.5) / N
    for x in np.flatnonzero(q):
        for ua, us in itertools.product(grid, grid[::16] - 7.5 / N):
            cm, _ = sp.verify(l, np.array([[x]]), np.array([[ua, us]]),
                              None if certain else np.broadcast_to(q, (1, 1, V)))
            got[cm[0, 0]] += q[x] / (N * (N // 16))
    assert np.abs(got - p).max() <= V * (1.0 / N + 16.0 / N), (got, p)


def test_route_matches_the_plain_router():
    g = np.random.default_rng(5)
    z = g.standard_normal((20, 16))
    idx, w = sp.route(z, 4)
    assert np.array_equal(idx, np.argsort(-z, axis=1, kind="stable")[:, :4])
    e = np.exp(z)
    assert np.allclose(w, np.take_along_axis(e / e.sum(1, keepdims=True), idx, 1))
    # one group left: its experts only
    idx, _ = sp.route(z, 4, n_groups=4, topk_groups=1)
    assert np.array_equal(np.sort(idx, axis=1) // 4, np.repeat(z.reshape(20, 4, 4).max(2).argmax(1)[:, None], 4, axis=1))
