"""The oracle of log probabilities against facts that do not depend on it: a direct sum on small rows, finite
differences of its forward, and the conventions for padding, ties and ruled-out tokens."""
import math

import numpy as np
import pytest

from oracle import logprob as O


def test_forward_small_row_by_hand():
    z = np.array([[0.0, math.log(2.0), math.log(5.0)]])
    r = O.forward(z, [[2, 0, -1, 3]], 2)
    assert np.isclose(r["lse"][0], math.log(8.0))
    assert np.allclose(r["logp"][0], [math.log(5 / 8), math.log(1 / 8), 0.0, 0.0])
    assert np.isclose(r["entropy"][0], -(1 / 8 * math.log(1 / 8) + 2 / 8 * math.log(2 / 8) + 5 / 8 * math.log(5 / 8)))
    assert r["top_ids"].tolist() == [[2, 1]]
    assert np.allclose(r["top_logp"], [[math.log(5 / 8), math.log(2 / 8)]])


def test_ties_and_ruled_out_tokens():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 1.0], [-np.inf] * 5, [-np.inf, 2.0, -np.inf, -np.inf, -np.inf]])
    r = O.forward(z, [[3], [0], [1]], 4)
    assert r["top_ids"].tolist() == [[1, 2, 0, 4], [-1] * 4, [1, -1, -1, -1]]
    assert r["logp"].tolist() == [[-np.inf], [-np.inf], [0.0]]
    assert r["lse"][1] == -np.inf and r["entropy"][1] == 0.0 and r["entropy"][2] == 0.0
    g, _ = O.backward(z, [[1], [0], [1]], [[1.0], [1.0], [1.0]], [0.5, 0.5, 0.5])
    assert np.all(g[1] == 0.0) and np.all(g[0][3] == 0.0) and np.allclose(g[2], 0.0)


@pytest.mark.parametrize("m", [0, 1, 4])
def test_gradient_against_differences(m):
    rng = np.random.default_rng(7 + m)
    T, V = 3, 11
    z = rng.normal(size=(T, V)) * 2
    ids = rng.integers(-1, V, size=(T, m)) if m else None
    if m == 4:
        ids[:, 1] = ids[:, 0]                             # the same id twice
    dl = rng.normal(size=(T, m)) if m else None
    de = rng.normal(size=T)

    def value(z):
        r = O.forward(z, ids)
        return (float(np.sum(r["logp"] * dl)) if m else 0.0) + float(np.sum(r["entropy"] * de))

    g, _ = O.backward(z, ids, dl, de)
    num = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        e = np.zeros_like(z)
        e[i] = 1e-5
        num[i] = (value(z + e) - value(z - e)) / 2e-5
    assert np.allclose(g, num, atol=1e-8)
    assert np.allclose(g.sum(-1), 0.0)                    # a shift of the row changes nothing
