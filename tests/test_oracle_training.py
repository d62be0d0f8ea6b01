"""Pins of the oracle of the router's training steps."""

import numpy as np
import pytest

from oracle import training


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_gate_backward_is_the_difference_quotient(renorm, masked):
    rng = np.random.default_rng(2)
    T, E, k = 5, 7, 3
    z = rng.standard_normal((T, E))
    z[1, 4] = -np.inf
    z[3, 1:] = -np.inf                       # one expert left of three
    z[4] = -np.inf                           # none
    mask = np.array([1, 1, 0, 1, 1]) if masked else None
    r = training.gate(z, k, renorm, mask)
    dw, dloss = rng.standard_normal((T, k)), 0.7
    got = training.gate_backward(z, r["ids"], renorm, dw, r["counts"], dloss)

    def value(v):
        q = training.gate(v, k, renorm, mask)
        assert np.array_equal(q["ids"], r["ids"])
        return np.sum(dw * q["w"]) + dloss * q["loss"]

    for t in range(T):
        for e in range(E):
            if not np.isfinite(z[t, e]):
                assert got[t, e] == 0
                continue
            d = np.zeros_like(z)
            d[t, e] = 1e-5
            assert abs((value(z + d) - value(z - d)) / 2e-5 - got[t, e]) < 1e-9


def test_balance_loss_of_known_routers():
    T, E, k = 12, 6, 2
    # every expert equally often, uniform probabilities: 1
    z = np.zeros((T, E))
    for t in range(T):
        z[t, [(2 * t) % E, (2 * t + 1) % E]] = 1e-12
    assert abs(training.gate(z, k)["loss"] - 1) < 1e-9
    # always the same two with all the probability: E / k
    z = np.full((T, E), -60.0)
    z[:, :2] = 0
    r = training.gate(z, k)
    assert abs(r["loss"] - E / k) < 1e-9
    assert list(r["counts"]) == [T, T, 0, 0, 0, 0, T]
    assert training.gate(z, k, mask=np.zeros(T))["loss"] == 0
