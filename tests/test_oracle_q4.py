"""Pins of the oracle of 4-bit integer matrices."""

import numpy as np
import pytest

from oracle import formats, q4


@pytest.mark.parametrize("N,K,group,zero", [(1, 1, 32, True), (16, 128, 128, False),
                                            (17, 129, 64, True), (40, 300, 32, False)])
def test_layout_and_parse_invert(N, K, group, zero):
    rng = np.random.default_rng(N * K)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    G = -(-K // group)
    s = formats.bf16_round(rng.uniform(0.01, 1, (N, G)).astype(np.float32))
    z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zero else None
    block = q4.layout(q, s, z, group)
    assert block.size == q4.sections(N, K, group, zero)[3]
    q2, s2, z2 = q4.parse(block, N, K, group, zero)
    assert np.array_equal(q, q2) and np.array_equal(s, s2)
    assert (z is None and z2 is None) or np.array_equal(z, z2)


def test_every_element_has_a_place_of_its_own():
    at, high = q4._places(32, 256)
    place = (at * 2 + high).ravel()
    assert np.array_equal(np.sort(place), np.arange(32 * 256))


@pytest.mark.parametrize("zero", [False, True])
def test_encode_is_within_half_a_step(zero):
    rng = np.random.default_rng(5)
    v = (rng.standard_normal((6, 200)) * 0.02 + (0.03 if zero else 0)).astype(np.float32)
    v[2] = 0
    q, s, z = q4.encode(v, 32, zero)
    step = np.repeat(formats.bf16_decode(s), 32, axis=1)[:, :200]
    # half a step, and where the BF16 scale came out low the end of the range
    # (15 steps of a scale up to 2^-8 low); a rounded zero point moves both ends
    # of its range by up to half a step
    slack = 0.5 + 15 * 2.0 ** -8 + (0.5 if zero else 0)
    assert np.all(np.abs(q4.decode(q, s, z, 32) - v) <= slack * step + 1e-12)


def test_encode_reproduces_the_grid():
    q = np.arange(16, dtype=np.uint8)[None].repeat(2, 0)
    q = np.concatenate([q, q[:, ::-1]], 1)[:, 1:31]          # codes 1..15: -7..7
    q = np.clip(q, 1, 15)
    v = (q.astype(np.float32) - 8) * np.float32(0.25)
    got, s, _ = q4.encode(v, 32, False)
    assert np.array_equal(got, q) and np.all(formats.bf16_decode(s) == 0.25)
