"""The float64 reference of the experts' operators against published vectors, differences and the identity (CPU)."""

import numpy as np
import pytest

from oracle import experts as ox


def test_philox_published_vectors():
    """The known-answer vectors that were published with the generator (10 rounds)."""
    f = 0xFFFFFFFF
    assert ox.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ox.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ox.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_rate():
    """Within five deviations of a binomial count."""
    n, p = 40000, 0.3
    m, q = ox.keep(n, p, 5, 9)
    assert abs(m.sum() - n * q) < 5 * (n * q * (1 - q)) ** 0.5
    assert ox.keep(64, 0.0, 1, 2)[0].all() and not ox.keep(64, 1.0, 1, 2)[0].any()
    assert np.array_equal(ox.keep(100, p, 5, 9, first=37)[0], m[37:100])


def test_sort_round_trip():
    rng = np.random.default_rng(0)
    idx = rng.integers(-2, 9, (50, 3))
    offsets, pos, slot = ox.sort(idx, 7)
    live = (idx >= 0) & (idx < 7)
    assert offsets[-1] == live.sum() and (pos[~live] == -1).all() and (slot[offsets[-1]:] == -1).all()
    assert np.array_equal(pos.reshape(-1)[slot[:offsets[-1]]], np.arange(offsets[-1]))
    assert (np.diff(idx.reshape(-1)[slot[:offsets[-1]]]) >= 0).all()


@pytest.mark.parametrize("name", ["none", "silu", "gelu", "swiglu"])
def test_slopes_are_differences(name):
    z = np.random.default_rng(1).standard_normal((5, 8))
    z += np.sign(z) * 0.1
    _, slopes = ox.act(z, name)
    h = 1e-6
    for part, s in enumerate(slopes):
        e = np.zeros_like(z)
        sl = slice(None) if len(slopes) == 1 else slice(part * 4, part * 4 + 4)
        e[:, sl] = h
        diff = (ox.act(z + e, name)[0] - ox.act(z - e, name)[0]) / (2 * h)
        assert np.abs(diff - s).max() < 1e-8    # h^2 of third derivatives, and 2^-52 / h
