"""Pins of the layers' binary64 oracle (CPU): the generator's published test
vectors, the mask's rate and independence, and the norm's gradient against
differences of the norm."""
import numpy as np
import pytest

from oracle import layers as L


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_gives_the_published_vectors(counter, key, words):
    got = L.philox_words([np.array([c]) for c in counter], key)
    assert [int(w[0]) for w in got] == words


def test_mask_rate_and_independence():
    """Kept shares within five standard deviations of 1 - t / 65536, between
    neighbours in every argument as between independent draws."""
    p, rows, size = 0.3, 512, 1000
    q = 1.0 - L.dropout_threshold(p) / 65536.0
    a = L.kept(rows, size, p, 1)
    n = rows * size
    assert abs(a.mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
    both = q * q
    for other in (L.kept(rows, size, p, 2), L.kept(rows, size, p, 1 + (1 << 32)), L.kept(rows, size, p, 1, step=1),
                  L.kept(rows, size, p, 1, site=1), np.roll(a, 1, 0), np.roll(a, 1, 1)):
        assert abs((a & other).mean() - both) < 5 * np.sqrt(both * (1 - both) / n)


def test_mask_of_a_slice_and_of_the_ends():
    a = L.kept(9, 40, 0.5, 77, 3, 4)
    assert np.array_equal(a[:5, :13], L.kept(5, 13, 0.5, 77, 3, 4))
    assert L.kept(3, 17, 0.0, 5).all() and not L.kept(3, 17, 1.0, 5).any()
    assert L.dropout_scale(0.0) == 1.0 and L.dropout_scale(1.0) == 0.0 and L.dropout_scale(0.5) == 2.0


@pytest.mark.parametrize("rows,size", [(1, 2), (3, 5), (4, 16)])
def test_norm_gradient_against_differences(rows, size):
    """Central differences of sum(dy * y): their error is O(step^2) times the
    third derivative, and rounding 2^-52 / step: 1e-7 relative bounds both at
    a step of 1e-5 and values around 1."""
    rng = np.random.default_rng(rows * 100 + size)
    x, dy = rng.standard_normal((rows, size)), rng.standard_normal((rows, size))
    w, b = 1 + 0.3 * rng.standard_normal(size), rng.standard_normal(size)
    eps, step = 1e-2, 1e-5
    f = lambda x, w, b: float((dy * L.norm(x, w, b, eps)[0]).sum())  # noqa: E731
    _, mean, rstd = L.norm(x, w, b, eps)
    dx, dw, db = L.norm_gradient(dy, x, mean, rstd, w)
    for grad, args, at in ((dx, (x, w, b), 0), (dw, (x, w, b), 1), (db, (x, w, b), 2)):
        for i in np.ndindex(grad.shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[at][i] += step
            lo[at][i] -= step
            assert abs((f(*hi) - f(*lo)) / (2 * step) - grad[i]) < 1e-7 * max(1.0, np.abs(grad).max())
