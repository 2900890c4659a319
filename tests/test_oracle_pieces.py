"""The oracles take a matrix in pieces of its rows: the same bits as whole, the
columns' sums but for their order."""
import numpy as np
import pytest

from oracle import block as B
from oracle import layers as L
from oracle import pieces


def special(rng, rows, size):
    x = 3 * rng.standard_normal((rows, size))
    x[rng.random((rows, size)) < 0.05] = -np.inf
    x[rows // 3, : size // 2] = x[rows // 3, 0]
    x[rows // 2, 0] = np.nan
    x[rows // 2 + 1] = -np.inf
    return x


def everything(x, rng):
    rows, size = x.shape
    dy, w, r = rng.standard_normal((rows, size)), rng.standard_normal(size), np.abs(rng.standard_normal(rows))
    plain = np.where(np.isfinite(x), x, 1.0)
    target = rng.integers(0, size, rows)
    target[::5] = -100
    m, s, z, p, h = B.log_probs(x)
    with np.errstate(invalid="ignore", over="ignore"):
        yield from (m, s, z, p, h, B.top(x, min(size, 7)), B.log_probs_gradient(x, target, r, dy[:, 0], m, s, h))
        yield from (B.e4m3_half_step(x), B.scales(x, "row"), B.scales(x, "block"), B.rms(plain, 1e-5))
    for kind in ("silu", "gelu", "gelu_tanh", "relu"):
        yield from B.act(kind, plain)
    yield from L.statistics(plain, 1e-5)
    yield L.kept(rows, size, 0.3, 12345678901, step=3, site=4)
    yield B.rms_gradient(dy, plain, r, w)[0]
    yield L.norm_gradient(dy, plain, r, r, w)[0]
    for sums in (B.rms_gradient(dy, plain, r, w)[1:], L.norm_gradient(dy, plain, r, r, w)[1:]):
        yield from ((v, rows * 2.0 ** -52 * np.abs(dy).max() * 30 * size) for v in sums)


@pytest.mark.parametrize("rows,size", [(40, 130), (9, 8), (33, 1)])
def test_pieces_have_the_bits_of_the_whole(rows, size, monkeypatch):
    x = special(np.random.default_rng([rows, size]), rows, size)
    got = []
    for elements in (1 << 30, 4 * size, 1):
        monkeypatch.setattr(pieces, "ELEMENTS", elements)
        got.append(list(everything(x, np.random.default_rng(7))))
    for other in got[1:]:
        for a, b in zip(got[0], other, strict=True):
            if isinstance(a, tuple):
                assert np.abs(a[0] - b[0]).max() <= a[1]
            else:
                assert a.dtype == b.dtype and np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def test_the_callers_error_state_holds_in_the_pieces(monkeypatch):
    monkeypatch.setattr(pieces, "ELEMENTS", 1)
    with np.errstate(divide="raise"), pytest.raises(FloatingPointError):
        pieces.by_rows(0)(lambda x: 1.0 / x)(np.zeros((3, 2)))


def test_the_half_step_is_that_of_the_table():
    """Half of the distance of a value to the next one away from zero."""
    v = B.E4M3[:127]
    assert np.array_equal(B.e4m3_half_step(v[:-1]), np.diff(v) / 2)
    assert np.array_equal(B.e4m3_half_step(np.array([np.inf, np.nan, -448.0, 0.0])), [0.0, 0.0, 16.0, 2.0 ** -10])


@pytest.mark.parametrize("seed", range(6))
def test_the_likeliest_by_a_sort_of_everything(seed):
    rng = np.random.default_rng(seed)
    x = rng.integers(-3, 4, (50, 40)).astype(float)
    x[rng.random(x.shape) < 0.1] = np.nan
    x[rng.random(x.shape) < 0.1] = np.inf
    x[rng.random(x.shape) < 0.2] = -np.inf
    x[rng.random(x.shape) < 0.1] = -0.0
    x[0], x[1], x[2] = np.nan, -np.inf, np.inf
    for k in (1, 3, 20, 40):
        want = [sorted(range(40), key=lambda c: (not np.isnan(r[c]), 0.0 if np.isnan(r[c]) else -r[c], c))[:k] for r in x]
        assert B.top(x, k).tolist() == want


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_long_lists_in_threads_have_the_bits_of_one(dtype, monkeypatch):
    """scale_ and accumulate_ element by element, over the tensors' ends."""
    import oracle
    from oracle import oracle as O
    from synth import gradsets as gs
    rng = np.random.default_rng(3)
    new = lambda: [gs.to_storage(rng.standard_normal(n), dtype) for n in (1000, 1, 0, 77, 5)]  # noqa: E731
    a, b = new(), new()
    got = []
    for apart in (1 << 30, 1):
        monkeypatch.setattr(O, "APART", apart)
        x = [t.copy() for t in a]
        oracle.scale_(x, dtype, 0.37)
        oracle.accumulate_(x, b, dtype)
        got.append(x)
        with pytest.raises(ValueError):
            oracle.accumulate_(x, b[:3], dtype)
        with pytest.raises(TypeError):
            oracle.scale_([t.astype(np.float64) for t in x], dtype, 0.5)
        with pytest.raises(TypeError):
            oracle.scale_([x[0][::2]], dtype, 0.5)
    for x, y, z in zip(*got, a, strict=True):
        assert np.array_equal(x, y) and (z.size < 5 or not np.array_equal(x, z))
