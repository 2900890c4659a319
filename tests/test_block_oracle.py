"""Pins of oracle/block.py: the 8-bit format against torch's, the gradients
against differences, the sums against library routines."""
import numpy as np
import pytest

from oracle import block as B


def test_e4m3_against_torch():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, B.E4M3, equal_nan=True)
    v = np.concatenate([B.E4M3[:127], (B.E4M3[:126] + B.E4M3[1:127]) / 2,
                        np.nextafter((B.E4M3[:126] + B.E4M3[1:127]) / 2, np.inf),
                        np.nextafter((B.E4M3[:126] + B.E4M3[1:127]) / 2, -np.inf)])
    v = np.concatenate([v, -v]).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.round_e4m3(v), want)


def test_scales_by_hand():
    v = np.zeros((1, 130))
    v[0, 3], v[0, 129] = -896.0, np.inf
    assert np.array_equal(B.scales(v, "block"), [[2.0, 2.0 ** -112]])
    assert np.array_equal(B.scales(v, "row"), [[2.0]])


def differences(f, x, h=1e-6):
    out = np.empty_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_rms_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, dy, w = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    loss = lambda x, w: (dy * (x * B.rms(x, 1e-3)[:, None] * w)).sum()  # noqa: E731
    dx, dw = B.rms_gradient(dy, x, B.rms(x, 1e-3), w)
    np.testing.assert_allclose(dx, differences(lambda v: loss(v, w), x), rtol=1e-7, atol=1e-8)
    np.testing.assert_allclose(dw, differences(lambda v: loss(x, v), w), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_activations_against_torch_and_differences(kind):
    import torch
    x = np.linspace(-9, 9, 57)
    y, slope = B.act(kind, x)
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[kind]
    np.testing.assert_allclose(y, f(torch.from_numpy(x)).numpy(), rtol=1e-12, atol=1e-14)
    off = x + 1e-3 * (x == 0)
    np.testing.assert_allclose(B.act(kind, off)[1], (B.act(kind, off + 1e-6)[0] - B.act(kind, off - 1e-6)[0]) / 2e-6,
                               rtol=1e-7, atol=1e-9)
    assert np.all(np.isfinite(slope))


def test_log_probs_against_torch_and_differences():
    import torch
    rng = np.random.default_rng(2)
    x = 3 * rng.normal(size=(5, 11))
    x[1, 4] = x[1, 6] = -np.inf
    m, s, z, p, h = B.log_probs(x)
    t = torch.from_numpy(x)
    np.testing.assert_allclose(z, torch.log_softmax(t, 1).numpy(), rtol=1e-13)
    np.testing.assert_allclose(h, torch.distributions.Categorical(probs=torch.softmax(t, 1)).entropy().numpy(), rtol=1e-6)
    target = np.array([0, 3, 10, 5, -100])
    dlogp, dh = rng.normal(size=5), rng.normal(size=5)

    def loss(x):
        _, _, z, _, h = B.log_probs(x)
        return sum(dlogp[r] * z[r, target[r]] + dh[r] * h[r] for r in range(4))
    got = B.log_probs_gradient(x, target, dlogp, dh, m, s, h)
    finite = np.isfinite(x)
    x0 = np.where(finite, x, -40.0)  # as good as -infinity
    np.testing.assert_allclose(got[finite], differences(loss, x0)[finite], rtol=1e-6, atol=1e-8)
    assert not got[~finite].any() and not got[4].any()


def test_log_probs_of_empty_rows_and_nans():
    x = np.array([[-np.inf] * 3, [0.0, np.nan, 1.0], [-3.4e38] * 3])
    m, s, z, p, h = B.log_probs(x)
    assert np.isneginf(m[0]) and np.isneginf(s[0]) and np.isneginf(z[0]).all() and h[0] == 0
    assert m[1] == 1.0 and np.isnan(s[1]) and np.isnan(z[1]).all() and np.isnan(h[1])
    np.testing.assert_allclose([h[2], s[2], *-z[2]], np.log(3))
    assert B.top(np.array([[2.0, np.nan, 5.0, 2.0, -0.0, 0.0, 5.0]]), 7).tolist() == [[1, 2, 6, 0, 3, 4, 5]]
