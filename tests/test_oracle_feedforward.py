"""The feed-forward references against differences of their own forward formulas."""
import numpy as np
import pytest

from oracle import feedforward as FF


@pytest.mark.parametrize("name", FF.ACTIVATIONS)
def test_slopes(name):
    z = np.concatenate((np.linspace(-30, 30, 4001) + 0.0037, [1e-3, -1e-3, 200.0, -200.0]))
    h = 1e-5 * np.maximum(1.0, np.abs(z))
    f, df = FF.activation64(name, z)
    num = (FF.activation64(name, z + h)[0] - FF.activation64(name, z - h)[0]) / (2 * h)
    # central differences: h^2 f''' / 6 with f''' below 3, and the rounding 2^-52 |f| / h
    assert np.all(np.abs(num - df) <= 3 * h ** 2 + 2.0 ** -50 * np.abs(f) / h)
    assert np.all(np.isfinite(FF.activation64(name, np.array([3e38, -3e38, 1e20, -1e20]))[1]))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", FF.ACTIVATIONS)
def test_epilogue_gradient(name, gated):
    g = np.random.RandomState(1)
    z, dy, d = g.randn(5, 12), g.randn(5, 6 if gated else 12), g.randn(5, 12)
    loss = lambda e: (dy * FF.epilogue64(z + e * d, name, gated)).sum()
    want = (FF.epilogue_bwd64(dy, z, name, gated) * d).sum()
    assert abs((loss(1e-6) - loss(-1e-6)) / 2e-6 - want) < 1e-6


@pytest.mark.parametrize("direct", [False, True])
def test_norm_gradient(direct):
    g = np.random.RandomState(2)
    h, w, dy, d, dw = g.randn(4, 33), g.randn(33), g.randn(4, 33), g.randn(4, 33), g.randn(33)
    dh = g.randn(4, 33) if direct else None
    eps = 1e-3
    loss = lambda e: ((dy * FF.rmsnorm64(h + e * d, w + e * dw, eps)[0]).sum()
                      + (0 if dh is None else (dh * (h + e * d)).sum()))
    dx, got_dw, _, _ = FF.rmsnorm_bwd64(dy, h, w, FF.rmsnorm64(h, w, eps)[1], dh)
    assert abs((loss(1e-6) - loss(-1e-6)) / 2e-6 - (dx * d).sum() - (got_dw * dw).sum()) < 1e-6
