"""CPU checks of the 64-bit definitions that the GPU tests of the norm and epilogue
operators compare with: gradients against central differences, and closed forms."""
import numpy as np
import pytest

from tests import _ops64 as ops


def difference(f, x, h=1e-5):
    return (f(x + h) - f(x - h)) / (2 * h)


@pytest.mark.parametrize("name", ops.ACTS)
def test_activation_slope_is_the_difference_quotient(name):
    x = np.linspace(-9, 9, 4001) + 1e-3  # off relu's corner
    # central differences: h^2/6 of the third derivative (< 4) and rounding 1e-16 * 9 / h
    assert np.max(np.abs(difference(lambda t: ops.act(t, name), x) - ops.act_slope(x, name))) < 3e-10


def test_activation_values():
    assert ops.act(np.array([0.0]), "gelu")[0] == 0
    assert abs(ops.act(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15
    assert abs(ops.act(np.array([1.0]), "silu")[0] - 1 / (1 + np.exp(-1))) < 1e-15
    u = np.sqrt(2 / np.pi) * (1 + 0.044715)
    assert abs(ops.act(np.array([1.0]), "gelu_tanh")[0] - (1 + np.tanh(u)) / 2) < 1e-15
    assert ops.act(np.array([-2.0, 2.0]), "relu").tolist() == [0.0, 2.0]


def test_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    M, K, eps, t = 3, 40, 1e-3, 1e-6
    h, dy, w = rng.normal(size=(M, K)), rng.normal(size=(M, K)), rng.normal(size=K)
    loss = lambda a, b: float((ops.rmsnorm(a, None, b, eps)[0] * dy).sum())  # noqa: E731
    rstd = ops.rmsnorm(h, None, w, eps)[2]
    dx, dw, _, _ = ops.rmsnorm_backward(dy, h, w, rstd)
    for _ in range(20):
        d, e = rng.normal(size=(M, K)), rng.normal(size=K)
        assert abs((loss(h + t * d, w) - loss(h - t * d, w)) / (2 * t) - (dx * d).sum()) < 1e-7
        assert abs((loss(h, w + t * e) - loss(h, w - t * e)) / (2 * t) - (dw * e).sum()) < 1e-7
    # the gradient along the residual stream adds to both summands' gradient
    dh = rng.normal(size=(M, K))
    assert np.allclose(ops.rmsnorm_backward(dy, h, w, rstd, dh)[0], dx + dh, rtol=0, atol=1e-15)


def test_norm_closed_forms():
    y, s, rstd = ops.rmsnorm(np.full((1, 128), 3.0), np.full((1, 128), 1.0), np.ones(128), 0.0)
    assert np.all(s == 4) and rstd[0] == 0.25 and np.all(y == 1)
