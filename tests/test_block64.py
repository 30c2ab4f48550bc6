"""CPU: the 64-bit definitions of the layer norm, the gated product and dropout against
published outputs of the generator, difference quotients and each other."""
import numpy as np
import pytest

from tests import _block64 as blk
from tests import _ops64 as ops


def test_philox_published_outputs():
    # Random123's known answers for the zero counter and key, the all-ones ones and digits of pi
    ones, pi = [0xFFFFFFFF] * 4, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]
    for counter, key, rounds, want in (
            ([0] * 4, [0] * 2, 7, "5f6fb709 0d893f64 4f121f81 4f730a48"),
            ([0] * 4, [0] * 2, 10, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            (ones, ones[:2], 10, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            (pi, [0xA4093822, 0x299F31D0], 10, "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join(f"{int(v[0]):08x}" for v in blk.philox(counter, key, rounds)) == want


@pytest.mark.parametrize("p", [2.0 ** -16, 0.1, 0.5, 0.9, 1 - 2.0 ** -16])
def test_share_of_kept_elements(p):
    n = 1 << 18
    k = blk.kept(0, n, p, 1234567890123, 42)
    q = 1 - blk.threshold(p) / 65536
    assert abs(k.mean() - q) <= 5 * np.sqrt(q * (1 - q) / n)
    assert np.array_equal(k[800:], blk.kept(800, n - 800, p, 1234567890123, 42))
    assert not np.array_equal(k, blk.kept(0, n, p, 1234567890123, 43)) or p < 1e-4 or p > 0.9999
    assert np.array_equal(blk.kept(0, n, p, 7, 40, 3), blk.kept(0, n, p, 7, 43))


def test_layernorm_backward_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    M, K = 5, 256
    s, w, b, dy = (rng.normal(size=t) for t in ((M, K), K, K, (M, K)))
    _, mean, rstd, *_ = blk.layernorm(s, 0 * s, w, b, 1e-5)
    dx, dw, db, *_ = blk.layernorm_backward(dy, s, w, mean, rstd)
    for _ in range(4):
        d, e, f, t = rng.normal(size=(M, K)), rng.normal(size=K), rng.normal(size=K), 1e-5
        loss = lambda a: float((blk.layernorm(s + a * d, 0 * s, w + a * e, b + a * f, 1e-5)[0] * dy).sum())  # noqa: E731
        slope = (loss(t) - loss(-t)) / (2 * t)
        want = (dx * d).sum() + (dw * e).sum() + (db * f).sum()
        assert abs(slope - want) <= 1e-7 * (np.abs(dx * d).sum() + np.abs(dw * e).sum())


@pytest.mark.parametrize("act", ops.ACTS)
def test_gated_backward_is_the_difference_quotient(act):
    rng = np.random.default_rng(2)
    z, dh = rng.normal(size=(4, 64)) + 0.01, rng.normal(size=(4, 32))
    z[np.abs(z) < 1e-3] = 0.5  # away from relu's corner
    p, _ = blk.gated_backward(dh, z, act)
    d, t = rng.normal(size=z.shape), 1e-6
    loss = lambda a: float((blk.gated(z + a * d, 0.0, act)[0] * dh).sum())  # noqa: E731
    assert abs((loss(t) - loss(-t)) / (2 * t) - (p * d).sum()) <= 1e-7 * np.abs(p * d).sum()
