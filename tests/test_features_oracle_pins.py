"""The fp64 oracle of linear, gated and rms_norm (oracle/features.py) against
closed forms and central differences (CPU only)."""
import numpy as np
import pytest

from oracle import features as O

KINDS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _differences(f, v, g, h=1e-6):
    """d/dv of sum(f(v) * g) by central differences."""
    out = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        e = np.zeros_like(v)
        e[i] = h
        out[i] = ((f(v + e) - f(v - e)) * g).sum() / (2 * h)
    return out


def test_activation_values():
    z = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    assert np.allclose(O.act(z, "relu")[0], [0, 0, 0, 1, 30])
    assert np.allclose(O.act(z, "silu")[0], [0, -1 / (1 + np.e), 0, 1 / (1 + np.exp(-1)), 30], atol=1e-9)
    assert np.allclose(O.act(z, "gelu")[0], [0, -0.15865525393, 0, 0.84134474607, 30], atol=1e-9)
    # the tanh form stays within 5e-4 of the other one
    grid = np.linspace(-6, 6, 1001)
    assert np.abs(O.act(grid, "gelu_tanh")[0] - O.act(grid, "gelu")[0]).max() < 5e-4


@pytest.mark.parametrize("kind", KINDS)
def test_activation_slopes(kind):
    z = np.linspace(-5, 5, 37) + 0.01
    h = 1e-6
    num = (O.act(z + h, kind)[0] - O.act(z - h, kind)[0]) / (2 * h)
    assert np.abs(num - O.act(z, kind)[1]).max() < 1e-8


@pytest.mark.parametrize("kind", KINDS)
def test_linear_gradients(kind):
    rng = np.random.default_rng(1)
    x, w, b, dy = (rng.standard_normal(s) for s in [(3, 4), (5, 4), (5,), (3, 5)])
    dx, dw, db = O.linear_bwd(dy, x, w, b, kind)
    assert np.allclose(dx, _differences(lambda v: O.linear(v, w, b, None, kind), x, dy), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: O.linear(x, v, b, None, kind), w, dy), atol=1e-7)
    assert np.allclose(db, _differences(lambda v: O.linear(x, w, v, None, kind), b, dy), atol=1e-7)


@pytest.mark.parametrize("kind", KINDS)
def test_gated_gradients(kind):
    rng = np.random.default_rng(2)
    x, wg, wu, dh = (rng.standard_normal(s) for s in [(3, 4), (5, 4), (5, 4), (3, 5)])
    dx, dg, du = O.gated_bwd(dh, x, wg, wu, kind)
    assert np.allclose(dx, _differences(lambda v: O.gated(v, wg, wu, kind), x, dh), atol=1e-7)
    assert np.allclose(dg, _differences(lambda v: O.gated(x, v, wu, kind), wg, dh), atol=1e-7)
    assert np.allclose(du, _differences(lambda v: O.gated(x, wg, v, kind), wu, dh), atol=1e-7)


def test_rms_norm_values_and_gradients():
    rng = np.random.default_rng(3)
    x, r, w, dy, ds = (rng.standard_normal(s) for s in [(3, 6), (3, 6), (6,), (3, 6), (3, 6)])
    y, s = O.rms_norm(x, np.ones(6), r, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1) and np.allclose(s, x + r)
    dx, dw = O.rms_norm_bwd(dy, s, w, ds)
    both = lambda v: np.concatenate(O.rms_norm(v, w, r), -1)  # noqa: E731
    assert np.allclose(dx, _differences(both, x, np.concatenate([dy, ds], -1)), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: O.rms_norm(x, v, r)[0], w, dy), atol=1e-7)
    assert O.row_scales(np.zeros((1, 4)))[0] == O.MIN_SCALE
    assert O.row_scales(np.array([[1.0, -896.0]]))[0] == 2.0
