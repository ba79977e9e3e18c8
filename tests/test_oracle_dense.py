"""The float64 oracle of the dense products and the orthogonalised update,
pinned by differences, closed forms and its two independent forms (CPU)."""

import numpy as np
import pytest

from oracle import dense_ref as ref

ACTS = ("none", "relu", "gelu", "silu")


@pytest.mark.parametrize("name", ACTS)
def test_slopes_by_differences(name):
    z = np.linspace(-6, 6, 241) + 0.013
    h = 1e-6
    d = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    assert np.abs(d - ref.slope(z, name)).max() < 1e-8


def test_activations_at_known_points():
    assert ref.act(np.array([-1.0, 0.0, 2.0]), "relu").tolist() == [0, 0, 2]
    assert abs(ref.act(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15
    assert abs(ref.act(np.array([1.0]), "silu")[0] - 1 / (1 + np.exp(-1.0))) < 1e-15


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_by_differences(name):
    g = np.random.default_rng(1)
    x, w, b, r, dy = (g.standard_normal(s) for s in ((5, 7), (4, 7), (4,), (5, 4), (5, 4)))
    _, z = ref.linear(x, w, b, r, name)
    dx, dw, db, _ = ref.linear_bwd(dy, x, w, z, name)
    loss = lambda x, w, b: (ref.linear(x, w, b, r, name)[0] * dy).sum()
    h = 1e-6
    for arr, grad, at in ((x, dx, (2, 3)), (w, dw, (1, 6)), (b, db, (2,))):
        up, dn = arr.copy(), arr.copy()
        up[at] += h
        dn[at] -= h
        pick = lambda a: [a if arr is v else v for v in (x, w, b)]
        assert abs((loss(*pick(up)) - loss(*pick(dn))) / (2 * h) - grad[at]) < 1e-7


@pytest.mark.parametrize("shape", [(6, 6), (5, 9), (9, 5), (1, 7), (7, 1)])
def test_orthogonalize_two_ways(shape):
    g = np.random.default_rng(3).standard_normal(shape)
    a, b = ref.orthogonalize(g), ref.iterate(g)
    assert np.abs(a - b).max() < 1e-12
    s = np.linalg.svd(a, compute_uv=False)
    assert s.max() < 1.3


def test_the_quintic_keeps_its_interval():
    """[0, 1.21] maps into itself, so no iterate's largest singular value passes 1.21."""
    s = np.linspace(0, 1.21, 100001)
    p = ref.quintic(s)
    assert p.min() >= 0 and p.max() < 1.21


def test_orthogonal_input_and_scale():
    q, _ = np.linalg.qr(np.random.default_rng(5).standard_normal((8, 8)))
    s = 1 / np.sqrt(8.0)
    for _ in range(5):
        s = ref.quintic(s)
    assert np.abs(ref.orthogonalize(q * 37.0) - q * s).max() < 1e-6  # eps / |G| = 1e-9, slope 485
    assert not ref.orthogonalize(np.zeros((3, 4))).any()


def test_storage_models():
    v = np.random.default_rng(7).uniform(-1.2, 1.2, 10000)
    assert np.abs(ref.store_f16(v) - v).max() <= 2.0 ** -11 * 1.2
    assert np.abs(ref.store_2f16(v) - v).max() <= 2.0 ** -22 * 1.2


def test_muon_step():
    g = np.random.default_rng(9)
    w, dw, buf = (g.standard_normal((4, 6)) for _ in range(3))
    for nesterov in (True, False):
        w1, b1 = ref.muon(w, dw, buf, 0.1, 0.01, 0.9, nesterov)
        assert np.allclose(b1, 0.9 * buf + dw)
        u = dw + 0.9 * b1 if nesterov else b1
        assert np.allclose(w1, 0.99 * w - 0.1 * ref.orthogonalize(u))
