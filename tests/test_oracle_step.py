"""The training step's oracle against differences, autograd's formulas and closed forms."""

import numpy as np
import pytest

from fp8_fine_grained_online_amd import synthetic as S
from oracle import step


def differences(f, x, dy, eps=1e-5):
    """d sum(f(x) dy) / dx by central differences."""
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += eps
        down[i] -= eps
        d[i] = ((f(up) - f(down)) * dy).sum() / (2 * eps)
    return d


@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("shape", [(3, 7), (1, 1), (4, 16)])
def test_norm_gradient_is_the_difference(centred, shape):
    rng = S.rng_for(3000, shape[1])
    x, dy, res = (rng.standard_normal(shape) for _ in range(3))
    g, b = 1 + 0.3 * rng.standard_normal(shape[1]), rng.standard_normal(shape[1])
    eps = 0.01
    beta = b if centred else None
    dx, dg, db = step.norm_bwd(dy, x, g, eps, centred)
    assert np.allclose(dx, differences(lambda v: step.norm(v, g, eps, beta, centred), x, dy), rtol=1e-6, atol=1e-8)
    assert np.allclose(dg, differences(lambda v: step.norm(x, v, eps, beta, centred), g, dy), rtol=1e-6, atol=1e-8)
    if centred:
        assert np.allclose(db, differences(lambda v: step.norm(x, g, eps, v, centred), b, dy), rtol=1e-6, atol=1e-8)
    assert np.allclose(step.norm_bwd(dy, x, g, eps, centred, res)[0], dx + res, rtol=1e-12)


def test_norm_of_known_rows():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    y = step.norm(x, np.array([1.0, 2.0]), 0.5)
    assert np.allclose(y[0], [3 / np.sqrt(13), 8 / np.sqrt(13)], rtol=1e-12) and not y[1].any()
    y = step.norm(x, np.ones(2), 0.0 + 2.0 ** -10, np.array([5.0, 6.0]), True)
    r = 1 / np.sqrt(0.25 + 2.0 ** -10)
    assert np.allclose(y, [[5 - 0.5 * r, 6 + 0.5 * r], [5, 6]], rtol=1e-12)


def test_swiglu_and_its_gradient():
    rng = S.rng_for(3001, 0)
    gu = 3 * rng.standard_normal((4, 10))
    dy = rng.standard_normal((4, 5))
    assert np.allclose(step.swiglu(gu), gu[:, :5] / (1 + np.exp(-gu[:, :5])) * gu[:, 5:], rtol=1e-13)
    assert np.allclose(step.swiglu_bwd(dy, gu), differences(step.swiglu, gu, dy), rtol=1e-6, atol=1e-9)
    far = np.array([[-800.0, 800.0, 0.0, 2.0, 3.0, 4.0]])
    assert np.array_equal(step.swiglu(far), [[-0.0, 2400.0, 0.0]])


@pytest.mark.parametrize("shape", [(6, 6), (5, 9), (9, 4), (1, 7), (2, 3, 5)])
def test_orthogonalize_maps_the_singular_values(shape):
    """X = U s V^T goes to U p(s) V^T, p the odd polynomial applied `steps` times to s / |s|."""
    g = S.rng_for(3002, shape[-1]).standard_normal(shape)
    coeffs = tuple(float(np.float32(v)) for v in (3.4445, -4.7750, 2.0315))
    got = step.orthogonalize(g, 4, coeffs, 0.5).reshape(-1, *shape[-2:])
    for m, o in zip(g.reshape(-1, *shape[-2:]), got):
        u, s, vt = np.linalg.svd(m, full_matrices=False)
        s = s / np.linalg.norm(s)
        for _ in range(4):
            s = coeffs[0] * s + coeffs[1] * s ** 3 + coeffs[2] * s ** 5
        assert np.allclose(o, 0.5 * (u * s) @ vt, rtol=1e-9, atol=1e-10)
    assert not step.orthogonalize(np.zeros((3, 4))).any()
