"""Pins of the float64 oracles of the router, the sorted rows and the int8 product."""

import numpy as np
import pytest

from fp8_fine_grained_online_amd import synthetic as S
from oracle import int8, moe, route, tokens


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    rng = S.rng_for(2100, 0)
    x = rng.standard_normal((5, 12))
    x[1, 3] = -np.inf
    ids, _ = route.route(x, 3, score=score, renormalize=renormalize)
    ids[2, 1] = -1          # a choice that was not filled
    ids[3] = [4, 4, 7]      # an expert listed twice
    g = rng.standard_normal(ids.shape)
    d = route.route_bwd(x, ids, g, score, renormalize, 2.5)

    def value(logits):
        return (g * route.weights_of(logits, ids, score, renormalize, 2.5)).sum()

    h = 1e-5
    for t in range(x.shape[0]):
        for e in range(x.shape[1]):
            if not np.isfinite(x[t, e]):
                assert d[t, e] == 0
                continue
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            # central difference: error h^2 times a third derivative below 10 |g|, plus rounding 1e-16 / h
            assert abs((value(up) - value(down)) / (2 * h) - d[t, e]) < 1e-8


def decimal_weights(x, ids, score, renormalize):
    """The weights by the formula, in 60 decimal digits."""
    from decimal import Decimal as D, getcontext
    getcontext().prec, getcontext().Emin = 60, -10 ** 6
    e = [D(float(v)) for v in x]
    if score == "sigmoid":
        p = [1 / (1 + (-v).exp()) for v in e]
    else:
        top = max(e)
        p = [(v - top).exp() for v in e]
        p = [v / sum(p) for v in p]
    w = [p[i] for i in ids]
    return [v / sum(w) for v in w] if renormalize else w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_of_far_logits(score):
    """Against the formula in 60 digits: dw_j / dl_e = q_j (delta - q_e), times 1 - p_e for sigmoids."""
    from decimal import Decimal as D
    g = np.array([[200.0, -200.0]])
    for pair in ((-707.0, -706.0), (-720.0, -721.0), (-745.5, -744.0), (-800.0, -801.0), (0.0, -750.0)):
        x = np.array([[1.0, pair[0], pair[1]]])
        ids = np.array([[2, 1]], np.int32)
        q = decimal_weights(x[0], ids[0], score, True)
        p = decimal_weights(x[0], ids[0], score, False)
        mean = sum(D(float(a)) * b for a, b in zip(g[0], q))
        want = [float(b * (D(float(a)) - mean) * ((1 - c) if score == "sigmoid" else 1)) for a, b, c in zip(g[0], q, p)]
        d = route.route_bwd(x, ids, g, score, True, 1.0)[0]
        assert d[0] == 0
        # float64: a few tens of roundings against |g|
        assert abs(d[2] - want[0]) < 1e-12 and abs(d[1] - want[1]) < 1e-12, (pair, d, want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalized_weights_that_underflow(score):
    """A bias steers the choice to experts whose probabilities are 0 in float64."""
    bias = np.array([-9.0, 0, 0])
    for pair in ((-707.0, -706.0), (-720.0, -721.0), (-745.5, -744.0), (-800.0, -801.0), (0.0, -750.0), (-3.0, 0.5)):
        x = np.array([[1.0, *pair]])
        ids, w = route.route(x, 2, bias, score=score)
        assert sorted(ids[0]) == [1, 2]
        want = [float(v) for v in decimal_weights(x[0], ids[0], score, True)]
        assert np.allclose(w[0], want, rtol=1e-13, atol=1e-300)
        assert np.allclose(route.weights_of(x, ids, score, True, 1.0)[0], want, rtol=1e-13, atol=1e-300)


def test_sigmoid_of_far_logits():
    x = np.array([-699.5, -700.5, -709.25, -709.75, -720.0, -744.0, -1.0, 30.0])
    want = decimal_weights(x, range(8), "sigmoid", False)
    # float64, and one unit of the smallest subnormal number
    assert all(abs(a - float(b)) <= 1e-15 * float(b) + 5e-324 for a, b in zip(route.scores(x[None], "sigmoid")[0], want))


def test_route_ties_groups_and_masks():
    x = np.zeros((4, 8))
    ids, w = route.route(x, 3)
    assert np.array_equal(ids[0], [0, 1, 2]) and np.allclose(w[0], 1 / 3)
    x[1] = -np.inf
    x[2] = [0, 0, 5, 0, 3, 3, 0, 0]  # groups of 2: scores by z = p
    x[3, :6] = np.nan
    ids, w = route.route(x, 3, n_groups=4, topk_groups=2)
    assert np.array_equal(ids[1], [-1, -1, -1]) and not w[1].any()
    assert np.array_equal(ids[2], [2, 4, 5])
    assert np.array_equal(ids[3], [6, 7, -1]) and w[3, 2] == 0


def test_layout_is_the_dispatch_layout():
    rng = S.rng_for(2101, 0)
    ids = rng.integers(-1, 6, (70, 3)).astype(np.int32)  # 5 is outside [0, 5)
    x = S.activations(70, 128, rng)
    _, _, off, rows, counts = moe.dispatch_1x128(x, ids, 5)
    rows2, off2, counts2 = tokens.layout(ids, 5)
    assert np.array_equal(rows, rows2) and np.array_equal(off, off2) and np.array_equal(counts, counts2)


def test_combine_gradient_against_differences():
    rng = S.rng_for(2102, 0)
    ids = rng.integers(-1, 3, (6, 2)).astype(np.int32)
    rows, off, _ = tokens.layout(ids, 3)
    c = rng.standard_normal((int(off[-1]), 4))
    w = rng.random((6, 2))
    dy = rng.standard_normal((6, 4))
    dc, dw, _ = tokens.combine_bwd(dy, c, rows, w, off)
    h = 1e-6
    for t, j in [(0, 0), (3, 1), (5, 0)]:
        up = w.copy()
        up[t, j] += h
        # linear in w: the difference quotient is exact up to rounding, 1e-16 * 10 / h
        assert abs(((tokens.combine(c, rows, up)[0] - tokens.combine(c, rows, w)[0]) * dy).sum() / h - dw[t, j]) < 1e-7
    for r in {int(v) for v in rows.reshape(-1) if v >= 0}:
        up = c.copy()
        up[r, 1] += h
        assert abs(((tokens.combine(up, rows, w)[0] - tokens.combine(c, rows, w)[0]) * dy).sum() / h - dc[r, 1]) < 1e-7


def test_permutes_gradient_is_the_unweighted_combine():
    rng = S.rng_for(2103, 0)
    ids = rng.integers(-1, 4, (9, 3)).astype(np.int32)
    x, g = rng.standard_normal((9, 5)), None
    xp, off, rows = tokens.permute(x, ids, 4)
    g = rng.standard_normal(xp.shape)
    # permute is linear: <g, permute(v)> = <its gradient, v> for every v
    dx = tokens.combine(g, rows)[0]
    v = rng.standard_normal(x.shape)
    assert abs((g * tokens.permute(v, ids, 4)[0]).sum() - (dx * v).sum()) < 1e-12


def test_int8_rows():
    x = np.array([[0, 0, 0], [127, -63.5, 1], [-2, 1, 0.0078125]], np.float32)
    q, s = int8.quant_rows(x)
    assert s[0] == 0 and not q[0].any()
    assert np.array_equal(q[1], [127, -64, 1])  # 63.5 is a tie: to even
    assert np.array_equal(q[2], [-127, 64, 0])  # 1 / (2/127): 63.5 in binary32, a tie
    acc = int8.gemm(np.array([[-128] * 16], np.int8), [1.0], np.array([[-128] * 16], np.int8), [0.5])
    assert acc[0, 0] == 128 * 128 * 16 / 2
