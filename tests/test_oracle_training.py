"""The float64 forms of the drafter-training operators: worked values, and their
gradients against central differences."""

import numpy as np
import pytest

from oracle import training as ot


def test_top_logits_order_ties_and_gaps():
    z = np.array([[1.0, 3.0, -np.inf, 3.0, np.nan, 2.0], [-np.inf] * 6])
    ids, values, lse = ot.top_logits(z[:, :4], 3)
    assert ids[0].tolist() == [1, 3, 0] and values[0].tolist() == [3.0, 3.0, 1.0]
    assert np.isclose(lse[0], np.log(2 * np.exp(3) + np.exp(1)))
    assert ids[1].tolist() == [-1] * 3 and np.all(np.isneginf(values[1])) and np.isneginf(lse[1])
    assert ot.top_logits(z, 6)[0][0].tolist() == [1, 3, 5, 0, -1, -1]


def test_distill_of_the_full_row_is_the_divergence():
    rng = np.random.default_rng(1)
    z, t = rng.normal(size=(2, 7)), rng.normal(size=(2, 7))
    ids = np.stack([rng.permutation(7) for _ in range(2)])
    loss, grad, *_ = ot.distill(z, ids, np.take_along_axis(t, ids, 1))
    p, q = (np.exp(x) / np.exp(x).sum(1, keepdims=True) for x in (t, z))
    assert np.allclose(loss, (p * np.log(p / q)).sum(1)) and np.allclose(grad, q - p)


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_distill_gradient_against_differences(lse, temperature):
    rng = np.random.default_rng(2)
    z, t = rng.normal(size=(3, 11)) * 2, rng.normal(size=(3, 4)) * 2
    ids = np.array([[0, 3, 3, 10], [5, -1, 2, 11], [1, 2, 3, 4]])   # repeated and empty slots
    L = rng.normal(size=3) + 4 if lse else None
    w = np.array([1.0, 0.3, 2.0])
    _, grad, *_ = ot.distill(z, ids, t, temperature, L, w)
    h = 1e-6
    for r, v in [(0, 0), (0, 3), (0, 7), (1, 2), (1, 9), (2, 4)]:
        up, down = z.copy(), z.copy()
        up[r, v] += h
        down[r, v] -= h
        d = (ot.distill(up, ids, t, temperature, L)[0] - ot.distill(down, ids, t, temperature, L)[0])[r]
        assert abs(w[r] * d / (2 * h) - grad[r, v]) < 1e-7


def test_linear_ce_gradients_against_differences():
    rng = np.random.default_rng(3)
    h, w = rng.normal(size=(4, 5)), rng.normal(size=(9, 5))
    y = np.array([2, -100, 8, 2])
    g = np.array([0.5, 3.0, 1.0, 2.0])
    loss, gh, gw, *_ = ot.linear_ce(h, w, y, g)
    assert loss[1] == 0.0 and np.all(gh[1] == 0)
    eps = 1e-6
    for x, grad in ((h, gh), (w, gw)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + eps
            up = (g * ot.linear_ce(h, w, y)[0]).sum()
            x[i] = keep - eps
            down = (g * ot.linear_ce(h, w, y)[0]).sum()
            x[i] = keep
            assert abs((up - down) / (2 * eps) - grad[i]) < 1e-7
