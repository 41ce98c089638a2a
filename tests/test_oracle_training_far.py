"""The float64 form of the distillation at teacher logits so large that their
log-normaliser is their value."""

import numpy as np
import pytest

from oracle import training as ot


@pytest.mark.parametrize("far", [-1e16, -1e20, -3.3895313892515355e38, 3e38])
def test_distill_teachers_of_one_far_value_share_their_mass(far):
    rng = np.random.default_rng(1)
    z, ids = rng.normal(size=(1, 9)), np.array([[0, 3, 5, 8]])
    a = ot.distill(z, ids, np.full((1, 4), far))
    b = ot.distill(z, ids, np.zeros((1, 4)))
    assert np.all(a[2] == 0.25) and all(np.array_equal(x, y) for x, y in zip(a, b))
