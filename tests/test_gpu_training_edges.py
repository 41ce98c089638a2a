"""Edges of the drafter-training kernels, against their float64 forms: what the
gradients keep of dz, finite masks, rows of NaN. Tolerances count roundings as in
tests/test_gpu_training.py (U: half a step of float32)."""

import numpy as np
import pytest

from oracle import training as ot
from tests.test_gpu_training import HALF, U, _dev, _head, _host, _sum_tol, _sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"


# ---------------------------------------------------------------- linear cross entropy


def _gradient_tol(h, w, z, dz, g):
    """Bounds of both gradients of bfloat16 matrices when dz reaches its products in two
    bfloat16 parts: what the second part leaves is at most 2^-8 of 2^-8 of dz. The rest:
    a logit's sum of D exact products (eight standard deviations of its roundings), the
    exponent, the sum over the vocabulary, the products' sums (two parts: 2 n terms) and
    one rounding of the result to bfloat16."""
    D, V = h.shape[1], w.shape[0]
    zt = 8 * np.sqrt(D) * U * (np.abs(h) @ np.abs(w).T).max(1)
    m, ls = ot.log_sum_exp(z)
    rel = 2 * zt + 8 * U * (np.abs(z).max(1) + 30) + _sum_tol(V)
    q = np.exp(z - (m + ls)[:, None])
    dt = np.abs(g)[:, None] * (rel[:, None] * q + 4 * U * (np.abs(dz) > 0)) + 2.0 ** -16 * np.abs(dz)

    def product(x, xt, y):
        return (xt @ np.abs(y) + 8 * np.sqrt(2 * x.shape[1]) * U * (np.abs(x) @ np.abs(y))
                + HALF["bf16"] * np.abs(x @ y) + 1e-37)
    return product(dz, dt, w), product(dz.T, dt.T, h)


@pytest.mark.parametrize("N,D,V,pad", [
    (1, 64, 1000, 0), (20, 72, 1500, 0), (31, 65, 700, 3), (100, 192, 2001, 0), (128, 1000, 515, 0),
    (200, 64, 127, 0), (300, 256, 4001, 0), (513, 129, 3000, 1), (777, 1000, 2500, 0),
])
def test_linear_ce_gradients_keep_dz_beyond_bfloat16(N, D, V, pad):
    """The only rounding to bfloat16 that the gradients of bfloat16 matrices show is
    their own."""
    import torch
    sv, rng = _sv(), np.random.default_rng(N + 3 * D + V)
    h, w, y = _head(rng, N, D, V, "bf16", pad)
    g = rng.uniform(0.2, 2.0, N).astype(np.float32) / N
    a = sv.spec_verify_linear_ce(h, w, _dev(y))
    b = sv.spec_verify_linear_ce_backward(h, w, _dev(y), a.stats, _dev(g))
    torch.cuda.synchronize()
    hh, ww = _host(h), _host(w)
    _, gh, gw, z, dz = ot.linear_ce(hh, ww, y, g)
    used = (y >= 0) & (y < V)
    for got, want, tol in zip((b.hidden, b.weight), (gh, gw),
                              _gradient_tol(hh, ww, z, dz, np.where(used, g, 0.0))):
        far = np.abs(_host(got) - want) - tol
        assert np.all(far <= 0), (far.max(), np.argwhere(far > 0)[:4], (far > 0).mean())
