"""Where the calls for the verification pass's rows have to keep small parts of a result beside large
ones, against the float64 forms of oracle/serving.py.

Attention's tolerances are relative to the sum of p |v|, with no part of the largest weight: a score
is off by (D + 8) U of sum |q k| scale, which counts twice in a probability's ratio to their sum;
base-2 exponents round at |t| U, twice; a weight enters the second product as two bfloat16 parts for
bfloat16 (2^-17 of it, each part half a step of 8 bits) and as three for float32 (U); sums of 32
tokens in a matrix instruction, then a block after the other: (64 + tokens / 16) U; then H of the result.
U = 2^-24 is half a step of float32, H half a step of the outputs' type.
"""

import numpy as np
import pytest

from oracle import serving as os_
from tests.test_gpu_serving import HALF, U, _dev, _filled, _host, _ints, _rows, _sv, _type

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import lossless_draft_verification_sample_amd._lib as L
    L.load()


def _weigh_tol(want, lse, size, reach, tokens, D, dtype):
    score = (D + 8) * U * reach + 2 * U * (reach + 30) * 1.5
    far = size * (2 * score[..., None] + (2.0 ** -17 if dtype == "bf16" else U) + (64 + tokens / 16) * U)
    return far + HALF[dtype] * (np.abs(want) + far), score + (70 + tokens / 16) * U + U * np.abs(lse)


def _same_as_formula(got, q, keys, vals, first, scale, dtype, window=0):
    want, lse, size, reach, _ = os_.attention(q, keys, vals, first, scale, window)
    tol, ltol = _weigh_tol(want, lse, size, reach, len(keys), q.shape[-1], dtype)
    far = np.abs(_host(got.out[0]) - want)
    assert np.all(far <= tol), ((far / tol).max(), (far / np.maximum(size, 1e-300)).max())
    assert np.all(np.abs(_host(got.lse[0]) - lse) <= ltol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [32, 300, 3000])
@pytest.mark.parametrize("N,qh,H,D", [(1, 2, 2, 32), (9, 8, 2, 128), (2, 1, 1, 256), (3, 6, 6, 80)])
@pytest.mark.parametrize("nats", [10.0, 13.0, 16.0, 17.0, 30.0, 60.0])
def test_attention_with_a_sink(dtype, T, N, qh, H, D, nats):
    """The first token takes nearly all of the weight and has the value 0, so that outputs are made of the
    other tokens' small weights alone."""
    rng = np.random.default_rng(int(nats) * 10 + D)
    cache, table, _, _ = _filled(rng, [T], H, D, 32)
    k = (rng.standard_normal((1, T, H, D)) * 0.25).astype(np.float32)
    k[..., 0] = 0.0
    k[0, 0] = 0.0
    k[0, 0, :, 0] = nats
    v, _ = _rows(rng, (1, T, H, D), "f32")
    v[0, 0] = 0.0
    _sv().spec_verify_cache_write(cache, _dev(table), _ints([0]), _dev(k), v)
    keys, vals = (_host(t)[0] for t in _sv().spec_verify_cache_read(cache, _dev(table), None, T, _type("f32")))
    assert (vals[0] == 0).all()
    q = (rng.standard_normal((1, N, qh, D)) / D ** 0.5).astype(np.float32)
    q[..., 0] = 1.0
    qt = _dev(q, dtype)
    got = _sv().spec_verify_attention(qt, cache, _dev(table), _ints([T - N]), 1.0, want_lse=True)
    _same_as_formula(got, _host(qt)[0], keys, vals, T - N, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low,high", [(-90, 0), (-40, 50), (0, 90)])
@pytest.mark.parametrize("T", [300, 2000])
def test_attention_beside_blocks_of_far_larger_values(dtype, low, high, T):
    """The first blocks' values are 2^90 times the others' and their weights nearly 0 (2^-115 or less): outputs are
    made of the small values. Then the other way round: the large values come last."""
    rng = np.random.default_rng(T + high)
    H, D = 2, 64
    for first in (True, False):
        cache, table, _, _ = _filled(rng, [T], H, D, 32)
        large = np.zeros(T, bool)
        end = T // 32 * 32
        large[slice(0, 128) if first else slice(end - 64, end)] = True
        k = (rng.standard_normal((1, T, H, D)) * 0.25).astype(np.float32)
        k[..., 0] = np.where(large, -80.0, 0.0)[None, :, None]
        v = rng.standard_normal((1, T, H, D)) * np.where(large, 2.0 ** high, 2.0 ** low)[None, :, None, None]
        _sv().spec_verify_cache_write(cache, _dev(table), _ints([0]), _dev(k), _dev(v.astype(np.float32)))
        keys, vals = (_host(t)[0] for t in _sv().spec_verify_cache_read(cache, _dev(table), None, T, _type("f32")))
        q = (rng.standard_normal((1, 3, 4, D)) / D ** 0.5).astype(np.float32)
        q[..., 0] = 1.0
        qt = _dev(q, dtype)
        got = _sv().spec_verify_attention(qt, cache, _dev(table), _ints([T - 3]), 1.0, want_lse=True)
        _same_as_formula(got, _host(qt)[0], keys, vals, T - 3, 1.0, dtype)


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotate_near_a_sine_or_cosine_of_zero(dtype, inter):
    """Pairs (1, 0) and (0, 1) become a cosine and a sine, which are right relative to themselves where the angle is
    near a multiple of a quarter of a turn: within 3 U (sine and cosine 2 U; what is left of the angle rounded to float32, U
    of the sine and 0.8 U of the cosine up to an eighth of a turn) and the float64 angle's own 2 pi t 2 2^-52 of t turns; then H."""
    import torch
    rng = np.random.default_rng(17)
    R, N = 32, 400
    # whole quarters of a turn a position, and a little more
    f = (rng.integers(0, 8, R // 2) + 10.0 ** -rng.uniform(3, 7, R // 2)) * np.pi / 2
    first = 3
    q = np.zeros((1, N, 2, R), np.float32)
    one = slice(0, R, 2) if inter else slice(0, R // 2)
    two = slice(1, R, 2) if inter else slice(R // 2, R)
    q[0, :, 0, one] = 1.0
    q[0, :, 1, two] = 1.0
    got = _host(_sv().spec_verify_rotate(_dev(q, dtype), None, _ints([first]), _dev(f), inter).q)[0]
    torch.cuda.synchronize()
    want = os_.rotate(q[0], first + np.arange(N), f, inter)
    turns = (first + np.arange(N))[:, None, None] * np.concatenate([f, f])[None, None] / (2 * np.pi)
    if inter:
        turns = (first + np.arange(N))[:, None, None] * np.repeat(f, 2)[None, None] / (2 * np.pi)
    exact = 3 * U * np.abs(want) + 2 * np.pi * 2 * turns * 2.0 ** -52
    tol = exact + HALF[dtype] * (np.abs(want) + exact)
    far = np.abs(got - want)
    assert np.all(far <= tol), (far / tol).max()
