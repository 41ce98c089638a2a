"""What rejected proposals leave in a block of the 8-bit cache: nothing in its scale, a coarser rounding of far
smaller committed values in its codes, and nothing at all where the block's committed rows are written again.

Proposals 2^k times the block's largest value L raise its scale from s to 2^k s. A value that is 2^e to 2^(e+1)
times s has a code that is a whole multiple of 2^(e-3), and stays exact where 2^(e-3-k) is no less than the smallest step
2^-9, so from 2^(k-6) s on, and L is above 224 s: from 2^(k-13) L on. Others are rounded to whole 2^(k-9) s: off by
2^(k-10) s at most.
"""

import numpy as np
import pytest

from oracle import serving as os_

SHAPE = (2, 40)     # heads, dimensions


def _rows(k, held=21, new=6):
    rng = np.random.default_rng(100 + k)
    x = rng.standard_normal((held, *SHAPE)) * 2.0 ** -rng.uniform(0, 12, (held, *SHAPE))
    x = x.clip(-2.5, 2.5).astype(np.float32).astype(np.float64)
    x[0, :, 0] = 3.0            # the largest: a code of its own, which decides the scale before and after rounding
    fresh = (rng.standard_normal((new, *SHAPE)) / 8).astype(np.float32).astype(np.float64)
    return x, fresh


def _proposals(before, k, n=3):
    """n rows that are 2^k times the largest value of each head."""
    return np.broadcast_to(np.abs(before).max((0, 2), keepdims=True) * 2.0 ** k, (n, *SHAPE)).copy()


def _check(write, read, scale, k):
    """write(first, rows), read(n), scale(): of one request's first block."""
    x, fresh = _rows(k)
    held = len(x)
    write(0, x)
    before, s = read(held), scale()
    write(held, _proposals(before, k))
    assert np.array_equal(scale(), s * 2.0 ** k)
    write(held, fresh)
    assert np.array_equal(scale(), s)                       # the scale is as if they had never been there
    after = read(held)
    large = np.abs(before).max((0, 2), keepdims=True)
    moved = before != after
    assert not moved[np.abs(before) >= 2.0 ** (k - 13) * large].any()
    assert np.all(np.abs(before - after) <= 2.0 ** (k - 10) * s[:, None])
    assert moved.any() == (k > 0), k      # values down to 2^-12 of the largest and below
    # the block's committed rows again, from the caller's own: as if written for the first time
    write(0, np.concatenate((x, fresh)))
    assert np.array_equal(read(held), before) and np.array_equal(scale(), s)


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("k", [0, 3, 8, 11, 13])
def test_in_the_formula(values, k):
    c = os_.Cache(np.zeros((1, SHAPE[0], 1, 2, 1024), np.uint8), np.zeros((1, SHAPE[0], 1), np.float32), SHAPE[1], values)
    _check(lambda first, x: c.write([0], first, x), lambda n: c.read([0], 0, n), lambda: c.scale[0, :, 0].astype(float), k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [0, 3, 8, 11, 13])
def test_in_the_cache(dtype, k):
    import torch
    import lossless_draft_verification_sample_amd as sv
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    kind = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    cache = sv.kv_cache(1, SHAPE[0], 32, SHAPE[1])
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def write(first, x):
        t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(kind)[None]
        sv.spec_verify_cache_write(cache, table, torch.tensor([first], dtype=torch.int32, device="cuda"), t, t)

    for name in ("k", "v"):
        def read(n, name=name):
            return getattr(sv.spec_verify_cache_read(cache, table, None, n, torch.float32), name)[0].double().cpu().numpy()

        _check(write, read, lambda name=name: getattr(cache, name + "_scale")[0, :, 0].double().cpu().numpy(), k)
