"""The drafter-training kernels against their float64 forms (oracle/training.py).

Tolerances count roundings. U = 2^-24 is half a step of float32, H half a step of
the outputs' type. A row's log-normaliser is off by at most
  _lse_tol: V/512 + 200 roundings of the running sum (a thread adds V/512 terms,
  then log-depth joins, each with a rescale), the exponents' own rounding
  (|z - m| / T <= 60 wherever a term matters: 60 * 2 U), and two roundings of the result.
"""

import numpy as np
import pytest

from oracle import training as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import lossless_draft_verification_sample_amd._lib as L
    L.load()


def _sv():
    import lossless_draft_verification_sample_amd as sv
    return sv


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    if dtype is not None:
        t = t.to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    return t


def _host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(rng, R, V, dtype, pad=0, shift=0):
    """Logits [R, V] on the device, and their float64 values: cut from a buffer
    that is `pad` columns wider, `shift` elements in."""
    z = (rng.standard_normal((R, V + pad)) * 3).astype(np.float32)
    hot = rng.integers(0, V + pad, (R, 6))
    np.put_along_axis(z, hot, rng.uniform(8, 20, hot.shape).astype(np.float32), 1)
    t = _dev(z, dtype)[:, shift: shift + V]
    return t, _host(t)


def _twin(t):
    """A copy with the same strides and alignment: the order of a row's sum follows
    where its 16-byte groups begin."""
    if t._base is None:
        return t.clone()
    return t._base.clone().as_strided(t.shape, t.stride(), t.storage_offset())


def _sum_tol(V):
    return (V / 512 + 200) * U + 120 * U


def _lse_tol(V, lse):
    return _sum_tol(V) + 2 * U * np.where(np.isfinite(lse), np.abs(lse), 0.0)


# ---------------------------------------------------------------- top logits

def _check_top(t, z, k, T=1.0, **kw):
    import torch
    out = _sv().spec_verify_top_logits(t, k, temperature=T, **kw)
    torch.cuda.synchronize()
    ids, values, lse = ot.top_logits(z.reshape(-1, z.shape[-1]), k, T)
    assert np.array_equal(out.ids.cpu().numpy().reshape(ids.shape), ids)
    assert np.array_equal(_host(out.values).reshape(values.shape), values)
    if out.lse is not None:
        got = _host(out.lse).reshape(-1)
        nan = np.isnan(z.reshape(-1, z.shape[-1])).any(1)
        assert np.all(np.isnan(got[nan]))
        with np.errstate(invalid="ignore"):
            far = np.abs(got - lse)
        ok = (got == lse) | (far <= _lse_tol(z.shape[-1], lse)) | nan
        assert np.all(ok), (got[~ok], lse[~ok])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,K,pad,shift,T", [
    (1, 1, 1, 0, 0, 1.0), (1, 7, 7, 0, 0, 1.0), (3, 9, 4, 5, 3, 0.5), (3, 1000, 1000, 0, 0, 1.0),
    (2, 1023, 64, 1, 1, 0.7), (5, 4097, 1, 0, 0, 1.0), (4, 8192, 33, 0, 0, 2.0),
    (4, 50257, 256, 3, 2, 1.0), (9, 151936, 32, 0, 0, 0.8), (2, 151936, 1024, 0, 0, 1.0),
    (3, 32000, 1000, 7, 5, 1.0), (600, 3001, 17, 0, 0, 1.3), (520, 20011, 300, 9, 4, 1.0),
    (700, 40003, 64, 0, 0, 1.0), (700, 40003, 65, 1, 0, 1.0), (1, 300007, 1024, 0, 0, 1.0),
])
def test_top_logits(dtype, R, V, K, pad, shift, T):
    rng = np.random.default_rng(R * 7919 + V + K)
    t, z = _rows(rng, R, V, dtype, pad, shift)
    _check_top(t, z, K, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [2, 513])
def test_top_logits_orders_and_ties(dtype, R):
    """Rows whose order defeats the running threshold, or whose values all tie."""
    V, rng = 12345, np.random.default_rng(5)
    ramp = np.linspace(-40, 40, V).astype(np.float32)
    low = np.float32(-3.3895313892515355e38)
    kinds = {
        "equal": np.full(V, 1.5, np.float32), "rising": ramp, "falling": ramp[::-1],
        "two values": (rng.random(V) < 0.5).astype(np.float32),
        "zeros of both signs": np.where(rng.random(V) < 0.5, -0.0, 0.0).astype(np.float32),
        "negative": -np.abs(ramp) - 1,
        "few": np.where(np.arange(V) % 4000 == 77, ramp, -np.inf).astype(np.float32),
        "one at the end": np.where(np.arange(V) == V - 1, 3.0, -np.inf).astype(np.float32),
        "none": np.full(V, -np.inf, np.float32),
        "lowest": np.full(V, low, np.float32),
        "lowest but three": np.where(np.isin(np.arange(V), (0, 5000, V - 1)), 2.0, low).astype(np.float32),
        "huge": np.where(np.arange(V) % 2 == 0, 3e38, -3e38).astype(np.float32),
    }
    z = np.stack([kinds[k] for k in kinds])
    z = np.concatenate([z] + [z[rng.integers(0, len(z), R)]])
    t = _dev(z, dtype)
    for K in (1, 40, 1024):
        _check_top(t, _host(t), K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_logits_orders_and_ties_of_long_rows(dtype):
    """Rows that go on long after the threshold's first stretches, one workgroup to a
    row and several: orders and ties that fill what is noted and listed."""
    import torch
    V, rng = 100003, np.random.default_rng(8)
    ramp = np.linspace(-40, 40, V).astype(np.float32)
    late = np.arange(V) > 70000
    z = np.stack([
        np.full(V, -2.5, np.float32), ramp, ramp[::-1],
        np.where(late, 3.0, rng.standard_normal(V)).astype(np.float32),      # ties behind the start
        np.where(late, ramp, 39.0).astype(np.float32),                       # ties first
        np.where(np.arange(V) % 9 == 0, 5.0, -1.0).astype(np.float32),       # a tie in every group
        np.where(late, rng.standard_normal(V), -np.inf).astype(np.float32),  # nothing at the start
    ])
    t = _dev(z, dtype)
    wide = t.repeat(100, 1)
    assert wide.shape[0] > 640   # at 2 workgroups a row and less
    for K in (1, 64, 65, 512, 513, 1024):
        few = _check_top(t, _host(t), K)
        many = _sv().spec_verify_top_logits(wide, K)
        torch.cuda.synchronize()
        assert torch.equal(many.ids, few.ids.repeat(100, 1)) and torch.equal(many.values, few.values.repeat(100, 1))
        assert ((many.lse - few.lse.repeat(100)).abs() <= 2 * _sum_tol(V) + 4 * U * 60).all()


def test_top_logits_nan_is_no_candidate():
    rng = np.random.default_rng(6)
    z = (rng.standard_normal((4, 9000)) * 3).astype(np.float32)
    z[1, ::7] = np.nan
    z[2, :] = np.nan
    for dtype in ("bf16", "f32"):
        t = _dev(z, dtype)
        _check_top(t, _host(t), 50)


def test_top_logits_takes_the_verifiers_target_rows():
    import torch
    rng = np.random.default_rng(7)
    t, z = _rows(rng, 3 * 5, 4099, "bf16")
    a = _check_top(t.view(3, 5, 4099), z, 20)
    assert a.ids.shape == (3, 5, 20) and a.lse.shape == (3, 5)
    b = _sv().spec_verify_top_logits(t.view(3, 5, 4099)[:, 2:3], 20, want_lse=False)   # one row a request
    torch.cuda.synchronize()
    assert b.lse is None and torch.equal(b.ids, a.ids[:, 2:3])


# ---------------------------------------------------------------- distillation

def _teacher(rng, z, K, spread=3.0):
    """Kept ids and logits of a teacher near the student z."""
    t = np.where(np.isfinite(z), z, 0.0) + rng.standard_normal(z.shape) * spread / 3
    ids, values, _ = ot.top_logits(t.astype(np.float32), min(K, z.shape[1]))
    if K > z.shape[1]:
        ids = np.pad(ids, ((0, 0), (0, K - z.shape[1])), constant_values=-1)
        values = np.pad(values, ((0, 0), (0, K - z.shape[1])))
    return ids, values.astype(np.float32)


def _distill_tol(z, ids, values, T, ref, dtype, w):
    """Bounds of loss and gradient from the exact p, q. A: the largest magnitude whose
    rounding enters an exponent."""
    _, _, ps, pv, qs = ref
    V, K = z.shape[1], values.shape[1]
    used = np.isfinite(values) & (ps > 0)
    with np.errstate(invalid="ignore"):
        gap = np.where(qs > 1e-30, z.max(1, keepdims=True) - z, 0).max(1) / T
    A = np.where(used, np.abs(values) / T, 0).max(1) + gap + 30
    rel = 8 * U * A + _sum_tol(V) + (K + 20) * U      # of p_k, q_v and each log
    P = ps.sum(1)
    # every term of the loss is p (log p - log q): p's error, and that of each log
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.take_along_axis(qs, np.where(ps > 0, ids, 0), 1)
        ratio = np.where(ps > 0, np.abs(np.log(ps) - np.log(q)), 0.0)
    loss = P * (A * 8 * U + 2 * rel) + (ps * ratio).sum(1) * (rel + 4 * U)
    g = (np.ones(len(P)) if w is None else np.abs(w)) / T
    size = g[:, None] * (P[:, None] * qs + pv)
    grad = HALF[dtype] * np.abs(ref[1]) + (rel + 4 * U)[:, None] * size + 1e-37
    return loss, grad


def _check_distill(t, z, ids, values, T=1.0, lse=None, w=None, dtype="bf16", in_place=False):
    import torch
    sv = _sv()
    di, dv = _dev(ids.astype(np.int32)), _dev(values)
    dl, dw = (None if x is None else _dev(np.asarray(x, np.float32)) for x in (lse, w))
    a = sv.spec_verify_distill(t, di, dv, temperature=T, teacher_lse=dl)
    assert a.grad is None
    b = sv.spec_verify_distill(t, di, dv, temperature=T, teacher_lse=dl, row_weight=dw, want_grad=True)
    c = sv.spec_verify_distill_backward(t, di, dv, a.stats, dw, temperature=T, teacher_lse=dl)
    torch.cuda.synchronize()
    ref = ot.distill(z, ids, values, T, lse, w)
    lt, gt = _distill_tol(z, ids, values, T, ref, dtype, w)
    assert torch.equal(a.loss.isnan(), b.loss.isnan())
    got = _host(a.loss)
    with np.errstate(invalid="ignore"):
        # a loss beyond float32's range is an infinity
        bad = ~((got == np.where(np.abs(ref[0]) > 3.4028236e38, np.inf, ref[0])) | (np.abs(got - ref[0]) <= lt))
    assert not bad.any(), (got[bad], ref[0][bad], lt[bad])
    for g in (b.grad, c):
        far = np.abs(_host(g) - ref[1]) - gt
        assert not (far > 0).any() and np.isfinite(_host(g)).all(), (far.max(), np.argwhere(far > 0)[:5])
    if in_place:
        t2, t3 = _twin(t), _twin(t)
        out = sv.DistillOut(torch.empty_like(a.loss), torch.empty_like(a.stats), t2)
        d = sv.spec_verify_distill(t2, di, dv, temperature=T, teacher_lse=dl, row_weight=dw, out=out)
        sv.spec_verify_distill_backward(t3, di, dv, a.stats, dw, temperature=T, teacher_lse=dl, out=t3)
        torch.cuda.synchronize()
        assert d.grad is t2 and torch.equal(t2, b.grad) and torch.equal(t3, c)
        assert torch.equal(d.loss, b.loss)
    return a, b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,K,pad,shift,T,lse,weighted", [
    (1, 1, 1, 0, 0, 1.0, False, False), (2, 5, 9, 0, 0, 1.0, False, True), (3, 17, 4, 6, 5, 2.0, True, True),
    (4, 1000, 16, 0, 0, 0.5, False, True), (7, 4099, 100, 3, 1, 1.0, True, False),
    (8, 32000, 16, 0, 0, 1.0, False, True), (3, 50257, 1024, 1, 0, 3.0, False, True),
    (1030, 1003, 33, 0, 0, 1.0, False, True), (1100, 515, 8, 5, 3, 1.5, True, True),
    (2, 151936, 64, 0, 0, 1.0, False, True), (1026, 8200, 5, 0, 0, 1.0, False, False),
    # rows held in registers, of each size, one and several to a workgroup; the last
    # is too long for that in float32
    (5, 90001, 40, 0, 0, 1.0, True, True), (3, 45001, 7, 2, 1, 0.7, False, False),
    (530, 20011, 9, 0, 0, 1.0, False, True), (270, 82001, 12, 3, 1, 2.0, True, True),
    (260, 80001, 6, 0, 0, 1.0, False, True),
])
def test_distill(dtype, R, V, K, pad, shift, T, lse, weighted):
    rng = np.random.default_rng(R + 31 * V + K)
    t, z = _rows(rng, R, V, dtype, pad, shift)
    ids, values = _teacher(rng, z, K)
    L = None
    if lse:   # the kept tokens hold nine tenths of the teacher's mass
        m, ls = ot.log_sum_exp(np.where(ids >= 0, values.astype(np.float64) / T, -np.inf))
        L = (m + ls + np.log(1 / 0.9)).astype(np.float32)
    w = rng.uniform(0.1, 2, R).astype(np.float32) if weighted else None
    _check_distill(t, z, ids, values, T, L, w, dtype, in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("copies,V", [(1, 9001), (200, 9001), (1, 20011), (80, 20011), (12, 82001)])
def test_distill_edges(dtype, copies, V):
    """Masked tokens, empty slots, repeated ids, rows that leave nothing; copies
    gives both one workgroup and several to a row, the longer rows are held in registers
    (the longest in bfloat16)."""
    rng = np.random.default_rng(9)
    K = 6
    z = (rng.standard_normal((8, V)) * 3).astype(np.float32)
    low = np.float32(-3.3895313892515355e38)
    ids = rng.integers(0, V, (8, K))
    values = (rng.standard_normal((8, K)) * 2).astype(np.float32)
    z[0, rng.random(V) < 0.5] = -np.inf
    z[0, ids[0]] = 1.0
    ids[1] = [4, 4, 9000, 4, 0, 9000]                 # masses add up
    ids[2] = [-1, V, 2 ** 31 - 1, -5, 7, 8]            # two filled slots
    ids[3] = -1                                        # nothing to learn from
    values[4, :4] = -np.inf                            # slots without mass
    z[5, :] = low                                      # uniform
    z[6, rng.random(V) < 0.9] = low
    z[7, :] = -np.inf                                  # no token possible, nothing kept
    ids[7] = -1
    z, ids, values = (np.repeat(x, copies, 0) for x in (z, ids, values))
    t = _dev(z, dtype)
    a, b = _check_distill(t, _host(t), ids, values, 0.8, None, None, dtype, in_place=True)
    assert np.all(_host(a.loss)[3 * copies: 4 * copies] == 0) and not b.grad[3 * copies: 4 * copies].any()


@pytest.mark.parametrize("copies,V", [(1, 9001), (300, 9001), (1, 20011), (150, 20011)])
def test_distill_impossible_tokens(copies, V):
    """A kept token the student rules out: loss +inf, a finite gradient; a row of -inf
    with a filled slot: loss +inf, no gradient; NaN stays in its row."""
    import torch
    rng = np.random.default_rng(10)
    z = (rng.standard_normal((4, V)) * 3).astype(np.float32)
    ids = np.array([[5, 6], [5, 6], [5, 6], [5, 6]], np.int32)
    values = np.ones((4, 2), np.float32)
    z[0, 5] = -np.inf
    z[1, :] = -np.inf
    z[2, 8000] = np.nan
    z, ids, values = (np.repeat(x, copies, 0) for x in (z, ids, values))
    for dtype in ("bf16", "f32"):
        t = _dev(z, dtype)
        out = _sv().spec_verify_distill(t, _dev(ids), _dev(values), want_grad=True)
        torch.cuda.synchronize()
        loss, grad = _host(out.loss), _host(out.grad)
        ref = ot.distill(_host(t)[:copies], ids[:copies], values[:copies])
        assert np.all(np.isposinf(loss[: 2 * copies])) and np.all(np.isnan(loss[2 * copies: 3 * copies]))
        assert np.all(np.isfinite(loss[3 * copies:]))
        assert np.abs(grad[:copies] - ref[1]).max() <= HALF[dtype] + 1e-4
        assert not grad[copies: 2 * copies].any() and np.isnan(grad[2 * copies: 3 * copies]).all()
        assert np.isfinite(grad[3 * copies:]).all()


@pytest.mark.parametrize("R,V", [(2, 20003), (1200, 301)])
def test_distill_gradient_columns_behind_the_row_stay(R, V):
    import torch
    sv, rng = _sv(), np.random.default_rng(11)
    t, z = _rows(rng, R, V, "bf16", 13, 6)
    ids, values = _teacher(rng, z, 12)
    wide = torch.full((R, V + 21), 7.0, dtype=torch.bfloat16, device="cuda:0")
    plain = sv.spec_verify_distill(t, _dev(ids), _dev(values), want_grad=True)
    for at in (0, 3, 6):   # as the input is aligned, and not
        wide.fill_(7.0)
        sv.spec_verify_distill_backward(t, _dev(ids), _dev(values), plain.stats, out=wide[:, at: at + V])
        torch.cuda.synchronize()
        assert torch.equal(wide[:, at: at + V], plain.grad)
        assert bool((wide[:, :at] == 7).all()) and bool((wide[:, at + V:] == 7).all())


def test_distill_gradient_against_differences():
    """The loss between z + h u and z - h u, along a random direction u of unit size."""
    import torch
    sv, rng = _sv(), np.random.default_rng(12)
    R, V, K, h = 3, 700, 20, 0.05
    z = rng.standard_normal((R, V)).astype(np.float32)
    ids, values = _teacher(rng, z, K)
    u = rng.standard_normal((R, V)).astype(np.float32)
    u /= np.linalg.norm(u, axis=1, keepdims=True)
    di, dv = _dev(ids), _dev(values)
    grad = _host(sv.spec_verify_distill(_dev(z), di, dv, want_grad=True).grad)
    up, down = ((z + s * h * u).astype(np.float32) for s in (1, -1))
    loss = [_host(sv.spec_verify_distill(_dev(x), di, dv).loss) for x in (up, down)]
    torch.cuda.synchronize()
    step = (up.astype(np.float64) - down)   # the directions as rounded
    slope = loss[0] - loss[1]
    # the third derivative along u is a third central moment of u under q, at most
    # (2 max |u|)^3; each loss has its own rounding
    third = (2 * np.abs(u).max(1) * h) ** 3 / 3
    tol = third + sum(_distill_tol(x.astype(np.float64), ids, values, 1.0, ot.distill(x, ids, values), "f32",
                                   None)[0] for x in (up, down))
    assert np.all(np.abs(slope - (grad * step).sum(1)) <= tol)
    assert np.abs(slope).max() > 2 * tol.max()   # a missing or doubled slope would show


# ---------------------------------------------------------------- linear cross entropy

def _head(rng, N, D, V, dtype, pad=0):
    w = _dev((rng.standard_normal((V, D + pad)) * 2 / np.sqrt(D)).astype(np.float32), dtype)[:, pad: pad + D]
    y = rng.integers(0, V, N)
    lean = (rng.random(N) < 0.6)[:, None] * 2.0
    h = rng.standard_normal((N, D + pad)).astype(np.float32)
    h[:, pad:] += (lean * _host(w)[y]).astype(np.float32)
    h = _dev(h, dtype)[:, pad:]
    y[rng.random(N) < 0.15] = -100
    return h, w, y.astype(np.int32)


def _ce_tol(h, w, z, dz, g, loss, dtype):
    """Bounds of loss, grad_hidden, grad_weight. A logit sums D exact products (float32:
    six part products each, and what is dropped is below 2^-22 of a product); its
    partial sums are below S = sum |h w|, and roundings of random sign add up to
    at most 8 sqrt(n) U S (eight standard deviations; n sums of them)."""
    N, D = h.shape
    V = w.shape[0]
    parts = 1 if dtype == "bf16" else 6
    S = (np.abs(h) @ np.abs(w).T).max(1)
    zt = 8 * np.sqrt(D * parts) * U * S + (0 if dtype == "bf16" else 2.0 ** -22) * S
    m, ls = ot.log_sum_exp(z)
    A = np.abs(z).max(1) + 30
    rel = 2 * zt + 8 * U * A + _sum_tol(V)       # of a probability
    lt = rel + 4 * U * np.abs(loss)
    gg = np.abs(g)
    q = np.exp(z - (m + ls)[:, None])
    # dz: its own error, and its rounding to bf16 (float32: three parts, 2^-24)
    dt = gg[:, None] * rel[:, None] * q + (HALF["bf16"] if dtype == "bf16" else 2 * U) * np.abs(dz) \
        + 4 * U * gg[:, None] * (np.abs(dz) > 0)
    out = HALF[dtype]

    def product(x, xt, y):
        full = np.abs(x) @ np.abs(y)
        n = x.shape[1] * parts
        return xt @ np.abs(y) + (8 * np.sqrt(n) * U + 2.0 ** -21) * full + out * np.abs(x @ y) + 1e-37
    return lt, product(dz, dt, w), product(dz.T, dt.T, h)


def _check_ce(h, w, y, g, dtype, check=None):
    import torch
    sv = _sv()
    dy, dg = _dev(y), None if g is None else _dev(g)
    a = sv.spec_verify_linear_ce(h, w, dy)
    b = sv.spec_verify_linear_ce_backward(h, w, dy, a.stats, dg)
    c = sv.spec_verify_linear_ce_backward(h, w, dy, a.stats, dg, want_weight=False)
    d = sv.spec_verify_linear_ce_backward(h, w, dy, a.stats, dg, want_hidden=False)
    torch.cuda.synchronize()
    assert c.weight is None and d.hidden is None
    hh, ww = _host(h), _host(w)
    loss, gh, gw, z, dz = ot.linear_ce(hh, ww, y, g)
    used = (y >= 0) & (y < ww.shape[0])
    gg = np.where(used, 1.0 if g is None else g, 0.0)
    lt, ht, wt = _ce_tol(hh, ww, z, dz, gg, loss, dtype)
    far = np.abs(_host(a.loss) - loss)
    assert np.all(far <= lt), (far.max(), lt.min())
    assert np.all(_host(a.loss)[~used] == 0)
    m, ls = ot.log_sum_exp(z)
    assert np.all(np.abs(_host(a.stats).sum(1) - m - ls) <= lt + 4 * U * np.abs(m + ls))
    for got in (b.hidden, c.hidden):
        far = np.abs(_host(got) - gh) - ht
        assert np.all(far <= 0), ("hidden", far.max(), np.argwhere(far > 0)[:4])
        assert np.all(_host(got)[~used] == 0)
    for got in (b.weight, d.weight):
        far = np.abs(_host(got) - gw) - wt
        assert np.all(far <= 0), ("weight", far.max(), np.argwhere(far > 0)[:4])
    return a, b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,V,pad", [
    (1, 1, 1, 0), (1, 64, 300, 0), (3, 7, 5, 0), (17, 128, 1000, 0), (32, 64, 257, 0), (33, 100, 1001, 0),
    (65, 192, 2500, 8), (100, 65, 513, 3), (129, 320, 4100, 0), (200, 64, 127, 64), (300, 96, 1536, 0),
    (513, 128, 700, 0), (31, 1000, 2049, 0),
])
def test_linear_ce(dtype, N, D, V, pad):
    rng = np.random.default_rng(N * 131 + D + V)
    h, w, y = _head(rng, N, D, V, dtype, pad)
    _check_ce(h, w, y, rng.uniform(0.2, 2.0, N).astype(np.float32) / N, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_ce_several_pieces(dtype):
    """A vocabulary longer than one piece of the backward pass, with a short last piece."""
    rng = np.random.default_rng(21)
    sv = _sv()
    N, D, V = 40, 64, (1 << 20) + 777
    small = sv.spec_verify_linear_ce_backward_workspace_bytes(N, D, V, sv.SV_BF16)
    assert small < 2 * V * D * 2 * 3   # not the whole head at once
    h, w, y = _head(rng, N, D, V, dtype)
    y[:3] = [V - 1, 1 << 20, (1 << 20) - 1]
    _check_ce(h, w, y, np.full(N, 1 / N, np.float32), dtype)


@pytest.mark.parametrize("N,D,V", [(385, 65, 129), (450, 200, 100), (400, 300, 1003), (700, 129, 257), (385, 7, 64)])
def test_linear_ce_float32_in_parts(N, D, V):
    """float32 with more states than the float32 instructions take, around its tiles."""
    rng = np.random.default_rng(N + D + V)
    h, w, y = _head(rng, N, D, V, "f32")
    _check_ce(h, w, y, rng.uniform(0.2, 2.0, N).astype(np.float32) / N, "f32")


def test_linear_ce_float32_short_last_piece():
    """A last piece of 100 tokens: lower than a tile of the pieces before it."""
    rng = np.random.default_rng(26)
    N, D, V = 385, 4000, 16384 + 100
    h, w, y = _head(rng, N, D, V, "f32")
    y[:4] = [V - 1, 16384, 16383, V - 36]
    _check_ce(h, w, y, np.full(N, 1 / N, np.float32), "f32")


def test_linear_ce_labels():
    """Left-out rows of every kind, the same label everywhere, no weights."""
    rng = np.random.default_rng(22)
    h, w, _ = _head(rng, 70, 64, 500, "bf16")
    y = np.full(70, 499, np.int32)
    _check_ce(h, w, y, None, "bf16")
    y[::2] = [-100, -1, 500, 2 ** 31 - 1, -2 ** 31] * 7
    _check_ce(h, w, y, None, "bf16")
    y[:] = -100
    _, b = _check_ce(h, w, y, None, "bf16")
    assert not b.hidden.any() and not b.weight.any()


def test_linear_ce_confident_and_far_logits():
    """Logits of a few hundred: probabilities of exactly one and zero."""
    rng = np.random.default_rng(23)
    for dtype in ("bf16", "f32"):
        h, w, y = _head(rng, 40, 64, 300, dtype)
        _check_ce(h * 32, w * 4, y, None, dtype)


def test_linear_ce_strided_outputs():
    import torch
    sv, rng = _sv(), np.random.default_rng(24)
    for dtype in ("bf16", "f32"):
        N, D, V = 37, 72, 600
        h, w, y = _head(rng, N, D, V, dtype, 5)
        dy = _dev(y)
        st = sv.spec_verify_linear_ce(h, w, dy).stats
        want = sv.spec_verify_linear_ce_backward(h, w, dy, st)
        gh = torch.full((N, D + 9), 3.0, dtype=h.dtype, device="cuda:0")
        gw = torch.full((V, D + 7), 3.0, dtype=h.dtype, device="cuda:0")
        sv.spec_verify_linear_ce_backward(h, w, dy, st, out=sv.LinearCeGrads(gh[:, 4: 4 + D], gw[:, 1: 1 + D]))
        torch.cuda.synchronize()
        assert torch.equal(gh[:, 4: 4 + D], want.hidden) and torch.equal(gw[:, 1: 1 + D], want.weight)
        assert bool((gh[:, :4] == 3).all()) and bool((gh[:, 4 + D:] == 3).all())
        assert bool((gw[:, :1] == 3).all()) and bool((gw[:, 1 + D:] == 3).all())


def test_linear_ce_gradient_against_differences():
    """As for the distillation: along u in the states, and along v in the head."""
    import torch
    sv, rng = _sv(), np.random.default_rng(25)
    N, D, V, eps = 5, 64, 300, 0.02
    h, w, y = _head(rng, N, D, V, "f32")
    dy = _dev(y)
    a = sv.spec_verify_linear_ce(h, w, dy)
    g = sv.spec_verify_linear_ce_backward(h, w, dy, a.stats)
    for x, grad in ((h, g.hidden), (w, g.weight)):
        u = _dev(rng.standard_normal(x.shape).astype(np.float32))
        u = u / u.norm()
        up, down = x + eps * u, x - eps * u
        pair = [(up, w) if x is h else (h, up), (down, w) if x is h else (h, down)]
        loss = [_host(sv.spec_verify_linear_ce(*p, dy).loss).sum() for p in pair]
        torch.cuda.synchronize()
        slope = loss[0] - loss[1]
        want = (_host(grad) * (_host(up) - _host(down))).sum()
        # a logit moves by at most eps |other factor| along u
        move = eps * max(_host(h if x is w else w).__abs__().max() * np.sqrt(D), 1e-3)
        tol = N * move ** 3 / 3 + 2 * N * 2e-5
        assert abs(slope - want) <= tol, (slope, want, tol)


# ---------------------------------------------------------------- offsets beyond 32 bits

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_further_apart_than_32_bits(dtype):
    """Three rows 2^32 + 24 bytes apart, and gradients that are as far apart."""
    import torch
    sv, rng = _sv(), np.random.default_rng(40)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    step, R, V, K, D = ((1 << 32) + 24) // dt.itemsize, 3, 20003, 40, 72

    def far(near):
        flat = torch.empty(2 * step + near.shape[1], dtype=dt, device="cuda:0")
        t = flat.as_strided(near.shape, (step, 1))
        t.copy_(near)
        return t

    z, _ = _rows(rng, R, V, dtype)
    zf = far(z)
    a, b = sv.spec_verify_top_logits(z, K), sv.spec_verify_top_logits(zf, K)
    ids, vals = _teacher(rng, _host(z), K)
    args = (_dev(ids), _dev(vals))
    c = sv.spec_verify_distill(z, *args, want_grad=True)
    d = sv.spec_verify_distill(zf, *args, out=sv.DistillOut(
        torch.empty_like(c.loss), torch.empty_like(c.stats), far(torch.zeros_like(z))))
    torch.cuda.synchronize()
    assert torch.equal(a.ids, b.ids) and torch.equal(a.values, b.values)
    # rows that start elsewhere in a group of 16 bytes are summed in another order
    assert ((a.lse - b.lse).abs() <= 2 * _sum_tol(V) + 4 * U * a.lse.abs()).all()
    ref = ot.distill(_host(z), ids, vals)
    lt, gt = _distill_tol(_host(z), ids, vals, 1.0, ref, dtype, None)
    assert np.all(np.abs(_host(d.loss) - ref[0]) <= lt) and np.all(np.abs(_host(d.grad) - ref[1]) <= gt)
    del zf, b, d
    h, w, y = _head(rng, R, D, 3, dtype)
    y[:] = [2, 0, 1]
    hf, wf = far(h), far(w)
    e = sv.spec_verify_linear_ce(hf, wf, _dev(y))
    out = sv.LinearCeGrads(far(torch.zeros_like(h)), far(torch.zeros_like(w)))
    f = sv.spec_verify_linear_ce_backward(hf, wf, _dev(y), e.stats, out=out)
    torch.cuda.synchronize()
    loss, gh, gw, zz, dz = ot.linear_ce(_host(h), _host(w), y)
    tol = _ce_tol(_host(h), _host(w), zz, dz, np.ones(R), loss, dtype)
    for got, want, t in ((e.loss, loss, tol[0]), (f.hidden, gh, tol[1]), (f.weight, gw, tol[2])):
        assert np.all(np.abs(_host(got) - want) <= t)


def test_more_rows_than_an_int32_are_refused():
    """2^32 + 5 rows of one column must not pass as five."""
    import torch
    t = torch.empty(((1 << 32) + 5, 1), dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ValueError):
        _sv().spec_verify_top_logits(t, 1)
    with pytest.raises(ValueError):
        _sv().spec_verify_linear_ce(t, t[:4], torch.zeros(5, dtype=torch.int32, device="cuda:0"))


# ---------------------------------------------------------------- together, streams, graphs

def test_verification_then_distillation_then_the_head():
    """One round as a drafter's training uses it: verify, record the target's top
    logits from the same rows, distil the drafter's rows against them, and take the
    cross entropy of its head at the tokens that were emitted."""
    import torch
    sv, rng = _sv(), np.random.default_rng(30)
    B, G, V, D, K = 6, 4, 5003, 96, 32
    h, w, _ = _head(rng, B * G, D, V, "bf16")
    draft = (h.float() @ w.float().t()).to(torch.bfloat16).view(B, G, V)
    target = torch.cat([draft, draft[:, :1]], 1) + _dev(
        rng.standard_normal((B, G + 1, V)).astype(np.float32)).to(torch.bfloat16)
    xs = torch.argmax(draft.float(), 2).to(torch.int32)
    out = sv.spec_verify_sample(target, draft, xs, seed=3)
    top = sv.spec_verify_top_logits(target, K)
    t_ids, t_vals, t_lse = (x[:, :G].contiguous() for x in top)
    dis = sv.spec_verify_distill(draft, t_ids, t_vals, teacher_lse=t_lse, want_grad=True)
    labels = out.tokens[:, :G].contiguous()     # -1 behind the emitted tokens: left out
    ce = sv.spec_verify_linear_ce(h.view(B, G, D), w, labels)
    grads = sv.spec_verify_linear_ce_backward(h.view(B, G, D), w, labels, ce.stats)
    torch.cuda.synchronize()
    rt = ot.top_logits(_host(target).reshape(-1, V), K)
    assert np.array_equal(top.ids.cpu().numpy().reshape(-1, K), rt[0])
    assert torch.all((top.lse - out.target_lse).abs() <= 1e-4)   # the verifier's own normaliser
    z = _host(draft).reshape(-1, V)
    L = t_lse.cpu().numpy().reshape(-1)
    ids, vals = t_ids.cpu().numpy().reshape(-1, K), t_vals.cpu().numpy().reshape(-1, K)
    ref = ot.distill(z, ids, vals, 1.0, L)
    lt, gt = _distill_tol(z, ids, vals, 1.0, ref, "bf16", None)
    assert np.all(np.abs(_host(dis.loss).reshape(-1) - ref[0]) <= lt)
    assert np.all(np.abs(_host(dis.grad).reshape(-1, V) - ref[1]) <= gt)
    y = labels.cpu().numpy().reshape(-1)
    loss, gh, gw, zz, dz = ot.linear_ce(_host(h), _host(w), y)
    ct = _ce_tol(_host(h), _host(w), zz, dz, (y >= 0) * 1.0, loss, "bf16")
    assert np.all(np.abs(_host(ce.loss).reshape(-1) - loss) <= ct[0])
    assert np.all(np.abs(_host(grads.hidden).reshape(-1, D) - gh) <= ct[1])
    assert np.all(np.abs(_host(grads.weight) - gw) <= ct[2])


def _all_calls(z, ids, vals, h, w, y, spaces):
    sv = _sv()
    top = sv.spec_verify_top_logits(z, 20, workspace=spaces and spaces[0])
    dis = sv.spec_verify_distill(z, ids, vals, want_grad=True, workspace=spaces and spaces[1])
    ce = sv.spec_verify_linear_ce(h, w, y, workspace=spaces and spaces[2])
    gr = sv.spec_verify_linear_ce_backward(h, w, y, ce.stats, workspace=spaces and spaces[3])
    return [*top, *dis, *ce, *gr]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_streams_repeats_and_graph_replays(dtype):
    """Another stream, dirty workspaces, and a captured round replayed on new inputs:
    the same bits every time."""
    import torch
    sv, rng = _sv(), np.random.default_rng(31)
    N, D, V = 50, 100, 20011
    t, z = _rows(rng, 5, V, dtype)
    t2, z2 = _rows(rng, 5, V, dtype)
    h, w, y = _head(rng, N, D, V, dtype)
    h2, _, y2 = _head(rng, N, D, V, dtype)
    ids, vals = _teacher(rng, z, 20)
    static = [t.clone(), _dev(ids), _dev(vals), h.clone(), w, _dev(y)]
    code = sv._dtype_code(h)
    need = [sv.spec_verify_top_logits_workspace_bytes(5, V, 20, code),
            sv.spec_verify_distill_workspace_bytes(5, V, code),
            sv.spec_verify_linear_ce_workspace_bytes(N, D, V, code),
            sv.spec_verify_linear_ce_backward_workspace_bytes(N, D, V, code)]
    spaces = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda:0") for n in need]
    first = [x.clone() for x in _all_calls(*static, None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _all_calls(*static, spaces)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all_calls(*static, spaces)
    for turn in range(3):
        new = (t2, h2, y2) if turn == 1 else (t, h, y)
        static[0].copy_(new[0])
        static[3].copy_(new[1])
        static[5].copy_(_dev(new[2]))
        for s in spaces:
            s.fill_(turn * 85)
        want = [x.clone() for x in _all_calls(*static, None)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), turn


def test_explicit_stream_argument():
    import torch
    sv, rng = _sv(), np.random.default_rng(32)
    t, z = _rows(rng, 4, 30011, "bf16")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = sv.spec_verify_top_logits(t, 9, stream=side)
    b = sv.spec_verify_top_logits(t, 9, stream=side.cuda_stream)
    side.synchronize()
    c = sv.spec_verify_top_logits(t, 9)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) and torch.equal(x, w) for x, y, w in zip(a, b, c))


def test_binding_refusals_on_device_tensors():
    import torch
    sv = _sv()
    z = torch.zeros(4, 64, device="cuda:0")
    ids = torch.zeros(4, 3, dtype=torch.int32, device="cuda:0")
    vals = torch.zeros(4, 3, device="cuda:0")
    y = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    w = torch.zeros(10, 64, device="cuda:0")
    bad = [
        (TypeError, lambda: sv.spec_verify_top_logits(z.half(), 3)),
        (ValueError, lambda: sv.spec_verify_top_logits(z.t(), 3)),
        (ValueError, lambda: sv.spec_verify_top_logits(z[:, ::2], 3)),
        (ValueError, lambda: sv.spec_verify_top_logits(z[:1].expand(4, 64), 3)),
        (ValueError, lambda: sv.spec_verify_top_logits(z[:0], 3)),
        (sv.SpecVerifyError, lambda: sv.spec_verify_top_logits(z, 65)),
        (sv.SpecVerifyError, lambda: sv.spec_verify_top_logits(z, 0)),
        (sv.SpecVerifyError, lambda: sv.spec_verify_top_logits(z, 3, temperature=0.0)),
        (ValueError, lambda: sv.spec_verify_distill(z, ids[:3], vals)),
        (ValueError, lambda: sv.spec_verify_distill(z, ids, None)),
        (ValueError, lambda: sv.spec_verify_distill(z, None, vals)),
        (ValueError, lambda: sv.spec_verify_distill(z, ids, vals[:, :2])),
        (TypeError, lambda: sv.spec_verify_distill(z, ids.long(), vals)),
        (ValueError, lambda: sv.spec_verify_distill(z, ids, vals, row_weight=vals)),
        (ValueError, lambda: sv.spec_verify_distill_backward(z, ids, vals, None)),
        (TypeError, lambda: sv.spec_verify_distill_backward(z, ids, vals, torch.zeros(4, 2, device="cuda:0"),
                                                            out=z.bfloat16())),
        (TypeError, lambda: sv.spec_verify_linear_ce(z, w.bfloat16(), y)),
        (ValueError, lambda: sv.spec_verify_linear_ce(z, w[:, :32], y)),
        (ValueError, lambda: sv.spec_verify_linear_ce(z, w, y[:2])),
        (sv.SpecVerifyError, lambda: sv.spec_verify_linear_ce_backward(
            z, w, y, torch.zeros(4, 2, device="cuda:0"), want_hidden=False, want_weight=False)),
        (sv.SpecVerifyError, lambda: sv.spec_verify_linear_ce(
            z, w, y, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda:0"))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
