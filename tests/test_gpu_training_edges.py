"""Edges of the drafter-training kernels, against their float64 forms: what the
gradients keep of dz, finite masks, rows of NaN. Tolerances count roundings as in
tests/test_gpu_training.py (U: half a step of float32)."""

import numpy as np
import pytest

from oracle import training as ot
from tests.test_gpu_training import HALF, U, _dev, _distill_tol, _head, _host, _lse_tol, _sum_tol, _sv

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


@pytest.mark.parametrize("N,D,V,pad,dtype", [(5, 4096, 40003, 3, "bf16"), (40, 2048, 40003, 1, "f32"),
                                             (150, 4096, 20100, 5, "bf16")])
def test_linear_ce_wide_heads_at_odd_strides(N, D, V, pad, dtype):
    """A head that is read in place but for its stride is packed in several pieces, the
    last of them short."""
    from tests.test_gpu_training import _check_ce
    rng = np.random.default_rng(N + D)
    h, w, y = _head(rng, N, D, V, dtype, pad)
    y[:4] = [V - 1, 16384, 16383, V - 100]
    _check_ce(h, w, y, np.full(N, 1 / N, np.float32), dtype)


@pytest.mark.parametrize("N,D,V,pad,border", [
    (129, 4096, 65636, 0, 65536), (129, 4095, 65636, 0, 65536),      # in place; packed, forward too
    (1030, 136, 52324, 0, 52224), (1030, 161, 52324, 0, 52224),      # several splits of dh
    (1030, 136, 52224 + 129, 3, 52224), (2050, 64, 28772, 0, 28672)])
def test_linear_ce_large_tiles_over_two_pieces(N, D, V, pad, border):
    """bfloat16 in the largest tile: dh added up over pieces of the vocabulary, the last of
    them of few tokens, with labels on both sides of the border. Exact values by float64
    products on the device; bounds as in _gradient_tol."""
    import torch
    sv, rng = _sv(), np.random.default_rng(N + D)
    h, w, y = _head(rng, N, D, V, "bf16", pad)
    y[:6] = [border - 1, border, border + 1, V - 1, 0, border]
    y, g = _dev(y), _dev(rng.uniform(0.2, 2.0, N).astype(np.float32) / N)
    a = sv.spec_verify_linear_ce(h, w, y)
    b = sv.spec_verify_linear_ce_backward(h, w, y, a.stats, g)
    torch.cuda.synchronize()
    hh, ww = h.double(), w.double()
    z = torch.mm(hh, ww.t().contiguous())
    m = z.amax(1)
    ls = torch.log(torch.exp(z - m[:, None]).sum(1))
    used = (y >= 0) & (y < V)
    at = torch.where(used, y, 0).long()[:, None]
    loss = torch.where(used, m + ls - z.gather(1, at)[:, 0], 0.0)
    zt = 8 * D ** 0.5 * U * torch.mm(hh.abs(), ww.abs().t().contiguous()).amax(1)
    rel = 2 * zt + 8 * U * (z.abs().amax(1) + 30) + _sum_tol(V)
    assert ((a.loss.double() - loss).abs() <= rel + 4 * U * loss.abs()).all()
    q = torch.exp(z - (m + ls)[:, None])
    gg = torch.where(used, g.double(), 0.0)[:, None]
    dz = q.scatter_add(1, at, torch.full((N, 1), -1.0, dtype=torch.float64, device=z.device)) * gg
    dt = gg * (rel[:, None] * q + 4 * U * (dz != 0)) + 2.0 ** -16 * dz.abs()
    del z, q
    for got, x, xt, other in ((b.hidden, dz, dt, ww), (b.weight, dz.t().contiguous(), dt.t().contiguous(), hh)):
        want = torch.mm(x, other)
        tol = (torch.mm(xt, other.abs()) + 8 * (2 * x.shape[1]) ** 0.5 * U * torch.mm(x.abs(), other.abs())
               + HALF["bf16"] * want.abs() + 1e-37)
        far = (got.double() - want).abs() - tol
        assert bool((far <= 0).all()), (far.max().item(), torch.nonzero(far > 0)[:4].tolist())


# ---------------------------------------------------------------- finite masks


def _masked(rng, V, fill):
    """Rows with a block of `fill` first, in the middle, last, and everywhere."""
    z = (rng.standard_normal((5, V)) * 3).astype(np.float32)
    z[0, : V // 2] = fill
    z[1, V // 3: V // 2] = fill
    z[2, V // 2:] = fill
    z[3] = fill
    z[4] = np.where(rng.random(V) < 0.9, fill, z[4])
    return z


MASKS = (-1e9, -1e10, -6e10, -1e12, -1e15, -1e20, -1e25, -1e30, 1e10, 1e20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("copies,V,T", [
    (1, 9001, 1.0), (120, 9001, 0.7), (1, 50003, 0.8), (20, 50003, 1.0), (1, 160001, 1.0)])
def test_top_logits_of_finite_masks(dtype, copies, V, T):
    """One workgroup to a row and several; masks of every size that the exponents'
    reference may be taken at."""
    import torch
    rng = np.random.default_rng(V + copies)
    z = np.concatenate([_masked(rng, V, f) for f in MASKS])
    t = _dev(z, dtype)
    want = ot.top_logits(_host(t), 5, T)
    out = _sv().spec_verify_top_logits(t.repeat(copies, 1), 5, temperature=T)
    torch.cuda.synchronize()
    tol = _lse_tol(V, want[2])
    for k in range(0, len(z) * copies, len(z)):
        assert np.array_equal(out.ids[k: k + len(z)].cpu().numpy(), want[0])
        far = np.abs(_host(out.lse[k: k + len(z)]) - want[2])
        assert np.all(far <= tol), (np.argwhere(~(far <= tol)).ravel(), far)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e-5, 1e-8, 1e-9, 1e-20, 1e-30])
def test_top_logits_at_small_temperatures(dtype, T):
    import torch
    rng = np.random.default_rng(3)
    z = np.concatenate([(rng.standard_normal((4, 20011)) * s) for s in (1.0, 10.0, 60.0, T, 30 * T)]).astype(np.float32)
    t = _dev(z, dtype)
    T = float(np.float32(T))
    lse = ot.top_logits(_host(t), 1, T)[2]
    for copies in (1, 80):
        out = _sv().spec_verify_top_logits(t.repeat(copies, 1), 1, temperature=T)
        torch.cuda.synchronize()
        far = np.abs(_host(out.lse).reshape(copies, -1) - lse)
        assert np.all(far <= _lse_tol(20011, lse)), far.max(0)


def _distill_case(rng, z, T, K=6):
    """Kept tokens among the row's, the rest of the teacher near them."""
    ids = np.stack([rng.choice(z.shape[1], K, replace=False) for _ in z]).astype(np.int32)
    return ids, (rng.standard_normal(ids.shape) * 2 * min(T, 1.0)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("copies,V", [(1, 9001), (120, 9001), (1, 30011), (20, 30011), (3, 82001), (1, 160001)])
def test_distill_loss_of_finite_masks(dtype, copies, V):
    """Streamed, split and (with the gradient) held rows."""
    import torch
    sv, rng = _sv(), np.random.default_rng(V + copies)
    for T in (1.0, 0.7):
        z = np.concatenate([_masked(rng, V, f) for f in MASKS])
        t = _dev(z, dtype)
        z = _host(t)
        ids, values = _distill_case(rng, z, T)
        ref = ot.distill(z, ids, values, T)
        tol = _distill_tol(z, ids, values, T, ref, dtype, None)[0]
        args = t.repeat(copies, 1), _dev(ids).repeat(copies, 1), _dev(values).repeat(copies, 1)
        for out in (sv.spec_verify_distill(*args, temperature=T),
                    sv.spec_verify_distill(*args, temperature=T, want_grad=True)):
            torch.cuda.synchronize()
            far = np.abs(_host(out.loss).reshape(copies, -1) - ref[0])
            assert np.all(far <= tol), (np.argwhere(~(far <= tol))[:5], far.max(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e-5, 1e-8, 1e-9, 1e-20])
def test_distill_loss_at_small_temperatures(dtype, T):
    import torch
    sv, rng = _sv(), np.random.default_rng(4)
    z = np.concatenate([(rng.standard_normal((4, 20011)) * s) for s in (1.0, 60.0, T, 30 * T)]).astype(np.float32)
    t = _dev(z, dtype)
    z, T = _host(t), float(np.float32(T))
    ids, values = _distill_case(rng, z, T)
    ref = ot.distill(z, ids, values, T)
    tol = _distill_tol(z, ids, values, T, ref, dtype, None)[0]
    for copies in (1, 40):
        args = t.repeat(copies, 1), _dev(ids).repeat(copies, 1), _dev(values).repeat(copies, 1)
        for out in (sv.spec_verify_distill(*args, temperature=T),
                    sv.spec_verify_distill(*args, temperature=T, want_grad=True)):
            torch.cuda.synchronize()
            far = np.abs(_host(out.loss).reshape(copies, -1) - ref[0])
            assert np.all(far <= tol), (np.argwhere(~(far <= tol))[:5], far.max(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("copies,V,T", [
    (1, 9001, 1.0), (120, 9001, 0.7), (1, 30011, 1.0), (20, 30011, 0.7), (1, 30011, 1e-5), (1, 30011, 1e-9),
    (3, 82001, 1.0), (1, 160001, 1.0), (120, 9001, 1e-9)])
def test_distill_gradient_of_finite_masks_and_small_temperatures(dtype, copies, V, T):
    """With the loss, and alone from its statistics."""
    import torch
    sv, rng = _sv(), np.random.default_rng(V + copies)
    T = float(np.float32(T))
    z = np.concatenate([_masked(rng, V, f) for f in MASKS] + [np.float32(T) * _masked(rng, V, -50.0)])
    t = _dev(z, dtype)
    z = _host(t)
    ids, values = _distill_case(rng, z, T)
    w = np.full(len(z), T, np.float32)   # a gradient of ordinary size
    ref = ot.distill(z, ids, values, T, None, w)
    tol = _distill_tol(z, ids, values, T, ref, dtype, w)[1]
    args = t.repeat(copies, 1), _dev(ids).repeat(copies, 1), _dev(values).repeat(copies, 1)
    dw = _dev(w).repeat(copies)
    a = sv.spec_verify_distill(*args, temperature=T, row_weight=dw, want_grad=True)
    b = sv.spec_verify_distill_backward(*args, a.stats, dw, temperature=T)
    torch.cuda.synchronize()
    for grad in (a.grad, b):
        for k in range(copies):
            far = np.abs(_host(grad[k * len(z): (k + 1) * len(z)]) - ref[1])
            assert np.all(far <= tol), (k, np.argwhere(~(far <= tol))[:5], np.nanmax(far - tol))


# ---------------------------------------------------------------- rows of NaN, teachers of the lowest value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("copies,V", [(1, 9001), (300, 9001), (1, 20011), (150, 20011), (3, 82001), (1, 160001)])
def test_distill_rows_of_nan_are_not_empty_rows(dtype, copies, V):
    """NaN makes a row's loss and gradient NaN also where no other logit is above -inf."""
    import torch
    sv = _sv()
    z = np.full((5, V), -np.inf, np.float32)
    z[0] = np.nan
    z[1, V // 2] = np.nan                     # NaN among -inf
    z[2, 0] = z[2, V - 1] = np.nan
    ids = np.array([[5, 6]] * 5, np.int32)
    ids[4] = -1                               # nothing kept: 0 whatever the row holds
    z[4] = np.nan
    args = [_dev(np.repeat(x, copies, 0)) for x in (z, ids, np.ones((5, 2), np.float32))]
    args[0] = args[0].to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    only = sv.spec_verify_distill(*args)
    both = sv.spec_verify_distill(*args, want_grad=True)
    alone = sv.spec_verify_distill_backward(*args, both.stats)
    torch.cuda.synchronize()
    for loss in (only.loss, both.loss):
        x = loss.reshape(5, copies)
        assert x[:3].isnan().all() and bool((x[3] == np.inf).all()) and not x[4].any()
    for grad in (both.grad, alone):
        x = grad.reshape(5, copies, V)
        assert x[:3].isnan().all() and not x[3:].any()


# ---------------------------------------------------------------- teachers of the lowest value


def _check_far_teacher(copies, V, values, T, want_p):
    """Loss and gradients of student rows against teachers with these exact masses."""
    import torch
    sv, rng = _sv(), np.random.default_rng(6)
    R = len(values)
    z = (rng.standard_normal((R, V)) * 3).astype(np.float32)
    ids = np.array([[3, 9, 4000, V - 1]] * R, np.int32)
    # the same masses from ordinary teacher logits: the exact results, and their bounds
    with np.errstate(divide="ignore"):
        near = np.log(np.array(want_p)) * float(np.float32(T))
    ref = ot.distill(z, ids, near, float(np.float32(T)))
    assert np.allclose(ref[2], want_p, rtol=1e-14, atol=0)
    lt, gt = _distill_tol(z.astype(np.float64), ids, near.astype(np.float32), T, ref, "f32", None)
    args = [_dev(np.repeat(x, copies, 0)) for x in (z, ids, np.array(values, np.float32))]
    a = sv.spec_verify_distill(*args, temperature=T, want_grad=True)
    b = sv.spec_verify_distill(*args, temperature=T)
    g = sv.spec_verify_distill_backward(*args, b.stats, temperature=T)
    torch.cuda.synchronize()
    for loss in (a.loss, b.loss):
        assert np.all(np.abs(_host(loss).reshape(R, copies) - ref[0][:, None]) <= lt[:, None])
    for grad in (a.grad, g):
        assert np.all(np.abs(_host(grad).reshape(R, copies, V) - ref[1][:, None]) <= gt[:, None])


LOW = -3.3895313892515355e38
INF = float("inf")


@pytest.mark.parametrize("copies,V", [(1, 9001), (300, 9001), (1, 30011), (150, 30011)])
def test_distill_teachers_of_one_far_value_share_their_mass(copies, V):
    """Equal teacher logits are a quarter each whatever their size: their log-normaliser
    is not their value."""
    far = [-1e10, -1e16, -1e20, LOW, 3e38]
    _check_far_teacher(copies, V, [[x] * 4 for x in far] + [[-1e20, -INF, -INF, -1e20]], 1.0,
                       [[0.25] * 4] * len(far) + [[0.5, 0, 0, 0.5]])


@pytest.mark.parametrize("copies,V", [(1, 9001), (300, 9001), (1, 30011), (150, 30011)])
@pytest.mark.parametrize("T", [0.5, 1e-3])
def test_distill_teachers_beyond_the_tempered_range(copies, V, T):
    """A finite teacher logit keeps its slot also where its tempered value passes
    float32's range; next to an ordinary one it has no mass."""
    _check_far_teacher(copies, V, [[LOW] * 4, [LOW, T, LOW, T], [-INF, LOW, -INF, LOW]], T,
                       [[0.25] * 4, [0, 0.5, 0, 0.5], [0, 0.5, 0, 0.5]])


# ---------------------------------------------------------------- autograd


def test_outputs_have_no_graph_and_count_as_changed_in_place():
    """The calls are not recorded; a tensor they overwrite raises its version, so that a
    backward pass which saved it refuses to use it."""
    import torch
    sv, rng = _sv(), np.random.default_rng(1)
    ids, values = _dev(np.zeros((4, 3), np.int32)), _dev(np.ones((4, 3), np.float32))
    x = _dev(rng.standard_normal((4, 700)).astype(np.float32)).requires_grad_()
    w = _dev(rng.standard_normal((50, 700)).astype(np.float32)).requires_grad_()
    y = _dev(np.arange(4, dtype=np.int32))

    def saved():
        z = x.exp()                 # exp keeps its result for the backward pass
        return z, z.sum()

    z, total = saved()
    kept = sv.spec_verify_distill(z, ids, values, want_grad=True)
    assert not (kept.loss.requires_grad or kept.grad.requires_grad)
    total.backward()                # nothing was overwritten
    z, total = saved()
    sv.spec_verify_distill(z, ids, values, out=sv.DistillOut(kept.loss, kept.stats, z.detach()))
    with pytest.raises(RuntimeError, match="inplace"):
        total.backward()
    z, total = saved()
    sv.spec_verify_distill_backward(z, ids, values, kept.stats, out=z.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        total.backward()
    ce = sv.spec_verify_linear_ce(x, w, y)
    assert not ce.loss.requires_grad
    top = sv.spec_verify_top_logits(x, 3)
    assert not top.values.requires_grad
    outs = [torch.zeros(4, 700, device="cuda:0"), torch.zeros(50, 700, device="cuda:0")]
    sv.spec_verify_linear_ce_backward(x, w, y, ce.stats, out=sv.LinearCeGrads(*outs))
    sv.spec_verify_linear_ce(x, w, y, out=ce)
    sv.spec_verify_top_logits(x, 3, out=top)
    torch.cuda.synchronize()
    assert all(t._version == 1 for t in (*outs, *ce, *top))
    with torch.inference_mode():
        sv.spec_verify_linear_ce(x, w, y, out=sv.spec_verify_linear_ce(x, w, y))


# ---------------------------------------------------------------- two streams, replays of the larger tiles


@pytest.mark.parametrize("N,D,V,dtype", [(300, 264, 30000, "bf16"), (20, 100, 30011, "bf16"), (400, 136, 9001, "f32")])
def test_steps_on_two_streams_and_in_a_graph(N, D, V, dtype):
    """Steps that run at once on two streams, and a captured one replayed on new inputs with
    eager steps between: the bits of a step alone."""
    import torch
    sv, rng = _sv(), np.random.default_rng(N)
    sets = []
    for _ in range(2):
        h, w, y = _head(rng, N, D, V, dtype)
        sets.append((h, w, _dev(y)))

    def step(h, w, y):
        a = sv.spec_verify_linear_ce(h, w, y)
        return [*a, *sv.spec_verify_linear_ce_backward(h, w, y, a.stats)]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(*sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for out in got[k] for a, b in zip(out, want[k]))
    static = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for turn in (1, 0, 1):
        for a, b in zip(static, sets[turn]):
            a.copy_(b)
        eager = step(*static)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(out, want[turn], eager))


def test_top_logits_pass_over_negative_ties():
    """bfloat16 rows of one negative value take about as long as those of a positive one:
    once k of them are listed, those that come later are not. (Listed again and again they
    took twelve times as long.)"""
    import torch
    sv, times = _sv(), []
    for value in (2.5, -2.5):
        t = torch.full((1152, 151936), value, dtype=torch.bfloat16, device="cuda:0")
        runs = []
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            out = sv.spec_verify_top_logits(t, 64)
            b.record()
            torch.cuda.synchronize()
            runs.append(a.elapsed_time(b))
        times.append(sorted(runs)[3])
        assert torch.equal(out.ids, torch.arange(64, dtype=torch.int32, device="cuda:0").repeat(1152, 1))
    assert times[1] < 4 * times[0], times
