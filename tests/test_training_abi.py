"""Argument checks of the drafter-training calls, on the CPU: everything here is
refused before any launch."""

import ctypes
import os
import re

import pytest

from tests.conftest import ROOT

FAKE = 4096   # non-null, aligned; never dereferenced because validation fails first


@pytest.fixture(scope="module")
def lib():
    from lossless_draft_verification_sample_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from lossless_draft_verification_sample_amd import build
        build.build()
    return _lib.load()


def _top(lib, **kw):
    a = dict(z=FAKE, stride=1000, dtype=1, R=4, V=1000, K=8, T=1.0, ids=FAKE, values=FAKE, lse=None,
             ws=None, ws_bytes=0)
    a.update(kw)
    return lib.spec_verify_top_logits(a["z"], a["stride"], a["dtype"], a["R"], a["V"], a["K"], a["T"],
                                      a["ids"], a["values"], a["lse"], a["ws"], a["ws_bytes"], None)


def _distill(lib, backward=False, **kw):
    a = dict(z=FAKE, stride=40000, dtype=1, R=2, V=40000, ids=FAKE, t=FAKE, lse=None, K=8, T=1.0,
             weight=None, loss=FAKE, stats=FAKE, grad=FAKE, gstride=40000, ws=None, ws_bytes=0)
    a.update(kw)
    head = [a[k] for k in ("z", "stride", "dtype", "R", "V", "ids", "t", "lse", "K", "T")]
    if backward:
        return lib.spec_verify_distill_backward(*head, a["stats"], a["weight"], a["grad"],
                                                a["gstride"], None)
    return lib.spec_verify_distill(*head, a["weight"], a["loss"], a["stats"], a["grad"],
                                   a["gstride"], a["ws"], a["ws_bytes"], None)


def _ce(lib, backward=False, **kw):
    a = dict(h=FAKE, hs=64, w=FAKE, ws=64, dtype=1, y=FAKE, N=5, D=64, V=100, loss=FAKE, stats=FAKE,
             g=None, gh=FAKE, ghs=64, gw=FAKE, gws=64, space=None, bytes=0)
    a.update(kw)
    head = [a[k] for k in ("h", "hs", "w", "ws", "dtype", "y")]
    if backward:
        return lib.spec_verify_linear_ce_backward(
            *head, a["stats"], a["g"], a["N"], a["D"], a["V"], a["gh"], a["ghs"], a["gw"], a["gws"],
            a["space"], a["bytes"], None)
    return lib.spec_verify_linear_ce(*head, a["N"], a["D"], a["V"], a["loss"], a["stats"], a["space"],
                                     a["bytes"], None)


def test_top_logits_refusals(lib):
    from lossless_draft_verification_sample_amd import _lib as L
    inf, nan = float("inf"), float("nan")
    for kw in (dict(z=None), dict(ids=None), dict(values=None), dict(R=0), dict(V=0), dict(K=0),
               dict(K=1001), dict(K=L.SV_MAX_TOP + 1, V=5000, stride=5000), dict(stride=999),
               dict(T=0.0), dict(T=-1.0), dict(T=inf), dict(T=nan), dict(z=FAKE + 1),
               dict(dtype=0, z=FAKE + 2)):
        assert _top(lib, **kw) == L.SV_EINVAL, kw
    assert _top(lib, dtype=2) == L.SV_EDTYPE
    assert _top(lib, T=1e-40) == L.SV_EINVAL and _top(lib, R=(1 << 22) + 1) == L.SV_ESIZE
    big = dict(V=151936, stride=151936, R=2)
    need = lib.spec_verify_top_logits_workspace_bytes(2, 151936, 8, 1)
    assert need > 0 and need % 256 == 0
    for kw in (dict(), dict(ws=FAKE, ws_bytes=need - 1), dict(ws=FAKE + 8, ws_bytes=need)):
        assert _top(lib, **big, **kw) == L.SV_EWORKSPACE, kw
    for bad in ((0, 100, 1), (1, 0, 1), (1, 100, 0), (1, 100, 101), (1, 5000, L.SV_MAX_TOP + 1)):
        assert lib.spec_verify_top_logits_workspace_bytes(*bad, 1) == 0


def test_distill_refusals(lib):
    from lossless_draft_verification_sample_amd import _lib as L
    for backward in (False, True):
        for kw in (dict(z=None), dict(ids=None), dict(t=None), dict(stats=None), dict(R=0), dict(V=0),
                   dict(K=0), dict(K=L.SV_MAX_TOP + 1), dict(T=0.0), dict(T=float("nan")),
                   dict(stride=39999), dict(gstride=39999), dict(z=FAKE + 1), dict(grad=FAKE + 1),
                   dict(stride=40008, gstride=40000)):   # in place at another stride
            assert _distill(lib, backward, **kw) == L.SV_EINVAL, (backward, kw)
        assert _distill(lib, backward, dtype=7) == L.SV_EDTYPE
        assert _distill(lib, backward, T=1e-40) == L.SV_EINVAL
        assert _distill(lib, backward, R=(1 << 22) + 1) == L.SV_ESIZE
    assert _distill(lib, loss=None) == L.SV_EINVAL
    assert _distill(lib, True, grad=None) == L.SV_EINVAL
    need = lib.spec_verify_distill_workspace_bytes(2, 200000, 1)
    assert need > 0
    big = dict(V=200000, stride=200000, gstride=200000)
    for kw in (dict(), dict(ws=FAKE, ws_bytes=need - 1), dict(ws=FAKE + 16, ws_bytes=need)):
        assert _distill(lib, **big, **kw) == L.SV_EWORKSPACE, kw
    assert lib.spec_verify_distill_workspace_bytes(0, 10, 1) == 0


def test_linear_ce_refusals(lib):
    from lossless_draft_verification_sample_amd import _lib as L
    for backward in (False, True):
        for kw in (dict(h=None), dict(w=None), dict(y=None), dict(stats=None), dict(N=0), dict(D=0),
                   dict(V=0), dict(hs=63), dict(ws=63), dict(h=FAKE + 1), dict(w=FAKE + 1)):
            assert _ce(lib, backward, **kw) == L.SV_EINVAL, (backward, kw)
        assert _ce(lib, backward, dtype=-1) == L.SV_EDTYPE
        assert _ce(lib, backward, N=1 << 23) == L.SV_ESIZE
        assert _ce(lib, backward, D=1 << 23, hs=1 << 23, ws=1 << 23) == L.SV_ESIZE
        assert _ce(lib, backward, N=1 << 22, V=1 << 30) == L.SV_ESIZE   # too many tiles
        assert _ce(lib, backward) == L.SV_EWORKSPACE
    assert _ce(lib, loss=None) == L.SV_EINVAL
    for kw in (dict(gh=None, gw=None), dict(ghs=63), dict(gws=63), dict(gh=FAKE + 1), dict(gw=FAKE + 1)):
        assert _ce(lib, True, **kw) == L.SV_EINVAL, kw
    f, b = lib.spec_verify_linear_ce_workspace_bytes, lib.spec_verify_linear_ce_backward_workspace_bytes
    assert f(5, 64, 100, 1) > 0 and b(5, 64, 100, 1, 1, 1) > b(5, 64, 100, 1, 0, 1) > 0
    assert f(0, 64, 100, 1) == 0 and f(5, 64, 100, 9) == 0 and b(5, 64, 100, 1, 0, 0) == 0
    need = b(5, 64, 100, 1, 1, 1)
    assert _ce(lib, True, space=FAKE, bytes=need - 1) == L.SV_EWORKSPACE


def test_binding_refuses_host_tensors_and_shapes():
    import torch
    import lossless_draft_verification_sample_amd as sv
    z = torch.zeros(2, 100)
    for call in (lambda: sv.spec_verify_top_logits(z, 4),
                 lambda: sv.spec_verify_distill(z, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)),
                 lambda: sv.spec_verify_linear_ce(z, z, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_constants_match_the_header():
    from lossless_draft_verification_sample_amd import _lib as L
    hdr = open(os.path.join(ROOT, "include", "spec_verify.h")).read()
    assert L.SV_MAX_TOP == int(re.search(r"#define SV_MAX_TOP (\d+)", hdr).group(1))
    assert ctypes.sizeof(ctypes.c_size_t) == 8
