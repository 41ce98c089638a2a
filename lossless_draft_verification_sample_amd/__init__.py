"""Lossless speculative-sampling verifier for AMD MI355X (gfx950), the losses its
drafter is trained with, and the operators that make and shape the rows it reads.

Thin Python binding over the C interface of include/spec_verify.h. The
functions below only marshal arguments (device pointers of torch tensors, the
current HIP stream) and allocate outputs; every step runs in the HIP kernels of
libspecverify.so. PyTorch supplies device memory and
streams. If the library is missing, every call raises.
"""

import functools
from collections import namedtuple

from . import _lib
from ._lib import (  # noqa: F401
    SV_BF16,
    SV_EDTYPE,
    SV_EHIP,
    SV_ESCRATCH,
    SV_EINVAL,
    SV_ESIZE,
    SV_EWORKSPACE,
    SV_F32,
    SV_FLAG_BAD_PARAM,
    SV_FLAG_EMPTY,
    SV_FLAG_NONFINITE,
    SV_FLAG_Q_ZERO,
    SV_FLAG_RESIDUAL_ZERO,
    SV_FLAG_TOKEN_RANGE,
    SV_MAX_BANNED,
    SV_MAX_HISTORY,
    SV_MAX_ROWS,
    SV_MAX_TOP,
    SV_NOALLOC_SCRATCH_BYTES,
    SV_OK,
    SvCache,
    SvRequests,
    SvSampler,
    SvStrides,
)

SampleOut = namedtuple("SampleOut",
                       "tokens num_accepted flags target_lse draft_lse overlap accept_hist",
                       defaults=(None, None))
GreedyOut = namedtuple("GreedyOut", "tokens num_accepted flags accept_hist", defaults=(None,))
CommitOut = namedtuple("CommitOut", "new_kv_len anchor n_free free_slots")
TopLogitsOut = namedtuple("TopLogitsOut", "ids values lse")
DistillOut = namedtuple("DistillOut", "loss stats grad")
LinearCeOut = namedtuple("LinearCeOut", "loss stats")
LinearCeGrads = namedtuple("LinearCeGrads", "hidden weight")
RotateOut = namedtuple("RotateOut", "q k")
CacheRows = namedtuple("CacheRows", "k v")
AttentionOut = namedtuple("AttentionOut", "out lse")
# A paged 8-bit cache (see sv_cache in include/spec_verify.h): k, v [pages, heads,
# page_size / 32, ceil(head_dim / 32), 1024] float8_e4m3fn, k_scale, v_scale [pages, heads,
# page_size / 32] float32. kv_cache() makes one.
KVCache = namedtuple("KVCache", "k v k_scale v_scale page_size head_dim")
# Per-request settings of a mixed batch (see sv_requests in include/spec_verify.h):
# gamma [B] int32, target / draft [B, 12] uint8 sv_sampler records (sampler_array),
# banned_draft [B, m] int32, history [B, H] int32, penalty / penalty_draft [B]
# float32 repetition penalties; None keeps the call-wide value (no penalty).
Requests = namedtuple("Requests",
                      "gamma target draft banned_draft history penalty penalty_draft",
                      defaults=(None,) * 7)


class SpecVerifyError(RuntimeError):
    def __init__(self, status, where):
        super().__init__(f"{where}: {spec_verify_strerror(status)} (status {status})")
        self.status = status


_TORCH = None


def _torch():
    """torch, imported when a call first needs it; the import statement takes 0.2 us even then."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _dtype_code(t, name="logits"):
    torch = _torch()
    dtype = t.dtype
    if dtype == torch.bfloat16:
        return SV_BF16
    if dtype == torch.float32:
        return SV_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _dev_ptr(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _checked(t, name, dtype, shape):
    """Device pointer of an optional output whose shape the library assumes."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _dev_ptr(t, name, dtype)


def _sampler(s):
    if isinstance(s, SvSampler):
        return s
    if isinstance(s, dict):
        return SvSampler(float(s.get("temperature", 1.0)), int(s.get("top_k", 0)),
                         float(s.get("top_p", 1.0)))
    t, k, p = s
    return SvSampler(float(t), int(k), float(p))


def sampler_array(samplers, device):
    """[B] sv_sampler records (float temperature, int32 top_k, float top_p) on
    `device`, as a [B, 12] uint8 tensor, from (temperature, top_k, top_p)
    tuples, dicts or SvSampler."""
    import numpy as np
    torch = _torch()
    rec = np.zeros(len(samplers), dtype=[("t", "<f4"), ("k", "<i4"), ("p", "<f4")])
    for j, smp in enumerate(samplers):
        c = _sampler(smp)
        rec[j] = (c.temperature, c.top_k, c.top_p)
    return torch.from_numpy(rec.view(np.uint8).reshape(len(samplers), 12).copy()).to(device)


def _requests(req, B):
    """ctypes sv_requests for a Requests tuple (or None)."""
    import ctypes
    if req is None:
        return None
    torch = _torch()
    for name, t in (("target", req.target), ("draft", req.draft)):
        if t is not None and (tuple(t.shape) != (B, 12) or t.dtype != torch.uint8):
            raise ValueError(f"requests.{name} must be a [B, 12] uint8 tensor (sampler_array)")
    if req.gamma is not None and tuple(req.gamma.shape) != (B,):
        raise ValueError("requests.gamma must be [B]")
    nbd = 0
    if req.banned_draft is not None:
        nbd = int(req.banned_draft.shape[1])
        if tuple(req.banned_draft.shape) != (B, nbd):
            raise ValueError("requests.banned_draft must be [B, n]")
    nh = 0
    if req.history is not None:
        nh = int(req.history.shape[1])
        if tuple(req.history.shape) != (B, nh):
            raise ValueError("requests.history must be [B, H]")
        if nh > SV_MAX_HISTORY:
            raise ValueError(f"requests.history holds {nh} > SV_MAX_HISTORY = {SV_MAX_HISTORY} "
                             "tokens per request")
    r = SvRequests(_dev_ptr(req.gamma, "requests.gamma", torch.int32),
                   _dev_ptr(req.target, "requests.target"), _dev_ptr(req.draft, "requests.draft"),
                   _dev_ptr(req.banned_draft, "requests.banned_draft", torch.int32), nbd,
                   _dev_ptr(req.history, "requests.history", torch.int32), nh,
                   _checked(req.penalty, "requests.penalty", torch.float32, (B,)),
                   _checked(req.penalty_draft, "requests.penalty_draft", torch.float32, (B,)))
    return ctypes.byref(r), r


def _stream(stream):
    """(hipStream_t handle, torch stream) of the call. None means torch's
    current stream; a raw handle is wrapped as an external stream. Outputs and
    the workspace the binding allocates are allocated on that stream, so the
    caching allocator keeps them until the call's kernels have run."""
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    elif not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.default_stream() if int(stream) == 0
                  else torch.cuda.ExternalStream(int(stream)))
    return stream.cuda_stream, stream


def spec_verify_strerror(status):
    return _lib.load().spec_verify_strerror(int(status)).decode()


def spec_verify_workspace_bytes(B, gamma, V):
    return int(_lib.load().spec_verify_workspace_bytes(int(B), int(gamma), int(V)))


def spec_verify_sample_noalloc(target_logits, draft_logits, draft_tokens,
                               target_sampler=(1.0, 0, 1.0), draft_sampler=(1.0, 0, 1.0),
                               banned_ids=None, seed=0, offset=0, uniforms=None, want_lse=True,
                               want_overlap=False, want_hist=False, requests=None, out=None,
                               stream=None, lib=None):
    """spec_verify_sample on the library's static per-GPU scratch instead of a
    workspace (see include/spec_verify.h). Pass `out` to avoid every
    allocation in this binding as well."""
    return spec_verify_sample(target_logits, draft_logits, draft_tokens, target_sampler,
                              draft_sampler, banned_ids, seed, offset, uniforms, want_lse,
                              want_overlap, want_hist, requests, None, out, stream, lib,
                              _noalloc=True)


def spec_verify_sample(target_logits, draft_logits, draft_tokens, target_sampler=(1.0, 0, 1.0),
                       draft_sampler=(1.0, 0, 1.0), banned_ids=None, seed=0, offset=0,
                       uniforms=None, want_lse=True, want_overlap=False, want_hist=False,
                       requests=None, workspace=None, out=None, stream=None, lib=None,
                       _noalloc=False):
    """Speculative-sampling verification of a batch (see include/spec_verify.h).

    target_logits [B, gamma+1, V] and draft_logits [B, gamma, V] (bf16 or fp32),
    draft_tokens [B, gamma] int32, banned_ids [B, n] int32 or None,
    uniforms [B, gamma+1] float64 or None (then Philox(seed, offset)).
    Samplers are (temperature, top_k, top_p) tuples, dicts or SvSampler.
    want_overlap adds the per-position overlaps [B, gamma] (float64; one more
    read of the rows), want_hist the accepted-prefix histogram [gamma+1]
    (int32 storage of the library's uint32 counts). requests: a Requests tuple
    of per-request settings (mixed batch) or None. stream: a torch stream, a
    raw hipStream_t handle or None (torch's current stream). lib: the loaded
    library to call (default libspecverify.so; bench.py passes the timing
    build).
    Returns SampleOut(tokens, num_accepted, flags, target_lse, draft_lse,
    overlap, accept_hist).
    """
    torch = _torch()
    lib = lib or _lib.load()
    B, G1, V = target_logits.shape
    gamma = G1 - 1
    if tuple(draft_logits.shape) != (B, gamma, V):
        raise ValueError("draft_logits must be [B, gamma, V]")
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must share a dtype")
    if tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("draft_tokens must be [B, gamma]")
    dt = _dtype_code(target_logits)
    n_banned = 0 if banned_ids is None else int(banned_ids.shape[1])
    if banned_ids is not None and tuple(banned_ids.shape) != (B, n_banned):
        raise ValueError("banned_ids must be [B, n_banned]")
    if uniforms is not None and tuple(uniforms.shape) != (B, G1):
        raise ValueError("uniforms must be [B, gamma+1]")
    dev = target_logits.device
    handle, strm = _stream(stream)
    with torch.cuda.stream(strm):
        if out is None:
            out = SampleOut(
                torch.empty((B, G1), dtype=torch.int32, device=dev),
                torch.empty((B,), dtype=torch.int32, device=dev),
                torch.empty((B,), dtype=torch.int32, device=dev),
                torch.empty((B, G1), dtype=torch.float32, device=dev) if want_lse else None,
                torch.empty((B, gamma), dtype=torch.float32, device=dev) if want_lse else None,
                torch.empty((B, gamma), dtype=torch.float64, device=dev) if want_overlap else None,
                torch.empty((G1,), dtype=torch.int32, device=dev) if want_hist else None,
            )
        if workspace is None and not _noalloc:
            need = lib.spec_verify_workspace_bytes(B, gamma, V)
            workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    req = _requests(requests, B)
    fn = lib.spec_verify_sample_noalloc if _noalloc else lib.spec_verify_sample
    ws_args = () if _noalloc else (_dev_ptr(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size())
    rc = fn(
        _dev_ptr(target_logits, "target_logits"), _dev_ptr(draft_logits, "draft_logits"), dt,
        _dev_ptr(draft_tokens, "draft_tokens", torch.int32),
        _dev_ptr(banned_ids, "banned_ids", torch.int32), n_banned, B, gamma, V,
        _sampler(target_sampler), _sampler(draft_sampler), None if req is None else req[0],
        int(seed), int(offset),
        _dev_ptr(uniforms, "uniforms", torch.float64),
        _dev_ptr(out.tokens, "out_tokens", torch.int32),
        _dev_ptr(out.num_accepted, "out_num_accepted", torch.int32),
        _dev_ptr(out.flags, "out_flags", torch.int32),
        _dev_ptr(out.target_lse, "out_target_lse", torch.float32),
        _dev_ptr(out.draft_lse, "out_draft_lse", torch.float32),
        _checked(out.overlap, "out_overlap", torch.float64, (B, gamma)),
        _checked(out.accept_hist, "out_accept_hist", torch.int32, (G1,)), *ws_args, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, fn.__name__)
    return out


def spec_verify_greedy(target_logits, draft_tokens, banned_ids=None, want_hist=False, out=None,
                       stream=None, lib=None):
    """Greedy verification (see include/spec_verify.h); banned_ids [B, n] int32
    or None; stream and lib as for spec_verify_sample.
    Returns GreedyOut(tokens, num_accepted, flags, accept_hist)."""
    torch = _torch()
    lib = lib or _lib.load()
    B, G1, V = target_logits.shape
    gamma = G1 - 1
    if tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("draft_tokens must be [B, gamma]")
    n_banned = 0 if banned_ids is None else int(banned_ids.shape[1])
    if banned_ids is not None and tuple(banned_ids.shape) != (B, n_banned):
        raise ValueError("banned_ids must be [B, n_banned]")
    dt = _dtype_code(target_logits)
    dev = target_logits.device
    handle, strm = _stream(stream)
    if out is None:
        with torch.cuda.stream(strm):
            out = GreedyOut(torch.empty((B, G1), dtype=torch.int32, device=dev),
                            torch.empty((B,), dtype=torch.int32, device=dev),
                            torch.empty((B,), dtype=torch.int32, device=dev),
                            torch.empty((G1,), dtype=torch.int32, device=dev) if want_hist else None)
    rc = lib.spec_verify_greedy(
        _dev_ptr(target_logits, "target_logits"), dt,
        _dev_ptr(draft_tokens, "draft_tokens", torch.int32),
        _dev_ptr(banned_ids, "banned_ids", torch.int32), n_banned, B, gamma, V,
        _dev_ptr(out.tokens, "out_tokens", torch.int32),
        _dev_ptr(out.num_accepted, "out_num_accepted", torch.int32),
        _dev_ptr(out.flags, "out_flags", torch.int32),
        _checked(out.accept_hist, "out_accept_hist", torch.int32, (G1,)), handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_greedy")
    return out


def spec_verify_commit(tokens, num_accepted, kv_len, slots=None, gamma_b=None, out=None,
                       stream=None, lib=None):
    """Chain KV-commit metadata of a verification round (see include/spec_verify.h).

    tokens [B, gamma+1] and num_accepted [B] from spec_verify_sample or
    spec_verify_greedy, kv_len [B] int32, slots [B, gamma+1] int32 or None,
    gamma_b [B] int32 proposals per request or None.
    Returns CommitOut(new_kv_len, anchor, n_free, free_slots); free_slots is
    None when slots is None. stream and lib as for spec_verify_sample.
    """
    torch = _torch()
    lib = lib or _lib.load()
    B, G1 = tokens.shape
    gamma = G1 - 1
    if tuple(num_accepted.shape) != (B,) or tuple(kv_len.shape) != (B,):
        raise ValueError("num_accepted and kv_len must be [B]")
    if slots is not None and tuple(slots.shape) != (B, G1):
        raise ValueError("slots must be [B, gamma+1]")
    dev = tokens.device
    handle, strm = _stream(stream)
    if out is None:
        with torch.cuda.stream(strm):
            out = CommitOut(torch.empty((B,), dtype=torch.int32, device=dev),
                            torch.empty((B,), dtype=torch.int32, device=dev),
                            torch.empty((B,), dtype=torch.int32, device=dev),
                            torch.empty((B, gamma), dtype=torch.int32, device=dev)
                            if slots is not None else None)
    rc = lib.spec_verify_commit(
        _dev_ptr(tokens, "tokens", torch.int32), _dev_ptr(num_accepted, "num_accepted", torch.int32),
        _dev_ptr(kv_len, "kv_len", torch.int32), _dev_ptr(slots, "slots", torch.int32),
        _checked(gamma_b, "gamma_b", torch.int32, (B,)), B, gamma,
        _checked(out.new_kv_len, "new_kv_len", torch.int32, (B,)),
        _checked(out.anchor, "anchor", torch.int32, (B,)),
        _checked(out.n_free, "n_free", torch.int32, (B,)),
        _checked(out.free_slots, "free_slots", torch.int32, (B, gamma)), handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_commit")
    return out


# ------------------------------------------------------- training the drafter
#
# Autograd records none of these calls: what they return has no graph, whether the
# inputs require gradients or not, and the gradients are those the *_backward calls and
# want_grad give. A program that trains through autograd makes the calls in the forward
# and backward of a torch.autograd.Function of its own.


_INT32_MAX = 2 ** 31 - 1


def _matrix(t, name, device=None, dtype=None, cols=None):
    """(pointer, row stride) of a tensor whose last dimension is consecutive and
    whose leading dimensions are rows at one stride."""
    if not _torch().is_tensor(t) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) < 2 or t.numel() == 0:
        raise ValueError(f"{name} must have at least one row and one column, got {tuple(shape)}")
    width = shape[-1]
    if cols is not None and width != cols:
        raise ValueError(f"{name} must have rows of {cols}, got {tuple(shape)}")
    if width > _INT32_MAX or t.numel() // width > _INT32_MAX:
        raise ValueError(f"{name} must have at most {_INT32_MAX} rows and columns, got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), width
    steps = t.stride()
    if width > 1 and steps[-1] != 1:
        raise ValueError(f"{name} must have consecutive elements in a row")
    stride, rows = None, 1
    for size, step in zip(reversed(shape[:-1]), reversed(steps[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = step
        elif step != stride * rows:
            raise ValueError(f"{name} must have its rows at one stride")
        rows *= size
    if stride is None:
        stride = width   # a single row
    if stride < width:
        raise ValueError(f"{name} must not have overlapping rows")
    return t.data_ptr(), stride


def _vector(t, name, dtype, shape, device):
    """Pointer of a contiguous tensor (or None) of this type, shape and device."""
    if t is None:
        return None
    # numbers of devices compare quicker than devices
    if t.get_device() == device.index and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class _Current:
    """The device and stream are torch's current ones already."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_CURRENT = _Current()


def _on(device, stream):
    """(context that makes the device and the call's stream current, stream handle)."""
    torch = _torch()
    # torch's own handle of the current stream: a Stream object around it costs 2 us a call
    if stream is None and torch.cuda.current_device() == device.index:
        return _CURRENT, torch._C._cuda_getCurrentRawStream(device.index)
    import contextlib
    with torch.cuda.device(device):
        handle, strm = _stream(stream)
    if strm.device != device:
        raise ValueError(f"the stream is one of {strm.device}, the tensors are on {device}")
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(device))
    ctx.enter_context(torch.cuda.stream(strm))
    return ctx, handle


def _space(workspace, need, device):
    """(pointer, bytes) of a workspace, allocated when the caller gave none; the
    tensor comes along so that it lives until the call is queued."""
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    return _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), workspace


def _written(out):
    """Tells autograd that a caller's outputs were written, as an operation in place would:
    a backward pass that had saved one of them (logits that were overwritten by their
    gradient) then raises instead of using what it holds now."""
    given = [t for t in out or () if t is not None]
    if given:
        _torch().autograd.graph.increment_version(given)


def spec_verify_top_logits_workspace_bytes(R, V, K, dtype=SV_BF16):
    return int(_lib.load().spec_verify_top_logits_workspace_bytes(int(R), int(V), int(K), int(dtype)))


def spec_verify_top_logits(logits, k, temperature=1.0, want_lse=True, workspace=None, out=None,
                           stream=None, lib=None):
    """The k largest logits of every row, descending, the lower id first among
    equals, and the row's log-normaliser at `temperature` (see
    include/spec_verify.h): what a drafter is distilled from.

    logits [..., V] bf16 or fp32, rows at one stride (the target logits
    [B, gamma+1, V] of spec_verify_sample as they are, or columns cut from a wider
    buffer).
    Returns TopLogitsOut(ids [..., k] int32, values [..., k] float32, lse [...]
    float32 or None).
    """
    torch = _torch()
    lib = lib or _lib.load()
    ptr, stride = _matrix(logits, "logits")
    dt, dev, lead, V = _dtype_code(logits), logits.device, tuple(logits.shape[:-1]), logits.shape[-1]
    R, k, given = logits.numel() // V, int(k), out is not None
    if not 1 <= k <= SV_MAX_TOP:
        raise SpecVerifyError(SV_EINVAL, "spec_verify_top_logits")
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            ids = torch.empty((*lead, k), dtype=torch.int32, device=dev)
            values = torch.empty((*lead, k), dtype=torch.float32, device=dev)
            lse = values.new_empty(lead) if want_lse else None
            out = TopLogitsOut(ids, values, lse)
            outs = ids.data_ptr(), values.data_ptr(), lse.data_ptr() if want_lse else None
        else:
            outs = (_vector(out.ids, "out.ids", torch.int32, (*lead, k), dev),
                    _vector(out.values, "out.values", torch.float32, (*lead, k), dev),
                    _vector(out.lse, "out.lse", torch.float32, lead, dev))
        ws, ws_bytes, keep = _space(
            workspace, lib.spec_verify_top_logits_workspace_bytes(R, V, k, dt), dev)
        rc = lib.spec_verify_top_logits(
            ptr, stride, dt, R, V, k, float(temperature), *outs, ws, ws_bytes, handle)
    del keep
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_top_logits")
    if given:
        _written(out)
    return out


def spec_verify_distill_workspace_bytes(R, V, dtype=SV_BF16):
    return int(_lib.load().spec_verify_distill_workspace_bytes(int(R), int(V), int(dtype)))


def _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse):
    torch = _torch()
    ptr, stride = _matrix(logits, "logits")
    dt, dev, lead, V = _dtype_code(logits), logits.device, tuple(logits.shape[:-1]), logits.shape[-1]
    if teacher_ids is None or teacher_logits is None:
        raise ValueError("teacher_ids and teacher_logits must be device tensors")
    if teacher_ids.dim() < 1 or tuple(teacher_ids.shape[:-1]) != lead:
        raise ValueError(f"teacher_ids must be {lead} rows of kept ids, got {tuple(teacher_ids.shape)}")
    K = int(teacher_ids.shape[-1])
    if not 1 <= K <= SV_MAX_TOP:
        raise SpecVerifyError(SV_EINVAL, "spec_verify_distill")
    return (ptr, stride, dt, logits.numel() // V, V,
            _vector(teacher_ids, "teacher_ids", torch.int32, (*lead, K), dev),
            _vector(teacher_logits, "teacher_logits", torch.float32, (*lead, K), dev),
            _vector(teacher_lse, "teacher_lse", torch.float32, lead, dev), K), dev, lead


def _loss_out(out, like, lead, dev):
    """Loss and statistics of rows `lead`, new ones (float32, as `like`) when out is
    None, and their pointers."""
    if out is None:
        loss, stats = like.new_empty(lead), like.new_empty((*lead, 2))
        return loss, stats, (loss.data_ptr(), stats.data_ptr())
    f32 = _torch().float32
    return out.loss, out.stats, (_vector(out.loss, "out.loss", f32, lead, dev),
                                 _vector(out.stats, "out.stats", f32, (*lead, 2), dev))


def _grad_out(t, like, name):
    """A gradient's tensor, its pointer and row stride; a new one when None."""
    if t is None:
        t = _torch().empty_like(like, memory_format=_torch().contiguous_format)
        return t, t.data_ptr(), like.shape[-1]
    if tuple(t.shape) != tuple(like.shape):
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    return (t, *_matrix(t, name, like.device, like.dtype))


def spec_verify_distill(logits, teacher_ids, teacher_logits, temperature=1.0, teacher_lse=None,
                        row_weight=None, want_grad=False, workspace=None, out=None, stream=None,
                        lib=None):
    """Distillation loss of student rows against a teacher's kept logits, and
    with want_grad its gradient in the same call (see include/spec_verify.h).

    logits [..., V] bf16 or fp32 (rows at one stride), teacher_ids [..., K] int32
    and teacher_logits [..., K] float32 as spec_verify_top_logits returns them,
    teacher_lse [...] float32 (its lse at the same temperature) or None to
    renormalise over the kept ids; row_weight [...] float32 scales the gradient's
    rows (not the loss). out: a DistillOut; its grad may be `logits` itself. Autograd
    records nothing here; outputs given by the caller count as changed in place.
    Returns DistillOut(loss [...], stats [..., 2], grad like logits or None);
    stats serve spec_verify_distill_backward.
    """
    torch = _torch()
    lib = lib or _lib.load()
    args, dev, lead = _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse)
    ctx, handle = _on(dev, stream)
    with ctx:
        grad, gptr, gstride = out and out.grad, None, 0
        loss, stats, outs = _loss_out(out, teacher_logits, lead, dev)
        if want_grad or grad is not None:
            grad, gptr, gstride = _grad_out(grad, logits, "out.grad")
        ws, ws_bytes, keep = _space(
            workspace, lib.spec_verify_distill_workspace_bytes(args[3], args[4], args[2]), dev)
        rc = lib.spec_verify_distill(
            *args, float(temperature),
            _vector(row_weight, "row_weight", torch.float32, lead, dev), *outs, gptr, gstride,
            ws, ws_bytes, handle)
    del keep
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_distill")
    _written(out)
    return DistillOut(loss, stats, grad)


def spec_verify_distill_backward(logits, teacher_ids, teacher_logits, stats, grad_loss=None,
                                 temperature=1.0, teacher_lse=None, out=None, stream=None, lib=None):
    """Gradient of spec_verify_distill's loss from its stats; grad_loss [...]
    float32 or None (1). out: the gradient's tensor, which may be `logits` (then changed
    in place, for autograd too).
    Returns the gradient, like logits."""
    torch = _torch()
    lib = lib or _lib.load()
    args, dev, lead = _distill_inputs(logits, teacher_ids, teacher_logits, teacher_lse)
    ctx, handle = _on(dev, stream)
    given = out is not None
    with ctx:
        out, gptr, gstride = _grad_out(out, logits, "out")
        if stats is None:
            raise ValueError("stats are those of spec_verify_distill")
        rc = lib.spec_verify_distill_backward(
            *args, float(temperature), _vector(stats, "stats", torch.float32, (*lead, 2), dev),
            _vector(grad_loss, "grad_loss", torch.float32, lead, dev), gptr, gstride, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_distill_backward")
    if given:
        _written((out,))
    return out


def spec_verify_linear_ce_workspace_bytes(N, D, V, dtype=SV_BF16):
    return int(_lib.load().spec_verify_linear_ce_workspace_bytes(int(N), int(D), int(V), int(dtype)))


def spec_verify_linear_ce_backward_workspace_bytes(N, D, V, dtype=SV_BF16, want_hidden=True,
                                                   want_weight=True):
    return int(_lib.load().spec_verify_linear_ce_backward_workspace_bytes(
        int(N), int(D), int(V), int(dtype), int(bool(want_hidden)), int(bool(want_weight))))


def _ce_inputs(hidden, weight, labels):
    torch = _torch()
    hptr, hstride = _matrix(hidden, "hidden")
    dt, dev, lead, D = _dtype_code(hidden), hidden.device, tuple(hidden.shape[:-1]), hidden.shape[-1]
    if weight.dim() != 2:
        raise ValueError(f"weight must be [V, D], got {tuple(weight.shape)}")
    wptr, wstride = _matrix(weight, "weight", dev, hidden.dtype, D)
    if labels is None:
        raise ValueError("labels must be a device tensor")
    return (hptr, hstride, wptr, wstride, dt,
            _vector(labels, "labels", torch.int32, lead, dev)), hidden.numel() // D, dev, lead


def spec_verify_linear_ce(hidden, weight, labels, workspace=None, out=None, stream=None, lib=None):
    """Softmax cross entropy of a linear head without storing its logits (see
    include/spec_verify.h).

    hidden [..., D] and weight [V, D] (bf16 or fp32, rows at one stride each),
    labels [...] int32; rows whose label lies outside [0, V), such as -100, are
    left out (loss 0). Autograd records nothing here: the gradients come from
    spec_verify_linear_ce_backward.
    Returns LinearCeOut(loss [...], stats [..., 2]), both float32; stats serve
    spec_verify_linear_ce_backward.
    """
    torch = _torch()
    lib = lib or _lib.load()
    args, N, dev, lead = _ce_inputs(hidden, weight, labels)
    V, D = weight.shape
    given = out is not None
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            loss = torch.empty(lead, dtype=torch.float32, device=dev)
            out = LinearCeOut(loss, loss.new_empty((*lead, 2)))
        ws, ws_bytes, keep = _space(
            workspace, lib.spec_verify_linear_ce_workspace_bytes(N, D, V, args[4]), dev)
        rc = lib.spec_verify_linear_ce(
            *args, N, D, V, _vector(out.loss, "out.loss", torch.float32, lead, dev),
            _vector(out.stats, "out.stats", torch.float32, (*lead, 2), dev), ws, ws_bytes, handle)
    del keep
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_linear_ce")
    if given:
        _written(out)
    return out


def spec_verify_linear_ce_backward(hidden, weight, labels, stats, grad_loss=None, want_hidden=True,
                                   want_weight=True, workspace=None, out=None, stream=None,
                                   lib=None):
    """Gradients of spec_verify_linear_ce's loss from its stats; grad_loss [...]
    float32 or None (1). want_hidden / want_weight: which ones (a frozen head needs
    the first alone). out: a LinearCeGrads of tensors for those wanted.
    Returns LinearCeGrads(hidden, weight), None where not wanted."""
    torch = _torch()
    lib = lib or _lib.load()
    args, N, dev, lead = _ce_inputs(hidden, weight, labels)
    V, D = weight.shape
    if stats is None:
        raise ValueError("stats are those of spec_verify_linear_ce")
    ctx, handle = _on(dev, stream)
    with ctx:
        gh, ghp, ghs, gw, gwp, gws = None, None, 0, None, None, 0
        if want_hidden:
            gh, ghp, ghs = _grad_out(out and out.hidden, hidden, "out.hidden")
        if want_weight:
            gw, gwp, gws = _grad_out(out and out.weight, weight, "out.weight")
        ws, ws_bytes, keep = _space(
            workspace, lib.spec_verify_linear_ce_backward_workspace_bytes(
                N, D, V, args[4], int(bool(want_hidden)), int(bool(want_weight))), dev)
        rc = lib.spec_verify_linear_ce_backward(
            *args, _vector(stats, "stats", torch.float32, (*lead, 2), dev),
            _vector(grad_loss, "grad_loss", torch.float32, lead, dev), N, D, V, ghp, ghs, gwp, gws,
            ws, ws_bytes, handle)
    del keep
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_linear_ce_backward")
    if out is not None:
        _written((gh, gw))
    return LinearCeGrads(gh, gw)


# ------------------------------------------- the verification pass's rows
#
# Row j of request b stands at position kv_len[b] + j. Autograd records none of these
# calls; outputs and caches given by the caller count as changed in place.


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original=None, low=1.0,
                       high=4.0, fast=32.0, slow=1.0, device="cuda"):
    """(freqs, scale) of spec_verify_rotate for a head's `rotary_dim` rotated dimensions:
    freqs [rotary_dim / 2] float64, radians a position, and the factor on rotated values.

    f_i = base^(-2i / rotary_dim), scaled for contexts `factor` times as long as the model was
    trained for:
      None      as they are.
      "linear"  f_i / factor: positions are interpolated.
      "base"    the base raised to base * factor^(R / (R - 2)), which leaves the fastest
                pair as it is and divides the slowest by factor.
      "smooth"  by wavelength w = 2 pi / f_i against the trained context `original`: w < original / high
                as it is, w > original / low divided by factor, between them
                f_i ((1 - s) / factor + s), s = (original / w - low) / (high - low).
      "ramp"    by the pair's index between those that turn `fast` and `slow` times over `original`
                positions: f_i (1 - r + r / factor), r rising from 0 to 1, and scale
                0.1 log(factor) + 1 (Peng et al. 2023, "YaRN", sections 3.2 to 3.4).
    """
    import math
    torch = _torch()
    R = int(rotary_dim)
    if R < 0 or R % 2:
        raise ValueError(f"rotary_dim must be even, got {rotary_dim}")
    if not base > 0 or not factor >= 1:
        raise ValueError("base must be positive, factor at least 1")
    if scaling in ("smooth", "ramp") and not (original and original > 0):
        raise ValueError(f"scaling {scaling!r} needs the trained context, original")
    if scaling == "base" and R > 2:
        base = base * factor ** (R / (R - 2))
    freqs = [float(base) ** (-2.0 * i / R) for i in range(R // 2)]
    scale = 1.0
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling == "smooth":
        if not high > low:
            raise ValueError("high must exceed low")
        share = [min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low))) for f in freqs]
        freqs = [f * ((1 - s) / factor + s) for f, s in zip(freqs, share)]
    elif scaling == "ramp":
        def index(turns):   # of the pair that turns so often
            return R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(0, math.floor(index(fast))), min(R - 1, math.ceil(index(slow)))
        width = max(last - first, 0.001)
        ramp = [min(1.0, max(0.0, (i - first) / width)) for i in range(R // 2)]
        freqs = [f * (1 - r + r / factor) for f, r in zip(freqs, ramp)]
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(freqs, dtype=torch.float64, device=device), scale


def _on_device(t, name, device, dtype, shape):
    """Raises what is wrong with a tensor of rows: not on a device, or on another device, of another
    type or shape than wanted (None: any)."""
    if not isinstance(t, _TORCH.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# What an int32 argument holds: ctypes would take a larger number's lower 32 bits.
_MOST = 2 ** 31 - 1

# sv_strides of these strides: made once, passed by value
_strides = functools.lru_cache(maxsize=1024)(SvStrides)


def _rows4(t, name, device=None, dtype=None, shape=None):
    """(pointer, strides) of a [B, N, heads, D] tensor with consecutive D."""
    _on_device(t, name, device, dtype, shape)
    size = t.shape
    if len(size) != 4 or 0 in size:
        raise ValueError(f"{name} must be [B, N, heads, D], none of them 0, got {tuple(size)}")
    if max(size) > _MOST:
        raise SpecVerifyError(SV_ESIZE, name)
    b, n, h, one = t.stride()
    if one != 1 and size[3] > 1:
        raise ValueError(f"{name} must have consecutive elements in a head")
    return t.data_ptr(), _strides(b, n, h)


def _out4(t, like, name):
    """An output like `like`, its pointer and strides; a new contiguous one when None."""
    if t is None:
        t = _TORCH.empty_like(like, memory_format=_TORCH.contiguous_format)
        b, n, h, _ = t.stride()
        return t, t.data_ptr(), _strides(b, n, h)
    return (t, *_rows4(t, name, like.device, like.dtype, like.shape))


_NO_STRIDES = SvStrides(0, 0, 0)


def spec_verify_rotate(q, k, kv_len, freqs, interleaved=False, scale=1.0, inverse=False, rows=None,
                       out=None, stream=None, lib=None):
    """Rotary positions of queries and keys (see include/spec_verify.h).

    q [B, N, q_heads, D] and k [B, N, k_heads, D] or None (bf16 or fp32, any strides with
    consecutive D), kv_len [B] int32 or None (positions from 0), freqs [R/2] float64 (see
    rotary_frequencies): the first R dimensions of a head are turned. inverse turns
    back: with it, gradients of the outputs become gradients of the inputs. rows [B] int32 or None.
    out: a RotateOut, whose tensors may be q and k themselves.
    Returns RotateOut(q, k)."""
    torch = _torch()
    lib = lib or _lib.load()
    qp, qs = _rows4(q, "q")
    dt, dev, (B, N, qh, D) = _dtype_code(q, "q"), q.device, q.shape
    kp, ks, kh = None, _NO_STRIDES, 0
    if k is not None:
        kh = k.shape[2] if k.dim() == 4 else 0
        kp, ks = _rows4(k, "k", dev, q.dtype, (B, N, kh, D))
    if freqs is None or freqs.dim() != 1:
        raise ValueError("freqs must be [R/2] float64")
    R = 2 * freqs.shape[0]
    ctx, handle = _on(dev, stream)
    with ctx:
        oq, oqp, oqs = _out4(out and out.q, q, "out.q")
        ok, okp, oks = (None, None, _NO_STRIDES) if k is None else _out4(out and out.k, k, "out.k")
        rc = lib.spec_verify_rotate(
            qp, qs, kp, ks, dt, B, N, qh, kh, D, R, int(bool(interleaved)), int(bool(inverse)),
            _vector(freqs, "freqs", torch.float64, freqs.shape, dev), float(scale),
            _vector(kv_len, "kv_len", torch.int32, (B,), dev),
            _vector(rows, "rows", torch.int32, (B,), dev), oqp, oqs, okp, oks, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_rotate")
    _written(out)
    return RotateOut(oq, ok)


def spec_verify_cache_bytes(pages, heads, page_size, head_dim):
    return int(_lib.load().spec_verify_cache_bytes(int(pages), int(heads), int(page_size), int(head_dim)))


def kv_cache(pages, heads, page_size, head_dim, device="cuda"):
    """An empty KVCache of this many pages (a power of two of tokens each, 32 or more)."""
    torch = _torch()
    if spec_verify_cache_bytes(pages, heads, page_size, head_dim) == 0:
        raise SpecVerifyError(SV_EINVAL, "kv_cache")
    per = page_size // 32
    k, v = (torch.empty((pages, heads, per, -(-head_dim // 32), 1024), dtype=torch.float8_e4m3fn,
                        device=device) for _ in range(2))
    ks, vs = (torch.empty((pages, heads, per), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs, page_size, head_dim)


def _cache(cache, device):
    """sv_cache of a KVCache."""
    k, v, ks, vs, page, D = cache
    code, f32 = _TORCH.float8_e4m3fn, _TORCH.float32
    shape, small = k.shape, ks.shape
    if len(shape) != 5 or shape[2] * 32 != page or shape[3] != -(-D // 32) or shape[4] != 1024:
        raise ValueError(f"cache.k must be [pages, heads, {page} / 32, ceil({D} / 32), 1024], got {tuple(shape)}")
    where = device.index                    # get_device is the quicker comparison
    if not (v.shape == shape and small == shape[:3] and vs.shape == small and k.dtype == code and v.dtype == code
            and ks.dtype == f32 and vs.dtype == f32 and k.get_device() == where and v.get_device() == where
            and ks.get_device() == where and vs.get_device() == where and k.is_contiguous() and v.is_contiguous()
            and ks.is_contiguous() and vs.is_contiguous()):
        for t, name, dtype, size in ((k, "cache.k", code, shape), (v, "cache.v", code, shape),
                                     (ks, "cache.k_scale", f32, shape[:3]), (vs, "cache.v_scale", f32, shape[:3])):
            _vector(t, name, dtype, size, device)      # which raises
    return SvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), shape[0], shape[1], page, D)


def _table(page_table, B, device):
    if page_table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, width] int32")
    width = page_table.shape[1]
    if width > _MOST:
        raise SpecVerifyError(SV_ESIZE, "page_table")
    return _vector(page_table, "page_table", _torch().int32, (B, width), device), width


def spec_verify_cache_write(cache, page_table, kv_len, k, v, rows=None, stream=None, lib=None):
    """Quantises the rows k, v [B, N, heads, D] (bf16 or fp32, any strides with consecutive D)
    into the cache at positions kv_len[b] .. (see include/spec_verify.h). Rejected rows are written over
    by the next round's; what they leave are coarser codes of far smaller rows in the same block, unless
    that block's committed rows are written again with the new ones.

    cache: a KVCache; page_table [B, width] int32, kv_len [B] int32, rows [B] int32 or None."""
    torch = _torch()
    lib = lib or _lib.load()
    kp, ks = _rows4(k, "k")
    dt, dev, (B, N, heads, D) = _dtype_code(k, "k"), k.device, k.shape
    vp, vs = _rows4(v, "v", dev, k.dtype, k.shape)
    c = _cache(cache, dev)
    if (heads, D) != (c.heads, c.head_dim):
        raise ValueError(f"k must have {c.heads} heads of {c.head_dim}, got {tuple(k.shape)}")
    table, width = _table(page_table, B, dev)
    if kv_len is None:
        raise ValueError("kv_len must be [B] int32")
    ctx, handle = _on(dev, stream)
    with ctx:
        rc = lib.spec_verify_cache_write(
            c, table, width, _vector(kv_len, "kv_len", torch.int32, (B,), dev),
            _vector(rows, "rows", torch.int32, (B,), dev), kp, ks, vp, vs, dt, B, N, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_cache_write")
    _written(cache[:4])


def spec_verify_cache_read(cache, page_table, first, N, dtype=None, rows=None, out=None, stream=None,
                           lib=None):
    """Rows first[b] .. first[b] + N - 1 of every request as values (see
    include/spec_verify.h).

    first [B] int32 or None (from position 0), rows [B] int32 or None; dtype of new outputs
    (torch.bfloat16 when None). out: a CacheRows of [B, N, heads, D] tensors, either may be None.
    Returns CacheRows(k, v)."""
    torch = _torch()
    lib = lib or _lib.load()
    dev = cache.k.device
    if dev.type != "cuda":
        raise ValueError("cache must be on a device")
    c = _cache(cache, dev)
    if page_table is None:
        raise ValueError("page_table must be [B, width] int32")
    B, N = page_table.shape[0], int(N)
    if N > _MOST:
        raise SpecVerifyError(SV_ESIZE, "spec_verify_cache_read")
    table, width = _table(page_table, B, dev)
    shape = (B, N, c.heads, c.head_dim)
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            given = None
            out = CacheRows(*(torch.empty(shape, dtype=dtype or torch.bfloat16, device=dev)
                              for _ in range(2)))
        else:
            given = out
        one = out.k if out.k is not None else out.v
        if one is None:
            raise ValueError("out must have k or v")
        kp, ks = (None, _NO_STRIDES) if out.k is None else _rows4(out.k, "out.k", dev, one.dtype, shape)
        vp, vs = (None, _NO_STRIDES) if out.v is None else _rows4(out.v, "out.v", dev, one.dtype, shape)
        rc = lib.spec_verify_cache_read(
            c, table, width, _vector(first, "first", torch.int32, (B,), dev),
            _vector(rows, "rows", torch.int32, (B,), dev), kp, ks, vp, vs, _dtype_code(one, "out"), B, N,
            handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_cache_read")
    _written(given)
    return out


def spec_verify_attention_workspace_bytes(B, N, q_heads, heads, head_dim, tokens, dtype=SV_BF16):
    return int(_lib.load().spec_verify_attention_workspace_bytes(
        int(B), int(N), int(q_heads), int(heads), int(head_dim), int(tokens), int(dtype)))


@functools.lru_cache(maxsize=256)
def _attention_space(*sizes):
    """The same by sizes alone, without a call into the library each time."""
    return _lib.load().spec_verify_attention_workspace_bytes(*sizes)


def spec_verify_attention(q, cache, page_table, kv_len, scale=None, window=0, rows=None, want_lse=False,
                          workspace=None, out=None, stream=None, lib=None):
    """Attention of a round's rows over the 8-bit cache, which holds them already (see
    include/spec_verify.h).

    q [B, N, q_heads, D] (bf16 or fp32, any strides with consecutive D), N up to SV_MAX_ROWS, q_heads
    a multiple of the cache's heads; page_table [B, width] int32, kv_len [B] int32: tokens
    before the rows; scale of the scores (None: D^-1/2); window: how many positions a row sees, its
    own included (0: all); rows [B] int32 or None. out: an AttentionOut, either of whose tensors may be
    None: out is made then, lse if want_lse is set.
    Returns AttentionOut(out like q, lse [B, N, q_heads] float32 or None)."""
    torch = _torch()
    lib = lib or _lib.load()
    qp, qs = _rows4(q, "q")
    dt, dev, (B, N, qh, D) = _dtype_code(q, "q"), q.device, q.shape
    c = _cache(cache, dev)
    if D != c.head_dim:
        raise ValueError(f"q must have heads of {c.head_dim}, got {tuple(q.shape)}")
    table, width = _table(page_table, B, dev)
    if kv_len is None:
        raise ValueError("kv_len must be [B] int32")
    window = int(window)
    if not 0 <= window <= _MOST:
        raise SpecVerifyError(SV_EINVAL, "spec_verify_attention")
    ctx, handle = _on(dev, stream)
    with ctx:
        o, op, os_ = _out4(out and out.out, q, "out.out")
        lse = out.lse if out is not None else None
        if lse is None and want_lse:
            lse = torch.empty((B, N, qh), dtype=torch.float32, device=dev)
        tokens = width * c.page_size
        if 0 < window + N + 31 < tokens and window:
            tokens = window + N + 31
        ws, ws_bytes, keep = _space(workspace, _attention_space(B, N, qh, c.heads, D, tokens, dt), dev)
        rc = lib.spec_verify_attention(
            qp, qs, dt, B, N, qh, c, table, width, _vector(kv_len, "kv_len", torch.int32, (B,), dev),
            _vector(rows, "rows", torch.int32, (B,), dev), D ** -0.5 if scale is None else float(scale),
            window, op, os_, _vector(lse, "out.lse", torch.float32, (B, N, qh), dev), ws, ws_bytes, handle)
    del keep
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_attention")
    _written(out)
    return AttentionOut(o, lse)


def _rows3(t, name, device=None, dtype=None, shape=None):
    """(pointer, strides) of a [B, N, V] tensor with consecutive V."""
    _on_device(t, name, device, dtype, shape)
    size = t.shape
    if len(size) != 3 or 0 in size:
        raise ValueError(f"{name} must be [B, N, V], none of them 0, got {tuple(size)}")
    if max(size) > _MOST:
        raise SpecVerifyError(SV_ESIZE, name)
    b, n, one = t.stride()
    if one != 1 and size[2] > 1:
        raise ValueError(f"{name} must have consecutive elements in a row")
    return t.data_ptr(), _strides(b, n, 0)


def _id_list(t, name, B, device):
    """(pointer, width) of a [B, n] int32 list, or of none."""
    if t is None or (t.dim() == 2 and t.shape[1] == 0):
        return None, 0
    if t.dim() != 2:
        raise ValueError(f"{name} must be [B, n] int32")
    if t.shape[1] > _MOST:
        raise SpecVerifyError(SV_ESIZE, name)
    return _vector(t, name, _torch().int32, (B, t.shape[1]), device), t.shape[1]


def spec_verify_adjust_logits(logits, tokens=None, history=None, prompt=None, repetition=None,
                              frequency=None, presence=None, bias_ids=None, bias=None, allowed=None,
                              rows=None, out=None, stream=None, lib=None):
    """Penalties, biases and a grammar's mask on a batch's logits (see include/spec_verify.h),
    before they are verified or drawn from: the target rows [B, gamma+1, V] and the
    drafter's [B, gamma, V] alike.

    logits [B, N, V] bf16 or fp32 (any strides with consecutive V), tokens [B, >= N - 1] int32: the
    proposals, of which row j counts those before it; history, prompt [B, n] int32 (-1: padding);
    repetition, frequency, presence [B] float32; bias_ids [B, n] int32 with bias [B, n]
    float32; allowed [B, N, ceil(V / 32)] int32, token v at bit v % 32 of word v / 32; rows [B] int32. All
    but logits may be None. out: a tensor like logits, or logits itself.
    Returns the adjusted logits."""
    torch = _torch()
    lib = lib or _lib.load()
    zp, zs = _rows3(logits, "logits")
    dt, dev, (B, N, V) = _dtype_code(logits), logits.device, logits.shape
    tp, nt = _id_list(tokens, "tokens", B, dev)
    hp, nh = _id_list(history, "history", B, dev)
    pp, np_ = _id_list(prompt, "prompt", B, dev)
    bp, nb = _id_list(bias_ids, "bias_ids", B, dev)
    if (bias is None) != (bias_ids is None):
        raise ValueError("bias_ids and bias come together")
    f32, given = torch.float32, out is not None
    weight = _vector(bias, "bias", f32, (B, nb), dev) if nb else None
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(logits, memory_format=torch.contiguous_format)
        op, os_ = _rows3(out, "out", dev, logits.dtype, (B, N, V))
        rc = lib.spec_verify_adjust_logits(
            zp, zs, dt, B, N, V, _vector(rows, "rows", torch.int32, (B,), dev), tp, nt, hp, nh, pp, np_,
            _vector(repetition, "repetition", f32, (B,), dev), _vector(frequency, "frequency", f32, (B,), dev),
            _vector(presence, "presence", f32, (B,), dev), bp, weight, nb,
            _vector(allowed, "allowed", torch.int32, (B, N, -(-V // 32)), dev), op, os_, handle)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_adjust_logits")
    if given:
        _written((out,))
    return out


def bench_profile_start(max_launches_per_kernel):
    """Starts per-kernel event timing in the benchmark build (_lib.load_bench());
    only calls made with lib=_lib.load_bench() are timed."""
    rc = _lib.load_bench().sv_bench_profile_start(int(max_launches_per_kernel))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "sv_bench_profile_start")


def bench_profile_stop():
    """Returns {kernel name: (total_ms, launches)} since bench_profile_start."""
    import ctypes
    ms = (ctypes.c_double * _lib.SV_NUM_KERNELS)()
    n = (ctypes.c_int32 * _lib.SV_NUM_KERNELS)()
    rc = _lib.load_bench().sv_bench_profile_stop(ctypes.cast(ms, ctypes.c_void_p),
                                                 ctypes.cast(n, ctypes.c_void_p))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "sv_bench_profile_stop")
    return {name: (ms[k], n[k]) for k, name in enumerate(_lib.KERNEL_NAMES)}
