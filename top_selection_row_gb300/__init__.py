"""Exact top-k / top-p candidate-set selection on GB300 (Python binding).

Thin wrappers over the C ABI of ``libqrita.so`` (include/qrita.h) with the
same names. They only marshal arguments: every step of the selection and of
the losses runs in the library's CUDA kernels. PyTorch provides device memory and streams.
"""

from __future__ import annotations

import ctypes
from collections import namedtuple

import numpy as np

from ._lib import EXPORTED, lib  # noqa: F401

DTYPE_F32 = 0
DTYPE_BF16 = 1

OK, EINVAL, EUNSUPPORTED, ECUDA = 0, 1, 2, 3
ROW_OK, ROW_NONFINITE, ROW_SEARCH_CAP, ROW_TIMEOUT = 0, 1, 2, 3

FLAG_NO_TRUNCATION = 0x1
FLAG_FORCE_FALLBACK = 0x2
FLAG_KEY_PIVOTS = 0x4
FLAG_FORCE_RETRY = 0x8
FLAG_HIST_MISS = 0x10
FLAG_CLUSTER_SET = 0x800
FLAG_TEST_GIVE_UP = 0x1000
FLAG_NO_KEY_HIST = 0x2000
FLAG_SEARCH_QUATERNARY = 0x4000
FLAG_SEARCH_BINARY = 0x8000
LOSS_FLAG_TEST_GIVE_BACK = 0x1


def flag_cluster(n_ctas: int) -> int:
    """Flags that force ``n_ctas`` (1, 2, 4, 8 or 16) CTAs per row."""
    shift = {1: 0, 2: 1, 4: 2, 8: 3, 16: 4}[n_ctas]
    return FLAG_CLUSTER_SET | (shift << 8)


PATH_TOPK, PATH_TOPP, PATH_TRUNC, PATH_HIT = 0x1, 0x2, 0x4, 0x8
PATH_FALLBACK, PATH_OVERFLOW, PATH_KEEP_ALL, PATH_RETRY = 0x10, 0x20, 0x40, 0x80
PATH_HIST = 0x100
PATH_SAMPLE_T = 0x200
PATH_KEYHIST = 0x400

# Layout of qrita_row_info_t (64 bytes).
ROW_INFO_DTYPE = np.dtype(
    [
        ("mu", "<f4"),
        ("sigma", "<f4"),
        ("threshold", "<f4"),
        ("row_max", "<f4"),
        ("survivors", "<u4"),
        ("path", "<u4"),
        ("rounds_k", "<u4"),
        ("rounds_p", "<u4"),
        ("boundary", "<f4"),
        ("n_boundary", "<u4"),
        ("kept", "<u4"),
        ("status", "<u4"),
        ("z", "<f8"),
        ("passes", "<u4"),
        ("reserved", "<u4"),
    ]
)
assert ROW_INFO_DTYPE.itemsize == 64


class QritaError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"qrita error {code}: {strerror(code)}")


def strerror(code: int) -> str:
    return lib().qrita_strerror(int(code)).decode()


def version() -> int:
    return int(lib().qrita_version())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _check_rows(logits):
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor (use qrita_select_host for host buffers)")
    B, V = logits.shape
    if B > 0 and (logits.stride(1) != 1 or (B > 1 and logits.stride(0) != V)):
        raise ValueError("logits must be row-major with leading dimension V")
    return B, V


def _vec(t, n, dtype, name, device):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        t = torch.as_tensor(t)
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")
    return t


def _tensors(values):
    """The CUDA tensors among values and the tuples they hold."""
    for v in values:
        if isinstance(v, (tuple, list)):
            yield from _tensors(v)
        elif isinstance(v, _torch().Tensor) and v.is_cuda:
            yield v


def _on_stream(stream, fn, *args):
    """fn(*args) with ``stream`` as the current one: what the call allocates
    comes from that stream's memory, whose last use is ordered before the
    call's kernels (a block of another stream may still be read or written
    there). The arguments are marked as used on ``stream`` and the results as
    used on the caller's, so that neither's memory is handed out again before
    that stream is done with it."""
    torch = _torch()
    dev = stream.device
    if args[0].is_cuda and args[0].device != dev:
        raise ValueError(f"stream must be one of the logits' device, not of {dev}")
    if stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev.index):
        return fn(*args)
    caller = torch.cuda.current_stream(dev)
    if torch.cuda.current_device() == dev.index:
        torch.cuda.set_stream(stream)  # (as the context below, some 6 us sooner)
        try:
            got = fn(*args)
        finally:
            torch.cuda.set_stream(caller)
    else:
        with torch.cuda.stream(stream):
            got = fn(*args)
    given = list(_tensors(args))
    for t in given:
        t.record_stream(stream)
    for t in _tensors((got,)):
        if not any(t is g for g in given):
            t.record_stream(caller)
    return got


def _wrote(*tensors):
    """Raises the versions of tensors that the caller gave and a call has written
    through their addresses, as an in-place operation does: autograd then refuses
    a backward pass that has saved one of them, instead of reading what is there
    now."""
    torch = _torch()
    torch.autograd.graph.increment_version([t for t in tensors if t is not None and not t.is_inference()])


def _stream_ptr(device):
    return ctypes.c_void_p(_torch()._C._cuda_getCurrentRawStream(device.index))


def qrita_select(logits, k=None, p=None, out=None, stream=None):
    """Keep-mask of the exact top-k / top-p candidate set of every row.

    logits: CUDA tensor [B, V], float32 or bfloat16, row-major.
    k: CUDA int32 [B] or None (top-k off); p: CUDA float32 [B] or None.
    out: optional CUDA bool/uint8 tensor [B, V]. Returns the mask (bool).
    The kernel is enqueued on ``stream`` (default: the current stream), where
    the caller sees to it that the inputs are ready.
    """
    return qrita_select_ex(logits, k, p, out=out, stream=stream)[0]


def qrita_select_ex(logits, k=None, p=None, out=None, stream=None, flags=0,
                    row_status=False, row_info=False):
    """qrita_select plus path flags, per-row status and per-row diagnostics.

    Returns (mask, status or None, info or None); ``status`` is a CUDA int32
    [B] tensor, ``info`` a CUDA uint8 [B, 64] tensor holding
    qrita_row_info_t records (decode with :func:`decode_row_info`).
    """
    if stream is not None:
        return _on_stream(stream, qrita_select_ex, logits, k, p, out, None, flags, row_status, row_info)
    torch = _torch()
    B, V = _check_rows(logits)
    dev = logits.device
    dt = _dtype_code(logits)
    kk = _vec(k, B, torch.int32, "k", dev)
    pp = _vec(p, B, torch.float32, "p", dev)
    given = out
    if out is None:
        out = torch.empty((B, V), dtype=torch.bool, device=dev)
    elif out.shape != (B, V) or out.dtype not in (torch.bool, torch.uint8) or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous bool/uint8 [B, V] tensor on the logits' device")
    st = torch.empty(B, dtype=torch.int32, device=dev) if row_status else None
    info = torch.empty((B, 64), dtype=torch.uint8, device=dev) if row_info else None
    rc = lib().qrita_select_ex(
        ctypes.c_void_p(logits.data_ptr() if B else 0),
        dt,
        B,
        V,
        ctypes.c_void_p(kk.data_ptr() if kk is not None else 0),
        ctypes.c_void_p(pp.data_ptr() if pp is not None else 0),
        ctypes.c_void_p(out.data_ptr() if B else 0),
        _stream_ptr(dev),
        ctypes.c_uint32(flags),
        ctypes.c_void_p(st.data_ptr() if st is not None else 0),
        ctypes.c_void_p(info.data_ptr() if info is not None else 0),
    )
    if rc != OK:
        raise QritaError(rc)
    if given is not None:
        _wrote(given)
    return out, st, info


def decode_row_info(info) -> np.ndarray:
    """qrita_row_info_t records (CUDA uint8 [B, 64]) as a numpy structured array."""
    raw = info.detach().cpu().numpy()
    return np.ascontiguousarray(raw).view(ROW_INFO_DTYPE).reshape(-1)


def qrita_topk_ids(logits, k, kmax, out_mask=None, out_ids=None, stream=None):
    """Top-k ids of every row in stable order (logit descending, lower id
    first among equals) through qrita_topk_ids.

    logits: CUDA [B, V] float32 / bfloat16; k: CUDA int32 [B]; kmax: 1..8192.
    Returns (ids int32 [B, kmax], padded with -1; mask bool [B, V]).
    """
    if stream is not None:
        return _on_stream(stream, qrita_topk_ids, logits, k, kmax, out_mask, out_ids)
    torch = _torch()
    B, V = _check_rows(logits)
    dev = logits.device
    kk = _vec(k, B, torch.int32, "k", dev)
    if kk is None:
        raise ValueError("k is required")
    given = out_ids, out_mask
    if out_mask is None:
        out_mask = torch.empty((B, V), dtype=torch.bool, device=dev)
    if out_ids is None:
        out_ids = torch.empty((B, int(kmax)), dtype=torch.int32, device=dev)
    elif out_ids.shape != (B, int(kmax)) or out_ids.dtype != torch.int32 or not out_ids.is_contiguous():
        raise ValueError("out_ids must be a contiguous int32 [B, kmax] tensor")
    rc = lib().qrita_topk_ids(
        ctypes.c_void_p(logits.data_ptr() if B else 0), _dtype_code(logits), B, V,
        ctypes.c_void_p(kk.data_ptr()), int(kmax), ctypes.c_void_p(out_mask.data_ptr() if B else 0),
        ctypes.c_void_p(out_ids.data_ptr() if B else 0), _stream_ptr(dev))
    if rc != OK:
        raise QritaError(rc)
    _wrote(*given)
    return out_ids, out_mask


def qrita_candidates(logits, mask, cap, u=None, stream=None, out=None):
    """Kept ids in id order with probabilities renormalised over the kept set,
    the kept count, and (with u: CUDA float32 [B]) one token drawn per row,
    through qrita_candidates. Returns (ids [B, cap], probs [B, cap], count [B],
    sample [B] or None). Without ``out`` the entries past a row's count are
    -1 / 0; ``out`` = (ids, probs, count, sample) reuses the caller's buffers
    (contiguous int32 [B, cap], float32 [B, cap], int32 [B], int32 [B] or
    None exactly when u is), whose entries past a row's count are left as
    they were."""
    if stream is not None:
        return _on_stream(stream, qrita_candidates, logits, mask, cap, u, None, out)
    torch = _torch()
    B, V = _check_rows(logits)
    dev = logits.device
    if mask.shape != (B, V) or mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous bool/uint8 [B, V] tensor")
    uu = _vec(u, B, torch.float32, "u", dev)
    if out is None:
        ids = torch.full((B, int(cap)), -1, dtype=torch.int32, device=dev)
        probs = torch.zeros((B, int(cap)), dtype=torch.float32, device=dev)
        count = torch.empty(B, dtype=torch.int32, device=dev)
        sample = torch.empty(B, dtype=torch.int32, device=dev) if uu is not None else None
    else:
        ids, probs, count, sample = out
        for t, shape, dt, name in ((ids, (B, int(cap)), torch.int32, "ids"), (probs, (B, int(cap)), torch.float32, "probs"),
                                   (count, (B,), torch.int32, "count")):
            if t.shape != shape or t.dtype != dt or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"out {name} must be a contiguous {dt} {list(shape)} tensor on {dev}")
        if (sample is None) != (uu is None):
            raise ValueError("out sample must be given exactly when u is")
        if sample is not None and (sample.shape != (B,) or sample.dtype != torch.int32 or not sample.is_contiguous()
                                   or sample.device != dev):
            raise ValueError(f"out sample must be a contiguous int32 [{B}] tensor on {dev}")
    rc = lib().qrita_candidates(
        ctypes.c_void_p(logits.data_ptr() if B else 0), _dtype_code(logits), B, V,
        ctypes.c_void_p(mask.data_ptr() if B else 0), int(cap), ctypes.c_void_p(ids.data_ptr() if B else 0),
        ctypes.c_void_p(probs.data_ptr() if B else 0), ctypes.c_void_p(count.data_ptr() if B else 0),
        ctypes.c_void_p(uu.data_ptr() if uu is not None else 0),
        ctypes.c_void_p(sample.data_ptr() if sample is not None else 0), _stream_ptr(dev))
    if rc != OK:
        raise QritaError(rc)
    if out is not None:
        _wrote(ids, probs, count, sample)
    return ids, probs, count, sample


def delta_table(which: int) -> np.ndarray:
    """The host-built truncation table the kernel receives: ``which`` 0 is the
    top-k table (entry i = Phi^-1(1 - 2^(-i/4))), 1 the top-p table (entry
    i = Phi^-1(2^(-i/4))). Returns float32 [length]."""
    n = int(lib().qrita_delta_table(int(which), None, 0))
    if n < 0:
        raise ValueError(f"unknown delta table {which}")
    out = np.zeros(n, np.float32)
    lib().qrita_delta_table(int(which), out.ctypes.data_as(ctypes.c_void_p), n)
    return out


def host_staging_bytes(dtype_code: int, B: int, V: int) -> int:
    return int(lib().qrita_host_staging_bytes(int(dtype_code), int(B), int(V)))


def qrita_select_host(logits, k=None, p=None, out=None, staging=None, stream=None):
    """End-to-end selection for HOST (CPU) tensors through qrita_select_host.

    logits: CPU tensor [B, V] float32 / bfloat16 (pinned for full-speed
    copies); k / p: CPU int32 / float32 [B] or None; out: CPU uint8/bool
    [B, V] or None; staging: CUDA uint8 tensor of at least
    host_staging_bytes(...) bytes (allocated here when None). Returns ``out``
    after the stream has finished.
    """
    if stream is not None:
        return _on_stream(stream, qrita_select_host, logits, k, p, out, staging)
    torch = _torch()
    if logits.dim() != 2 or logits.is_cuda:
        raise ValueError("logits must be a host [B, V] tensor")
    B, V = logits.shape
    if B > 0 and (logits.stride(1) != 1 or (B > 1 and logits.stride(0) != V)):
        raise ValueError("logits must be row-major with leading dimension V")
    dt = _dtype_code(logits)
    cpu = torch.device("cpu")
    kk = _vec(k, B, torch.int32, "k", cpu)
    pp = _vec(p, B, torch.float32, "p", cpu)
    given = out
    if out is None:
        out = torch.empty((B, V), dtype=torch.bool, pin_memory=logits.is_pinned())
    need = host_staging_bytes(dt, B, V)
    dev = torch.device("cuda", torch.cuda.current_device())
    if staging is None:
        staging = torch.empty(need, dtype=torch.uint8, device=dev)
    elif staging.numel() < need or not staging.is_cuda:
        raise ValueError(f"staging must be a CUDA tensor of at least {need} bytes")
    rc = lib().qrita_select_host(
        ctypes.c_void_p(logits.data_ptr() if B else 0),
        dt,
        B,
        V,
        ctypes.c_void_p(kk.data_ptr() if kk is not None else 0),
        ctypes.c_void_p(pp.data_ptr() if pp is not None else 0),
        ctypes.c_void_p(out.data_ptr() if B else 0),
        ctypes.c_void_p(staging.data_ptr()),
        ctypes.c_size_t(staging.numel()),
        _stream_ptr(staging.device),
    )
    if rc != OK:
        raise QritaError(rc)
    if given is not None:
        _wrote(given)
    return out


# ---------------------------------------------------------------------------
# Losses over rows of logits
# ---------------------------------------------------------------------------
PolicyLoss = namedtuple("PolicyLoss", "loss grad row_loss logp kl entropy")
PreferenceLoss = namedtuple("PreferenceLoss", "loss grad pair_loss log_ratio seq_logp logp")


# stream= runs a call on another stream than the current one. The caller sees to
# it that its inputs are ready there, and waits for it before the results are used
# elsewhere; both may be dropped at any time.
#
# (These calls take 3 to 13 us on the GPU for a small batch, so what they do on
# the host is kept short: plain integers as pointers, one test per property.)
def _padded_rows(t, name="logits"):
    """B, V and the leading dimension of [B, V] rows that may be padded."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [B, V]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    B, V = t.shape
    ld, unit = t.stride()
    if B < 2:
        ld = V
    if V < 1 or (B > 0 and ((V > 1 and unit != 1) or ld < V)):
        raise ValueError(f"{name} must be row-major: unit stride within a row, a leading dimension of at least V")
    return B, V, ld


def _at(t, n, dtype, name, device):
    """Address of a contiguous vector of n elements; 0 for None or an empty one."""
    if t is None:
        return 0
    if not isinstance(t, _torch().Tensor) or t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")
    return t.data_ptr()


def _needed(t, n, dtype, name, device):
    if t is None:
        raise ValueError(f"{name} is required")
    return _at(t, n, dtype, name, device)


def _mask_at(mask, B, V, device):
    torch = _torch()
    if mask is None:
        return 0
    if mask.shape != (B, V) or mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous() or mask.device != device:
        raise ValueError("mask must be a contiguous bool/uint8 [B, V] tensor on the logits' device")
    return mask.data_ptr()


def _grad_rows(out, logits, B, V):
    """The gradient's tensor and its leading dimension."""
    if out is None:
        return _torch().empty((B, V), dtype=logits.dtype, device=logits.device), V
    if out.shape != (B, V) or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError("the gradient must be a [B, V] tensor of the logits' type on their device")
    return out, _padded_rows(out, "the gradient")[2]


def _call(fn, device, *args):
    """Calls fn(*args, stream) on the current stream, with the logits' device
    as the current one."""
    torch = _torch()
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != OK:
        raise QritaError(rc)


def qrita_token_logprobs(logits, tokens, mask=None, inv_temperature=1.0, entropy=False, stream=None, out=None):
    """Log-probability of one given token per row, and the row's entropy.

    logits: CUDA [B, V] float32 / bfloat16 (rows may be padded: any leading
    dimension >= V); tokens: CUDA int32 [B], a token outside [0, V) ignores
    its row; mask: bool/uint8 [B, V] or None, the kept set the softmax runs
    over (e.g. qrita_select's output). Returns (logp float32 [B], entropy
    float32 [B] or None); ``out`` = such a pair reuses the caller's buffers.
    include/qrita.h states the row contract.
    """
    if stream is not None:
        return _on_stream(stream, qrita_token_logprobs, logits, tokens, mask, inv_temperature, entropy, None, out)
    torch = _torch()
    B, V, ld = _padded_rows(logits)
    dev = logits.device
    dt = _dtype_code(logits)
    tok = _needed(tokens, B, torch.int32, "tokens", dev)
    keep = _mask_at(mask, B, V, dev)
    if out is None:
        logp = torch.empty(B, dtype=torch.float32, device=dev)
        ent = torch.empty(B, dtype=torch.float32, device=dev) if entropy else None
    else:
        logp, ent = out
        _needed(logp, B, torch.float32, "out logp", dev)
        if entropy:
            _needed(ent, B, torch.float32, "out entropy", dev)
    _call(lib().qrita_token_logprobs, dev, logits.data_ptr(), dt, B, V, ld, keep, tok,
          inv_temperature, logp.data_ptr(), ent.data_ptr() if entropy else 0)
    ent = ent if entropy else None
    if out is not None:
        _wrote(logp, ent)
    return logp, ent


def qrita_token_logprobs_grad(logits, tokens, grad_logp=None, grad_entropy=None, mask=None, inv_temperature=1.0,
                              out_grad=None, stream=None):
    """Gradient with respect to the logits of any function of
    qrita_token_logprobs' outputs, from the gradients of those outputs
    (float32 [B] each; one may be None). Returns the gradient, [B, V] of the
    logits' type; ``out_grad`` gives its tensor (rows may be padded, and it
    may be the logits themselves)."""
    if stream is not None:
        return _on_stream(stream, qrita_token_logprobs_grad, logits, tokens, grad_logp, grad_entropy, mask,
                          inv_temperature, out_grad)
    torch = _torch()
    B, V, ld = _padded_rows(logits)
    dev = logits.device
    dt = _dtype_code(logits)
    tok = _needed(tokens, B, torch.int32, "tokens", dev)
    keep = _mask_at(mask, B, V, dev)
    gl = _at(grad_logp, B, torch.float32, "grad_logp", dev)
    ge = _at(grad_entropy, B, torch.float32, "grad_entropy", dev)
    if grad_logp is None and grad_entropy is None:
        raise ValueError("one of grad_logp and grad_entropy is required")
    grad, ldg = _grad_rows(out_grad, logits, B, V)
    _call(lib().qrita_token_logprobs_grad, dev, logits.data_ptr(), dt, B, V, ld, keep, tok, inv_temperature, gl, ge,
          grad.data_ptr(), ldg)
    if out_grad is not None:
        _wrote(grad)
    return grad


def qrita_policy_loss(logits, tokens, old_logp, advantages, ref_logp=None, weights=None, mask=None, inv_temperature=1.0,
                      clip_low=0.2, clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, grad_loss=None, grad=True,
                      entropy=False, out_grad=None, stream=None, out=None, flags=0):
    """The clipped policy loss with a KL term over rows of logits, and its
    gradient with respect to them, in one call.

    logits, tokens, mask, inv_temperature: as qrita_token_logprobs.
    old_logp (None: on-policy), ref_logp (None: no KL term), advantages,
    weights (None: 1 / B): CUDA float32 [B]. grad_loss: CUDA float32 of one
    element that multiplies the gradient, or None. grad=False leaves the
    gradient out; entropy=True returns the entropies even where entropy_coef
    is 0. Returns PolicyLoss(loss [], grad [B, V] or None, row_loss [B],
    logp [B], kl [B], entropy [B] or None); ``out`` = such a tuple, as an
    earlier call returned it, reuses its tensors. flags: qrita_policy_loss_ex's.
    """
    if stream is not None:
        return _on_stream(stream, qrita_policy_loss, logits, tokens, old_logp, advantages, ref_logp, weights, mask,
                          inv_temperature, clip_low, clip_high, kl_coef, entropy_coef, grad_loss, grad, entropy,
                          out_grad, None, out, flags)
    torch = _torch()
    B, V, ld = _padded_rows(logits)
    dev = logits.device
    f32 = torch.float32
    dt = _dtype_code(logits)
    tok = _needed(tokens, B, torch.int32, "tokens", dev)
    keep = _mask_at(mask, B, V, dev)
    old = _at(old_logp, B, f32, "old_logp", dev)
    ref = _at(ref_logp, B, f32, "ref_logp", dev)
    adv = _needed(advantages, B, f32, "advantages", dev)
    w = _at(weights, B, f32, "weights", dev)
    gl = _at(grad_loss, 1, f32, "grad_loss", dev)
    want_ent = entropy or entropy_coef != 0
    if out is None:
        # (a tensor each: a view of a shared one takes longer to make and free)
        loss = torch.empty((), dtype=f32, device=dev)
        row_loss = torch.empty(B, dtype=f32, device=dev)
        logp = torch.empty_like(row_loss)
        kl = torch.empty_like(row_loss)
        ent = torch.empty_like(row_loss) if want_ent else None
    else:
        loss, given, row_loss, logp, kl, ent = out
        _needed(loss, 1, f32, "out loss", dev)
        for name, t in (("row_loss", row_loss), ("logp", logp), ("kl", kl), ("entropy", ent)):
            if name != "entropy" or want_ent:
                _needed(t, B, f32, "out " + name, dev)
        out_grad = given if out_grad is None else out_grad
        ent = ent if want_ent else None
    g, ldg = _grad_rows(out_grad, logits, B, V) if grad else (None, 0)
    fn, more = (lib().qrita_policy_loss, ()) if flags == 0 else (lib().qrita_policy_loss_ex, (flags,))
    _call(fn, dev, logits.data_ptr(), dt, B, V, ld, keep, tok, inv_temperature, old,
          ref, adv, w, clip_low, clip_high, kl_coef, entropy_coef, gl, loss.data_ptr(),
          row_loss.data_ptr(), logp.data_ptr(), kl.data_ptr(), ent.data_ptr() if want_ent else 0,
          g.data_ptr() if grad else 0, ldg, *more)
    if out is not None:
        _wrote(loss, row_loss, logp, kl, ent, g)
    elif out_grad is not None:
        _wrote(g)
    return PolicyLoss(loss, g, row_loss, logp, kl, ent)


def preference_workspace_bytes(B: int, P: int) -> int:
    return int(lib().qrita_preference_workspace_bytes(int(B), int(P)))


def qrita_preference_loss(logits, tokens, starts, ref_logp=None, weights=None, inv_temperature=1.0, beta=0.1,
                          label_smoothing=0.0, margin=0.0, length_norm=False, grad_loss=None, grad=True, out_grad=None,
                          workspace=None, stream=None, out=None):
    """The preference loss on paired log ratios over rows of logits, and its
    gradient with respect to them.

    logits, tokens, inv_temperature: as qrita_token_logprobs, the rows of all
    sequences one after another. starts: CUDA int32 [2 P + 1], sequence s owns
    rows [starts[s], starts[s + 1]); sequence 2i is the preferred one of pair
    i, 2i + 1 the rejected one. ref_logp: float32 [2 P] or None; weights:
    float32 [P] or None (1 / P); grad_loss as qrita_policy_loss. workspace:
    CUDA uint8 of at least preference_workspace_bytes(B, P), one for each call
    that may run at the same time (allocated here when None). Returns
    PreferenceLoss(loss [], grad [B, V] or None, pair_loss [P], log_ratio [P],
    seq_logp [2 P], logp [B]); ``out`` as qrita_policy_loss.
    """
    if stream is not None:
        return _on_stream(stream, qrita_preference_loss, logits, tokens, starts, ref_logp, weights, inv_temperature, beta,
                          label_smoothing, margin, length_norm, grad_loss, grad, out_grad, workspace, None, out)
    torch = _torch()
    B, V, ld = _padded_rows(logits)
    dev = logits.device
    f32 = torch.float32
    dt = _dtype_code(logits)
    tok = _needed(tokens, B, torch.int32, "tokens", dev)
    if starts is None:
        raise ValueError("starts is required")
    n = starts.numel()
    if n % 2 == 0:
        raise ValueError("starts must hold 2 P + 1 elements")
    P = n // 2
    at = _at(starts, n, torch.int32, "starts", dev)
    ref = _at(ref_logp, 2 * P, f32, "ref_logp", dev)
    w = _at(weights, P, f32, "weights", dev)
    gl = _at(grad_loss, 1, f32, "grad_loss", dev)
    need = preference_workspace_bytes(B, P)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {dev}")
    if out is None:
        loss = torch.empty((), dtype=f32, device=dev)
        pair_loss = torch.empty(P, dtype=f32, device=dev)
        ratio = torch.empty_like(pair_loss)
        seq = torch.empty(2 * P, dtype=f32, device=dev)
        logp = torch.empty(B, dtype=f32, device=dev)
    else:
        loss, given, pair_loss, ratio, seq, logp = out
        for name, t, n in (("loss", loss, 1), ("pair_loss", pair_loss, P), ("log_ratio", ratio, P), ("seq_logp", seq, 2 * P),
                           ("logp", logp, B)):
            _needed(t, n, f32, "out " + name, dev)
        out_grad = given if out_grad is None else out_grad
    g, ldg = _grad_rows(out_grad, logits, B, V) if grad else (None, 0)
    _call(lib().qrita_preference_loss, dev, logits.data_ptr(), dt, B, V, ld, tok, inv_temperature, at,
          P, ref, w, beta, label_smoothing, margin, 1 if length_norm else 0, gl,
          loss.data_ptr(), pair_loss.data_ptr(), ratio.data_ptr(), seq.data_ptr(), logp.data_ptr(),
          g.data_ptr() if grad else 0, ldg, workspace.data_ptr(), workspace.numel())
    if out is not None:
        _wrote(loss, pair_loss, ratio, seq, logp, g)
    elif out_grad is not None:
        _wrote(g)
    return PreferenceLoss(loss, g, pair_loss, ratio, seq, logp)
