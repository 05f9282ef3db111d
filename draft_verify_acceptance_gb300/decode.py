"""ctypes binding of the decode-side operators (include/spec_decode.h).

    paged_attention   the newest Q tokens' attention over a paged key-value cache
    cache_append      new tokens' keys and values into their pages
    cache_fork        the next step's sequences: fork, trim, end, reorder, reserve
    cache_compact     pages in use to the front of the pool
    filtered_sample   temperature, top-k, min-p and top-p from given uniforms

As in ``binding``, every step runs in the library's CUDA kernels; this module checks
tensors, owns a workspace per (device, stream) and passes pointers.  There is no CPU
fallback.  The workspaces (spec_decode.h gives their sizes) are kept for good, or may be
the caller's by ``workspace``.  Calls are queued on ``stream`` (default: the current stream); with
``debug=True`` they also return the device status word (OR of DATA_* bits).

A cache tensor is [pages, page_size, heads, head_dim], or with a leading layers
dimension for cache_fork and cache_compact; the last two dimensions are contiguous, the
other strides free (a layer of a larger tensor, K and V interleaved), the same for K
and V.

These are operators of inference: their results carry no gradient, also where an input requires
one, and grad mode makes no difference.  What they write in place (a cache's tensors, ``out``) counts
as changed for autograd, so a backward pass that needs the earlier values raises.

A page table is int32 [B, max_pages]; its rows may be strided or one row
expanded to all sequences, but not overlap otherwise.
"""
import ctypes
import threading
from typing import NamedTuple

import torch

from . import _decode_calls
from .binding import (DTYPE_BF16, DTYPE_F32, ERR_INVALID_ARG, ERR_UNSUPPORTED, LIB_PATH, MAX_V, OK,
                      SpecVerifyError)

# Most calls are several launches on one kept workspace, and threads on one stream share it.  So a call keeps
# the interpreter's lock from its first launch to its last (PyDLL), as the native ones do.
_lib = ctypes.PyDLL(LIB_PATH)

DATA_PAGE_RANGE = 64
DATA_LENGTH_RANGE = 128
DATA_CACHE_FULL = 256
DATA_PARAM_RANGE = 512

EXPORTS = ("spec_attention_workspace_size", "spec_paged_attention", "spec_cache_append",
           "spec_cache_fork_workspace_size", "spec_cache_fork", "spec_cache_compact_workspace_size",
           "spec_cache_compact", "spec_filtered_sample_workspace_size", "spec_filtered_sample")


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("layers", ctypes.c_int),
                ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


def _declare():
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    C = ctypes.POINTER(_Cache)
    sig = {
        "spec_attention_workspace_size": (Z, [I] * 6),
        "spec_paged_attention": (I, [P, L, L, L, C, P, L, I, P, I, I, I, F, P, P, P, Z, P, P]),
        "spec_cache_append": (I, [P, P, L, I, P, C, P, L, I, P, I, P, P]),
        "spec_cache_fork_workspace_size": (Z, [I, I]),
        "spec_cache_fork": (I, [C, P, L, I, P, I, P, P, I, I, P, P, P, P, P, P, Z, P, P]),
        "spec_cache_compact_workspace_size": (Z, [I]),
        "spec_cache_compact": (I, [C, P, L, I, I, P, P, P, P, Z, P, P]),
        "spec_filtered_sample_workspace_size": (Z, [I, I, I]),
        "spec_filtered_sample": (I, [P, L, P, I, I, I, F, I, F, F, P, P, P, P, P, P, P, P, P, Z, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = res, args


_declare()
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_ws_lock = threading.Lock()
_ws = {}
# the native calls' number of a kind of workspace, and how many of its first bytes are zero between calls
_KINDS = {"attention": (0, 2048), "fork": (1, 0), "compact": (2, 0), "sample": (3, 64)}


class ForkResult(NamedTuple):
    page_table: torch.Tensor  # int32 [C, max_pages]
    lengths: torch.Tensor     # int32 [C]
    ref_counts: torch.Tensor  # int32 [pages]
    free_pages: torch.Tensor  # int32 [pages]: ascending, then -1
    n_free: torch.Tensor      # int32 [1]
    status: torch.Tensor      # int32 [1] with debug, else None


class CompactResult(NamedTuple):
    page_table: torch.Tensor  # int32 [B, max_pages]
    ref_counts: torch.Tensor  # int32 [pages]
    n_live: torch.Tensor      # int32 [1]
    status: torch.Tensor      # int32 [1] with debug, else None


class SampleResult(NamedTuple):
    tokens: torch.Tensor      # int32 [...]
    p: torch.Tensor           # float32 [...]
    n_kept: torch.Tensor      # int32 [...]
    filtered: torch.Tensor    # [..., V] in the logits' dtype, or None
    status: torch.Tensor      # int32 [1] with debug, else None


_decode_calls.bind(tuple(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in EXPORTS), ForkResult, CompactResult,
                   SampleResult)

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object


def _fit_workspace(kind, nbytes, index):
    """A workspace whose first bytes are zero as far as its kind needs it (filled whole, a captured call's tens of
    megabytes took longer than the call)."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
    zero = _KINDS[kind][1]
    if zero:
        ws[:zero].zero_()
    return ws


def _workspace(kind, index, stream, nbytes, given):
    """(pointer, bytes, what owns them): the caller's workspace, or one kept for this kind of call, device and
    stream; every call leaves it fit for the next.  A call that a CUDA graph captures gets one of its own, made fit
    by the graph: a kept one may be replaced by a larger one before a replay."""
    if given is not None:
        if given.get_device() != index or not given.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{index}")
        if given.numel() * given.element_size() < nbytes:
            raise ValueError(f"workspace holds {given.numel() * given.element_size()} bytes, {nbytes} are needed")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if nbytes == 0:
        return None, 0, None
    if torch.cuda.is_current_stream_capturing():
        ws = _fit_workspace(kind, nbytes, index)
        return ws.data_ptr(), nbytes, ws
    key = (kind, index, stream)
    kept = _ws.get(key)
    if kept is None or kept[2] < nbytes:
        with _ws_lock:
            kept = _ws.get(key)
            if kept is None or kept[2] < nbytes:
                ws = _fit_workspace(kind, nbytes, index)
                kept = _ws[key] = (ws, ws.data_ptr(), nbytes)
                _decode_calls.register_workspace(_KINDS[kind][0], index, stream, kept[1], nbytes)
    return kept[1], kept[2], kept[0]


def _on_stream(fn):
    """Runs a call with its device and, when one is given, its stream current, so that what it allocates
    belongs to the stream that uses it; passes the device's index and the stream's handle."""
    native = getattr(_decode_calls, fn.__name__)

    def call(*args, **kw):
        r = native(*args, **kw)  # the ordinary call; what it does not do comes back
        return slow(*args, **kw) if r is NotImplemented else r

    def slow(first, *args, stream=None, **kw):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            where = first.device if isinstance(first, torch.Tensor) else type(first).__name__
            raise ValueError(f"{fn.__name__} takes CUDA tensors (got {where})")
        index = first.get_device()
        if stream is not None:
            with torch.cuda.stream(stream):
                return fn((index, stream.cuda_stream), first, *args, **kw)
        if index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return fn((index, _raw_stream(index)), first, *args, **kw)
        return fn((index, _raw_stream(index)), first, *args, **kw)
    call.__name__, call.__doc__, call.__wrapped__ = fn.__name__, fn.__doc__, fn
    return call


def _ints(t, name, shape, index):
    """The pointer of a contiguous int32 tensor of a shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)} on cuda:{index}, "
                         f"got {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, B, index):
    """(pointer, row stride, max_pages) of a page table.  Its rows may be strided, or one row expanded to all."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError("page_table must be an int32 tensor")
    if t.dim() != 2 or t.shape[0] != B or t.get_device() != index:
        raise ValueError(f"page_table must be [{B}, max_pages] on cuda:{index}, got {tuple(t.shape)} on {t.device}")
    M = t.shape[1]
    if t.is_contiguous():
        return t.data_ptr(), M, M
    if M > 1 and t.stride(1) != 1:
        raise ValueError("page_table rows must be contiguous")
    stride = t.stride(0) if B > 1 else M
    if 0 < stride < M:
        raise ValueError("page_table rows must not overlap")
    return t.data_ptr(), stride, M


def _cache(k, v, layered, index):
    dtype = k.dtype
    dt = _DTYPES.get(dtype)
    if dt is None or v.dtype is not dtype:
        raise TypeError(f"k_pages and v_pages must both be float32 or bfloat16, got {k.dtype} and {v.dtype}")
    shape, stride = k.shape, k.stride()
    dims = len(shape)
    if dims != 4 and not (layered and dims == 5):
        raise ValueError("a cache tensor is [pages, page_size, heads, head_dim]"
                         + (" or [layers, pages, page_size, heads, head_dim]" if layered else ""))
    if v.shape != shape or v.stride() != stride or k.get_device() != index or v.get_device() != index:
        raise ValueError("k_pages and v_pages must have the same shape, strides and device")
    if dims == 5:
        L, P, S, H, D = shape
        ls, ps, ts, hs, ds = stride
    else:
        (P, S, H, D), (ps, ts, hs, ds) = shape, stride
        L, ls = 1, 0
    if (D > 1 and ds != 1) or (H > 1 and hs != D):
        raise ValueError("the last two dimensions (heads, head_dim) of a cache tensor must be contiguous")
    return _Cache(k.data_ptr(), v.data_ptr(), ls, ps, ts if S > 1 else max(ts, H * D), L, P, S, H, D, dt)


def _written(*tensors):
    """Tells autograd that tensors were changed in place."""
    for t in tensors:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _raise(rc, what):
    raise SpecVerifyError(rc, what)


def _status(debug, device):
    """The status word (None without debug) and its pointer."""
    if not debug:
        return None, None
    t = torch.zeros(1, dtype=torch.int32, device=device)
    return t, t.data_ptr()


def attention_workspace_size(B, Q, Hq, heads, head_dim, dtype):
    """Bytes of workspace that a paged_attention call with these sizes needs (0: not supported): zero-filled once,
    used by one call at a time."""
    return int(_lib.spec_attention_workspace_size(B, Q, Hq, heads, head_dim, _DTYPES[dtype]))


@_on_stream
def paged_attention(at, q, k_pages, v_pages, page_table, lengths, scale=None, *, return_lse=False, out=None,
                    workspace=None, debug=False):
    """Attention of the newest Q tokens of each sequence over its paged cache.

    q [B, Q, Hq, D] (strides free but the last; D 64 or 128), k_pages / v_pages
    [pages, page_size, heads, D] of the same dtype (float32 or bfloat16), page_table int32
    [B, max_pages], lengths int32 [B] (the Q new tokens included: cache_append comes
    first).  Query i of a sequence of n tokens stands at n - Q + i and sees the tokens up to
    itself; query head h reads cache head h * heads // Hq.  ``scale`` defaults to
    1 / sqrt(D).  Returns out [B, Q, Hq, D], with ``return_lse`` (out, lse float32
    [B, Q, Hq]); a query that sees nothing gets 0 and -inf.
    """
    index, stream = at
    shape, st = q.shape, q.stride()
    if len(shape) != 4:
        raise ValueError("q must be [B, Q, Hq, D]")
    B, Q, Hq, D = shape
    c = _cache(k_pages, v_pages, False, index)
    if q.dtype is not k_pages.dtype:
        raise TypeError(f"q is {q.dtype}, the cache {k_pages.dtype}")
    heads = c.heads
    if D != c.head_dim or Hq % heads:
        raise ValueError(f"q has {Hq} heads of {D}, the cache {heads} of {c.head_dim}")
    if D > 1 and st[3] != 1:
        raise ValueError("q's last dimension must be contiguous")
    table, ts, M = _table(page_table, B, index)
    lens = _ints(lengths, "lengths", (B,), index)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    elif out.shape != shape or out.dtype is not q.dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be contiguous, shaped and typed as q")
    else:
        _written(out)
    lse = lse_at = None
    if return_lse:
        lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device)
        lse_at = lse.data_ptr()
    status, status_at = _status(debug, q.device)
    need = _lib.spec_attention_workspace_size(B, Q, Hq, heads, D, c.dtype)
    if need == 0:
        _raise(ERR_UNSUPPORTED, f"paged_attention with head_dim {D}")
    ws, nbytes, held = _workspace("attention", index, stream, need, workspace)
    # the stride of a dimension of one element is free in torch
    rc = _lib.spec_paged_attention(
        q.data_ptr(), st[0] if B > 1 else 0, st[1] if Q > 1 else 0, st[2] if Hq > 1 else 0, c, table, ts, M, lens, B, Q, Hq,
        D ** -0.5 if scale is None else scale, out.data_ptr(), lse_at, ws, nbytes, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_paged_attention")
    if debug:
        return (out, lse, status) if return_lse else (out, status)
    return (out, lse) if return_lse else out


@_on_stream
def cache_append(at, k_new, v_new, k_pages, v_pages, page_table, lengths, starts=None, *, debug=False):
    """Writes new tokens' keys and values into their pages (in place).

    k_new / v_new [T, heads, head_dim] with ``starts`` int32 [B + 1] (sequence b's new
    tokens are rows starts[b] .. starts[b+1] - 1), or [B, n, heads, head_dim] without;
    lengths int32 [B] counts the new tokens in: they become the last ones of their
    sequence.  Rows may be strided (a slice of a fused projection).  Returns the status
    word with ``debug``, else None.
    """
    index, stream = at
    c = _cache(k_pages, v_pages, False, index)
    if k_new.dtype is not k_pages.dtype or v_new.dtype is not k_pages.dtype:
        raise TypeError(f"the new tokens are {k_new.dtype}, {v_new.dtype}, the cache {k_pages.dtype}")
    shape, st = k_new.shape, k_new.stride()
    if v_new.shape != shape or v_new.stride() != st or v_new.get_device() != index:
        raise ValueError("k_new and v_new must have the same shape, strides and device")
    B = lengths.shape[0]
    H, D = c.heads, c.head_dim
    if starts is not None:
        if len(shape) != 3 or shape[1] != H or shape[2] != D:
            raise ValueError(f"with starts, k_new must be [T, {H}, {D}]")
        T, row = shape[0], st[0]
        first = _ints(starts, "starts", (B + 1,), index)
    else:
        if len(shape) != 4 or shape[0] != B or shape[2] != H or shape[3] != D:
            raise ValueError(f"without starts, k_new must be [{B}, n, {H}, {D}]")
        T, row = B * shape[1], st[1] if shape[1] > 1 else st[0]
        if B > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError("without starts, the rows of k_new must lie at one stride")
        first = None
    if (D > 1 and st[-1] != 1) or (H > 1 and st[-2] != D):
        raise ValueError("heads and head_dim of k_new must be contiguous")
    table, ts, M = _table(page_table, B, index)
    lens = _ints(lengths, "lengths", (B,), index)
    status, status_at = _status(debug, k_new.device)
    rc = _lib.spec_cache_append(k_new.data_ptr(), v_new.data_ptr(), row if T > 1 else H * D, T, first, c, table, ts, M, lens,
                                B, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_cache_append")
    _written(k_pages, v_pages)
    return status


@_on_stream
def cache_fork(at, k_pages, v_pages, page_table, lengths, parents, keep, room=0, *, workspace=None, debug=False):
    """The next step's sequences from the current ones.

    Sequence c of the next step continues sequence ``parents[c]`` (-1: a new one) with its
    first ``keep[c]`` tokens, and gets pages for ``room`` tokens more.  Full pages are
    shared; a partly filled one stays with one sequence, the others that end in it get
    copies (all layers of k_pages / v_pages, in place); sequences that nobody continues
    end, and their pages are free.  Returns a ForkResult: the new page table and lengths,
    the references to each page, and the free pages.
    """
    index, stream = at
    c = _cache(k_pages, v_pages, True, index)
    B, C = lengths.shape[0], parents.shape[0]
    table, ts, M = _table(page_table, B, index)
    lens = _ints(lengths, "lengths", (B,), index)
    par, kp = _ints(parents, "parents", (C,), index), _ints(keep, "keep", (C,), index)
    P = c.pages
    device = k_pages.device
    new = torch.empty((C, M), dtype=torch.int32, device=device)
    lens_new = torch.empty(C, dtype=torch.int32, device=device)
    refs = torch.empty(P, dtype=torch.int32, device=device)
    free = torch.empty(P, dtype=torch.int32, device=device)
    n_free = torch.empty(1, dtype=torch.int32, device=device)
    status, status_at = _status(debug, device)
    ws, nbytes, held = _workspace("fork", index, stream, _lib.spec_cache_fork_workspace_size(P, C), workspace)
    rc = _lib.spec_cache_fork(c, table, ts, M, lens, B, par, kp, C, room, new.data_ptr(), lens_new.data_ptr(),
                              refs.data_ptr(), free.data_ptr(), n_free.data_ptr(), ws, nbytes, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_cache_fork")
    _written(k_pages, v_pages)
    return ForkResult(new, lens_new, refs, free, n_free, status)


@_on_stream
def cache_compact(at, k_pages, v_pages, page_table, *, workspace=None, debug=False):
    """Moves the pages in use (entries >= 0 of the page table) to the front of the pool, in place,
    all layers: with n in use, those at or above n fill the unused ones below n, in
    ascending order.  Returns a CompactResult: the rewritten page table, the references
    to each page, and n.
    """
    index, stream = at
    c = _cache(k_pages, v_pages, True, index)
    B = page_table.shape[0]
    table, ts, M = _table(page_table, B, index)
    P = c.pages
    device = k_pages.device
    new = torch.empty((B, M), dtype=torch.int32, device=device)
    refs = torch.empty(P, dtype=torch.int32, device=device)
    n_live = torch.empty(1, dtype=torch.int32, device=device)
    status, status_at = _status(debug, device)
    ws, nbytes, held = _workspace("compact", index, stream, _lib.spec_cache_compact_workspace_size(P), workspace)
    rc = _lib.spec_cache_compact(c, table, ts, M, B, new.data_ptr(), refs.data_ptr(), n_live.data_ptr(), ws, nbytes, stream,
                                 status_at)
    if rc != OK:
        _raise(rc, "spec_cache_compact")
    _written(k_pages, v_pages)
    return CompactResult(new, refs, n_live, status)


def _setting(v, off, kind, name, R, index):
    """(scalar, pointer) of a sampling setting: None, a number for every row, or one a row."""
    if v is None:
        return off, None
    if not isinstance(v, torch.Tensor):
        return v, None
    if v.dtype is not kind:
        raise TypeError(f"{name} must be {kind}, got {v.dtype}")
    if v.numel() != R or v.get_device() != index or not v.is_contiguous():
        raise ValueError(f"{name} must hold one value a row on cuda:{index}")
    return off, v.data_ptr()


@_on_stream
def filtered_sample(at, logits, uniforms, temperature=1.0, *, top_k=None, top_p=None, min_p=None, return_filtered=False,
                    out=None, workspace=None, debug=False):
    """One token per row of ``logits`` [..., V] (float32 or bfloat16; rows may be strided when
    two-dimensional) from its truncated softmax, by the given uniforms [...].

    temperature, top_k, top_p and min_p are numbers or tensors with one value a row
    (float32; top_k int32).  top_k keeps the largest logits; min_p those of at least
    min_p times the largest one's probability; top_p then the most likely ones up to
    that share of what is left.  Temperature 0 takes the largest logit.  Returns a
    SampleResult: tokens, p (the token's probability among the kept ones), n_kept and, with
    ``return_filtered``, the logits with -inf for what was not kept -- rows for ``verify``,
    whose accept test then holds for the truncated distributions.  ``out`` may give a
    preallocated tensor for those: the logits themselves, or one that does not overlap them.
    """
    index, stream = at
    shape, device = logits.shape, logits.device
    if len(shape) < 1:
        raise ValueError("logits must be [..., V]")
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    V = shape[-1]
    if V < 1:
        _raise(ERR_INVALID_ARG, "filtered_sample with an empty vocabulary")
    if V > MAX_V:
        _raise(ERR_UNSUPPORTED, f"filtered_sample with {V} tokens")
    rows = shape[:-1]
    R = rows.numel()
    if logits.is_contiguous():
        stride = V
    elif len(shape) == 2 and logits.stride(1) == 1 and logits.stride(0) >= V:
        stride = logits.stride(0)
    else:
        raise ValueError("the rows of logits must be contiguous, and at one stride")
    if uniforms.dtype is not torch.float32 or uniforms.shape != rows or uniforms.get_device() != index or not uniforms.is_contiguous():
        raise ValueError(f"uniforms must be contiguous float32 {tuple(rows)} on {device}")
    T, Tp = _setting(temperature, 1.0, torch.float32, "temperature", R, index)
    k, kp = _setting(top_k, 0, torch.int32, "top_k", R, index)
    p, pp = _setting(top_p, 1.0, torch.float32, "top_p", R, index)
    m, mp = _setting(min_p, 0.0, torch.float32, "min_p", R, index)
    tokens = torch.empty(rows, dtype=torch.int32, device=device)
    prob = torch.empty(rows, dtype=torch.float32, device=device)
    n_kept = torch.empty(rows, dtype=torch.int32, device=device)
    out_at = None
    if out is not None:
        if out.shape != shape or out.dtype is not logits.dtype or out.get_device() != index or not out.is_contiguous():
            raise ValueError("out must be contiguous, shaped and typed as logits")
        out_at = out.data_ptr()
        _written(out)
    elif return_filtered:
        out = torch.empty(shape, dtype=logits.dtype, device=device)
        out_at = out.data_ptr()
    status, status_at = _status(debug, device)
    need = _lib.spec_filtered_sample_workspace_size(R, V, dt)
    ws, nbytes, held = _workspace("sample", index, stream, need, workspace)
    rc = _lib.spec_filtered_sample(
        logits.data_ptr(), stride, uniforms.data_ptr(), R, V, dt, T, k, p, m, Tp, kp, pp, mp, tokens.data_ptr(),
        prob.data_ptr(), n_kept.data_ptr(), out_at, ws, nbytes, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_filtered_sample")
    return SampleResult(tokens, prob, n_kept, out, status)
