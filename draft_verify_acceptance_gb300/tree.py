"""ctypes binding of speculation over trees of drafted tokens (include/spec_tree.h).

    cache_append_rotated  new keys, rotated by position, and values into their pages; queries rotated
    tree_attention        a tree's nodes over the paged cache: the context, their ancestors, themselves
    tree_accept           the path that the target's tokens take through each tree
    cache_keep            the path's keys and values to the front of the tree's slots

A tree of N nodes is the newest N tokens of its sequence, and ``parents`` int32 [B, N] (or one row
for every sequence, [N] or expanded) holds each node's parent: a lower index, -1 for a child of the
context, less for no node (padding).  Everything else is as in ``decode``: caches, page tables, streams,
workspaces, ``debug`` and autograd.
"""
import ctypes
from typing import NamedTuple

import torch

from . import _decode_calls
from .binding import ERR_UNSUPPORTED, OK
from .decode import _Cache, _DTYPES, _cache, _ints, _lib, _on_stream, _raise, _status, _table, _workspace, _written

MAX_NODES = 256
DATA_TREE_PARENT = 1024
DATA_PATH_RANGE = 2048

EXPORTS = ("spec_tree_attention_workspace_size", "spec_tree_attention", "spec_cache_append_rotated", "spec_tree_accept",
           "spec_cache_keep")


def _declare():
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    C = ctypes.POINTER(_Cache)
    sig = {
        "spec_tree_attention_workspace_size": (Z, [I] * 6),
        "spec_tree_attention": (I, [P, L, L, L, C, P, L, I, P, P, L, I, I, I, F, P, P, P, Z, P, P]),
        "spec_cache_append_rotated": (I, [P, P, L, I, P, P, L, I, P, L, P, P, I, I, C, P, L, I, P, I, P, P]),
        "spec_tree_accept": (I, [P, P, L, P, I, I, P, P, P, P, P]),
        "spec_cache_keep": (I, [C, P, L, I, P, I, P, I, P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = res, args


_declare()


class AcceptResult(NamedTuple):
    accepted_len: torch.Tensor  # int32 [B]: nodes behind the root, -1 where there is no root
    out_tokens: torch.Tensor    # int32 [B, N]: the emitted tokens, then -1
    path: torch.Tensor          # int32 [B, N]: the accepted nodes, the root first, then -1
    status: torch.Tensor        # int32 [1] with debug, else None


_decode_calls.bind_tree(tuple(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in EXPORTS), AcceptResult)


def _parents(t, B, N, index):
    """(pointer, row stride) of the parents: one row a sequence, or one for all."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError("parents must be an int32 tensor")
    if t.get_device() != index or t.shape not in ((B, N), (N,)) or (N > 1 and t.stride(-1) != 1):
        raise ValueError(f"parents must be [{B}, {N}] or [{N}] with contiguous rows on cuda:{index}, "
                         f"got {tuple(t.shape)} on {t.device}")
    if t.dim() == 1:
        return t.data_ptr(), 0
    stride = t.stride(0) if B > 1 else N
    if 0 < stride < N:
        raise ValueError("the rows of parents must not overlap")
    return t.data_ptr(), stride


def attention_workspace_size(B, N, Hq, heads, head_dim, dtype):
    """Bytes of workspace that a tree_attention call with these sizes needs (0: not supported): zero-filled once,
    used by one call at a time."""
    return int(_lib.spec_tree_attention_workspace_size(B, N, Hq, heads, head_dim, _DTYPES[dtype]))


@_on_stream
def tree_attention(at, q, k_pages, v_pages, page_table, lengths, parents, scale=None, *, return_lse=False, out=None,
                   workspace=None, debug=False):
    """Attention of a tree's nodes over their sequence's paged cache.

    q [B, N, Hq, D] (N up to 256; strides free but the last; D 64 or 128), k_pages / v_pages
    [pages, page_size, heads, D] of the same dtype (float32 or bfloat16), page_table int32
    [B, max_pages], lengths int32 [B] (the N nodes included: cache_append_rotated comes
    first), parents int32 [B, N] or [N].  Node i of a sequence of n tokens is its token n - N + i
    and sees the tokens before n - N, its ancestors and itself; query head h reads cache head
    h * heads // Hq.  ``scale`` defaults to 1 / sqrt(D).  Returns out [B, N, Hq, D], with
    ``return_lse`` (out, lse float32 [B, N, Hq]); no node gets 0 and -inf.  What a node sees that is
    not finite makes its result not finite (infinite or NaN); what it does not see never reaches it.
    ``out`` may give a preallocated tensor that does not overlap q.
    """
    index, stream = at
    shape, st = q.shape, q.stride()
    if len(shape) != 4:
        raise ValueError("q must be [B, N, Hq, D]")
    B, N, Hq, D = shape
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
    par, ps = _parents(parents, B, N, index)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    elif out.shape != shape or out.dtype is not q.dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be contiguous, shaped and typed as q")
    else:
        _written(out)
    lse = lse_at = None
    if return_lse:
        lse = torch.empty((B, N, Hq), dtype=torch.float32, device=q.device)
        lse_at = lse.data_ptr()
    status, status_at = _status(debug, q.device)
    need = _lib.spec_tree_attention_workspace_size(B, N, Hq, heads, D, c.dtype)
    if need == 0:
        _raise(ERR_UNSUPPORTED, f"tree_attention with {N} nodes, head_dim {D}")
    ws, nbytes, held = _workspace("tree", index, stream, need, workspace)
    # the stride of a dimension of one element is free in torch
    rc = _lib.spec_tree_attention(
        q.data_ptr(), st[0] if B > 1 else 0, st[1] if N > 1 else 0, st[2] if Hq > 1 else 0, c, table, ts, M, lens, par, ps, B, N,
        Hq, D ** -0.5 if scale is None else scale, out.data_ptr(), lse_at, ws, nbytes, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_tree_attention")
    if debug:
        return (out, lse, status) if return_lse else (out, status)
    return (out, lse) if return_lse else out


def _rows(t, name, lead, heads, D):
    """(row stride, rows) of new tokens' heads [*lead, heads, D], their heads contiguous and rows at one stride."""
    shape, st = t.shape, t.stride()
    if shape != (*lead, heads, D):
        raise ValueError(f"{name} must be {(*lead, heads, D)}, got {tuple(shape)}")
    if (D > 1 and st[-1] != 1) or (heads > 1 and st[-2] != D):
        raise ValueError(f"heads and head_dim of {name} must be contiguous")
    T = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    if T <= 1:
        return heads * D, T
    if len(lead) == 1:
        return st[0], T
    if lead[0] > 1 and lead[1] > 1 and st[0] != lead[1] * st[1]:
        raise ValueError(f"the rows of {name} must lie at one stride")
    return st[1] if lead[1] > 1 else st[0], T


@_on_stream
def cache_append_rotated(at, k_new, v_new, k_pages, v_pages, page_table, lengths, inv_freq, q=None, positions=None, starts=None, *,
                         interleaved=False, out=None, debug=False):
    """``cache_append`` with the position rotation on the way: keys are rotated and written into their pages,
    values as they are (both in place), and the queries ``q`` of the same tokens are rotated too.

    k_new / v_new [T, heads, head_dim] with ``starts`` int32 [B + 1], or [B, n, heads, head_dim]
    without; q [T, Hq, head_dim] or [B, n, Hq, head_dim]; rows may be strided (slices of a fused
    projection).  lengths int32 [B] counts the new tokens in.  ``inv_freq`` float32 [F]: pair i of a head
    turns by position * inv_freq[i]; pair i is dimensions i and F + i, or 2i and 2i + 1 with
    ``interleaved``; dimensions from 2 F on stay.  ``positions`` int32 [T] or [B, n] gives the tokens'
    positions (of a tree's nodes: the context's tokens and their depth), else they are their
    places in their sequences.  Returns the rotated queries (``out`` if it is given: q itself, which then shares
    nothing with k_new and v_new, or a tensor that overlaps none of the new rows; None without q), with ``debug`` (queries, status).
    """
    index, stream = at
    c = _cache(k_pages, v_pages, False, index)
    if k_new.dtype is not k_pages.dtype or v_new.dtype is not k_pages.dtype:
        raise TypeError(f"the new tokens are {k_new.dtype}, {v_new.dtype}, the cache {k_pages.dtype}")
    if v_new.shape != k_new.shape or v_new.stride() != k_new.stride() or v_new.get_device() != index:
        raise ValueError("k_new and v_new must have the same shape, strides and device")
    if lengths.dim() != 1:
        raise ValueError("lengths must be [B]")
    B = lengths.shape[0]
    H, D = c.heads, c.head_dim
    first = None
    if starts is not None:
        first = _ints(starts, "starts", (B + 1,), index)
        lead = k_new.shape[:1]
    else:
        lead = k_new.shape[:2]
        if lead[:1] != (B,):
            raise ValueError(f"without starts, k_new must be [{B}, n, {H}, {D}]")
    row, T = _rows(k_new, "k_new", lead, H, D)
    table, ts, M = _table(page_table, B, index)
    lens = _ints(lengths, "lengths", (B,), index)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not torch.float32:
        raise TypeError("inv_freq must be a float32 tensor")
    if inv_freq.dim() != 1 or inv_freq.get_device() != index or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be contiguous [F] on cuda:{index}")
    F = inv_freq.shape[0]
    pos = None
    if positions is not None:
        pos = _ints(positions, "positions", tuple(lead), index)
    q_at, q_row, Hq, out_at, out_row = None, 0, 0, None, 0
    if q is not None:
        if q.dtype is not k_pages.dtype:
            raise TypeError(f"q is {q.dtype}, the cache {k_pages.dtype}")
        if q.dim() != k_new.dim() or q.get_device() != index:
            raise ValueError(f"q must hold the new tokens' queries on cuda:{index}")
        Hq = q.shape[-2]
        q_row, _ = _rows(q, "q", lead, Hq, D)
        q_at = q.data_ptr()
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            if out.dtype is not q.dtype or out.get_device() != index:
                raise ValueError("out must be on q's device, of q's dtype")
            _written(out)
        out_row, _ = _rows(out, "out", lead, Hq, D)
        out_at = out.data_ptr()
    elif out is not None:
        raise ValueError("out is for the rotated q")
    status, status_at = _status(debug, k_new.device)
    rc = _lib.spec_cache_append_rotated(
        k_new.data_ptr(), v_new.data_ptr(), row, T, first, q_at, q_row, Hq, out_at, out_row, pos, inv_freq.data_ptr(), F,
        int(bool(interleaved)), c, table, ts, M, lens, B, stream, status_at)
    if rc != OK:
        _raise(rc, "spec_cache_append_rotated")
    _written(k_pages, v_pages)
    return (out, status) if debug else out


@_on_stream
def tree_accept(at, tokens, parents, drawn, *, debug=False):
    """The path that the target's tokens take through each tree.

    tokens int32 [B, N] (node 0 is the root, the token that the step before emitted), parents
    int32 [B, N] or [N], drawn int32 [B, N]: the target's token after each node (its argmax, or
    ``filtered_sample`` of its rows).  The walk goes from the root on to the child whose
    token is the one drawn after the node.  Returns an AcceptResult.
    """
    index, stream = at
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, N]")
    B, N = tokens.shape
    if N > MAX_NODES:
        _raise(ERR_UNSUPPORTED, f"tree_accept with {N} nodes")
    tok = _ints(tokens, "tokens", (B, N), index)
    par, ps = _parents(parents, B, N, index)
    dr = _ints(drawn, "drawn", (B, N), index)
    device = tokens.device
    n = torch.empty(B, dtype=torch.int32, device=device)
    out, path = (torch.empty((B, N), dtype=torch.int32, device=device) for _ in range(2))
    status, status_at = _status(debug, device)
    rc = _lib.spec_tree_accept(tok, par, ps, dr, B, N, n.data_ptr(), out.data_ptr(), path.data_ptr(), stream, status_at)
    if rc != OK:
        _raise(rc, "spec_tree_accept")
    return AcceptResult(n, out, path, status)


@_on_stream
def cache_keep(at, k_pages, v_pages, page_table, lengths, path, *, debug=False):
    """Of each sequence's newest N tokens keeps those of ``path`` int32 [B, N] (ascending indexes, ended by -1:
    tree_accept's), moved to the front, in place, all layers.  The pages that hold those N tokens must be the
    sequence's own.  Returns the new lengths int32 [B], with ``debug`` (lengths, status); cache_fork then gives the
    pages behind them away, or to the next tree.
    """
    index, stream = at
    c = _cache(k_pages, v_pages, True, index)
    if lengths.dim() != 1 or path.dim() != 2:
        raise ValueError("lengths must be [B] and path [B, N]")
    B, N = lengths.shape[0], path.shape[1]
    table, ts, M = _table(page_table, B, index)
    lens = _ints(lengths, "lengths", (B,), index)
    pth = _ints(path, "path", (B, N), index)
    new = torch.empty(B, dtype=torch.int32, device=k_pages.device)
    status, status_at = _status(debug, k_pages.device)
    rc = _lib.spec_cache_keep(c, table, ts, M, lens, B, pth, N, new.data_ptr(), stream, status_at)
    if rc != OK:
        _raise(rc, "spec_cache_keep")
    _written(k_pages, v_pages)
    return (new, status) if debug else new
