"""Decoding with trees of drafted tokens over the paged MXFP4 cache (C ABI in include/mx_draft.h).

The functions carry the C ABI's names, check their tensors (device, type, shape, strides) and pass
pointers, sizes and strides to the library.  They allocate nothing: outputs and workspaces are the
caller's.  The nodes of all sequences lie one after the other in every [nodes] tensor; q_starts (int32
[batch + 1], with max_q) says where each sequence's begin, and without it every sequence has the same
number.  Node 0 of a sequence is the last token of its text, the others are drafted.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import MX_ERR_DEVICE, MX_ERR_SHAPE, MX_ERR_STRIDE, MX_OK, MxError, load
from .attention import (MxKvCacheFp4, _Tensor, _attn, _cache, _current_device, _f32, _flat, _i32, _need,
                        _starts, _stream, _table, _workspace)

# The argument structs of the header: pointers, then int64 fields, then a double.
_TREE_MASK = struct.Struct("=5Q5q")
_ATTN_TREE = struct.Struct("=10Q14qd")
_VERIFY = struct.Struct("=11Q10q")
_ACCEPT = struct.Struct("=7Q7q")

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _nodes(fn: str, t, what: str, dtype, dev: int):
    """Pointer and length of a contiguous tensor [nodes]."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev >= 0 and t.dim() == 1 and \
            t.is_contiguous():
        return t.data_ptr(), t.numel()
    _need(fn, t, what, dtype, dev)                # what is wrong with it
    if t.dim() != 1:
        raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected [nodes]")
    return _flat(fn, t, what, dtype, dev, t.shape), t.shape[0]


def _batch(fn: str, q_starts, max_q, nodes: int):
    """Sequences of a call that no other argument counts: by q_starts, or nodes / max_q."""
    if q_starts is not None:
        if not isinstance(q_starts, _Tensor):
            raise TypeError(f"{fn}: q_starts must be a torch tensor, got {type(q_starts).__name__}")
        return max(q_starts.numel() - 1, 0)
    if max_q is None:
        raise TypeError(f"{fn}: needs q_starts or max_q")
    return nodes // max_q if max_q > 0 else 0


def _mask(fn: str, mask, nodes: int, dev: int):
    """Pointer, row stride and words of a mask [nodes, words]."""
    if isinstance(mask, _Tensor) and mask.dtype is _i32 and mask.get_device() == dev >= 0:
        sh, st = mask.shape, mask.stride()
        if len(sh) == 2 and sh[0] == nodes and (st[1] == 1 or sh[1] <= 1):
            return mask.data_ptr(), st[0] if nodes > 1 else sh[1], sh[1]
    _need(fn, mask, "mask", _i32, dev)            # what is wrong with it
    if mask.dim() != 2 or mask.shape[0] != nodes:
        raise MxError(fn, MX_ERR_SHAPE, f"mask has shape {tuple(mask.shape)}, expected [{nodes}, words]")
    raise MxError(fn, MX_ERR_STRIDE, f"mask's rows are not contiguous ({mask.stride()})")


def _rows(fn: str, t, what: str, dtype, dev: int, shape=None):
    """Pointer and row stride of probabilities [nodes, vocab]."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev >= 0:
        sh, st = t.shape, t.stride()
        if len(sh) == 2 and (shape is None or sh == shape) and (st[1] == 1 or sh[1] <= 1):
            return t.data_ptr(), st[0] if sh[0] > 1 else sh[1]
    _need(fn, t, what, dtype, dev)                # what is wrong with it
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        want = "[nodes, vocab]" if shape is None else list(shape)
        raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected {want}")
    raise MxError(fn, MX_ERR_STRIDE, f"{what}'s rows are not contiguous ({t.stride()})")


def _path(fn: str, path, B: int, dev: int):
    """Pointer and shape of a path [batch, width]."""
    if not isinstance(path, _Tensor) or path.dim() != 2 or path.shape[0] != B:
        _need(fn, path, "path", _i32, dev)
        raise MxError(fn, MX_ERR_SHAPE, f"path has shape {tuple(path.shape)}, expected [{B}, width]")
    sh = path.shape
    return _flat(fn, path, "path", _i32, dev, sh), sh


def mx_tree_mask(parents, mask, seq_lens=None, positions=None, q_starts=None, max_q=None, stream=None):
    """Masks and positions of trees.

    parents: int32 [nodes], each node's parent's number in its sequence (less than its own; otherwise it
    has none).  mask: int32 [nodes, words], words at least max_q / 32: bit j of a row is set where node j
    is the row's node or an ancestor.  positions: int32 [nodes], seq_lens - nodes + depth, with seq_lens
    int32 [batch] counting the nodes; both or neither.  At most 1024 nodes a sequence."""
    fn, dev = "mx_tree_mask", _current_device()
    pp, N = _nodes(fn, parents, "parents", _i32, dev)
    B = seq_lens.shape[0] if isinstance(seq_lens, _Tensor) and seq_lens.dim() == 1 else \
        _batch(fn, q_starts, max_q, N)
    starts, max_q = _starts(fn, q_starts, max_q, N, B, dev)
    mp, stride, words = _mask(fn, mask, N, dev)
    lp = 0 if seq_lens is None else _flat(fn, seq_lens, "seq_lens", _i32, dev, (B,))
    op = 0 if positions is None else _flat(fn, positions, "positions", _i32, dev, (N,))
    st = load().mx_tree_mask(_TREE_MASK.pack(pp, lp, starts, mp, op, stride, words, B, N, max_q),
                             _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_attn_tree_fp4(cache, q, mask, page_table, seq_lens, out, workspace, q_starts=None, max_q=None,
                     scale=None, window=0, positions=None, lse=None, stream=None):
    """Attention of trees' nodes over the cache that holds them as each sequence's last tokens.

    Arguments as in mx_attn_fp4 (the workspace and its size too), with `mask` in place of the causal one:
    int32 [nodes, words], bit j of a row set where its query sees node j of its sequence (as mx_tree_mask
    writes it; any row stride).  Of the tokens before the tree a query sees all, or with a window those
    past its position (int32 [nodes], needed then) less the window."""
    fn, dev = "mx_attn_tree_fp4", _current_device()
    (qp, op, lp, tp, lens, starts, wp, wb, strides, table, B, N, max_q, H, scale) = _attn(
        fn, dev, cache, q, page_table, seq_lens, out, workspace, q_starts, max_q, scale, lse)
    mp, stride, words = _mask(fn, mask, N, dev)
    pp = 0 if positions is None else _flat(fn, positions, "positions", _i32, dev, (N,))
    st = load().mx_attn_tree_fp4(
        _ATTN_TREE.pack(cache._addr, qp, op, lp, mp, pp, tp, lens, starts, wp, wb, *strides, stride, words,
                        *table, B, N, max_q, H, window, scale), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_tree_verify_workspace_size(batch) -> int:
    """Bytes of workspace mx_tree_verify needs; an mx_attn_fp4 workspace that is as large serves too."""
    return int(load().mx_tree_verify_workspace_size(batch))


def mx_tree_verify(target, draft, tokens, parents, accept_u, sample_u, path, tokens_out, count, workspace,
                   q_starts=None, max_q=None, replacement=True, stream=None):
    """Which drafted tokens stand, and the token after them.

    target: probabilities [nodes, vocab], fp32, bf16 or fp16, of the token after each node; draft: the same
    (and of the same type) of what each node's children were drawn from, with or without `replacement`, or
    None where drafts were chosen; rows contiguous, any row stride.  tokens, parents: int32 [nodes];
    accept_u: fp32 [nodes], sample_u: fp32 [batch], random numbers in [0, 1).  Written: path, int32
    [batch, width], the accepted nodes from the root on, then -1; tokens_out, the same shape, their
    tokens without the root's, the next token, then -1; count, int32 [batch], the number of either.
    workspace: a tensor of mx_tree_verify_workspace_size bytes, zero before its first use, reusable."""
    fn, dev = "mx_tree_verify", _current_device()
    if not isinstance(target, _Tensor) or target.dtype not in _TYPES:
        raise TypeError(f"{fn}: target must be a torch tensor of fp32, bf16 or fp16")
    gp, gs = _rows(fn, target, "target", target.dtype, dev)
    shape = target.shape
    N, V = shape
    dp, ds = (0, 0) if draft is None else _rows(fn, draft, "draft", target.dtype, dev, shape)
    nodes = (N,)
    tp = _flat(fn, tokens, "tokens", _i32, dev, nodes)
    pp = _flat(fn, parents, "parents", _i32, dev, nodes)
    up = _flat(fn, accept_u, "accept_u", _f32, dev, nodes)
    sp, B = _nodes(fn, sample_u, "sample_u", _f32, dev)
    starts, max_q = _starts(fn, q_starts, max_q, N, B, dev)
    op, sh = _path(fn, path, B, dev)
    np_ = _flat(fn, tokens_out, "tokens_out", _i32, dev, sh)
    cp = _flat(fn, count, "count", _i32, dev, (B,))
    wp, wb = _workspace(fn, workspace, dev)
    st = load().mx_tree_verify(
        _VERIFY.pack(gp, dp, tp, pp, up, sp, starts, op, np_, cp, wp, wb, gs, ds, B, N, max_q, V, sh[1],
                     _TYPES[target.dtype], bool(replacement)), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_kv_accept_fp4(caches, page_table, seq_lens, path, count, lens_out=None, q_starts=None, max_q=None,
                     stream=None):
    """Moves the accepted path's keys and values behind the text in every layer's cache.

    caches: MxKvCacheFp4, or any iterable of them (one a layer, of one shape and the same strides) that share
    page_table (int32 [batch, width]).  seq_lens: int32 [batch], tokens cached with the nodes; path int32
    [batch, width] and count int32 [batch] as mx_tree_verify writes them.  Node path[i] becomes the i-th
    token after the text; lens_out (int32 [batch], not seq_lens, or None): the lengths with the accepted
    nodes alone, written without any cache too (an empty sequence, on a stage that has no attention).  Without
    q_starts, max_q nodes each."""
    fn, dev = "mx_kv_accept_fp4", _current_device()
    caches = (caches,) if isinstance(caches, MxKvCacheFp4) else tuple(caches)     # gone over more than once
    if any(type(c) is not MxKvCacheFp4 or c.device_index != dev for c in caches):
        for c in caches:
            _cache(fn, c, dev)
    packed = [c._packed for c in caches]
    tp, stride, B, width = _table(fn, page_table, dev)
    lens = _flat(fn, seq_lens, "seq_lens", _i32, dev, (B,))
    pp, sh = _path(fn, path, B, dev)
    cp = _flat(fn, count, "count", _i32, dev, (B,))
    op = 0 if lens_out is None else _flat(fn, lens_out, "lens_out", _i32, dev, (B,))
    if max_q is None:
        raise TypeError(f"{fn}: needs max_q")
    starts, max_q = _starts(fn, q_starts, max_q, 0, B, dev)
    rows = (1 << 31) - 1 if starts else B * max_q        # no tensor of nodes: q_starts alone says
    array = ctypes.create_string_buffer(b"".join(packed))
    st = load().mx_kv_accept_fp4(
        _ACCEPT.pack(ctypes.addressof(array), tp, lens, starts, pp, cp, op, len(packed), stride, width, B,
                     rows, max_q, sh[1]), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)
