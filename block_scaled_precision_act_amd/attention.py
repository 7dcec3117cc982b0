"""Attention around a paged MXFP4 key/value cache (C ABI in include/mx_attention.h).

The functions carry the C ABI's names, check their tensors (device, type, shape, strides) and pass
pointers, sizes and strides to the library.  They allocate nothing: outputs and workspaces are the
caller's.  `MxKvCacheFp4` holds a cache's four tensors, checked once.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import MX_ERR_DEVICE, MX_ERR_SHAPE, MX_ERR_STRIDE, MX_OK, MxError, load
from . import _current_device as _any_device
from . import _stream as _any_stream

# The argument structs of the header: pointers, then int64 fields, then a double.
_CACHE = struct.Struct("=4Q8q")
_NORM_ROPE = struct.Struct("=9Q15qd")
_NORM_ROPE_BACK = struct.Struct("=14Q20qd")
_APPEND = struct.Struct("=9Q8q")
_ATTN = struct.Struct("=8Q13qd")

_Tensor, _bf16, _f32, _u8 = torch.Tensor, torch.bfloat16, torch.float32, torch.uint8
_i32, _i64 = torch.int32, torch.int64

# torch's raw getters, where it has them: 0.1 us each in a call of a few microseconds.
_raw_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_device() -> int:
    """The current GPU's index, or -1 when no GPU is visible (every tensor is then refused)."""
    if _raw_device is not None and torch.cuda.is_initialized():
        return _raw_device()
    return _any_device()


def _stream(stream, dev: int):
    """The hipStream_t to launch on: `stream`, or torch's current one on GPU `dev`."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _any_stream(stream)


def _need(fn: str, t, what: str, dtype, dev: int):
    """`t` is a tensor of `dtype` on GPU `dev`: the library sees pointers only."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{fn}: {what} must be a torch tensor, got {type(t).__name__}")
    d = t.get_device()
    if d < 0 or d != dev:
        raise MxError(fn, MX_ERR_DEVICE, f"{what} is on {t.device}, not the current GPU")
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {what} must be {dtype}, got {t.dtype}")


def _heads(fn: str, t, what: str, dev: int, shape=None):
    """Pointer, token and head stride of bf16 heads [tokens, heads, dim] with contiguous values."""
    if isinstance(t, _Tensor) and t.dtype is _bf16 and t.get_device() == dev >= 0:
        sh, st = t.shape, t.stride()
        if len(sh) == 3 and (shape is None or sh == shape) and (st[2] == 1 or sh[2] <= 1):
            return t.data_ptr(), st[0] if sh[0] > 1 else 0, st[1] if sh[1] > 1 else 0
    _need(fn, t, what, _bf16, dev)                # what is wrong with it
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        want = "[tokens, heads, head_dim]" if shape is None else list(shape)
        raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected {want}")
    raise MxError(fn, MX_ERR_STRIDE, f"{what}'s head values are not contiguous ({t.stride()})")


def _flat(fn: str, t, what: str, dtype, dev: int, shape):
    """Pointer of a contiguous tensor of exactly `shape`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev >= 0 and \
            t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need(fn, t, what, dtype, dev)                # what is wrong with it
    if t.shape != shape:
        raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected {list(shape)}")
    raise MxError(fn, MX_ERR_STRIDE, f"{what} is not contiguous ({t.stride()})")


def _rotation(fn: str, positions, cos, sin, tokens: int, dev: int):
    """(positions, cos, sin) pointers, table rows and rotated values; all None: no rotation."""
    if positions is None:
        if cos is not None or sin is not None:
            raise TypeError(f"{fn}: cos and sin need positions")
        return 0, 0, 0, 0, 0
    if not isinstance(cos, _Tensor):
        raise TypeError(f"{fn}: cos must be a torch tensor, got {type(cos).__name__}")
    sh = cos.shape
    if len(sh) != 2:
        raise MxError(fn, MX_ERR_SHAPE, f"cos has shape {tuple(sh)}, expected [positions, rot / 2]")
    return (_flat(fn, positions, "positions", _i32, dev, (tokens,)),
            _flat(fn, cos, "cos", _f32, dev, sh), _flat(fn, sin, "sin", _f32, dev, sh),
            sh[0], 2 * sh[1])


def _workspace(fn: str, ws, dev: int):
    """Pointer and bytes of a workspace tensor (None: none)."""
    if ws is None:
        return 0, 0
    if not isinstance(ws, _Tensor) or ws.get_device() < 0 or ws.get_device() != dev:
        raise MxError(fn, MX_ERR_DEVICE, "the workspace must be a tensor on the current GPU")
    if not ws.is_contiguous():
        raise MxError(fn, MX_ERR_STRIDE, "the workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _table(fn: str, page_table, dev: int):
    """Pointer and row stride of a page table, sequences, pages of a sequence."""
    if isinstance(page_table, _Tensor) and page_table.dtype is _i32 and page_table.get_device() == dev >= 0:
        sh, st = page_table.shape, page_table.stride()
        if len(sh) == 2 and (st[1] == 1 or sh[1] <= 1):
            return page_table.data_ptr(), st[0] if sh[0] > 1 else sh[1], *sh
    _need(fn, page_table, "page_table", _i32, dev)            # what is wrong with it
    if page_table.dim() != 2:
        raise MxError(fn, MX_ERR_SHAPE, f"page_table has shape {tuple(page_table.shape)}, expected "
                                        "[batch, pages of a sequence]")
    raise MxError(fn, MX_ERR_STRIDE, f"page_table's rows are not contiguous "
                                     f"({page_table.stride()})")


def _starts(fn: str, q_starts, max_q, rows: int, B: int, dev: int):
    """Pointer of q_starts (None: rows / B each) and max_q."""
    if q_starts is not None:
        if max_q is None:
            raise TypeError(f"{fn}: q_starts needs max_q")
        return _flat(fn, q_starts, "q_starts", _i32, dev, (B + 1,)), max_q
    return 0, (rows // B if B else 0) if max_q is None else max_q


class MxKvCacheFp4:
    """A paged MXFP4 key/value cache over the caller's tensors: codes k, v uint8
    [pages, kv_heads, page_size, head_dim / 2] and E8M0 scales k_scale, v_scale uint8
    [pages, kv_heads, page_size, head_dim / 32], with any page and head strides that are multiples
    of 16 bytes (the same for k and v, and for their scales).  page_size: a multiple of 16; appending
    takes any, mx_attn_fp4 pages of fewer than 2^20 tokens and page tables with
    width * (page_size / 16) ** 2 < 2 ** 32."""

    def __init__(self, k, k_scale, v, v_scale):
        fn, dev = "MxKvCacheFp4", _current_device()
        for t, what in ((k, "k"), (k_scale, "k_scale"), (v, "v"), (v_scale, "v_scale")):
            _need(fn, t, what, _u8, dev)
        if k.dim() != 4:
            raise MxError(fn, MX_ERR_SHAPE, f"k has shape {tuple(k.shape)}, expected "
                                            "[pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, size, half = k.shape
        dim = 2 * half
        codes, scales = (pages, heads, size, half), (pages, heads, size, dim // 32)
        for t, what, want in ((v, "v", codes), (k_scale, "k_scale", scales),
                              (v_scale, "v_scale", scales)):
            if tuple(t.shape) != want:
                raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected "
                                                f"{list(want)}")
        # 2^31 slots at most: slots and lengths are counted in 32 bits
        if dim not in (64, 128, 256) or size <= 0 or size % 16 or heads <= 0 or \
                pages * size >= 1 << 31:
            raise MxError(fn, MX_ERR_SHAPE, f"head_dim {dim}, page_size {size}, {heads} heads, "
                                            f"{pages} pages")

        def strides(t, width):
            p, h, a, b = t.stride()
            if pages and (a != width or b != 1 and width > 1):
                raise MxError(fn, MX_ERR_STRIDE, "a page's tokens are not contiguous "
                                                 f"({t.stride()})")
            return p if pages > 1 else size * width * heads, h if heads > 1 else size * width

        code, scale = strides(k, half), strides(k_scale, dim // 32)
        if strides(v, half) != code or strides(v_scale, dim // 32) != scale:
            raise MxError(fn, MX_ERR_STRIDE, "k and v (or their scales) differ in strides")
        self.k, self.k_scale, self.v, self.v_scale = k, k_scale, v, v_scale
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, size, dim
        self.device_index = dev
        self._packed = _CACHE.pack(k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr(),
                                   pages, heads, size, dim, *code, *scale)
        self._struct = ctypes.create_string_buffer(self._packed, _CACHE.size)
        self._addr = ctypes.addressof(self._struct)


def _cache(fn: str, cache, dev: int):
    if not isinstance(cache, MxKvCacheFp4):
        raise TypeError(f"{fn}: cache must be an MxKvCacheFp4, got {type(cache).__name__}")
    if dev < 0 or cache.device_index != dev:
        raise MxError(fn, MX_ERR_DEVICE, "the cache is not on the current GPU")
    return cache


def mx_qk_norm_rope(q, k, positions, cos, sin, q_out, k_out, q_weight=None, k_weight=None,
                    eps=1e-6, interleaved=False, stream=None):
    """Per-head norm of queries and keys and their rotation in one pass.

    q, q_out: bf16 [tokens, q_heads, head_dim]; k, k_out: bf16 [tokens, k_heads, head_dim] or None;
    any token and head strides that are multiples of 4, an output may be its input.  positions:
    int32 [tokens]; cos, sin: fp32 [positions, rot / 2] (all three None: no rotation).
    q_weight, k_weight: bf16 [head_dim], or None for no norm."""
    fn, dev = "mx_qk_norm_rope", _current_device()
    qp, qt, qh = _heads(fn, q, "q", dev)
    T, Hq, D = q.shape
    qop, qot, qoh = _heads(fn, q_out, "q_out", dev, q.shape)
    kp = kt = kh = kop = kot = koh = Hk = 0
    if k is not None:
        kp, kt, kh = _heads(fn, k, "k", dev)
        Hk = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise MxError(fn, MX_ERR_SHAPE, f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
        kop, kot, koh = _heads(fn, k_out, "k_out", dev, k.shape)
    qw = 0 if q_weight is None else _flat(fn, q_weight, "q_weight", _bf16, dev, (D,))
    kw = 0 if k_weight is None else _flat(fn, k_weight, "k_weight", _bf16, dev, (D,))
    pp, cp, sp, rows, rot = _rotation(fn, positions, cos, sin, T, dev)
    st = load().mx_qk_norm_rope(
        _NORM_ROPE.pack(qp, kp, qop, kop, qw, kw, pp, cp, sp, qt, qh, kt, kh, qot, qoh, kot, koh,
                        T, Hq, Hk, D, rows, rot, interleaved, eps), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_qk_norm_rope_backward_workspace_size(tokens, q_heads, k_heads, head_dim) -> int:
    """Bytes of the workspace mx_qk_norm_rope_backward needs where it writes a weight gradient."""
    return int(load().mx_qk_norm_rope_backward_workspace_size(tokens, q_heads, k_heads, head_dim))


def mx_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, cos, sin, dq, dk, q_weight=None,
                             k_weight=None, dq_weight=None, dk_weight=None, workspace=None,
                             eps=1e-6, interleaved=False, stream=None):
    """Gradients of mx_qk_norm_rope: dq, dk (bf16, may be dq_out, dk_out) from those of its outputs,
    and dq_weight, dk_weight (fp32 [head_dim], written; None: not wanted).  workspace: a tensor of
    mx_qk_norm_rope_backward_workspace_size bytes, zero before its first use, reusable (by this call, not
    by mx_attn_fp4)."""
    fn, dev = "mx_qk_norm_rope_backward", _current_device()
    qp, qt, qh = _heads(fn, q, "q", dev)
    T, Hq, D = q.shape
    gqp, gqt, gqh = _heads(fn, dq_out, "dq_out", dev, q.shape)
    dqp, dqt, dqh = _heads(fn, dq, "dq", dev, q.shape)
    kp = kt = kh = gkp = gkt = gkh = dkp = dkt = dkh = Hk = 0
    if k is not None:
        kp, kt, kh = _heads(fn, k, "k", dev)
        Hk = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise MxError(fn, MX_ERR_SHAPE, f"k has shape {tuple(k.shape)}, q {tuple(q.shape)}")
        gkp, gkt, gkh = _heads(fn, dk_out, "dk_out", dev, k.shape)
        dkp, dkt, dkh = _heads(fn, dk, "dk", dev, k.shape)
    qw = 0 if q_weight is None else _flat(fn, q_weight, "q_weight", _bf16, dev, (D,))
    kw = 0 if k_weight is None else _flat(fn, k_weight, "k_weight", _bf16, dev, (D,))
    dqw = 0 if dq_weight is None else _flat(fn, dq_weight, "dq_weight", _f32, dev, (D,))
    dkw = 0 if dk_weight is None else _flat(fn, dk_weight, "dk_weight", _f32, dev, (D,))
    pp, cp, sp, rows, rot = _rotation(fn, positions, cos, sin, T, dev)
    wp, wb = _workspace(fn, workspace, dev)
    st = load().mx_qk_norm_rope_backward(
        _NORM_ROPE_BACK.pack(gqp, gkp, qp, kp, dqp, dkp, qw, kw, dqw, dkw, pp, cp, sp, wp, wb,
                             gqt, gqh, gkt, gkh, qt, qh, kt, kh, dqt, dqh, dkt, dkh, T, Hq, Hk, D,
                             rows, rot, interleaved, eps), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_kv_append_fp4(cache, k, v, slots, positions=None, cos=None, sin=None, k_out=None,
                     v_out=None, interleaved=False, stream=None):
    """Writes keys (rotated by positions, cos, sin where given) and values of new tokens into the
    cache's slots, as MXFP4.

    cache: MxKvCacheFp4; k, v: bf16 [tokens, kv_heads, head_dim], strides multiples of 8; slots:
    int64 [tokens], page * page_size + token (outside the cache: the token is skipped).
    k_out, v_out: bf16 [tokens, kv_heads, head_dim], the values as stored, or None."""
    fn, dev = "mx_kv_append_fp4", _current_device()
    _cache(fn, cache, dev)
    kp, kt, kh = _heads(fn, k, "k", dev)
    T, H, D = k.shape
    if H != cache.kv_heads or D != cache.head_dim:
        raise MxError(fn, MX_ERR_SHAPE, f"k has shape {tuple(k.shape)}, the cache "
                                        f"{cache.kv_heads} heads of {cache.head_dim}")
    vp, vt, vh = _heads(fn, v, "v", dev, k.shape)
    sp_ = _flat(fn, slots, "slots", _i64, dev, (T,))
    pp, cp, sp, rows, rot = _rotation(fn, positions, cos, sin, T, dev)
    ko = 0 if k_out is None else _flat(fn, k_out, "k_out", _bf16, dev, k.shape)
    vo = 0 if v_out is None else _flat(fn, v_out, "v_out", _bf16, dev, k.shape)
    st = load().mx_kv_append_fp4(
        _APPEND.pack(cache._addr, kp, vp, sp_, pp, cp, sp, ko, vo, kt, kh, vt, vh, T, rows, rot,
                     interleaved), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def mx_attn_fp4_workspace_size(batch, max_q, q_heads, kv_heads, head_dim) -> int:
    """Bytes of workspace mx_attn_fp4 and mx_attn_tree_fp4 need for these sizes and all smaller batch and
    max_q, whatever the lengths (mx_attn_fp4 alone is content with 26 MB at 33 to 64 rows of heads of 128 and
    17 to 32 of 256, where trees make it 43 and 77)."""
    return int(load().mx_attn_fp4_workspace_size(batch, max_q, q_heads, kv_heads, head_dim))


def mx_attn_fp4(cache, q, page_table, seq_lens, out, workspace, q_starts=None, max_q=None,
                scale=None, causal=True, window=0, lse=None, stream=None):
    """Attention of new queries over the cache.

    q, out: bf16 [total_q, q_heads, head_dim], strides multiples of 8; page_table: int32
    [batch, width]; seq_lens: int32 [batch], tokens cached, the new ones included.  q_starts: int32
    [batch + 1], where each sequence's queries begin (at most max_q each); None: max_q of every
    sequence (default total_q / batch).  scale: default head_dim ** -0.5.  window: keys that a query
    sees, itself included (0: all).  lse: fp32 [total_q, q_heads] or None.  workspace: a tensor of
    mx_attn_fp4_workspace_size bytes, zero before its first use, reusable."""
    fn, dev = "mx_attn_fp4", _current_device()
    (qp, op, lp, tp, lens, starts, wp, wb, strides, table, B, N, max_q, H, scale) = _attn(
        fn, dev, cache, q, page_table, seq_lens, out, workspace, q_starts, max_q, scale, lse)
    st = load().mx_attn_fp4(
        _ATTN.pack(cache._addr, qp, op, lp, tp, lens, starts, wp, wb, *strides, *table, B, N, max_q, H,
                   causal, window, scale), _stream(stream, dev))
    if st != MX_OK:
        raise MxError(fn, st)


def _attn(fn, dev, cache, q, page_table, seq_lens, out, workspace, q_starts, max_q, scale, lse):
    """What every attention call checks and passes: pointers, strides of q and out, of the table, sizes."""
    _cache(fn, cache, dev)
    qp, qt, qh = _heads(fn, q, "q", dev)
    N, H, D = q.shape
    if D != cache.head_dim:
        raise MxError(fn, MX_ERR_SHAPE, f"q has head_dim {D}, the cache {cache.head_dim}")
    op, ot, oh = _heads(fn, out, "out", dev, q.shape)
    tp, stride, B, width = _table(fn, page_table, dev)
    lens = _flat(fn, seq_lens, "seq_lens", _i32, dev, (B,))
    starts, max_q = _starts(fn, q_starts, max_q, N, B, dev)
    lp = 0 if lse is None else _flat(fn, lse, "lse", _f32, dev, (N, H))
    wp, wb = _workspace(fn, workspace, dev)
    return (qp, op, lp, tp, lens, starts, wp, wb, (qt, qh, ot, oh), (stride, width), B, N, max_q, H,
            D ** -0.5 if scale is None else scale)
