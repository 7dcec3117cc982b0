"""Plain CPU reference of the attention operators (numpy, float64): test infrastructure only.

Written from the definitions in include/mx_attention.h, row by row and sequence by sequence; shares
nothing with the HIP path.  Only the append's rotation is carried in float32, because the codes it
stores are defined by that arithmetic (each product rounded, then their sum).
"""
from __future__ import annotations

import numpy as np

from . import mx_oracle as O


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, positions, cos, sin, interleaved=False, back=False, dtype=np.float64):
    """x [T, H, D] with the first 2 * cos.shape[1] values of each head turned by the tokens'
    positions (back: by the transpose)."""
    y = np.array(x, dtype=dtype)
    if positions is None:
        return y
    a, b = _pairs(2 * cos.shape[1], interleaved)
    c = cos[positions].astype(dtype)[:, None]
    s = sin[positions].astype(dtype)[:, None] * dtype(-1 if back else 1)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = (xa * c).astype(dtype) - (xb * s).astype(dtype)
    y[..., b] = (xb * c).astype(dtype) + (xa * s).astype(dtype)
    return y


def norm_rope(x, w, positions, cos, sin, eps=1e-6, interleaved=False):
    """(result, bound on the pair's magnitudes) in float64."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y = rotate(x, positions, cos, sin, interleaved)
    size = np.abs(x)
    if positions is not None:
        a, b = _pairs(2 * cos.shape[1], interleaved)
        size[..., a] = size[..., b] = size[..., a] + size[..., b]
    return y, size


def norm_rope_backward(dy, x, w, positions, cos, sin, eps=1e-6, interleaved=False):
    """dx, dw (None without a weight) and the magnitudes that their sums' errors scale with."""
    dn = rotate(dy, positions, cos, sin, interleaved, back=True)
    size = np.abs(np.asarray(dy, np.float64))
    if positions is not None:
        a, b = _pairs(2 * cos.shape[1], interleaved)
        size[..., a] = size[..., b] = size[..., a] + size[..., b]
    if w is None:
        return dn, None, size, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dn * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    sx = r * (size * np.abs(w) + np.abs(x) * r * r * (size * np.abs(w * x)).mean(-1, keepdims=True))
    return dx, (dn * x * r).sum((0, 1)), sx, (size * np.abs(x) * r).sum((0, 1))


def quantize_fp4(x):
    """float32 [..., D] -> packed codes [..., D / 2], E8M0 bytes [..., D / 32], stored values."""
    x = np.asarray(x, np.float32).astype(np.float64)
    lead, d = x.shape[:-1], x.shape[-1]
    b = x.reshape(-1, 32)
    top = np.maximum(np.abs(b).max(-1), np.float64(np.float32(1e-4)))
    m, e = np.frexp(top / 6.0)
    # the smallest E with top <= 6 * 2^E, decided on exact values
    E = np.where(np.ldexp(6.0, e - 1) >= top, e - 1, e)
    y = np.ldexp(b, -E[:, None])
    codes = O.e2m1_encode_rne(y)
    vals = np.ldexp(np.array(O.FP4_TABLE)[codes], E[:, None])
    packed = O.fp4_pack(codes.reshape(-1, d))
    return (packed.reshape(*lead, d // 2), (E + 127).astype(np.uint8).reshape(*lead, d // 32),
            vals.reshape(*lead, d))


def cache_rows(codes, scales, table_row, length):
    """float64 [kv_heads, length, D] of a sequence, through its row of the page table."""
    pages, heads, size, half = codes.shape
    t = np.arange(length)
    page = np.asarray(table_row)[t // size] if length else np.zeros(0, int)
    c, s = codes[page, :, t % size], scales[page, :, t % size]           # [length, heads, .]
    nib = np.stack([c & 15, c >> 4], -1).reshape(length, heads, 2 * half)
    table = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    v = np.where(nib >= 8, -1.0, 1.0) * table[nib & 7]
    v = v * np.ldexp(1.0, np.repeat(s.astype(int), 32, -1) - 127)
    v[np.repeat(s == 255, 32, -1)] = np.nan
    return v.transpose(1, 0, 2)


def attention(q, k_codes, k_scales, v_codes, v_scales, page_table, seq_lens, q_starts, scale,
              causal=True, window=0):
    """out [N, Hq, D], lse [N, Hq] and, for error bounds, the weighted mean of |v| [N, Hq, D] and
    the largest scale * sum |q k| of a row [N, Hq]."""
    N, hq, D = q.shape
    q = np.asarray(q, np.float64)
    hk = k_codes.shape[1]
    out, lse = np.zeros((N, hq, D)), np.full((N, hq), -np.inf)
    mag, top = np.zeros((N, hq, D)), np.zeros((N, hq))
    for b, L in enumerate(seq_lens):
        k = cache_rows(k_codes, k_scales, page_table[b], L)
        v = cache_rows(v_codes, v_scales, page_table[b], L)
        n = q_starts[b + 1] - q_starts[b]
        for i in range(n):
            row, pos = q_starts[b] + i, L - n + i
            hi = min(L, pos + 1) if causal else L
            lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(hq):
                kk, vv = k[h // (hq // hk), lo:hi], v[h // (hq // hk), lo:hi]
                s = scale * (kk @ q[row, h])
                m = s.max()
                p = np.exp(s - m)
                out[row, h] = p @ vv / p.sum()
                mag[row, h] = p @ np.abs(vv) / p.sum()
                lse[row, h] = m + np.log(p.sum())
                top[row, h] = abs(scale) * (np.abs(kk) @ np.abs(q[row, h])).max()
    return out, lse, mag, top
