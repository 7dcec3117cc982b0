"""Pins of the attention oracle (CPU): central differences of the norm's gradients, the rotation as
complex products, brute-force softmax over explicitly listed keys, and the quantizer against the
library's own oracle of the MXFP4 producer."""
import math

import numpy as np
import pytest

from oracle import attention_oracle as A
from oracle import mx_oracle as O


def _tables(rows, rot):
    a = np.arange(rows)[:, None] * 7.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_complex_product_and_its_transpose_undoes_it(inter):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 64))
    cos, sin = _tables(9, 32)
    pos = np.array([0, 3, 8, 8, 1])
    y = A.rotate(x, pos, cos, sin, inter)
    for t in range(5):
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 16)
            z = (x[t, 1, a] + 1j * x[t, 1, b]) * (float(cos[pos[t], i]) + 1j * float(sin[pos[t], i]))
            assert abs(y[t, 1, a] - z.real) < 1e-12 and abs(y[t, 1, b] - z.imag) < 1e-12
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(A.rotate(y, pos, cos, sin, inter, back=True), x, atol=1e-6)   # fp32 tables


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 32, 64])
def test_gradients_against_differences(inter, rot):
    rng = np.random.default_rng(2)
    T, H, D, eps = 3, 2, 64, 1e-3
    x, w, dy = rng.standard_normal((T, H, D)), rng.standard_normal(D), rng.standard_normal((T, H, D))
    cos, sin = _tables(5, rot) if rot else (None, None)
    pos = np.array([4, 0, 2]) if rot else None

    def loss(x, w):
        return (A.norm_rope(x, w, pos, cos, sin, eps, inter)[0] * dy).sum()

    dx, dw, _, _ = A.norm_rope_backward(dy, x, w, pos, cos, sin, eps, inter)
    step = 1e-6
    for _ in range(40):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[i]) < 1e-7
    for j in range(0, D, 7):
        e = np.zeros_like(w)
        e[j] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[j]) < 1e-7
    # without a weight: the rotation alone
    dx, none, _, _ = A.norm_rope_backward(dy, x, None, pos, cos, sin, eps, inter)
    assert none is None and np.allclose(dx, A.rotate(dy, pos, cos, sin, inter, back=True))


def test_quantizer_is_the_mxfp4_producers_rule():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 128)) * np.exp(5 * rng.standard_normal((40, 1)))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)                 # truncated to bf16 patterns
    xb = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales, vals = A.quantize_fp4(xb)
    want, want_s = O.act_quant_fp4(bits)
    assert np.array_equal(codes, want) and np.array_equal(scales, want_s)
    assert np.array_equal(vals, O.decode_fp4_rows(codes, scales))
    # values that are no bf16: the nearest code, the smallest scale that clips nothing
    y = rng.standard_normal((50, 64)).astype(np.float32)
    y[0, :32] = 6 * 0.25
    y[0, 32:] = np.nextafter(np.float32(1.5), np.float32(2))
    codes, scales, vals = A.quantize_fp4(y)
    s = np.ldexp(1.0, scales.astype(int) - 127)
    top = np.abs(y).reshape(50, 2, 32).max(-1)
    assert (top <= 6 * s).all() and (top > 3 * s).all()
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    near = np.abs(np.abs(y.reshape(50, 2, 32, 1)) / s[..., None, None] - grid).min(-1)
    assert np.allclose(np.abs(vals - y).reshape(50, 2, 32) / s[..., None], near, atol=1e-12)
    assert scales[0, 0] + 1 == scales[0, 1]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 5)])
def test_attention_brute_force(causal, window):
    rng = np.random.default_rng(4)
    pages, hk, size, D, G = 7, 2, 16, 64, 2
    kc, vc = (rng.integers(0, 256, (pages, hk, size, D // 2), dtype=np.uint8) for _ in "kv")
    ks, vs = (rng.integers(122, 130, (pages, hk, size, D // 32), dtype=np.uint8) for _ in "kv")
    lens, starts = [0, 3, 37], [0, 1, 6, 9]                # 5 queries on 3 keys: two see nothing
    table = np.array([[0, 0, 0], [5, 0, 0], [3, 6, 1]])
    q = rng.standard_normal((9, hk * G, D))
    out, lse, _, _ = A.attention(q, kc, ks, vc, vs, table, lens, starts, 0.2, causal, window)
    for b in range(3):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            for h in range(hk * G):
                num, den = np.zeros(D), 0.0
                for t in range(lens[b]):
                    p = lens[b] - n + i
                    if causal and t > p or window and t <= p - window:
                        continue
                    at = (table[b][t // size], h // G, t % size)
                    k = O.decode_fp4_rows(kc[at][None], ks[at][None])[0]
                    v = O.decode_fp4_rows(vc[at][None], vs[at][None])[0]
                    e = math.exp(0.2 * sum(float(x) * float(y) for x, y in zip(k, q[starts[b] + i, h])))
                    num, den = num + e * v, den + e
                row = starts[b] + i
                if den == 0:
                    assert not out[row, h].any() and lse[row, h] == -np.inf
                else:
                    assert np.allclose(out[row, h], num / den, rtol=1e-10, atol=1e-12)
                    assert abs(lse[row, h] - math.log(den)) < 1e-9
