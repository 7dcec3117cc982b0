"""The gradients of the per-head norm with rotation (mx_qk_norm_rope_backward) where there are no rows,
and where there are very many."""
import numpy as np
import pytest
import torch

from attention_util import bf16, f64
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,hq,hk", [(0, 4, 2), (3, 0, 2), (3, 4, 0), (3, 0, 0)])
def test_weight_gradients_without_rows_are_zero(mx, D, T, hq, hk):
    # through a workspace of just what the size query asks for
    q, k = (torch.ones((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dw = [torch.full((D,), 7.0, device="cuda") for _ in "qk"]
    n = mx.mx_qk_norm_rope_backward_workspace_size(T, hq, hk, D)
    assert n == 0 if T == 0 else n > 0
    note(f"norm_rope_backward T={T} hq={hq} hk={hk} D={D}")
    mx.mx_qk_norm_rope_backward(q, k, q, k, None, None, None, dq, dk, w, w, *dw,
                                torch.zeros(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert T * hq > 0 or not dw[0].any()
    assert T * hk > 0 or not dw[1].any()
    for d, h in zip(dw, (hq, hk)):                    # rows of ones: x r = 1 / sqrt(1 + eps), one each
        if T * h > 0:
            assert (np.abs(f64(d) - T * h / np.sqrt(1 + 1e-6)) <= 2.0 ** -15 * T * h).all()


@pytest.mark.parametrize("D,inter", [(64, False), (64, True), (128, False), (256, True)])
def test_the_gradient_of_very_many_rows(mx, D, inter):
    """2^34 values in rows that are all alike (token strides of 0): 511 workgroups' lanes of 8 values add
    2^34 / (511 * 2048) = 16416 equal terms each.

    In one plain fp32 chain their rounding errors add up to parts in 10^4 (checked below); in chains of at
    most 2^9 additions the gradient is within 2^-15 of the sum of the terms' magnitudes, here the sum."""
    T = (1 << 34) // D
    rng = np.random.default_rng(5)
    x, g = (bf16(rng.uniform(0.5, 2, (1, 1, D))).cuda() for _ in "xg")
    w = bf16(1 + 0.3 * rng.standard_normal(D)).cuda()
    x1, g1 = f64(x)[0, 0], f64(g)[0, 0]
    term = g1 * x1 / np.sqrt((x1 * x1).mean() + 1e-6)
    chain = np.cumsum(np.repeat(term[None].astype(np.float32), 16416, 0), 0, dtype=np.float32)[-1]
    plain = np.abs(chain.astype(np.float64) - 16416 * term.astype(np.float32).astype(np.float64)) / (16416 * term)
    assert plain.max() > 2.0 ** -13
    dw, dx = torch.empty(D, device="cuda"), torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mx.mx_qk_norm_rope_backward_workspace_size(T, 1, 0, D), dtype=torch.uint8, device="cuda")
    note(f"norm_rope_backward of {T} rows, D={D} inter={inter}")
    mx.mx_qk_norm_rope_backward(g.expand(T, 1, D), None, x.expand(T, 1, D), None, None, None, None, dx, None, w, None,
                                dw, None, ws, interleaved=inter)
    torch.cuda.synchronize()
    assert (np.abs(f64(dw) - T * term) <= 2.0 ** -15 * T * term).all()


def test_an_infinite_gradient_stays_infinite(mx):
    # past the first fold: a weight gradient that overflows is an infinity, not NaN
    D, T = 64, 1 << 24
    x = torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda")
    g = torch.full((1, 1, D), 1e36, dtype=torch.bfloat16, device="cuda")
    g[..., 1] = 1.0
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    dw, dx = torch.empty(D, device="cuda"), torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(mx.mx_qk_norm_rope_backward_workspace_size(T, 1, 0, D), dtype=torch.uint8, device="cuda")
    note("norm_rope_backward overflowing")
    mx.mx_qk_norm_rope_backward(g.expand(T, 1, D), None, x.expand(T, 1, D), None, None, None, None, dx, None, w, None,
                                dw, None, ws)
    torch.cuda.synchronize()
    out = f64(dw)
    assert np.isposinf(np.delete(out, 1)).all() and abs(out[1] - T) <= T * 2.0 ** -15
