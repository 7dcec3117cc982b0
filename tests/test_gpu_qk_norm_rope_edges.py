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
