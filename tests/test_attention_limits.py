"""The attention operators' limits on the host, with no GPU: what lies on both sides of each."""
import pytest
import torch

import block_scaled_precision_act_amd as mx
from test_attention_abi import A, ATTN, _cache_address, _pack, lib  # noqa: F401 (lib: a fixture)

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")


@host_only
@pytest.mark.parametrize("page_size", [16, 48, 496])
def test_tokens_that_a_table_row_covers(lib, page_size):  # noqa: F811
    # token numbers up to two tiles past a length stay within 31 bits
    keep = []
    block = page_size * 64
    cache = _cache_address(keep, page_size=page_size, code_head_stride=block, code_page_stride=2 * block,
                           scale_head_stride=block // 16, scale_page_stride=block // 8)
    most = (2 ** 31 - 1024) // page_size
    for width, status in ((most, mx.MX_ERR_DEVICE), (most + 1, mx.MX_ERR_SHAPE), (2 ** 31 // page_size, mx.MX_ERR_SHAPE)):
        args = {**ATTN, "cache": cache, "batch": 1, "total_q": 1, "table_width": width, "table_stride": width}
        assert lib.mx_attn_fp4(_pack("mx_attn_fp4_args", args), None) == status, width


@host_only
def test_weight_gradients_without_rows_need_no_workspace(lib):  # noqa: F811
    # what the size query asks for is enough: 0 bytes without tokens, and nothing for a tensor without heads
    assert mx.mx_qk_norm_rope_backward_workspace_size(0, 4, 2, 128) == 0
    base = dict(q_weight=A, k_weight=A, dq_weight=A, dk_weight=A, positions=A, cos=A, sin=A, q_heads=4, k_heads=2,
                head_dim=128, table_rows=9, rot=64, eps=1e-6, k=A)

    def status(**change):
        return lib.mx_qk_norm_rope_backward(_pack("mx_qk_norm_rope_backward_args", {**base, **change}), None)

    assert status(tokens=0) == mx.MX_ERR_DEVICE
    assert status(tokens=0, k=0, dk_weight=0) == mx.MX_ERR_DEVICE
    assert status(tokens=5, q_heads=0, k=0) == mx.MX_ERR_DEVICE
    rows = dict(dk_out=A, dk=A, **{f"{t}_{s}_stride": 256 for t in ("dk_out", "k", "dk") for s in ("token", "head")})
    assert status(tokens=5, q_heads=0, k_heads=1, **rows) == mx.MX_ERR_WORKSPACE
    assert status(tokens=5, q_heads=0, k_heads=1, dk_weight=0, **rows) == mx.MX_ERR_DEVICE
