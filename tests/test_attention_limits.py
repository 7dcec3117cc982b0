"""The attention operators' limits on the host, with no GPU: what lies on both sides of each."""
import pytest
import torch

import block_scaled_precision_act_amd as mx
from test_attention_abi import ATTN, _cache_address, _pack, lib  # noqa: F401 (lib: a fixture)

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
