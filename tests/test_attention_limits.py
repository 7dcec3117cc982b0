"""The attention operators' limits on the host, with no GPU: what lies on both sides of each."""
import re

import pytest
import torch

import block_scaled_precision_act_amd as mx
from test_attention_abi import A, APPEND, ATTN, HEADER, NORM, _cache_address, _pack, lib  # noqa: F401 (lib: a fixture)

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


def _meet(n, a, m, b, size):
    at = sorted(i * a + j * b for i in range(n) for j in range(m))
    return any(y - x < size for x, y in zip(at, at[1:]))


@host_only
def test_outputs_whose_rows_lie_on_each_other_are_refused(lib):  # noqa: F811
    # every pair of strides of up to 9 rows, against all rows' places written out
    D, keep = 64, []
    cache = _cache_address(keep, kv_heads=1, head_dim=D)
    seen = set()
    for tokens, heads in ((2, 2), (3, 2), (2, 5), (4, 3), (3, 7)):
        for a in range(D // 2, 9 * D + 1, D // 2):
            for b in range(D // 2, 9 * D + 1, D // 2):
                want = mx.MX_ERR_STRIDE if _meet(tokens, a, heads, b, D) else mx.MX_ERR_DEVICE
                out = dict(q_out_token_stride=a, q_out_head_stride=b)
                args = {**NORM, **out, "k": 0, "tokens": tokens, "q_heads": heads, "head_dim": D, "rot": D}
                assert lib.mx_qk_norm_rope(_pack("mx_qk_norm_rope_args", args), None) == want, (tokens, heads, a, b)
                args = {**ATTN, "cache": cache, "total_q": tokens, "batch": 1, "max_q": tokens, "q_heads": heads,
                        "out_token_stride": a, "out_head_stride": b}
                assert lib.mx_attn_fp4(_pack("mx_attn_fp4_args", args), None) == want, (tokens, heads, a, b)
                seen.add((want, a < b, a >= D and b >= D))
    assert len(seen) == 6                                  # each answer on either side, also where no stride is short
    for huge in (1 << 62, (1 << 62) + 64):                 # products beyond 64 bits
        args = {**NORM, "k": 0, "q_out_token_stride": huge, "q_out_head_stride": huge}
        assert lib.mx_qk_norm_rope(_pack("mx_qk_norm_rope_args", args), None) == mx.MX_ERR_STRIDE


@host_only
@pytest.mark.parametrize("kind,block", [("code", 16 * 64), ("scale", 16 * 4)])
def test_caches_whose_blocks_lie_on_each_other_are_not_written(lib, kind, block):  # noqa: F811
    for page, head, status in ((block, block, mx.MX_ERR_STRIDE), (2 * block, 4 * block, mx.MX_ERR_STRIDE),
                               (2 * block, block, mx.MX_ERR_DEVICE), (block, 10 * block, mx.MX_ERR_DEVICE),
                               (2 * block, 3 * block, mx.MX_ERR_DEVICE), (3 * block, 2 * block, mx.MX_ERR_DEVICE)):
        keep = []
        c = _cache_address(keep, **{f"{kind}_page_stride": page, f"{kind}_head_stride": head})
        assert lib.mx_kv_append_fp4(_pack("mx_kv_append_fp4_args", {**APPEND, "cache": c}), None) == status, (page, head)


def test_the_limits_of_pages_and_tables_are_documented():
    text = " ".join(re.sub(r"^ \* ", "", HEADER, flags=re.M).split())
    for said in ("table_width * page_size at most 2^31 - 1024", "table_width * (page_size / 16)^2 < 2^32",
                 "Attention takes no page of 2^20 tokens or more"):
        assert said in text
    assert "width * (page_size / 16) ** 2 < 2 ** 32" in mx.MxKvCacheFp4.__doc__


@host_only
@pytest.mark.parametrize("page_size,most", [((1 << 20) - 16, 1), (1 << 16, 255), (1 << 14, 4095), (496, (2 ** 31 - 1024) // 496)])
def test_the_widest_table_of_large_pages(lib, page_size, most):  # noqa: F811
    keep = []
    block = page_size * 64
    cache = _cache_address(keep, page_size=page_size, code_head_stride=block, code_page_stride=2 * block,
                           scale_head_stride=block // 16, scale_page_stride=block // 8)
    for width, status in ((most, mx.MX_ERR_DEVICE), (most + 1, mx.MX_ERR_SHAPE)):
        args = {**ATTN, "cache": cache, "batch": 1, "total_q": 1, "table_width": width, "table_stride": width}
        assert lib.mx_attn_fp4(_pack("mx_attn_fp4_args", args), None) == status, width
