"""The draft operators' C ABI on the host, with no GPU: the library exports what include/mx_draft.h declares,
the binding packs its structs, and every argument error is a status before any device work."""
import ctypes
import os
import re
import struct

import pytest
import torch

import block_scaled_precision_act_amd as mx
from block_scaled_precision_act_amd import attention as at
from block_scaled_precision_act_amd import drafts as dr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "mx_draft.h")).read()
A = 1 << 20            # fake aligned addresses: never dereferenced by these calls
B = 1 << 24


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        from block_scaled_precision_act_amd import build
        build.build()
    return mx.load()


def _fields(name):
    """Field names of a struct of the header, in order, with their types' struct codes."""
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), HEADER, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    out = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        if "*" in decl:
            out.append((decl.split("*")[-1].strip(), "Q"))
            continue
        kind, names = decl.split(" ", 1)
        out += [(n.strip(), {"int64_t": "q", "double": "d"}[kind]) for n in names.split(",")]
    return out


STRUCTS = {"mx_tree_mask_args": dr._TREE_MASK, "mx_attn_tree_fp4_args": dr._ATTN_TREE,
           "mx_tree_verify_args": dr._VERIFY, "mx_kv_accept_fp4_args": dr._ACCEPT}


@pytest.mark.parametrize("name", STRUCTS)
def test_the_binding_packs_the_headers_structs(name):
    fields = _fields(name)
    assert 8 * len(fields) == STRUCTS[name].size
    assert re.sub(r"(\d+)(\w)", lambda m: m[2] * int(m[1]), STRUCTS[name].format[1:]) == "".join(c for _, c in fields)


def test_library_exports_and_binding_covers_every_declared_symbol(lib):
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(mx_\w+)\s*\(", HEADER, re.M)))
    assert names == ["mx_attn_tree_fp4", "mx_kv_accept_fp4", "mx_tree_mask", "mx_tree_verify",
                     "mx_tree_verify_workspace_size"]
    for n in names:
        assert hasattr(lib, n) and n in mx._SIGS and callable(getattr(mx, n))


def _call(lib, fn, good, change, keep=()):
    fields = _fields(fn + "_args")
    values = {**good, **change}
    assert set(values) <= {n for n, _ in fields}
    return getattr(lib, fn)(STRUCTS[fn + "_args"].pack(*(values.get(n, 0) for n, _ in fields)), None)


def _expect(status):
    """The status; to be asked for before the call, which goes on to the GPU where there is one."""
    if status == "device":
        if torch.cuda.is_available():
            pytest.skip("a GPU is visible: fake addresses must not reach it")
        return mx.MX_ERR_DEVICE
    return status


CACHE = dict(k=A, k_scale=A, v=A, v_scale=A, pages=10, kv_heads=2, page_size=16, head_dim=128,
             code_page_stride=2 * 16 * 64, code_head_stride=16 * 64, scale_page_stride=2 * 16 * 4,
             scale_head_stride=16 * 4)
NAMES = ["k", "k_scale", "v", "v_scale", "pages", "kv_heads", "page_size", "head_dim", "code_page_stride",
         "code_head_stride", "scale_page_stride", "scale_head_stride"]


def _caches(*changes):
    """Address of an array of caches; each later one's tensors lie elsewhere."""
    data = b"".join(at._CACHE.pack(*({**CACHE, **{n: A + (i << 16) + 4096 * k for k, n in enumerate(NAMES[:4])}, **c}[n]
                                     for n in NAMES)) for i, c in enumerate(changes))
    buf = ctypes.create_string_buffer(data)
    return buf, ctypes.addressof(buf)


S, N, AL, ST, W, OK = (mx.MX_ERR_SHAPE, mx.MX_ERR_NULL, mx.MX_ERR_ALIGN, mx.MX_ERR_STRIDE, mx.MX_ERR_WORKSPACE,
                       mx.MX_OK)
MASK = dict(parents=A, seq_lens=A, mask=B, positions=2 * B, mask_stride=2, mask_words=2, batch=2, total_q=80, max_q=40)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), S), (dict(batch=65536), S), (dict(max_q=41), S), (dict(q_starts=A, max_q=1025, mask_words=40,
                                                                            mask_stride=40), S),
    (dict(total_q=1 << 31, q_starts=A), S), (dict(mask_words=1), S), (dict(mask_words=-1), S), (dict(mask_words=1 << 31), S),
    (dict(mask_stride=1), ST), (dict(mask_stride=-2), ST), (dict(parents=0), N), (dict(mask=0), N),
    (dict(seq_lens=0), N), (dict(positions=0), N), (dict(parents=A + 2), AL), (dict(mask=A + 1), AL),
    (dict(q_starts=A + 2), AL), (dict(positions=A + 2), AL), (dict(mask=A), ST), (dict(positions=A + 80 * 4 - 4), ST),
    (dict(positions=B + 4), ST), (dict(positions=A + 80 * 4), "device"), (dict(batch=0, total_q=0, parents=0), OK),
    (dict(total_q=0, q_starts=A, mask=0), OK), ({}, "device"), (dict(seq_lens=0, positions=0), "device"),
    (dict(q_starts=A, max_q=64), "device")])
def test_tree_mask(lib, change, status):
    expected = _expect(status)
    assert _call(lib, "mx_tree_mask", MASK, change) == expected
    assert lib.mx_tree_mask(None, None) == N


ATTN = dict(q=A, out=A, mask=A, page_table=A, seq_lens=A, workspace=A, workspace_bytes=1 << 30, q_token_stride=512,
            q_head_stride=128, out_token_stride=512, out_head_stride=128, mask_stride=2, mask_words=2, table_stride=8,
            table_width=8, batch=2, total_q=80, max_q=40, q_heads=4, scale=0.1)


@pytest.mark.parametrize("change,status", [
    (dict(cache=0), N), (dict(q_heads=3), S), (dict(batch=-1), S), (dict(max_q=41), S), (dict(window=-3), S),
    (dict(window=1 << 31, positions=A), S), (dict(window=5), N), (dict(scale=float("nan")), S), (dict(mask=0), N),
    (dict(mask_words=1), S), (dict(mask_words=1 << 31), S), (dict(mask_stride=-1), ST), (dict(mask=A + 2), AL),
    (dict(window=5, positions=A + 1), AL), (dict(q_starts=A, max_q=65537, mask_words=4000), S), (dict(table_stride=7), ST),
    (dict(page_table=0), N), (dict(seq_lens=0), N), (dict(q=0), N), (dict(out=0), N), (dict(q=A + 8), AL),
    (dict(out_head_stride=120), ST), (dict(workspace=0), W), (dict(workspace_bytes=1 << 23), W),
    (dict(batch=0, total_q=0, q=0, mask=0), OK), ({}, "device"), (dict(mask_stride=0), "device"),
    (dict(window=5, positions=A), "device"), (dict(q_starts=A, max_q=64), "device")])
def test_attn_tree(lib, change, status):
    keep, c = _caches({})
    expected = _expect(status)
    assert _call(lib, "mx_attn_tree_fp4", {**ATTN, "cache": c}, change) == expected
    assert lib.mx_attn_tree_fp4(None, None) == N


def test_attn_tree_refuses_what_a_cache_may_not_be(lib):
    for change, status in ((dict(head_dim=32), S), (dict(page_size=24), S), (dict(k=A + 8), AL), (dict(k=0), N),
                           (dict(code_head_stride=512), ST)):
        keep, c = _caches(change)
        assert _call(lib, "mx_attn_tree_fp4", {**ATTN, "cache": c}, {}) == status


VERIFY = dict(target=A, draft=A, tokens=A, parents=A, accept_u=A, sample_u=A, path=B, tokens_out=2 * B, count=3 * B, workspace=A,
              workspace_bytes=1 << 24, target_stride=100, draft_stride=100, batch=2, total_q=10, max_q=5, vocab=100,
              width=5)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), S), (dict(batch=65536), S), (dict(max_q=6), S), (dict(max_q=1025, q_starts=A), S), (dict(vocab=0), S),
    (dict(vocab=(1 << 30) + 1), S), (dict(width=0), S), (dict(width=1 << 31), S), (dict(type=3), S), (dict(type=-1), S),
    (dict(target_stride=99), ST), (dict(target_stride=0), ST), (dict(target_stride=-1), ST), (dict(draft_stride=99), ST),
    (dict(draft_stride=-100), ST), (dict(target=0), N), (dict(tokens=0), N), (dict(parents=0), N), (dict(accept_u=0), N),
    (dict(sample_u=0), N), (dict(path=0), N), (dict(tokens_out=0), N), (dict(count=0), N), (dict(target=A + 2), AL),
    (dict(type=1, draft=A + 1), AL), (dict(path=A + 2), AL), (dict(accept_u=A + 1), AL), (dict(path=A), ST), (dict(path=A + 3999), AL),
    (dict(path=A + 3996), ST), (dict(tokens_out=B + 36), ST), (dict(tokens_out=B + 40), "device"), (dict(count=2 * B), ST),
    (dict(target_stride=(1 << 30) + 1), ST), (dict(batch=3, total_q=15, width=1 << 30), S), (dict(workspace=0), W),
    (dict(workspace=A + 64), W), (dict(workspace_bytes=1 << 23), W), (dict(batch=0, total_q=0, path=0), OK),
    (dict(total_q=0, max_q=0, target=0, tokens=0), "device"), ({}, "device"), (dict(draft=0, draft_stride=0), "device"),
    (dict(draft_stride=0), "device"), (dict(type=2, target=A + 2, draft=A + 2), "device")])
def test_verify(lib, change, status):
    expected = _expect(status)
    assert _call(lib, "mx_tree_verify", VERIFY, change) == expected
    assert lib.mx_tree_verify(None, None) == N


def test_verify_workspace_size(lib):
    size = mx.mx_tree_verify_workspace_size
    assert size(1) == size(65535) > 0 and size(0) == size(-1) == size(65536) == 0
    # an attention workspace is as large whatever its call
    assert min(mx.mx_attn_fp4_workspace_size(1, 1, 1, 1, d) for d in (64, 128, 256)) >= size(1)


ACCEPT = dict(page_table=A, seq_lens=A, path=A, count=A, lens_out=B, layers=2, table_stride=8, table_width=8, batch=2,
              total_q=10, max_q=5, width=5)


@pytest.mark.parametrize("change,status", [
    (dict(caches=0), N), (dict(layers=-1), S), (dict(layers=1025), S), (dict(batch=-1), S), (dict(max_q=6), S),
    (dict(q_starts=A, max_q=1025), S), (dict(width=-1), S), (dict(table_width=-1), S), (dict(table_width=1 << 28,
                                                                                             table_stride=1 << 28), S),
    (dict(table_stride=7), ST), (dict(table_stride=-8), ST), (dict(seq_lens=0), N), (dict(count=0), N), (dict(path=0), N),
    (dict(page_table=0), N), (dict(path=A + 2), AL), (dict(lens_out=B + 1), AL), (dict(lens_out=A), ST),
    (dict(lens_out=A + 4), ST), (dict(lens_out=A - 4), ST), (dict(lens_out=B, count=B), ST), (dict(lens_out=B, path=B - 36), ST), (dict(layers=0, caches=0), OK), (dict(batch=0, total_q=0), OK),
    ({}, "device"), (dict(lens_out=0), "device"), (dict(lens_out=A + 64), "device"),
    (dict(table_width=0, page_table=0, table_stride=0), "device"), (dict(width=0, path=0), "device")])
def test_accept(lib, change, status):
    keep, c = _caches({}, {})
    expected = _expect(status)
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "caches": c}, change) == expected
    assert lib.mx_kv_accept_fp4(None, None) == N


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=64, code_page_stride=4096), S), (dict(pages=9), S), (dict(kv_heads=1), S), (dict(head_dim=96), S),
    (dict(code_page_stride=4096), ST), (dict(scale_page_stride=4096), ST), (dict(k=A), ST), (dict(v_scale=A + 12288), ST),
    (dict(v=0), N), (dict(k=A + 65536 + 8), AL), ({}, "device")])
def test_accept_layers_have_one_shape(lib, change, status):
    keep, c = _caches({}, change)
    expected = _expect(status)
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "caches": c}, {}) == expected


@pytest.mark.parametrize("change", [dict(k=A + 8192 + 65536), dict(v=A), dict(v_scale=A + 4096), dict(k_scale=A + 12288)])
def test_accept_refuses_keys_that_lie_on_values(lib, change):
    keep, c = _caches({}, change)
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "caches": c}, {}) == ST


def test_rows_longer_than_any_memory_meet_what_lies_behind_them(lib):
    assert _call(lib, "mx_tree_mask", MASK, dict(mask=A - 4096, mask_stride=1 << 60)) == ST


def test_accept_refuses_blocks_that_lie_on_each_other(lib):
    # pages one block apart with two heads half a block apart from a page's
    meet = dict(code_page_stride=16 * 64 * 3 // 2, code_head_stride=16 * 64)
    keep, c = _caches(meet, meet)
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "caches": c}, {}) == ST


def test_host_tensors_are_refused_before_any_library_call():
    i, f = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    u = [torch.zeros((2, 2, 16, n), dtype=torch.uint8) for n in (64, 4)]
    for call in (lambda: mx.mx_tree_mask(i, i.view(3, 1), max_q=3),
                 lambda: mx.mx_tree_verify(f.view(1, 3), None, i, i, f, f, i, i, i, None),
                 lambda: mx.mx_kv_accept_fp4([], i.view(1, 3), i, i, i, max_q=3)):
        with pytest.raises(mx.MxError) as e:
            call()
        assert e.value.status == mx.MX_ERR_DEVICE
    for call in (lambda: mx.mx_attn_tree_fp4(u[0], f, i, None, None, f, None),
                 lambda: mx.mx_kv_accept_fp4([u[0]], i.view(1, 3), i, i, i, max_q=3)):
        with pytest.raises(TypeError):
            call()
