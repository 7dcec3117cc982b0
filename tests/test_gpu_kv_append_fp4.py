"""Appending to the paged MXFP4 cache (mx_kv_append_fp4): the stored bytes equal the oracle's, bytes
of other slots stay, tokens that no finite code stands for become NaN tokens."""
import numpy as np
import pytest
import torch

from attention_util import bf16, f64, tables
from gpu_util import note
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu


def _cache(pages, h, page, D, fill=0xC3):
    return [torch.full((pages, h, page, D // n), fill, dtype=torch.uint8, device="cuda") for n in (2, 32, 2, 32)]


def _expected(cache, k, v, slots, pos, cos, sin, inter, page):
    want = [t.cpu().numpy().copy() for t in cache]
    kr = A.rotate(k.astype(np.float32), pos, cos, sin, inter, dtype=np.float32)
    kc, kb, kv = A.quantize_fp4(kr)
    vc, vb, vv = A.quantize_fp4(v.astype(np.float32))
    for t, s in enumerate(slots):
        if 0 <= s < want[0].shape[0] * page:
            for a, new in zip(want, (kc, kb, vc, vb)):
                a[s // page, :, s % page] = new[t]
    return want, kv, vv


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (128, 128), (128, 48), (256, 256), (256, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,h,page", [(1, 8, 16), (41, 12, 16), (150, 1, 48), (77, 3, 64)])
def test_bytes(mx, D, rot, inter, T, h, page):
    rng = np.random.default_rng(D + rot + T)
    kv = rng.standard_normal((T, 2 * h, D)) * np.exp(rng.standard_normal((T, 2 * h, D)) * 2)
    kv[0, :, :32] = 0
    kv[T // 2] *= 1e-6
    x = bf16(kv).cuda()
    k, v = x[:, :h], x[:, h:]                                  # strided: keys and values side by side
    pages = -(-T // page) + 2
    cache = _cache(pages, h, page, D)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 3] = -1 if T > 3 else slots[T // 3]             # padding
    if T > 20:
        slots[20] = pages * page                               # past the end: skipped
    cos, sin = tables(rng, 512, rot) if rot else (None, None)
    pos = rng.integers(0, 512, T).astype(np.int32) if rot else None
    want, kval, vval = _expected(cache, f64(k), f64(v), slots, pos, cos, sin, inter, page)
    ko, vo = (torch.full((T, h, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    dev = [None if a is None else torch.from_numpy(a).cuda() for a in (pos, cos, sin)]
    note(f"append D={D} rot={rot} inter={inter} T={T} h={h} page={page}")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), k, v, torch.from_numpy(slots).cuda(), *dev, k_out=ko,
                        v_out=vo, interleaved=inter)
    torch.cuda.synchronize()
    for got, a, name in zip(cache, want, ("k", "k_scale", "v", "v_scale")):
        assert np.array_equal(got.cpu().numpy(), a), name
    live = (slots >= 0) & (slots < pages * page)
    assert np.array_equal(f64(ko)[live], kval[live]) and np.array_equal(f64(vo)[live], vval[live])
    assert (f64(ko)[~live] == 9).all() and (f64(vo)[~live] == 9).all()


@pytest.mark.parametrize("D,rot,T", [(64, 64, 22003), (128, 64, 11003), (256, 256, 5503)])
@pytest.mark.parametrize("inter", [False, True])
def test_bytes_of_many_rows(mx, D, rot, inter, T):
    """From 2^22 values on, two heads of a token at once: three heads leave one short."""
    test_bytes(mx, D, rot, inter, T, 3, 32)


def test_codes_of_values_between_codes(mx):
    # every E2M1 code, midpoint and their bf16 neighbours, at several scales, both signs
    base = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 0.1])
    rows = []
    for e in range(-12, 100, 7):
        for f in (1, 1 + 2.0 ** -7, 1 - 2.0 ** -8):
            row = np.concatenate([base * f, -base * f, base, -base])
            rows.append(np.ldexp(row, e))
    x = bf16(np.stack(rows)[:, None, :]).cuda()                # [T, 1, 64]
    T = x.shape[0]
    cache = _cache(T // 16 + 1, 1, 16, 64)
    slots = np.arange(T, dtype=np.int64)
    want, kval, _ = _expected(cache, f64(x), f64(x), slots, None, None, None, False, 16)
    note("append midpoints")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), x, x, torch.from_numpy(slots).cuda())
    for got, a in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), a)


def test_rotated_values_round_from_fp32(mx):
    # many rotated keys: the codes are those of the fp32 results, products rounded before their sum
    rng = np.random.default_rng(4)
    T, h, D = 600, 4, 128
    k, v = bf16(rng.standard_normal((T, h, D)) * 3).cuda(), bf16(rng.standard_normal((T, h, D))).cuda()
    cos, sin = tables(rng, T, D)
    pos, slots = np.arange(T, dtype=np.int32), np.arange(T, dtype=np.int64)
    cache = _cache(T // 16 + 1, h, 16, D)
    want, _, _ = _expected(cache, f64(k), f64(v), slots, pos, cos, sin, False, 16)
    note("append rotated")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), k, v, *(torch.from_numpy(a).cuda() for a in (slots, pos, cos, sin)))
    for got, a in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), a)


def test_values_without_a_finite_code(mx):
    T, h, D = 8, 2, 128
    x = torch.ones((T, 2 * h, D), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 5] = float("nan")
    x[2, 1, 100] = float("inf")
    x[3, 2, 0] = float("-inf")                                  # a value of head 0
    x[4, 3, 127] = float("nan")                                 # a value of head 1
    x[5, 0, 0] = 3e38                                           # above 6 * 2^125
    x[6, 0, 0] = 2.55e38                                        # 6 * 2^125 itself is stored
    cos, sin = (torch.ones((4, 64), device="cuda"), torch.zeros((4, 64), device="cuda"))
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[7] = 4                                                  # outside the table
    cache = _cache(1, h, 16, D, fill=0)
    ko, vo = (torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    note("append NaN tokens")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), x[:, :h], x[:, h:], torch.arange(T, device="cuda"), pos, cos, sin,
                        k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    bad = np.zeros((T, h), bool)
    bad[1, 0] = bad[2, 1] = bad[3, 0] = bad[4, 1] = bad[5, 0] = True
    bad[7] = True
    ks = cache[1][0].permute(1, 0, 2).cpu().numpy()[:T]
    vs = cache[3][0].permute(1, 0, 2).cpu().numpy()[:T]
    assert np.array_equal((ks == 255).all(-1), bad) and np.array_equal((ks == 255).any(-1), bad)
    assert (vs != 255).all()
    for o in (ko, vo):
        nan = torch.isnan(o).cpu().numpy()
        assert np.array_equal(nan.all(-1), bad) and np.array_equal(nan.any(-1), bad)
    assert f64(ko)[6, 0, 0] == 6 * 2.0 ** 125


def test_offsets_beyond_32_bits(mx):
    h, page, D, stride = 1, 16, 128, 1 << 31
    rng = np.random.default_rng(1)
    k, v = (bf16(rng.standard_normal((2, h, D))).cuda() for _ in "kv")
    big = torch.zeros(3 * stride, dtype=torch.uint8, device="cuda")
    cache = [torch.as_strided(big, (3, h, page, w), (stride, page * w, w, 1), storage_offset=i << 20)
             for i, w in enumerate((D // 2, D // 32, D // 2, D // 32))]
    slots = np.array([2 * page + 3, page - 1], np.int64)
    want, _, _ = _expected(cache, f64(k), f64(v), slots, None, None, None, False, page)
    note("append beyond 4 GiB")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), k, v, torch.from_numpy(slots).cuda())
    for got, a in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), a)


def test_binding_refusals(mx):
    c = mx.MxKvCacheFp4(*_cache(2, 2, 16, 128))
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")

    def refused(status, *args, **kw):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_kv_append_fp4(*args, **kw)
        assert e.type is TypeError if status is None else e.value.status == status

    refused(None, c.k, k, k, slots)
    refused(mx.MX_ERR_SHAPE, c, k[:, :1], k[:, :1], slots)
    refused(mx.MX_ERR_SHAPE, c, k, k[:2], slots)
    refused(None, c, k, k, slots.int())
    refused(mx.MX_ERR_SHAPE, c, k, k, slots[:2])
    refused(mx.MX_ERR_DEVICE, c, k.cpu(), k, slots)
    refused(mx.MX_ERR_SHAPE, c, k, k, slots, k_out=k[:2])
    refused(mx.MX_ERR_ALIGN, c, torch.zeros(3 * 256 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 2, 128), k, slots)
    refused(mx.MX_ERR_ALIGN, c, torch.zeros((3, 2, 132), dtype=torch.bfloat16, device="cuda")[..., :128], k, slots)
