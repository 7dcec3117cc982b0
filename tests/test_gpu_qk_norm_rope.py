"""Per-head norm with rotation (mx_qk_norm_rope) and its gradients against the float64 oracle.

Bounds.  A result is one bf16 rounding (2^-8 of it) of fp32 arithmetic whose sums (the row's mean
square, at most 256 terms; the two products of a rotation) are off by at most 2^-18 of their terms'
magnitudes; `size` holds those magnitudes.  A weight's gradient is an fp32 sum in chains of at most
2^9 additions: 2^-15 of the sum of its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from attention_util import bf16, f64, tables
from gpu_util import note
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu


def _close(got, want, size, what):
    g = f64(got)
    bad = ~(np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"


def _setup(seed, T, hq, hk, D, rot, norm, rows=64):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((T, hq + 2 * hk, D)) * 2).cuda()
    w = [bf16(1 + 0.3 * rng.standard_normal(D)).cuda() if norm else None for _ in "qk"]
    cos, sin = tables(rng, rows, rot) if rot else (None, None)
    pos = rng.integers(0, rows, T).astype(np.int32) if rot else None
    dev = [None if a is None else torch.from_numpy(a).cuda() for a in (pos, cos, sin)]
    return rng, x, w, pos, cos, sin, dev


def _np(t):
    return None if t is None else f64(t)


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48), (256, 256), (256, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,hq,hk", [(1, 32, 8), (5, 3, 1), (41, 12, 12), (130, 7, 2)])
def test_forward(mx, D, rot, inter, norm, T, hq, hk):
    rng, x, w, pos, cos, sin, dev = _setup(D + rot + T, T, hq, hk, D, rot, norm)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    qo, ko = (torch.full((T, h, D), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    note(f"norm_rope D={D} rot={rot} inter={inter} norm={norm} T={T} hq={hq} hk={hk}")
    mx.mx_qk_norm_rope(q, k, *dev, qo, ko, *w, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    for got, a, b, name in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want, size = A.norm_rope(f64(a), _np(b), pos, cos, sin, 1e-5, inter)
        _close(got, want, size, name)
    # in place, queries alone: the rest of the packed buffer stays
    y = x.clone()
    mx.mx_qk_norm_rope(y[:, :hq], None, *dev, y[:, :hq], None, w[0], eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :hq], qo) and torch.equal(y[:, hq:], x[:, hq:])


@pytest.mark.parametrize("D,rot,T", [(64, 32, 9401), (128, 128, 4703), (256, 192, 2351)])
@pytest.mark.parametrize("inter", [False, True])
def test_forward_of_many_rows(mx, D, rot, T, inter):
    """From 2^22 values on, four heads of a token at once: 5 and 2 heads leave three and two short."""
    rng, x, w, pos, cos, sin, dev = _setup(D + T, T, 5, 2, D, rot, True)
    q, k = x[:, :5], x[:, 5:7]
    qo, ko = (torch.full((T, h, D), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (5, 2))
    note(f"norm_rope of many rows D={D} rot={rot} inter={inter} T={T}")
    mx.mx_qk_norm_rope(q, k, *dev, qo, ko, *w, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    for got, a, b, name in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want, size = A.norm_rope(f64(a), _np(b), pos, cos, sin, 1e-5, inter)
        _close(got, want, size, name)


def test_rows_of_zeros_huge_and_tiny_values(mx):
    D, T = 128, 4
    x = torch.zeros((T, 2, D), dtype=torch.bfloat16, device="cuda")
    x[1], x[2], x[3] = 1e15, 1e-15, -3.0
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    note("norm of zeros, huge, tiny rows")
    mx.mx_qk_norm_rope(x, None, None, None, None, out, None, w, eps=1e-6)
    want, size = A.norm_rope(f64(x), f64(w), None, None, None, 1e-6)
    _close(out, want, size, "rows")
    assert not out[0].any()


def test_a_position_outside_the_table_gives_nan_rows(mx):
    rng, x, w, pos, cos, sin, dev = _setup(3, 6, 4, 2, 128, 64, True)
    dev[0][1], dev[0][4] = -1, 64
    qo, ko = (torch.empty((6, h, 128), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    note("positions out of range")
    mx.mx_qk_norm_rope(x[:, :4], x[:, 4:6], *dev, qo, ko, *w)
    for o in (qo, ko):
        nan = torch.isnan(o).flatten(1)
        assert nan[[1, 4]].all() and not nan[[0, 2, 3, 5]].any()


@pytest.mark.parametrize("D,rot", [(64, 32), (128, 128), (256, 128), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (3, 5, 1), (41, 12, 12), (1500, 6, 2)])
def test_backward(mx, D, rot, inter, norm, T, hq, hk):
    rng, x, w, pos, cos, sin, dev = _setup(2 * D + rot + T, T, hq, hk, D, rot, norm)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    g = bf16(rng.standard_normal((T, hq + hk, D))).cuda()
    dq, dk = (torch.full((T, h, D), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    dw = [torch.full((D,), float("nan"), device="cuda") if norm else None for _ in "qk"]
    ws = torch.zeros(mx.mx_qk_norm_rope_backward_workspace_size(T, hq, hk, D), dtype=torch.uint8, device="cuda")
    note(f"norm_rope_backward D={D} rot={rot} inter={inter} norm={norm} T={T}")
    args = (g[:, :hq], g[:, hq:], q, k, *dev, dq, dk, *w, *dw, ws)
    mx.mx_qk_norm_rope_backward(*args, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    first = [t.clone() for t in (dq, dk, *dw) if t is not None]
    for got, gw, dy, a, b, name in ((dq, dw[0], g[:, :hq], q, w[0], "q"), (dk, dw[1], g[:, hq:], k, w[1], "k")):
        dx, want_w, size, size_w = A.norm_rope_backward(f64(dy), f64(a), _np(b), pos, cos, sin, 1e-5, inter)
        _close(got, dx, size, "d" + name)
        if norm:
            assert (np.abs(f64(gw) - want_w) <= 2.0 ** -15 * size_w).all(), "dw " + name
    # again through the same workspace, in place over the incoming gradients: the same bits
    mx.mx_qk_norm_rope_backward(g[:, :hq], g[:, hq:], q, k, *dev, g[:, :hq], g[:, hq:], *w, *dw, ws,
                                eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    again = [g[:, :hq], g[:, hq:]] + [t for t in dw if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_weight_gradient_alone_of_one_tensor_and_without_rows(mx):
    rng, x, w, pos, cos, sin, dev = _setup(9, 20, 3, 2, 128, 128, True)
    g = bf16(rng.standard_normal((20, 3, 128))).cuda()
    dq, dw = torch.empty_like(g), torch.empty(128, device="cuda")
    ws = torch.zeros(mx.mx_qk_norm_rope_backward_workspace_size(20, 3, 0, 128), dtype=torch.uint8, device="cuda")
    note("norm_rope_backward queries alone")
    mx.mx_qk_norm_rope_backward(g, None, x[:, :3], None, *dev, dq, None, w[0], None, dw, None, ws)
    _, want, _, size = A.norm_rope_backward(f64(g), f64(x[:, :3]), f64(w[0]), pos, cos, sin)
    assert (np.abs(f64(dw) - want) <= 2.0 ** -15 * size).all()
    dw.fill_(7)
    empty = [t[:0] for t in (g, x[:, :3], dq)]
    note("norm_rope_backward without tokens")
    mx.mx_qk_norm_rope_backward(empty[0], None, empty[1], None, dev[0][:0], dev[1], dev[2], empty[2], None,
                                w[0], None, dw, None, ws)
    torch.cuda.synchronize()
    assert not dw.any()


def test_binding_refusals(mx):
    x = torch.zeros((4, 6, 128), dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(x)
    cos = torch.zeros((16, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")

    def refused(status, *args, **kw):
        with pytest.raises((mx.MxError, TypeError)) as e:
            mx.mx_qk_norm_rope(*args, **kw)
        assert e.type is TypeError if status is None else e.value.status == status

    refused(mx.MX_ERR_DEVICE, x.cpu(), None, pos, cos, cos, o, None)
    refused(None, x.float(), None, pos, cos, cos, o, None)
    refused(None, x, None, pos.long(), cos, cos, o, None)
    refused(None, x, None, None, cos, cos, o, None)
    refused(mx.MX_ERR_SHAPE, x, None, pos[:3], cos, cos, o, None)
    refused(mx.MX_ERR_SHAPE, x, None, pos, cos, cos[:8], o, None)
    refused(mx.MX_ERR_SHAPE, x, None, pos, cos[:, :60].contiguous(), cos[:, :60].contiguous(), o, None)
    refused(mx.MX_ERR_STRIDE, x, None, pos, cos[:, :32], cos[:, :32], o, None)
    refused(mx.MX_ERR_SHAPE, x[..., :96], None, None, None, None, o[..., :96], None)
    refused(mx.MX_ERR_SHAPE, x, None, pos, cos, cos, o, None, w[:64])
    refused(mx.MX_ERR_SHAPE, x, x[:3], pos, cos, cos, o, o)
    refused(mx.MX_ERR_STRIDE, x, None, pos, cos, cos, o[:1].expand(4, 6, 128), None)
    refused(mx.MX_ERR_STRIDE, x.transpose(1, 2), None, None, None, None, o, None)
    refused(mx.MX_ERR_SHAPE, x, None, pos, cos, cos, o, None, w, eps=-1.0)
    with pytest.raises(mx.MxError) as e:
        mx.mx_qk_norm_rope_backward(x, None, x, None, pos, cos, cos, o, None, w, None,
                                    torch.empty(128, device="cuda"))
    assert e.value.status == mx.MX_ERR_WORKSPACE
    with pytest.raises(mx.MxError) as e:                     # a gradient of no weight
        mx.mx_qk_norm_rope_backward(x, None, x, None, pos, cos, cos, o, None, None, None,
                                    torch.empty(128, device="cuda"))
    assert e.value.status == mx.MX_ERR_NULL
