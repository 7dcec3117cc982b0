"""The attention operators' calls of more workgroups than one dimension of a grid holds (2^32 threads),
caches of very large pages, and the longest sequence."""
import numpy as np
import pytest
import torch

from attention_util import Paged, attention_close, bf16, f64, oracle, tables
from gpu_util import note
from oracle import attention_oracle as A
from test_gpu_attn_fp4 import queries, run

pytestmark = pytest.mark.gpu


def test_norm_of_more_rows_than_a_grid_holds(mx):
    # 2^27 + 5 rows of 256, 32 lanes each; the input one row (a token stride of 0), the output 64 GiB
    D, T = 256, (1 << 27) + 5
    rng = np.random.default_rng(1)
    x = bf16(rng.standard_normal((1, 1, D))).cuda()
    cos, sin = tables(rng, 2, D)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-1] = 1
    w = bf16(1 + 0.3 * rng.standard_normal(D)).cuda()
    out = torch.full((T, 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    note(f"norm_rope of {T} rows")
    mx.mx_qk_norm_rope(x.expand(T, 1, D), None, pos, torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), out, None, w)
    torch.cuda.synchronize()
    for row, p in ((0, 0), (T - 1, 1)):
        want, size = A.norm_rope(f64(x), f64(w), np.array([p]), cos, sin)
        assert (np.abs(f64(out[row:row + 1]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size).all()
    for part in out[:-1].view(torch.int64).split(1 << 23):      # all others are row 0's bits
        assert bool((part == out[:1].view(torch.int64)).all())


def test_append_of_more_tokens_than_a_grid_holds(mx):
    # 2^27 + 5 tokens, 32 lanes each, all but six of them padding
    D, T, page = 256, (1 << 27) + 5, 16
    rng = np.random.default_rng(2)
    kv = bf16(rng.standard_normal((2, 1, D))).cuda()
    cache = [torch.full((1, 1, page, D // n), 0xC3, dtype=torch.uint8, device="cuda") for n in (2, 32, 2, 32)]
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    at = {0: 3, 77: 0, (1 << 27) - 9: 5, (1 << 27) - 8: 6, (1 << 27) - 1: 15, T - 1: 9}
    for t, s in at.items():
        slots[t] = s
    note(f"append of {T} tokens")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), kv[:1].expand(T, 1, D), kv[1:].expand(T, 1, D), slots)
    torch.cuda.synchronize()
    kc, kb, _ = A.quantize_fp4(f64(kv[0]).astype(np.float32))
    vc, vb, _ = A.quantize_fp4(f64(kv[1]).astype(np.float32))
    for got, new in zip(cache, (kc, kb, vc, vb)):
        want = np.full(got.shape, 0xC3, np.uint8)
        for s in at.values():
            want[0, :, s] = new
        assert np.array_equal(got.cpu().numpy(), want)


def test_attention_of_more_blocks_than_a_grid_holds(mx):
    # a bound on queries far above most sequences': 1100 x 8 heads x 1000 blocks of 256 rows
    rng = np.random.default_rng(3)
    B, hk, group, max_q, D = 1100, 8, 8, 32000, 64
    news = [1] * B
    news[5], news[900], news[B - 1] = 70, 0, 3
    lens = [int(n) + 2 for n in news]
    lens[900], lens[7] = 9, 0
    starts = [0, *np.cumsum(news).tolist()]
    paged = Paged(rng, lens, hk, D, 16)
    q = queries(rng, starts[-1], hk * group, D)
    note("attn of 8.8 million blocks")
    out, lse = run(mx, paged, q, starts=starts, max_q=max_q)
    attention_close(out, lse, oracle(paged, q, starts, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_into_a_page_of_more_than_4_gib(mx, D):
    # one page of one head, whose codes pass 2^32 bytes
    page = (1 << 33) // D + 160
    rng = np.random.default_rng(D)
    k, v = (bf16(rng.standard_normal((5, 1, D))).cuda() for _ in "kv")
    cache = [torch.zeros((1, 1, page, D // n), dtype=torch.uint8, device="cuda") for n in (2, 32, 2, 32)]
    at = (1 << 33) // D                                        # its codes begin at byte 2^32
    slots = np.array([at + 5, 7, page - 1, at - 1, at], np.int64)
    note(f"append into a page of {page} tokens, D={D}")
    mx.mx_kv_append_fp4(mx.MxKvCacheFp4(*cache), k, v, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    kc, kb, _ = A.quantize_fp4(f64(k).astype(np.float32))
    vc, vb, _ = A.quantize_fp4(f64(v).astype(np.float32))
    for got, new in zip(cache, (kc, kb, vc, vb)):
        for i, s in enumerate(slots):
            assert np.array_equal(got[0, 0, s].cpu().numpy(), new[i, 0]), s
        got[0, 0, torch.from_numpy(slots).cuda()] = 0          # nothing else is written
        assert not any(bool(part.any()) for part in got.view(-1).split(1 << 30))


def test_attention_at_the_longest_length(mx):
    """2^31 - 1024 tokens through a table of 2^27 - 64 entries, all of them one page of 16 tokens: the mean is
    that page's, and the log-sum-exp larger by ln of the entries.

    Each of 768 workgroups' four wavefronts walks about 21845 steps of 32 tokens.  A lane's sum of weights is a
    chain of 8 additions a step, less than 2^18 in all: 2^-6 of it at most; the sums of values are chains of
    less than 2^15 products of 32 tokens, 2^-8 with the weights' rounding and the result's 2^-8."""
    D, page, width = 64, 16, (1 << 27) - 64
    rng = np.random.default_rng(4)
    paged = Paged(rng, [page], 1, D, page, spare=0, width_extra=0)
    q = queries(rng, 1, 4, D)
    o, l, mag, _ = oracle(paged, q, [0, 1], D ** -0.5)
    paged.lens, paged.table = [page * width], np.zeros((1, width), np.int32)
    note("attn of 2^31 - 1024 tokens")
    out, lse = run(mx, paged, q)
    assert (np.abs(f64(out) - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -6 + 2.0 ** -7) * mag).all()
    assert (np.abs(f64(lse) - l - np.log(width)) <= 2.0 ** -6).all()
